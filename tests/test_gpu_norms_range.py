"""Gates far from zero: the output gate down to FP32's smallest values, decays
down to them, and the same rates for both kinds of gate."""
import pytest

from tests.test_gpu_norms import DT, HALF, U, B, randn, within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149  # FP32's smallest value


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
@pytest.mark.parametrize("d", [64, 128])
def test_output_gates_far_from_zero(d, gate, dtype):
    """f32: a library exponential (2 units of 2^-23), a sum, a quotient and the
    products beside the norm's d / 2 + 8 roundings of 2^-24.  bf16: 1e-5 for the
    gate.  Results below the normal numbers: half a step of FP32's smallest for
    the gate, times what it is multiplied by, and half a step for the result."""
    b = B()
    m, h = 64, 3
    cfg = b.make_config(1, h, d, d, bits=32, in_dtype=dtype)
    o = 1 + 0.2 * randn(1, m, h, d)
    g = torch.linspace(-102, 30, m * h * d, device="cuda").view(m, h, d).to(DT[dtype])
    y = torch.empty(m, h, d, dtype=DT[dtype], device="cuda")
    b.lq_out_norm(cfg, o, y, gate=g, gate_kind=gate, eps=0.0)
    x = o.double()
    norm = x / x.square().mean(-1, keepdim=True).sqrt()
    factor = norm * (g.double() if gate == "silu" else 1)
    want = factor * torch.sigmoid(g.double())
    rel = HALF[dtype] + (d / 2 + 16) * U + (1e-5 if dtype == "bf16" else 0)
    # a value of the output's type below its normal ones: half of its smallest
    small = TINY / 2 if dtype == "f32" else 2.0 ** -134
    within(y, want, rel * want.abs() + 3 * TINY * factor.abs() + small, "y")
