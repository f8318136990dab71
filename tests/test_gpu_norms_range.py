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


def gates(dtype, kda, a, a_log, dt_bias=None, d=64):
    """Decays of logits a [m, h] (the same for every channel), as [m, h]."""
    b = B()
    m, h = a.shape
    cfg = b.make_config(1, h, d, d, bits=8, in_dtype=dtype, decay_kind="kda" if kda else "gdn")
    ch = (d,) if kda else ()
    x = a.to(DT[dtype])
    if kda:
        x = x[..., None].expand(m, h, d).contiguous()
    rows = torch.ones(m, h, d, dtype=DT[dtype], device="cuda")
    bias = torch.zeros(h, device="cuda") if dt_bias is None else dt_bias
    bias = bias[:, None].expand(h, d).contiguous() if kda else bias
    decay, beta = torch.empty(m, h, *ch, device="cuda"), torch.empty(m, h, device="cuda")
    b.lq_qk_norm(cfg, rows, rows, x, torch.zeros(m, h, device="cuda").to(DT[dtype]), a_log, bias, torch.empty_like(rows),
                 torch.empty_like(rows), decay, beta)
    if kda:
        assert torch.equal(decay, decay[..., :1].expand_as(decay)) or decay.isnan().any()
        decay = decay[..., 0]
    return decay


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kda", [False, True])
def test_strong_decays(kda, dtype):
    """Logits of 18 and more with a rate of 1: softplus is the logit itself (what
    is left out is below half a unit), so the decay is exp(-a) and nothing of a's
    size is rounded before the exponential: 2 units of 2^-23 for it, one rounding
    of 2^-24 for the correction, one for the sum."""
    m, h = 512, 4
    a = torch.linspace(18, 87, m * h, device="cuda").view(m, h).to(DT[dtype])
    want = torch.exp(-a.double())
    within(gates(dtype, kda, a, torch.zeros(h, device="cuda")), want, 8 * U * want, "decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_both_kinds_of_gate_agree(dtype):
    """A gate per key channel with equal channels has the bits of a gate per head."""
    m, h = 301, 7
    a, a_log, bias = 4 * randn(3, m, h), 2 * randn(4, h), randn(5, h) - 2
    assert torch.equal(gates(dtype, True, a, a_log, bias), gates(dtype, False, a, a_log, bias))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kda", [False, True])
def test_logits_and_rates_at_their_ends(kda, dtype):
    """Infinite and NaN logits, and rates so small or large that products leave
    FP32: exp(-exp(a_log) softplus(a)) in 64 bits, within 14 units of 2^-24 of the
    exponent and 8 of the result."""
    inf = float("inf")
    logits = [inf, -inf, float("nan"), 1e38, -1e38, 0.0, -80.0, 3.0]
    rates = [0.0, 45.0, 60.0, -42.0, -80.0]
    a = torch.tensor(logits, device="cuda")[:, None].expand(len(logits), len(rates)).contiguous()
    a_log = torch.tensor(rates, device="cuda")
    got = gates(dtype, kda, a, a_log)
    z = a.to(DT[dtype]).double()
    x = a_log.double().exp() * torch.logaddexp(z, torch.zeros_like(z))
    want = torch.exp(-x)
    assert got[2].isnan().all()
    keep = [i for i in range(len(logits)) if i != 2]
    got, want, x = got[keep], want[keep], x[keep]
    far = x > 1000                     # the decay is 0 there
    assert (got[far] == 0).all()
    want, x, got = want[~far], x[~far], got[~far]
    # exp(-|a|) below is within (4 + 2.4 |a|) units where softplus is that small: 200 at -80
    within(got, want, want * U * (214 * x + 8) + 2.0 ** -125, "decay")
    assert (gates(dtype, kda, torch.tensor([[-inf]], device="cuda"), torch.zeros(1, device="cuda")) == 1).all()
