"""A padded row so long that its zeros, counted in values, pass 2^31."""
import pytest

from tests.test_gpu_linear import DT, reference, near, run_prefill, state_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,d,t,cut", [("f32", 64, 2 ** 25 + 2 ** 16, False), ("f32", 64, 2 ** 25 + 2 ** 16, True),
                                           ("bf16", 128, 2 ** 26 + 2 ** 16, False)])
def test_zeros_behind_a_short_row_of_a_very_long_call(dtype, d, t, cut):
    """One head, a few tokens, padding to the end; q, k and v are one tensor."""
    length = 5
    g = torch.Generator(device="cuda").manual_seed(90)
    x = torch.empty(1, t, 1, d, dtype=DT[dtype], device="cuda")
    x[:, :128] = torch.randn(1, 128, 1, d, generator=g, device="cuda").to(DT[dtype]) * d ** -0.5
    a = torch.full((1, t, 1), 0.5, device="cuda")
    call = dict(q=x, k=x, v=x, decay=a, S0=None)
    st = state_of(1, 1, d, DT[dtype])
    out = run_prefill(st, call, lengths=torch.tensor([length], dtype=torch.int32, device="cuda"), cut=cut)
    want, S = reference({k: v[:, :length] for k, v in call.items() if v is not None}, None)
    near(out[:, :length], want)
    near(st.dequant(), S)
    assert st.check() == 0
    rows = out.view(t, d)
    for at in range(length, t, 2 ** 22):    # run_prefill gives outputs full of 7
        assert not rows[at:at + 2 ** 22].any()
