"""Gates above 1 in the linear-attention calls: refused like negative ones, by
tokens and by every form of a prompt."""
import pytest

from tests.test_gpu_linear import DT, inputs, near, reference, run_prefill, state_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ABOVE = [1.0 + 2.0 ** -23, 1.5, 1e30, 3e38]   # the first is the next FP32 value


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()


def statuses(st, n, h):
    return st.blobs()[:, 4:8].contiguous().view(torch.int32).view(n, h).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_token_with_a_gate_above_one_is_skipped(d, dtype):
    n, h = len(ABOVE) + 1, 2
    x = inputs(100, n, 1, h, h, d, DT[dtype])
    x["decay"][:, 0, 0] = torch.tensor(ABOVE + [1.0], device="cuda")
    st = state_of(n, h, d, DT[dtype])
    st.init(x["S0"])
    before = st.buf.clone().view(n, h, -1)
    out = torch.full((n, h, d), float("nan"), device="cuda")
    st.linear_step(*(x[name][:, 0].contiguous() for name in ("q", "k", "v", "decay")), out)
    bad = len(ABOVE)
    assert statuses(st, n, h) == [[2, 0]] * bad + [[0, 0]]
    assert (out[:bad, 0] == 0).all()
    assert torch.equal(st.buf.view(n, h, -1)[:bad, 0, 128:], before[:bad, 0, 128:])
    x["decay"][:bad, 0, 0] = 0
    want, S = reference(x, x["S0"])
    near(out[:, 1], want[:, 0, 1])
    near(out[bad:], want[bad:, 0])
    near(st.dequant()[bad:], S[bad:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [9, 150, 1500])
@pytest.mark.parametrize("cont", [False, True])
def test_a_prompt_ends_before_a_gate_above_one(t, cont, d, dtype):
    n, h = len(ABOVE) + 1, 2
    x = inputs(101, n, t, h, h, d, DT[dtype])
    ends = [0, 1, t // 2, t - 1, t]
    y = dict(x, decay=x["decay"].clone())
    for i, (e, a) in enumerate(zip(ends, ABOVE)):
        y["decay"][i, e:, 0] = a            # and all behind it
    y["decay"][n - 1, :, 1] = 1.0
    x["decay"][n - 1, :, 1] = 1.0
    st = state_of(n, h, d, DT[dtype])
    if cont:
        st.init(x["S0"])
    out = run_prefill(st, y, S0=None if cont else x["S0"], cont=cont)
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    first = {k: v[:, :, :1].contiguous() if k != "S0" else v[:, :1] for k, v in x.items()}
    want, S = reference(first, first["S0"], lengths)
    near(out[:, :, :1], want, "before the gate")
    for i, e in enumerate(ends):
        assert (out[i, e:, 0] == 0).all()
    near(st.dequant()[:, :1], S, "state before the gate")
    second = {k: v[:, :, 1:].contiguous() if k != "S0" else v[:, 1:] for k, v in x.items()}
    want, S = reference(second, second["S0"])
    near(out[:, :, 1:], want, "the head beside it")
    near(st.dequant()[:, 1:], S, "its state")
    assert statuses(st, n, h) == [[2, 0]] * len(ABOVE) + [[0, 0]]
