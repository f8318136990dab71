"""Linear-attention prompts in which a wait gives up: the heads it concerns end
with LQ_DEV_TIMEOUT, every other head is right, and the context stays usable.

A copy of the library is built in which one chosen commit is not made
(lost_commit.cu), so its waiters run into their limit of a second."""
import ctypes
import os
import subprocess

import pytest

from tests.test_gpu_linear import inputs, near, reference, state_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TIMEOUT = 4  # LQ_DEV_TIMEOUT


@pytest.fixture(scope="module")
def lossy(tmp_path_factory):
    """The binding's library with the linear-attention calls of the copy, and
    the function that chooses the commit to leave out."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()
    from linear_attention_recurrent_lq_b200 import binding as b
    out = str(tmp_path_factory.mktemp("lossy") / "lossy.so")
    subprocess.run(["nvcc", *build.NVCC_FLAGS, "-shared", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(build.HERE, "csrc"), "-o", out, os.path.join(ROOT, "tests", "lost_commit.cu")], check=True)
    so = ctypes.CDLL(out)
    for name in ("lq_linear_prefill", "lq_linear_prefill_workspace"):
        getattr(so, name).argtypes = getattr(b.lib, name).argtypes
        getattr(so, name).restype = getattr(b.lib, name).restype
    so.lose_commit.argtypes = [ctypes.c_char_p] + [ctypes.c_int] * 3
    real = b.lib

    class Lib:
        def __getattr__(self, name):
            return getattr(so if name.startswith("lq_linear_prefill") else real, name)

    b.lib = Lib()
    yield lambda name, block=0, segment=0, nth=0: so.lose_commit(name.encode(), block, segment, nth)
    b.lib = real


def statuses(st, n, h):
    return st.blobs()[:, 4:8].contiguous().view(torch.int32).view(n, h).tolist()


def segments(st, work, need, d):
    return (need // 4 - work) // (work * (d * d + 2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cont", [False, True])
@pytest.mark.parametrize("name,nth", [("&bars->all_done", 0), ("&bars->d_done[i & 1]", 0),
                                      ("&bars->empty[i % kLsStages]", 1)])
def test_a_lost_segment_is_reported(lossy, name, nth, cont, d):
    """The first pass of a prompt cut along time loses a segment of one head:
    zero outputs, the state as it was, and the status, which no later pass
    clears."""
    from linear_attention_recurrent_lq_b200 import binding as b
    n, h, t, head = 1, 24, 2500, 1
    x = inputs(80, n, t, h, h, d, torch.bfloat16)
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, torch.bfloat16)
    st.init(x["S0"])
    nseg = segments(st, n * h, b.lq_linear_prefill_workspace(st.cfg, n, t), d)
    assert 4 <= nseg <= 8  # several chunks each, more than there are stages
    before = st.dequant()
    out = torch.full_like(want, float("nan"), dtype=torch.float32)
    call = dict(tokens=t, q=x["q"], k=x["k"], v=x["v"], decay=x["decay"], out=out)
    assert lossy(name, block=head, segment=nseg // 2, nth=nth) == 0
    st.linear_prefill(**call, S0=None if cont else x["S0"], cont=cont)
    torch.cuda.synchronize()
    assert statuses(st, n, h) == [[TIMEOUT if i == head else 0 for i in range(h)]]
    assert st.check() == b.LQ_ERR_TIMEOUT
    assert (out[:, :, head] == 0).all()
    others = [i for i in range(h) if i != head]
    near(out[:, :, others], want[:, :, others], "the other heads")
    state = st.blobs()[:, 128:128 + 4 * d * d].contiguous().view(torch.float32).view(n, h, d, d)
    near(state[:, others], S[:, others], "the other states")
    assert torch.equal(state[:, head], before[:, head])
    # nothing is lost any more: the next call from a given state is right
    assert lossy("") == 0
    st.linear_prefill(**call, S0=x["S0"])
    near(out, want)
    near(st.dequant(), S)
    assert st.check() == 0
