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
    subprocess.run([os.environ.get("NVCC", "nvcc"), *build.NVCC_FLAGS, "-shared", "-I", os.path.join(ROOT, "include"), "-I",
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


@pytest.mark.parametrize("cont,d", [(False, 64), (False, 128), (True, 128)])
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


QK, D_DONE, Y_DONE, O_DONE, EMPTY = ("&bars->qk_done", "&bars->d_done[c % NK]", "&bars->y_done", "&bars->o_done[c & 1u]",
                                     "&bars->empty[st]")


def check_heads(st, out, want, S, n, h, d):
    """Every head is right or has LQ_DEV_TIMEOUT; returns how many have it."""
    state = st.blobs()[:, 128:128 + 4 * d * d].contiguous().view(torch.float32).view(n, h, d, d)
    status = st.blobs()[:, 4:8].contiguous().view(torch.int32).view(n, h)
    assert ((status == 0) | (status == TIMEOUT)).all()
    good = status == 0
    near(out.transpose(1, 2)[good], want.transpose(1, 2)[good], "outputs of the other heads")
    near(state[good], S[good], "states of the other heads")
    assert (st.blobs()[:, 12:16].contiguous().view(torch.int32) == 0x4C515354).all()
    return int((~good).sum())


@pytest.mark.parametrize("cont,d", [(False, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("name,n,h,t,nth", [
    # many heads: one SM takes several, one after the other
    (QK, 50, 12, 130, 4), (D_DONE, 50, 12, 130, 4), (Y_DONE, 50, 12, 130, 4), (O_DONE, 50, 12, 130, 4), (EMPTY, 50, 12, 130, 4),
    (O_DONE, 50, 12, 130, 0),
    # one head, the last of its chunks: its state is complete where its outputs are not
    (QK, 1, 1, 200, 3), (Y_DONE, 1, 1, 200, 3), (O_DONE, 1, 1, 200, 3)])
def test_lost_chunks_are_reported(lossy, name, n, h, t, nth, cont, d):
    """A chunk whose products are not seen to end: whatever it leaves unfinished
    has the status, whichever role gave up."""
    x = inputs(81, n, t, h, h, d, torch.bfloat16)
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, torch.bfloat16)
    if cont:
        st.init(x["S0"])
    out = torch.full_like(want, float("nan"), dtype=torch.float32)
    call = dict(tokens=t, q=x["q"], k=x["k"], v=x["v"], decay=x["decay"], out=out)
    assert lossy(name, nth=nth) == 0
    st.linear_prefill(**call, S0=None if cont else x["S0"], cont=cont)
    torch.cuda.synchronize()
    # at most the described ones, the one being fed and the one claimed
    assert 1 <= check_heads(st, out, want, S, n, h, d) <= 6
    assert lossy("") == 0
    st.linear_prefill(**call, S0=x["S0"])
    assert check_heads(st, out, want, S, n, h, d) == 0


@pytest.mark.parametrize("cont,d", [(False, 64), (False, 128), (True, 128)])
def test_a_chunk_lost_in_a_segment_is_reported(lossy, cont, d):
    """A prompt cut along time: the segment that loses a chunk is not the one that
    holds the prompt's end, whose CTA goes on."""
    from linear_attention_recurrent_lq_b200 import binding as b
    n, h, t = 1, 24, 2500
    x = inputs(82, n, t, h, h, d, torch.bfloat16)
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, torch.bfloat16)
    if cont:
        st.init(x["S0"])
    nseg = segments(st, n * h, b.lq_linear_prefill_workspace(st.cfg, n, t), d)
    out = torch.full_like(want, float("nan"), dtype=torch.float32)
    call = dict(tokens=t, q=x["q"], k=x["k"], v=x["v"], decay=x["decay"], out=out)
    assert lossy(O_DONE, block=nseg + 1) == 0   # the second segment of the second head
    st.linear_prefill(**call, S0=None if cont else x["S0"], cont=cont)
    torch.cuda.synchronize()
    assert st.blobs()[1, 4:8].view(torch.int32).item() == TIMEOUT
    assert 1 <= check_heads(st, out, want, S, n, h, d) <= 6
    assert lossy("") == 0
    st.linear_prefill(**call, S0=x["S0"])
    assert check_heads(st, out, want, S, n, h, d) == 0
