"""Linear attention with one decay per head on the GPU: one token, prompts,
slot lists and prompts cut along time, against the recurrence in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Relative 2-norm of an output or state.  A value is a sum of terms, each
# rounded once or twice per token it is carried (about 1 / (1 - gate) = 40 to
# 64 tokens here) and once per key channel it is summed over (<= 128): some
# 256 independent roundings of at most 2^-24, so 16 x 2^-24 = 2^-20; twice
# that where an accumulator truncates.
REL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()


def B():
    from linear_attention_recurrent_lq_b200 import binding
    return binding


def inputs(seed, n, t, h, hk, d, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda")

    q, k = randn(n, t, hk, d), randn(n, t, hk, d)
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    a = torch.exp(-torch.nn.functional.softplus(randn(n, t, h) - 4))
    return dict(q=q.to(dtype), k=k.to(dtype), v=randn(n, t, h, d).to(dtype), decay=a, S0=randn(n, h, d, d))


def reference(x, S0, lengths=None):
    """Outputs and final state in 64 bits, token by token; tokens behind a
    row's length leave its state as it is and give zeros."""
    n, t, h, d = x["v"].shape
    g = h // x["q"].shape[2]
    q, k = (x[name].double().repeat_interleave(g, 2) for name in ("q", "k"))
    v, a = x["v"].double(), x["decay"].double()
    S = torch.zeros(n, h, d, d, dtype=torch.float64, device="cuda") if S0 is None else S0.double().clone()
    out = torch.zeros(n, t, h, d, dtype=torch.float64, device="cuda")
    for i in range(t):
        new = S * a[:, i, :, None, None] + k[:, i, :, :, None] * v[:, i, :, None, :]
        o = (q[:, i, :, :, None] * new).sum(-2)
        live = torch.ones(n, dtype=torch.bool, device="cuda") if lengths is None else lengths > i
        S = torch.where(live[:, None, None, None], new, S)
        out[:, i] = torch.where(live[:, None, None], o, torch.zeros_like(o))
    return out, S


def near(got, want, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    err, ref = (got - want).norm().item(), want.norm().item()
    assert err <= REL * ref, f"{what}: relative error {err / ref if ref else err:.2e}"


def state_of(n, h, d, dtype, slots=None):
    b = B()
    st = b.LQState(b.make_config(slots or n, h, d, d, bits=32, in_dtype="bf16" if dtype == torch.bfloat16 else "f32"))
    st.buf.fill_(0xA5)
    return st


def run_prefill(st, x, S0=None, lengths=None, cont=False, cut=True, out=True, slots=None):
    """The call, with outputs laid between guard rows and an unused workspace
    full of NaN."""
    b = B()
    n, t, h, d = x["v"].shape
    size = n * t * h * d
    guard = torch.full((size + 256,), 7.0, device="cuda")
    o = guard[128:128 + size].view(n, t, h, d) if out else None
    need = b.lq_linear_prefill_workspace(st.cfg, n, t) if cut else 0
    ws = torch.full((max(need, 4) // 4,), float("nan"), device="cuda").view(torch.uint8) if need else None
    args = dict(S0=S0, lengths=lengths, out=o, qk_heads=x["q"].shape[2], cont=cont)
    if cut:
        args["workspace"] = ws
    else:
        args["workspace"] = None
    call = dict(state=st.buf, tokens=t, q=x["q"], k=x["k"], v=x["v"], decay=x["decay"])
    if not cut:  # a null workspace reaches the library as it is
        real = b._linear_workspace
        b._linear_workspace = lambda *a: (None, None, 0)
    try:
        if slots is None:
            b.lq_linear_prefill(st.cfg, **call, **args)
        else:
            b.lq_linear_prefill_slots(st.cfg, slots=slots, **call, **args)
    finally:
        if not cut:
            b._linear_workspace = real
    torch.cuda.synchronize()
    assert (guard[:128] == 7.0).all() and (guard[128 + size:] == 7.0).all()
    return o


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h,hk,d", [(1, 1, 1, 128), (3, 6, 2, 64), (2, 8, 8, 128), (37, 9, 3, 128), (100, 12, 1, 64)])
def test_step(n, h, hk, d, dtype):
    x = inputs(1, n, 3, h, hk, d, DT[dtype])
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    st.init(x["S0"])
    out = torch.full((n, h, d), float("nan"), device="cuda")
    for t in range(3):
        st.linear_step(*(x[name][:, t].contiguous() for name in ("q", "k", "v", "decay")), out, qk_heads=hk)
        near(out, want[:, t], f"token {t}")
    near(st.dequant(), S, "state")
    assert st.check() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_step_gates_at_their_ends_and_bad_ones(d):
    """Gates of 0 and 1 are exact; a negative, infinite or NaN gate, a set
    status and a wrong header skip their head alone."""
    b = B()
    n, h = 8, 2
    x = inputs(2, n, 1, h, h, d, torch.bfloat16)
    x["decay"][:, 0, 0] = torch.tensor([0.0, 1.0, -1e-30, float("nan"), float("inf"), -0.0, 0.5, 0.5])
    st = state_of(n, h, d, torch.bfloat16)
    st.init(x["S0"])
    st.blobs()[6 * h].view(torch.int32)[1] = 2     # status
    st.blobs()[7 * h].view(torch.int32)[3] = 1     # magic
    before = st.buf.clone().view(n, h, -1)
    out = torch.full((n, h, d), float("nan"), device="cuda")
    st.linear_step(*(x[name][:, 0].contiguous() for name in ("q", "k", "v", "decay")), out)
    torch.cuda.synchronize()
    skip = [2, 3, 4, 6, 7]
    rest = [i for i in range(n) if i not in skip]
    after = st.buf.view(n, h, -1)
    assert (out[skip, 0] == 0).all()
    assert torch.equal(after[skip, 0, 128:], before[skip, 0, 128:])
    status = after[:, 0, 4:8].contiguous().view(torch.int32).flatten().tolist()
    assert status == [0, 0, 2, 2, 2, 0, 2, 8]
    good = {k: (v[rest] if k != "S0" else v[rest]) for k, v in x.items()}
    want, S = reference(good, good["S0"])
    near(out[rest], want[:, 0])
    near(st.dequant()[rest], S)
    y = {k: v[skip] for k, v in x.items()}
    y["decay"] = y["decay"].clone()
    y["decay"][:, 0, 0] = 0
    near(out[skip, 1], reference(y, y["S0"])[0][:, 0, 1], "the head beside a skipped one")
    assert st.check() == b.LQ_ERR_RANGE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_step_slots(d, dtype):
    N, h, hk = 9, 6, 3
    rows = [5, 0, -1, 8, 9, 2]
    x = inputs(3, len(rows), 1, h, hk, d, DT[dtype])
    st = state_of(N, h, d, DT[dtype])
    S0 = inputs(4, N, 1, h, hk, d, DT[dtype])["S0"]
    st.init(S0)
    before = st.buf.clone().view(N, -1)
    out = torch.full((len(rows), h, d), float("nan"), device="cuda")
    slots = torch.tensor(rows, dtype=torch.int32, device="cuda")
    st.linear_step_slots(slots, *(x[name][:, 0].contiguous() for name in ("q", "k", "v", "decay")), out, qk_heads=hk)
    live = [i for i, s in enumerate(rows) if 0 <= s < N]
    at = [rows[i] for i in live]
    want, S = reference({k: v[live] for k, v in x.items()}, S0[at])
    near(out[live], want[:, 0])
    near(st.dequant()[at], S)
    assert (out[[2, 4]] == 0).all()
    others = [i for i in range(N) if i not in at]
    assert torch.equal(st.buf.view(N, -1)[others], before[others])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 63, 64, 65, 130, 300])
def test_prefill_lengths_of_a_prompt(t, d, dtype):
    n, h, hk = 2, 4, 2
    x = inputs(5, n, t, h, hk, d, DT[dtype])
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    near(run_prefill(st, x, S0=x["S0"]), want, "out")
    near(st.dequant(), S, "state")
    assert st.check() == 0
    near(run_prefill(st, x), reference(x, None)[0], "from zero")
    before = st.buf.clone()
    run_prefill(st, x, out=False)                       # without outputs: the same state
    assert torch.equal(st.buf, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h,hk,d,t", [(40, 12, 4, 128, 70), (80, 12, 12, 64, 100), (300, 1, 1, 128, 65), (1, 1, 1, 64, 200),
                                        (40, 12, 4, 128, 5), (100, 1, 1, 128, 17), (90, 2, 1, 64, 33),
                                        (5, 36, 12, 128, 130)])
def test_prefill_head_layouts(n, h, hk, d, t, dtype):
    x = inputs(6, n, t, h, hk, d, DT[dtype])
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    st.init(x["S0"])
    near(run_prefill(st, x, cont=True), want, "out")
    near(st.dequant(), S, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,t", [(9, 150), (7, 1100)])
def test_prefill_ragged_rows_with_padding_full_of_nan(n, t, d, dtype):
    h, hk = 3, 3
    x = inputs(7, n, t, h, hk, d, DT[dtype])
    lengths = torch.tensor([0, 1, t, t + 5, -3, t // 2, 64, 128, t - 1][:n], dtype=torch.int32, device="cuda")
    pad = torch.arange(t, device="cuda") >= lengths[:, None].clamp(0, t)
    want, S = reference(x, x["S0"], lengths)
    for name in ("q", "k", "v", "decay"):
        x[name] = x[name].masked_fill(pad.view(n, t, *[1] * (x[name].dim() - 2)), float("nan"))
    st = state_of(n, h, d, DT[dtype])
    out = run_prefill(st, x, S0=x["S0"], lengths=lengths)
    near(out, want, "out")
    assert (out[pad] == 0).all()
    near(st.dequant(), S, "state")
    assert st.check() == 0
    st.init(x["S0"])
    near(run_prefill(st, x, lengths=lengths, cont=True), want, "continued")
    near(st.dequant(), S, "continued state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_strong_and_resetting_gates(d, dtype):
    """Gates of 0, products far below the smallest float, and runs of 1."""
    n, t, h = 2, 200, 4
    x = inputs(8, n, t, h, h, d, DT[dtype])
    a = x["decay"]
    a[0, ::37, 0] = 0
    a[0, 63:66, 1] = 0
    a[0, :, 2] = 1e-3
    a[0, :, 3] = 1
    a[1, :, 0] = 1e-30
    a[1, ::2, 1] = 1e-20
    a[1, 64:128, 2] = 0
    a[1, :, 3] = 0
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    out = run_prefill(st, x, S0=x["S0"])
    for i in range(n):
        for j in range(h):
            near(out[i, :, j], want[i, :, j], f"out {i} {j}")
            near(st.dequant()[i, j], S[i, j], f"state {i} {j}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [100, 1500])
@pytest.mark.parametrize("cont", [False, True])
def test_prefill_ends_before_a_bad_gate(t, cont, d, dtype):
    b = B()
    n, h = 6, 2
    x = inputs(9, n, t, h, h, d, DT[dtype])
    ends = [0, 1, 17, t // 2, t - 1, t]
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    bad = [-1.0, float("nan"), float("inf"), -1e-38, float("-inf")]
    y = dict(x, decay=x["decay"].clone())
    for i, e in enumerate(ends[:5]):
        y["decay"][i, e, 0] = bad[i]
    st = state_of(n, h, d, DT[dtype])
    if cont:
        st.init(x["S0"])
    out = run_prefill(st, y, S0=None if cont else x["S0"], cont=cont)
    cut = {k: v[:, :, :1].contiguous() if k != "S0" else v[:, :1] for k, v in x.items()}
    want, S = reference(cut, cut["S0"], lengths)
    near(out[:, :, :1], want, "out before the gate")
    for i, e in enumerate(ends):
        assert (out[i, e:, 0] == 0).all()
    near(st.dequant()[:, :1], S, "state before the gate")
    side = {k: v[:, :, 1:].contiguous() if k != "S0" else v[:, 1:] for k, v in x.items()}
    near(out[:, :, 1:], reference(side, side["S0"])[0], "the head beside it")
    status = st.blobs()[:, 4:8].contiguous().view(torch.int32).view(n, h).tolist()
    assert status == [[2, 0]] * 5 + [[0, 0]]
    # a set status: the next call that goes on from the blobs skips these heads
    before = st.buf.clone().view(n, h, -1)
    out = run_prefill(st, x, cont=True)
    assert (out[:5, :, 0] == 0).all()
    assert torch.equal(st.buf.view(n, h, -1)[:5, 0], before[:5, 0])
    assert st.check() == b.LQ_ERR_RANGE
    # a wrong header is refused too
    st.blobs()[5 * h].view(torch.int32)[3] = 0
    out = run_prefill(st, x, cont=True)
    assert (out[5, :, 0] == 0).all()
    assert st.blobs()[5 * h, 4:8].view(torch.int32).item() == 8
    # and a call from a given state writes the headers anew
    run_prefill(st, x, S0=x["S0"])
    assert st.check() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h,d,t", [(1, 3, 128, 1031), (2, 2, 64, 2048), (1, 1, 128, 3001)])
def test_prefill_cut_along_time(n, h, d, t, dtype):
    """Few heads and a long prompt: with and without the cut."""
    b = B()
    x = inputs(10, n, t, h, h, d, DT[dtype])
    x["decay"][:, 700, :] = 0
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    assert b.lq_linear_prefill_workspace(st.cfg, n, t) > 0
    for cut in (True, False):
        near(run_prefill(st, x, S0=x["S0"], cut=cut), want, f"out, cut {cut}")
        near(st.dequant(), S, f"state, cut {cut}")
        st.init(x["S0"])
        near(run_prefill(st, x, cont=True, cut=cut), want, f"continued, cut {cut}")
        near(st.dequant(), S, f"continued state, cut {cut}")
    o = torch.empty_like(x["v"], dtype=torch.float32)
    st.linear_prefill(t, x["q"], x["k"], x["v"], x["decay"], S0=x["S0"], out=o)   # the binding's own workspace
    near(o, want, "own workspace")


@pytest.mark.parametrize("n,h,hk,d,t,dtype", [
    (10, 10, 5, 128, 19, "f32"), (23, 10, 10, 128, 5, "f32"), (15, 10, 2, 128, 37, "f32"), (4, 10, 10, 128, 40, "f32"),
    (2, 12, 12, 128, 70, "f32"), (7, 11, 11, 64, 33, "f32"), (8, 2, 1, 128, 700, "f32"), (5, 8, 8, 128, 515, "f32"),
    (6, 10, 10, 64, 300, "f32"), (1, 8, 8, 128, 777, "f32"), (10, 14, 7, 64, 256, "f32"), (1, 25, 25, 128, 31, "bf16"),
    (1, 25, 25, 128, 32, "bf16"), (10, 10, 10, 128, 19, "bf16"), (10, 10, 10, 128, 20, "bf16"), (30, 10, 10, 128, 7, "bf16"),
    (30, 10, 10, 128, 8, "bf16"), (1, 12, 12, 128, 96, "bf16"), (1, 12, 12, 128, 97, "bf16"),
    (2, 16, 8, 64, 128, "bf16"), (2, 16, 8, 64, 129, "bf16"), (20, 10, 10, 64, 63, "bf16")])
def test_prefill_on_both_sides_of_each_choice(n, h, hk, d, t, dtype):
    """Head counts and lengths around those that change a prompt's kernel or its
    cut: given, continued and with a bad gate in two heads."""
    x = inputs(11, n, t, h, hk, d, DT[dtype])
    x["decay"][:, t // 3, ::3] = 0
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, DT[dtype])
    near(run_prefill(st, x, S0=x["S0"]), want, "given")
    near(st.dequant(), S, "state")
    st.init(x["S0"])
    near(run_prefill(st, x, cont=True), want, "continued")
    near(st.dequant(), S, "continued state")
    assert st.check() == 0
    for row, head, at in ((0, 0, t - 1), (n - 1, h - 1, t // 2)):
        x["decay"][row, at, head] = -1.0
        early, Se = reference({k: v[row:row + 1, :at] if k != "S0" else v for k, v in x.items()}, x["S0"][row:row + 1])
        want[row, :, head] = 0
        want[row, :at, head] = early[0, :, head]
        S[row, head] = Se[0, head]
    near(run_prefill(st, x, S0=x["S0"]), want, "bad gates")
    near(st.dequant(), S, "state before the bad gates")
    assert st.check() == B().LQ_ERR_RANGE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [40, 1200])
def test_prefill_slots(t, dtype):
    N, h, hk, d = 6, 4, 2, 128
    rows = [4, -1, 0, 6]
    x = inputs(11, len(rows), t, h, hk, d, DT[dtype])
    S0 = inputs(12, N, 1, h, hk, d, DT[dtype])["S0"]
    st = state_of(N, h, d, DT[dtype])
    slots = torch.tensor(rows, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([t, t, t - 9, t], dtype=torch.int32, device="cuda")
    live, at = [0, 2], [4, 0]
    others = [i for i in range(N) if i not in at]
    for cont in (False, True):
        st.init(S0)
        before = st.buf.clone().view(N, -1)
        out = run_prefill(st, x, lengths=lengths, cont=cont, slots=slots)
        want, S = reference({k: v[live] for k, v in x.items()}, S0[at] if cont else None, lengths[live])
        near(out[live], want)
        assert (out[[1, 3]] == 0).all()
        near(st.dequant()[at], S)
        assert torch.equal(st.buf.view(N, -1)[others], before[others])


@pytest.mark.parametrize("t", [0, 5])
def test_prefill_of_no_tokens(t):
    n, h, d = 2, 3, 64
    x = inputs(13, n, t, h, h, d, torch.bfloat16)
    st = state_of(n, h, d, torch.bfloat16)
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    run_prefill(st, x, S0=x["S0"], lengths=zero)
    assert torch.equal(st.dequant(), x["S0"]) and st.check() == 0
    run_prefill(st, x, lengths=zero, cont=True)
    assert torch.equal(st.dequant(), x["S0"])
    run_prefill(st, x, lengths=zero)
    assert (st.dequant() == 0).all() and st.check() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_tokens_equals_one_prompt(d):
    n, h, hk, t = 3, 6, 2, 90
    x = inputs(14, n, t, h, hk, d, torch.bfloat16)
    want, S = reference(x, None)
    st = state_of(n, h, d, torch.bfloat16)
    head = {k: v[:, :77].contiguous() if k != "S0" else v for k, v in x.items()}
    near(run_prefill(st, head), want[:, :77])
    mid = {k: v[:, 77:85].contiguous() if k != "S0" else v for k, v in x.items()}
    near(run_prefill(st, mid, cont=True), want[:, 77:85])
    out = torch.empty(n, h, d, device="cuda")
    for i in range(85, t):
        st.linear_step(*(x[name][:, i].contiguous() for name in ("q", "k", "v", "decay")), out, qk_heads=hk)
        near(out, want[:, i])
    near(st.dequant(), S)


def test_captured_calls_replay_on_another_stream():
    """A prompt cut along time and a token step in one graph, replayed twice;
    two such graphs of different states run side by side."""
    n, h, d, t = 1, 2, 128, 1500
    graphs, states, outs, wants = [], [], [], []
    for i in range(2):
        x = inputs(20 + i, n, t, h, h, d, torch.bfloat16)
        y = inputs(30 + i, n, 1, h, h, d, torch.bfloat16)
        st = state_of(n, h, d, torch.bfloat16)
        o, o1 = torch.empty(n, t, h, d, device="cuda"), torch.empty(n, h, d, device="cuda")

        def calls():
            st.linear_prefill(t, x["q"], x["k"], x["v"], x["decay"], S0=x["S0"], out=o)
            st.linear_step(y["q"][:, 0].contiguous(), y["k"][:, 0].contiguous(), y["v"][:, 0].contiguous(),
                           y["decay"][:, 0].contiguous(), o1)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        both = {k: (torch.cat([x[k], y[k]], 1) if k != "S0" else x[k]) for k in x}
        wants.append(reference(both, x["S0"]))
        graphs.append(g); states.append((st, x, y)); outs.append((o, o1))
    for _ in range(2):
        for o, o1 in outs:
            o.fill_(float("nan")); o1.fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, o1), (st, _, _), (want, S) in zip(outs, states, wants):
            near(o, want[:, :t])
            near(o1, want[:, t])
            near(st.dequant(), S)


def test_call_on_a_given_stream():
    n, h, d, t = 1, 2, 128, 1500
    x = inputs(40, n, t, h, h, d, torch.bfloat16)
    want, S = reference(x, x["S0"])
    st = state_of(n, h, d, torch.bfloat16)
    out = torch.empty(n, t, h, d, device="cuda")
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        out.zero_()
        torch.cuda.synchronize()
        st.linear_prefill(t, x["q"], x["k"], x["v"], x["decay"], S0=x["S0"], out=out, stream=s)
        torch.cuda.synchronize()
        near(out, want)
        near(st.dequant(), S)


@pytest.mark.parametrize("n,h,d,t", [(1, 5, 128, 4000), (1, 8, 64, 3000), (150, 2, 128, 200)])
def test_the_same_inputs_give_the_same_bits(n, h, d, t):
    """Nothing in a prompt depends on which warp or copy comes first."""
    x = inputs(50, n, t, h, h, d, torch.bfloat16)
    st = state_of(n, h, d, torch.bfloat16)
    o = run_prefill(st, x, S0=x["S0"])
    state = st.buf.clone()
    again = torch.empty_like(o)
    for _ in range(40):
        for _ in range(10):
            st.linear_prefill(t, x["q"], x["k"], x["v"], x["decay"], S0=x["S0"], out=again)
        assert torch.equal(again, o) and torch.equal(st.buf, state)


def test_offsets_beyond_32_bits():
    """A state buffer of more than 2^32 bytes, and a prompt whose outputs have
    more than 2^31 elements: the last head and the last tokens are right."""
    b = B()
    n, h, d = 1100, 60, 128
    st = state_of(n, h, d, torch.bfloat16)
    assert st.buf.numel() > 2 ** 32
    st.buf.zero_()
    blobs = st.blobs()
    blobs[:, 12:16].view(torch.int32)[:] = 0x4C515354
    S0 = torch.randn(d, d, device="cuda")
    blobs[-1, 128:128 + 4 * d * d].view(torch.float32).view(d, d).copy_(S0)
    x = inputs(60, n, 1, h, 1, d, torch.bfloat16)["q"]
    y = inputs(61, n, 1, 1, 1, d, torch.bfloat16)
    v = y["v"].expand(n, 1, h, d).contiguous()
    a = torch.full((n, h), 0.5, device="cuda")
    out = torch.empty(n, h, d, device="cuda")
    st.linear_step(x[:, 0].contiguous(), y["k"][:, 0].contiguous(), v[:, 0].contiguous(), a, out, qk_heads=1)
    S = 0.5 * S0.double() + torch.outer(y["k"][-1, 0, 0].double(), v[-1, 0, -1].double())
    near(blobs[-1, 128:128 + 4 * d * d].view(torch.float32).view(d, d), S, "last state")
    near(out[-1, -1], S.T @ x[-1, 0, 0].double(), "last output")
    del st, blobs, v, out, S
    torch.cuda.empty_cache()
    h, t, tail = 16, 2 ** 31 // (16 * 128) + 1000, 7
    x = inputs(62, 1, t, 1, 1, d, torch.bfloat16)
    v = torch.randn(1, t, h, d, device="cuda", dtype=torch.bfloat16)
    a = torch.rand(1, t, h, device="cuda")
    a[:, t - tail] = 0
    out = torch.empty(1, t, h, d, device="cuda")
    assert out.numel() > 2 ** 31
    st = state_of(1, h, d, torch.bfloat16)
    st.linear_prefill(t, x["q"], x["k"], v, a, out=out, qk_heads=1)
    end = dict(q=x["q"][:, -tail:], k=x["k"][:, -tail:], v=v[:, -tail:], decay=a[:, -tail:])
    want, S = reference(end, None)
    near(out[:, -tail:], want, "last tokens")
    near(st.dequant(), S, "last state")
    assert st.check() == b.LQ_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,t", [(1, 64, 40), (2, 128, 150), (60, 128, 70), (130, 128, 33), (1, 128, 700), (1, 64, 700)])
@pytest.mark.parametrize("gate", [0.06, 0.3, 0.9])
def test_large_values_under_strong_gates(n, d, t, gate, dtype):
    """Values of 2^55 stay finite whatever the gates: the state is held over a
    product of gates of 2^-64 or more."""
    x = inputs(72, n, t, 2, 2, d, DT[dtype])
    x["v"] = x["v"] * 2.0 ** 55
    x["S0"] = x["S0"] * 2.0 ** 55
    x["decay"] = gate * x["decay"]
    want, S = reference(x, x["S0"])
    st = state_of(n, 2, d, DT[dtype])
    near(run_prefill(st, x, S0=x["S0"]), want)
    near(st.dequant(), S)
    assert st.check() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [3, 70, 150])
def test_non_finite_rows_stay_in_their_head(t, d, dtype):
    """Infinities and NaN in some heads' q, k or v leave every other head right,
    also where one SM takes them one after the other."""
    n, h = 170, 2
    x = inputs(70, n, t, h, h, d, DT[dtype])
    want, S = reference(x, x["S0"])
    bad = torch.zeros(n, h, dtype=torch.bool, device="cuda")
    for i, (row, head, name, value) in enumerate([(0, 0, "v", float("nan")), (3, 1, "k", float("inf")), (90, 0, "q", float("-inf")),
                                                  (150, 1, "v", float("inf")), (169, 0, "k", float("nan"))]):
        x[name][row, min(i, t - 1), head, 5] = value
        bad[row, head] = True
    st = state_of(n, h, d, DT[dtype])
    for S0 in (x["S0"], None):
        if S0 is None:
            want, S = reference({k: v[~bad.any(1)] for k, v in x.items()}, None)
            out = run_prefill(st, x)
            near(out[~bad.any(1)], want)
            near(st.dequant()[~bad.any(1)], S)
        else:
            out = run_prefill(st, x, S0=S0)
            good = ~bad
            near(out.transpose(1, 2)[good], want.transpose(1, 2)[good])
            near(st.dequant()[good], S[good])
    assert st.check() == 0


def test_a_state_on_a_given_buffer():
    b = B()
    cfg = b.make_config(2, 3, 64, 64, bits=32)
    buf = torch.zeros(2 * 3 * b.lq_state_bytes(cfg) + 256, dtype=torch.uint8, device="cuda")
    st = b.LQState(cfg, buf=buf)
    x = inputs(71, 2, 1, 3, 3, 64, torch.bfloat16)
    st.init(x["S0"])
    assert st.ptr == buf.data_ptr() and torch.equal(st.dequant(), x["S0"])
    short = b.LQState(cfg, buf=buf[:1024])
    with pytest.raises(ValueError, match="state"):
        short.init(x["S0"])
