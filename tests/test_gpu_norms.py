"""The norms and gates around the recurrence against the same formulas in 64
bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # one FP32 rounding
HALF = {"bf16": 2.0 ** -8, "f32": U}   # one rounding to the output's type
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()


def B():
    from linear_attention_recurrent_lq_b200 import binding
    return binding


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def within(got, want, tol, what):
    bad = (got.double() - want).abs() > tol
    assert not bad.any() and torch.isfinite(got).all(), f"{what}: {int(bad.sum())} values off"


def run_qk(cfg, m, h, hk, d, dtype, kda, seed=0, scale=0.125, eps=1e-6, alias=False, magnitude=1.0):
    b, dt, ch = B(), DT[dtype], ((d,) if kda else ())
    q, k = (magnitude * randn(seed, m, hk, d)).to(dt), (magnitude * randn(seed + 1, m, hk, d)).to(dt)
    a, bb = (3 * randn(seed + 2, m, h, *ch)).to(dt), (3 * randn(seed + 3, m, h)).to(dt)
    a_log, dt_bias = randn(seed + 4, h), randn(seed + 5, h, *ch) - 2
    if m > 1:
        q[m // 2] = 0                       # a zero row stays zero
        a.view(-1)[:4] = torch.tensor([80.0, -80.0, 20.0, -20.0], device="cuda")
        bb.view(-1)[:2] = torch.tensor([90.0, -90.0], device="cuda")
    q0, k0 = q.clone(), k.clone()
    qo, ko = (q, k) if alias else (torch.empty_like(q), torch.empty_like(k))
    decay, beta = torch.empty(m, h, *ch, device="cuda"), torch.empty(m, h, device="cuda")
    b.lq_qk_norm(cfg, q, k, a, bb, a_log, dt_bias, qo, ko, decay, beta, q_scale=scale, eps=eps, qk_heads=hk)
    # a sum of d squares, a root and a quotient: d + 4 roundings of the sum count half
    rel = HALF[dtype] + (d / 2 + 6) * U
    for got, x, s, name in ((qo, q0, scale, "q"), (ko, k0, 1.0, "k")):
        x = x.double()
        want = s * x / (x.square().sum(-1, keepdim=True) + eps).sqrt()
        within(got, want, rel * want.abs(), name)
    z = a.double() + dt_bias.double()
    soft = torch.logaddexp(z, torch.zeros_like(z))
    x = a_log.double().exp().view(-1, *[1] * len(ch)) * soft
    # exponent: its two factors by library functions within 2 units each, a
    # product, and the sum a + dt_bias whose rounding moves softplus by up to |z| units
    want = torch.exp(-x)
    within(decay, want, want * U * ((14 + 2 * z.abs()) * x + 6) + 2.0 ** -125, "decay")
    want = torch.sigmoid(bb.double())
    within(beta, want, 8 * U * want + 2.0 ** -125, "beta")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("m,h,hk,d", [(1, 1, 1, 128), (1, 4, 2, 64), (7, 6, 3, 128), (64, 32, 32, 128), (333, 12, 4, 64),
                                      (1000, 9, 9, 128)])
def test_qk_norm(m, h, hk, d, kda, dtype):
    b = B()
    cfg = b.make_config(1, h, d, d, bits=8, in_dtype=dtype, decay_kind="kda" if kda else "gdn")
    run_qk(cfg, m, h, hk, d, dtype, kda)
    run_qk(cfg, m, h, hk, d, dtype, kda, alias=True, magnitude=1e-3, seed=9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("m,h,d", [(1, 1, 64), (1, 3, 128), (31, 5, 128), (257, 12, 64)])
def test_out_norm(m, h, d, weight, gate, dtype):
    b = B()
    cfg = b.make_config(1, h, d, d, bits=32, in_dtype=dtype)
    o = randn(1, m, h, d)
    o[0] *= 1e-4
    o[-1, -1] = 0
    w = 1 + 0.1 * randn(2, d) if weight else None
    g = None if gate == "none" else (3 * randn(3, m, h, d)).to(DT[dtype])
    if g is not None:
        g.view(-1)[:2] = torch.tensor([95.0, -95.0], device="cuda")
    y = torch.empty(m, h, d, dtype=DT[dtype], device="cuda")
    b.lq_out_norm(cfg, o, y, weight=w, gate=g, gate_kind=gate, eps=1e-6)
    x = o.double()
    want = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    if weight:
        want = want * w.double()
    if g is not None:
        want = want * torch.sigmoid(g.double()) * (g.double() if gate == "silu" else 1)
    within(y, want, (HALF[dtype] + (d / 2 + 16) * U) * want.abs() + 2.0 ** -125, "y")


def test_rows_of_every_leading_shape_and_none():
    b = B()
    cfg = b.make_config(2, 4, 64, 64, bits=32)
    o = randn(5, 2, 3, 4, 64)
    y = torch.full((2, 3, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    b.lq_out_norm(cfg, o, y)
    flat = torch.empty(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    b.lq_out_norm(cfg, o.view(6, 4, 64), flat)
    assert torch.equal(y.view(6, 4, 64), flat)
    b.lq_out_norm(cfg, o[:0], y[:0])


def test_a_layer_from_raw_projections():
    """Norms and gates, a prompt, tokens and the output norm in a row, on the
    linear-attention calls and on the delta-rule calls, against 64 bits."""
    b = B()
    n, h, d, t = 2, 4, 128, 70
    raw = [randn(50 + i, n, t + 2, h, d).bfloat16() for i in range(4)]
    q, k, v, gate = raw
    a, bb = randn(60, n, t + 2, h).bfloat16(), randn(61, n, t + 2, h).bfloat16()
    a_log, dt_bias, w = randn(62, h).abs(), randn(63, h) - 4, 1 + 0.1 * randn(64, d)
    for delta in (False, True):
        cfg = b.make_config(n, h, d, d, bits=32, window=16)
        qn, kn = torch.empty_like(q), torch.empty_like(k)
        decay, beta = torch.empty(n, t + 2, h, device="cuda"), torch.empty(n, t + 2, h, device="cuda")
        b.lq_qk_norm(cfg, q, k, a, bb, a_log, dt_bias, qn, kn, decay, beta, q_scale=d ** -0.5)
        o = torch.empty(n, t + 2, h, d, device="cuda")
        st = b.LQState(cfg)
        head = [x[:, :t].contiguous() for x in (qn, kn, v, decay)]
        if delta:
            st.init(torch.zeros(n, h, d, d, device="cuda"))
            for i in range(t + 2):
                row = torch.empty(n, h, d, device="cuda")
                st.step(*(x[:, i].contiguous() for x in (qn, kn, v, beta, decay)), row)
                o[:, i] = row
        else:
            oh = torch.empty(n, t, h, d, device="cuda")
            st.linear_prefill(t, *head, out=oh)
            o[:, :t] = oh
            for i in (t, t + 1):
                row = torch.empty(n, h, d, device="cuda")
                st.linear_step(*(x[:, i].contiguous() for x in (qn, kn, v, decay)), row)
                o[:, i] = row
        y = torch.empty_like(q)
        b.lq_out_norm(cfg, o, y, weight=w, gate=gate, gate_kind="silu")
        # 64 bits from the normalised rows the kernel gave (they were checked above)
        S = torch.zeros(n, h, d, d, dtype=torch.float64, device="cuda")
        want = torch.empty(n, t + 2, h, d, dtype=torch.float64, device="cuda")
        for i in range(t + 2):
            S = S * decay[:, i, :, None, None].double()
            ki, vi = kn[:, i].double(), v[:, i].double()
            u = beta[:, i, :, None].double() * (vi - torch.einsum("nhi,nhij->nhj", ki, S)) if delta else vi
            S = S + ki[..., None] * u[..., None, :]
            want[:, i] = torch.einsum("nhi,nhij->nhj", qn[:, i].double(), S)
        want = want / (want.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        g = gate.double()
        want = want * g * torch.sigmoid(g)
        err = (y.double() - want).norm() / want.norm()
        assert err < 2.0 ** -8, f"delta {delta}: {err:.2e}"
