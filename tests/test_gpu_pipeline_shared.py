"""A captured layer that is given to a second host pipeline goes on giving the
bits of the plain calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_two_pipelines_over_one_captured_layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()
    from linear_attention_recurrent_lq_b200 import binding as B
    from linear_attention_recurrent_lq_b200.pipeline import HostIOPipeline, Layer, Projections
    N, H, d, W = 3, 4, 128, 4
    g = torch.Generator().manual_seed(3)

    def rand(*s):
        return torch.randn(s, generator=g)

    cfg = B.make_config(N, H, d, d, window=W, bits=32)
    shapes = dict(q=(W, N, H, d), k=(W, N, H, d), v=(W, N, H, d), a=(W, N, H), b=(W, N, H))
    host = {n: rand(*s).bfloat16().pin_memory() for n, s in shapes.items()}
    p = Projections(rand(H).abs().cuda(), (rand(H) - 3).cuda(), None, "none", d ** -0.5, linear=True)
    S0 = rand(N, H, d, d).cuda()
    st, ref = B.LQState(cfg), B.LQState(cfg)
    out = torch.empty(W, N, H, d, dtype=torch.bfloat16, device="cuda")
    lay = Layer(st, {n: h.cuda() for n, h in host.items()}, out, host, torch.empty(out.shape, dtype=out.dtype).pin_memory(), proj=p)
    first = HostIOPipeline([lay], W)
    st.init(S0)
    first.capture()
    second = HostIOPipeline([lay], W)
    # memory that a replaced scratch would have left to others
    others = [torch.full((W, N, H, d), 3.0, device="cuda") for _ in range(64)]
    ref.init(S0)
    st.buf.copy_(ref.buf)
    torch.cuda.synchronize()
    x = lay.dev_in
    q, k = torch.empty_like(x["q"]), torch.empty_like(x["k"])
    decay, beta, rows = (torch.empty(s, device="cuda") for s in ((W, N, H), (W, N, H), (W, N, H, d)))
    y = torch.empty_like(out)
    for pipe in (first, second, first):
        pipe.fork()
        pipe.step()
        pipe.join()
        B.lq_qk_norm(cfg, x["q"], x["k"], x["a"], x["b"], p.a_log, p.dt_bias, q, k, decay, beta, q_scale=p.q_scale)
        for t in range(W):
            ref.linear_step(q[t], k[t], x["v"][t], decay[t], rows[t])
        B.lq_out_norm(cfg, rows, y)
        torch.cuda.synchronize()
        assert torch.equal(lay.host_out, y.cpu()) and torch.equal(st.buf, ref.buf)
        assert all((o == 3.0).all() for o in others)
