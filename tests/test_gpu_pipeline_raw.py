"""The host-I/O pipeline on raw projections: norms and gates, a window of
tokens and the output norm give, step after step, the bits of the plain calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrent_lq_b200 import build
    build.build()


@pytest.mark.parametrize("kind,bits,linear,gate", [("gdn", 8, False, "silu"), ("kda", 8, False, "none"),
                                                   ("gdn", 32, True, "sigmoid")])
def test_pipeline_on_raw_projections_equals_plain_calls(kind, bits, linear, gate):
    from linear_attention_recurrent_lq_b200 import binding as B
    from linear_attention_recurrent_lq_b200.pipeline import HostIOPipeline, Layer, Projections
    N, H, d, W, steps = 3, 4, 128, 4, 3
    hk = 2 if linear else H
    g = torch.Generator().manual_seed(1)
    cfg = B.make_config(N, H, d, d, window=W, bits=bits, decay_kind=kind)
    ch = (d,) if kind == "kda" else ()
    shapes = dict(q=(W, N, hk, d), k=(W, N, hk, d), v=(W, N, H, d), a=(W, N, H, *ch), b=(W, N, H))
    if gate != "none":
        shapes["gate"] = (W, N, H, d)

    def rand(*s):
        return torch.randn(s, generator=g)

    layers, plain = [], []
    for _ in range(2):
        host = {n: rand(*s).bfloat16().pin_memory() for n, s in shapes.items()}
        p = Projections(rand(H).abs().cuda(), (rand(H, *ch) - 3).cuda(), (1 + 0.1 * rand(d)).cuda(), gate, d ** -0.5,
                        linear=linear)
        st, ref = B.LQState(cfg), B.LQState(cfg)
        S0 = rand(N, H, d, d).cuda()
        for s in (st, ref):
            s.buf.zero_()
            s.init(S0)
        out = torch.empty(W, N, H, d, dtype=torch.bfloat16, device="cuda")
        layers.append(Layer(st, {n: h.cuda() for n, h in host.items()}, out, host,
                            torch.empty(out.shape, dtype=out.dtype).pin_memory(), proj=p))
        plain.append(ref)
    pipe = HostIOPipeline(layers, W)
    snap = [lay.state.buf.clone() for lay in layers]
    pipe.capture()
    for lay, s0 in zip(layers, snap):
        lay.state.buf.copy_(s0)
    torch.cuda.synchronize()
    assert pipe.bytes_per_step()[1] == 2 * W * N * H * d * 2
    for _ in range(steps):
        pipe.fork()
        pipe.step()
        pipe.join()
        torch.cuda.synchronize()
        for lay, ref in zip(layers, plain):
            x, p = {n: h.cuda() for n, h in lay.host_in.items()}, lay.proj
            q, k = torch.empty_like(x["q"]), torch.empty_like(x["k"])
            decay, beta = torch.empty(W, N, H, *ch, device="cuda"), torch.empty(W, N, H, device="cuda")
            B.lq_qk_norm(cfg, x["q"], x["k"], x["a"], x["b"], p.a_log, p.dt_bias, q, k, decay, beta,
                         q_scale=p.q_scale, qk_heads=hk)
            rows = torch.empty(W, N, H, d, device="cuda")
            for t in range(W):
                if linear:
                    ref.linear_step(q[t], k[t], x["v"][t], decay[t], rows[t], qk_heads=hk)
                else:
                    ref.step(q[t], k[t], x["v"][t], beta[t], decay[t], rows[t])
            ref.flush()
            y = torch.empty(W, N, H, d, dtype=torch.bfloat16, device="cuda")
            B.lq_out_norm(cfg, rows, y, weight=p.weight, gate=x.get("gate"), gate_kind=gate)
            torch.cuda.synchronize()
            assert torch.equal(lay.host_out, y.cpu())
            assert torch.equal(lay.state.buf, ref.buf) and lay.state.check() == 0
            for n, h in lay.host_in.items():   # the next step's projections
                h.copy_(rand(*h.shape).bfloat16())
