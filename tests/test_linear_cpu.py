"""Host-side checks of the linear-attention and norm entry points that need no
GPU: bad arguments are refused before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from linear_attention_recurrent_lq_b200 import build
    build.build()
    from linear_attention_recurrent_lq_b200 import binding
    return binding


def cfg_of(B, **over):
    return B.make_config(**{**dict(num_slots=4, num_heads=4, bits=32), **over})


def test_step_arguments_rejected_before_launch(B):
    L, c = B.lib, ctypes.byref(cfg_of(B))
    assert L.lq_linear_step(None, 256, 4, 16, 16, 16, 16, 16, None) == 1
    assert L.lq_linear_step(c, None, 4, 16, 16, 16, 16, 16, None) == 1
    for hk in (0, -1, 3, 8):                       # H % Hk != 0
        assert L.lq_linear_step(c, 256, hk, 16, 16, 16, 16, 16, None) == 1
    for at in range(5):                            # q, k, v, decay, out
        p = [16] * 5
        p[at] = None
        assert L.lq_linear_step(c, 256, 4, *p, None) == 1
        p[at] = 2 if at == 3 else 8
        assert L.lq_linear_step(c, 256, 4, *p, None) == 6
    assert L.lq_linear_step(c, 128, 4, 16, 16, 16, 16, 16, None) == 6
    for other in (dict(bits=8), dict(bits=8, per_step=True), dict(decay_kind="kda")):
        assert L.lq_linear_step(ctypes.byref(cfg_of(B, **other)), 256, 4, 16, 16, 16, 16, 16, None) == 2


def test_step_slots_arguments_rejected_before_launch(B):
    L, c = B.lib, ctypes.byref(cfg_of(B))
    assert L.lq_linear_step_slots(c, 256, None, 0, 4, None, None, None, None, None, None) == 0
    assert L.lq_linear_step_slots(c, 256, None, 2, 4, 16, 16, 16, 16, 16, None) == 1
    assert L.lq_linear_step_slots(c, 256, 64, -1, 4, 16, 16, 16, 16, 16, None) == 1
    assert L.lq_linear_step_slots(c, 256, 66, 2, 4, 16, 16, 16, 16, 16, None) == 6
    assert L.lq_linear_step_slots(c, 256, 64, 0x7FFFFFFF, 4, 16, 16, 16, 16, 16, None) == 2


def test_prefill_arguments_rejected_before_launch(B):
    L, cfg = B.lib, cfg_of(B)
    c = ctypes.byref(cfg)

    def call(c=c, state=256, tokens=4, lengths=None, S0=None, hk=4, inp=(16, 16, 16, 16), out=None, flags=0, ws=None,
             n=0):
        return L.lq_linear_prefill(c, state, tokens, lengths, S0, hk, *inp, out, flags, ws, n, None)

    assert call(tokens=-1) == 1
    assert call(state=None) == 1
    assert call(hk=3) == 1
    assert call(flags=2) == 1                      # unknown flag
    assert call(flags=1, S0=16) == 1               # go on from the blobs, or from S0
    for at in range(4):
        assert call(inp=[None if i == at else 16 for i in range(4)]) == 1
        assert call(inp=[(2 if at == 3 else 8) if i == at else 16 for i in range(4)]) == 6
    assert call(state=128) == 6
    assert call(lengths=2) == 6
    assert call(S0=8) == 6
    assert call(out=8) == 6
    assert call(ws=8) == 6
    assert call(tokens=0x7FFFFFFF) == 2
    need = B.lq_linear_prefill_workspace(cfg, 4, 4096)
    assert need > 0
    assert call(tokens=4096, ws=256, n=need - 1) == 1
    for other in (dict(bits=4), dict(bits=16, per_step=True), dict(decay_kind="kda")):
        assert call(c=ctypes.byref(cfg_of(B, **other))) == 2
    assert L.lq_linear_prefill_slots(c, 256, 64, 0, 4, None, None, 4, None, None, None, None, None, 0, None, 0, None) == 0
    assert L.lq_linear_prefill_slots(c, 256, None, 2, 4, None, None, 4, 16, 16, 16, 16, None, 0, None, 0, None) == 1


def test_workspace_is_asked_for_where_heads_are_few(B):
    one = cfg_of(B, num_slots=1)
    assert B.lq_linear_prefill_workspace(one, 1, 1) == 0
    assert B.lq_linear_prefill_workspace(one, 1, 0) == 0
    assert B.lq_linear_prefill_workspace(one, 0, 4096) == 0
    long = B.lq_linear_prefill_workspace(one, 1, 16384)
    assert long > 0 and long % 4 == 0
    assert B.lq_linear_prefill_workspace(cfg_of(B, num_slots=1, dk=64, dv=64), 1, 16384) < long
    assert B.lq_linear_prefill_workspace(cfg_of(B, num_slots=512), 512, 16384) == 0
    assert B.lq_linear_prefill_workspace(cfg_of(B, bits=8), 1, 16384) == 0


def test_norm_arguments_rejected_before_launch(B):
    L = B.lib
    for kind in ("gdn", "kda"):
        c = ctypes.byref(cfg_of(B, decay_kind=kind, bits=8))

        def call(rows=2, hk=4, eps=1e-6, **over):
            p = dict.fromkeys(("q", "k", "a", "b", "a_log", "dt_bias", "q_out", "k_out", "decay", "beta"), 16)
            p.update(over)
            return L.lq_qk_norm(c, rows, hk, p["q"], p["k"], p["a"], p["b"], p["a_log"], p["dt_bias"], 1.0, eps,
                                p["q_out"], p["k_out"], p["decay"], p["beta"], None)

        assert call(rows=-1) == 1
        assert call(hk=3) == 1
        assert call(eps=-1.0) == 1
        assert call(eps=float("nan")) == 1
        assert call(rows=0, q=None) == 0
        for name in ("q", "k", "a", "b", "a_log", "dt_bias", "q_out", "k_out", "decay", "beta"):
            assert call(**{name: None}) == 1
            assert call(**{name: 1}) == 6
        for name in ("q", "k", "q_out", "k_out"):
            assert call(**{name: 8}) == 6
        for name in ("a", "dt_bias", "decay") if kind == "kda" else ():
            assert call(**{name: 8}) == 6
        assert call(rows=0x7FFFFFFF) == 2
    c = ctypes.byref(cfg_of(B, bits=8))
    assert L.lq_out_norm(c, -1, 16, None, None, 0, 1e-6, 16, None) == 1
    assert L.lq_out_norm(c, 2, None, None, None, 0, 1e-6, 16, None) == 1
    assert L.lq_out_norm(c, 2, 16, None, None, 0, 1e-6, None, None) == 1
    assert L.lq_out_norm(c, 2, 16, None, 16, 0, 1e-6, 16, None) == 1     # a gate that is not used
    assert L.lq_out_norm(c, 2, 16, None, None, 1, 1e-6, 16, None) == 1   # no gate to use
    assert L.lq_out_norm(c, 2, 16, None, 16, 3, 1e-6, 16, None) == 1
    assert L.lq_out_norm(c, 2, 16, None, None, 0, -1.0, 16, None) == 1
    assert L.lq_out_norm(c, 2, 8, None, None, 0, 1e-6, 16, None) == 6
    assert L.lq_out_norm(c, 2, 16, 8, None, 0, 1e-6, 16, None) == 6
    assert L.lq_out_norm(c, 2, 16, None, 8, 1, 1e-6, 16, None) == 6
    assert L.lq_out_norm(c, 0, None, None, None, 0, 1e-6, None, None) == 0


def test_binding_checks_tensors_before_any_call(B, monkeypatch):
    torch = pytest.importorskip("torch")
    calls, real = [], B.lib

    class Spy:
        def __getattr__(self, name):
            if name in ("lq_state_bytes", "lq_linear_prefill_workspace"):
                return getattr(real, name)
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(B, "lib", Spy())
    N, H, Hk, d, T = 2, 6, 2, 64, 3
    cfg = B.make_config(N, H, d, d, bits=32)
    state = torch.zeros(N * H * B.lq_state_bytes(cfg), dtype=torch.uint8)
    bf, f = torch.bfloat16, torch.float32
    good = dict(q=torch.zeros(N, T, Hk, d, dtype=bf), k=torch.zeros(N, T, Hk, d, dtype=bf),
                v=torch.zeros(N, T, H, d, dtype=bf), decay=torch.zeros(N, T, H), out=torch.zeros(N, T, H, d))

    def prefill(hk=Hk, S0=None, lengths=None, workspace=None, **over):
        a = {**good, **over}
        B.lq_linear_prefill(cfg, state, T, a["q"], a["k"], a["v"], a["decay"], S0=S0, lengths=lengths, out=a["out"],
                            qk_heads=hk, workspace=workspace, stream=0)

    for why, over in [("q: 768 elements", dict(hk=H)), ("dtype", dict(v=good["v"].float())),
                      ("elements", dict(decay=torch.zeros(N, T, H, d))), ("out", dict(out=torch.zeros(N, T, H, d + 1))),
                      ("S0", dict(S0=torch.zeros(N, H, d, d - 1))), ("lengths", dict(lengths=torch.zeros(N, dtype=torch.int64))),
                      ("workspace", dict(workspace=torch.zeros(8))), ("CUDA tensor", {})]:
        with pytest.raises(ValueError, match=why):
            prefill(**over)
    with pytest.raises(ValueError, match="contiguous|CUDA"):
        prefill(q=good["q"].transpose(0, 1))
    with pytest.raises(ValueError, match="q"):
        B.lq_linear_step(cfg, state, good["q"], good["k"], good["v"], good["decay"], good["out"], Hk, stream=0)
    with pytest.raises(ValueError, match="slots"):
        B.lq_linear_step_slots(cfg, state, torch.zeros(1, dtype=torch.int64), good["q"], good["k"], good["v"],
                               good["decay"], good["out"], Hk, stream=0)
    with pytest.raises(ValueError, match="multiple"):
        B.lq_qk_norm(cfg, torch.zeros(d + 1, dtype=bf), *[None] * 9, qk_heads=Hk, stream=0)
    with pytest.raises(ValueError, match="rows is needed"):
        B.lq_out_norm(cfg, 256, 256, stream=0)
    with pytest.raises(ValueError, match="gate_kind"):
        B.lq_out_norm(cfg, torch.zeros(N, H, d), torch.zeros(N, H, d, dtype=bf), gate_kind="relu", stream=0)
    with pytest.raises(ValueError, match="weight"):
        B.lq_out_norm(cfg, torch.zeros(N, H, d), torch.zeros(N, H, d, dtype=bf), weight=torch.zeros(d + 1), stream=0)
    assert calls == []
    B.lq_out_norm(cfg, 256, 512, rows=2, stream=0)
    B.lq_linear_step(cfg, 256, 256, 256, 256, 256, 256, stream=0)
    assert calls == ["lq_out_norm", "lq_linear_step"]
