"""Cases for timing the linear-attention operators beside the delta-rule calls.

Four operators of one layer: ``step`` (one token of linear attention with a
decay per head), ``prefill`` (a prompt of it), ``qk_norm`` (what comes before
the recurrence: normalised queries and keys, gates from logits) and
``out_norm`` (what comes after it: the head's norm and output gate).

A case is a dict of plain values; ``run`` makes one pass, through the library
where ``own`` is true and in elementary torch operations otherwise.
"""
import math

import torch

own = False

_HEADER = 128  # bytes of a dense state blob before its matrix


def listed():
    return [
        # one conversation, one token: launch latency and a 4 MB state
        dict(name="step 1x32", op="step", n=1, h=32, hk=32, d=128, dtype="bf16", slots=False),
        # a layer of a 64-sequence decode batch
        dict(name="step 64x32", op="step", n=64, h=32, hk=32, d=128, dtype="bf16", slots=False),
        # continuous batching: three quarters of 512 slots run, in any order
        dict(name="step 512x36 slots", op="step", n=512, h=36, hk=36, d=128, dtype="bf16", slots=True),
        # narrow heads, q and k shared by three value heads, f32 inputs
        dict(name="step 200x12 shared f32", op="step", n=200, h=12, hk=4, d=64, dtype="f32", slots=False),
        # a chat turn's few tokens appended to a running state
        dict(name="prefill 1x12x17 continued", op="prefill", n=1, h=12, hk=12, d=128, t=17, dtype="bf16", lengths=False, start="continue", resets=False),
        # a batch of ordinary prompts
        dict(name="prefill 64x32x256", op="prefill", n=64, h=32, hk=32, d=128, t=256, dtype="bf16", lengths=False, start="zero", resets=False),
        # one long document: few heads, many tokens
        dict(name="prefill 1x32x16384", op="prefill", n=1, h=32, hk=32, d=128, t=16384, dtype="bf16", lengths=False, start="zero", resets=False),
        # padded batch of unequal prompts with packed documents (a gate of 0
        # starts each), q and k shared by three heads, from a given state
        dict(name="prefill 9x36x1000 ragged", op="prefill", n=9, h=36, hk=12, d=128, t=1000, dtype="bf16", lengths=True, start="given", resets=True),
        # narrow heads in f32, a length that fits no tile
        dict(name="prefill 3x12x777 f32", op="prefill", n=3, h=12, hk=12, d=64, t=777, dtype="f32", lengths=False, start="zero", resets=False),
        # the projections of a 64-sequence decode batch, before the recurrence
        dict(name="qk_norm 64x32", op="qk_norm", m=64, h=32, hk=32, d=128, dtype="bf16", kda=False),
        # the same for a batch of prompts with a gate per key channel
        dict(name="qk_norm 16384x12 channels", op="qk_norm", m=16384, h=12, hk=12, d=128, dtype="bf16", kda=True),
        # a batch of prompts after the recurrence
        dict(name="out_norm 16384x32", op="out_norm", m=16384, h=32, d=128, dtype="bf16", gate="silu", weight=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "prefill", "qk_norm", "out_norm"])
    h = rng.choice([1, 3, 4, 8, 12, 16, 24, 32, 36, 48])
    hk = rng.choice([x for x in (1, 2, 3, 4, 6, 8, 12, 16, 18, 24, 32, 36, 48) if h % x == 0 and 4 * x >= h])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        n = _log_int(rng, 1, 512)
        return dict(op=op, n=min(n, 13824 // h), h=h, hk=hk, d=d, dtype=dtype, slots=rng.random() < 0.5)
    if op == "prefill":
        t = _log_int(rng, 1, 16384)
        n = min(_log_int(rng, 1, 64), max(1, 262144 // (t * h)))
        h, hk = (h, hk) if n * t * h <= 524288 else (16, 16)
        return dict(op=op, n=n, h=h, hk=hk, d=d, t=t, dtype=dtype, lengths=rng.random() < 0.5,
                    start=rng.choice(["zero", "given", "continue"]), resets=rng.random() < 0.3)
    m = min(_log_int(rng, 1, 16384), 16384 * 12 // h)
    if op == "qk_norm":
        return dict(op=op, m=m, h=h, hk=hk, d=d, dtype=dtype, kda=rng.random() < 0.4)
    return dict(op=op, m=m, h=h, d=d, dtype=dtype, gate=rng.choice(["silu", "sigmoid", "none"]), weight=rng.random() < 0.8)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _unit(g, shape, dtype):
    """Normalised rows, as queries and keys reach the recurrence."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _blobs(case, n):
    """The state buffer of n sequences: a 128-byte header and the FP32 matrix,
    rounded up to 256 bytes, for each head."""
    size = (_HEADER + 4 * case["d"] ** 2 + 255) // 256 * 256
    buf = torch.zeros(n * case["h"], size, dtype=torch.uint8, device="cuda")
    head = buf[:, :_HEADER].view(torch.int32)
    head[:, 3] = 0x4C515354  # the header's magic
    head[:, 4] = 0x3F800000  # 1.0
    return buf


def _matrix(buf, d):
    return buf[:, _HEADER:_HEADER + 4 * d * d].view(torch.float32).view(-1, d, d)


def _config(case, n):
    from linear_attention_recurrent_lq_b200 import binding as B
    if case["op"] in ("step", "prefill"):
        return B.make_config(n, case["h"], case["d"], case["d"], bits=32, in_dtype=case["dtype"])
    return B.make_config(1, case["h"], case["d"], case["d"], in_dtype=case["dtype"], decay_kind="kda" if case.get("kda") else "gdn")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, h, d = _dtype(case), case["h"], case["d"]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def gates(*shape):
        return torch.exp(-torch.nn.functional.softplus(randn(*shape) - 4))

    if case["op"] in ("step", "prefill"):
        n, hk = case["n"], case["hk"]
        s["buf"] = _blobs(case, n)
        rows, tokens = n, (case["t"],) if case["op"] == "prefill" else ()
        if case.get("slots"):
            rows = max(1, 3 * n // 4)
            s["slots"] = torch.randperm(n, generator=g, device="cuda")[:rows].to(torch.int32)
        if case["op"] == "step" or case["start"] == "continue":
            _matrix(s["buf"], d).normal_(0, 0.1, generator=g)
        if case.get("start") == "given":
            s["S0"] = 0.1 * randn(n, h, d, d)
        s["q"] = _unit(g, (rows, *tokens, hk, d), dt)
        s["k"] = _unit(g, (rows, *tokens, hk, d), dt)
        s["v"] = randn(rows, *tokens, h, d).to(dt)
        s["decay"] = gates(rows, *tokens, h)
        if case.get("resets"):
            s["decay"].masked_fill_(torch.rand((rows, *tokens, 1), generator=g, device="cuda") < 0.005, 0.0)
        if case.get("lengths"):
            s["lengths"] = torch.randint(0, case["t"] + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty(s["v"].shape, dtype=torch.float32, device="cuda")
        rows_of = s["slots"].long() if "slots" in s else None
        s["heads"] = None if rows_of is None else (rows_of[:, None] * h + torch.arange(h, device="cuda")).view(-1)
    elif case["op"] == "qk_norm":
        m, hk = case["m"], case["hk"]
        s["q"], s["k"] = randn(m, hk, d).to(dt), randn(m, hk, d).to(dt)
        channels = (d,) if case["kda"] else ()
        s["a"], s["b"] = randn(m, h, *channels).to(dt), randn(m, h).to(dt)
        s["a_log"] = torch.log(1 + 15 * torch.rand(h, generator=g, device="cuda"))
        s["dt_bias"] = randn(h, *channels) - 4
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["decay"] = torch.empty(s["a"].shape, device="cuda")
        s["beta"] = torch.empty(s["b"].shape, device="cuda")
    else:
        m = case["m"]
        s["o"] = randn(m, h, d)
        s["weight"] = 1 + 0.1 * randn(d) if case["weight"] else None
        s["gate"] = None if case["gate"] == "none" else randn(m, h, d).to(dt)
        s["y"] = torch.empty(m, h, d, dtype=dt, device="cuda")
    return s


_EPS = 1e-6


def run(s):
    case = s["case"]
    return {"step": _step, "prefill": _prefill, "qk_norm": _qk_norm, "out_norm": _out_norm}[case["op"]](s, case)


def _state(s, case):
    from linear_attention_recurrent_lq_b200 import binding as B
    if "state" not in s:
        s["state"] = B.LQState(_config(case, case["n"]), buf=s["buf"].view(-1))
    return s["state"]


def _spread(x, h):
    """Queries or keys of the head each of the h value heads reads."""
    return x.float().repeat_interleave(h // x.shape[-2], dim=-2)


def _step(s, case):
    d = case["d"]
    S = _matrix(s["buf"], d)
    if own:
        st = _state(s, case)
        if "slots" in s:
            st.linear_step_slots(s["slots"], s["q"], s["k"], s["v"], s["decay"], s["out"], qk_heads=case["hk"])
        else:
            st.linear_step(s["q"], s["k"], s["v"], s["decay"], s["out"], qk_heads=case["hk"])
        return s["out"], S
    q, k = (_spread(s[x], case["h"]).view(-1, d, 1) for x in ("q", "k"))
    v = s["v"].float().view(-1, 1, d)
    a = s["decay"].view(-1, 1, 1)
    if s["heads"] is None:
        S.mul_(a).add_(k * v)
        new = S
    else:
        new = S[s["heads"]].mul_(a).add_(k * v)
        S[s["heads"]] = new
    return (new * q).sum(1).view(s["out"].shape), S


def _prefill(s, case):
    d = case["d"]
    if own:
        st = _state(s, case)
        st.linear_prefill(case["t"], s["q"], s["k"], s["v"], s["decay"], S0=s.get("S0"), lengths=s.get("lengths"),
                          out=s["out"], qk_heads=case["hk"], cont=case["start"] == "continue")
        return s["out"], _matrix(s["buf"], d)
    n, t, h = s["v"].shape[:3]
    c = 64
    pieces = (t + c - 1) // c
    pad = pieces * c - t

    def split(x):  # [n, t, h, ...] -> [n, h, pieces, c, ...]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)) if pad else x
        return x.view(n, pieces, c, h, -1).permute(0, 3, 1, 2, 4)

    live = torch.ones(n, t, 1, 1, dtype=torch.bool, device="cuda")
    if "lengths" in s:
        live = (torch.arange(t, device="cuda") < s["lengths"][:, None]).view(n, t, 1, 1)
    q = split(_spread(s["q"], h) * live)
    k = split(_spread(s["k"], h) * live)
    v = split(s["v"].float() * live)
    # sums of logarithms in 64 bits: only their differences are used
    log = torch.log(s["decay"].double()).clamp(min=-1e6).unsqueeze(-1) * live
    log = split(log).squeeze(-1).cumsum(-1)                                   # [n, h, pieces, c]
    total = log[..., -1]
    inside = torch.exp(log.unsqueeze(-1) - log.unsqueeze(-2)).tril().float()  # [n, h, pieces, c, c]
    left = torch.exp(total.unsqueeze(-1) - log).float().unsqueeze(-1)
    own_state = (k * left).transpose(-1, -2) @ v                              # [n, h, pieces, d, d]
    if "S0" in s:
        S0 = s["S0"]
    elif case["start"] == "continue":
        S0 = _matrix(s["buf"], d).view(n, h, d, d)
    else:
        S0 = torch.zeros(n, h, d, d, device="cuda")
    # the state before each piece and after the last: one product with the
    # lower triangle of decays between pieces
    along = torch.nn.functional.pad(total.cumsum(-1), (1, 0))
    between = torch.exp(along.unsqueeze(-1) - along.unsqueeze(-2)).tril().float()  # [n, h, pieces + 1, pieces + 1]
    parts = torch.cat([S0.unsqueeze(2), own_state], 2).view(n, h, pieces + 1, d * d)
    states = (between @ parts).view(n, h, pieces + 1, d, d)
    o = (q @ k.transpose(-1, -2) * inside) @ v + torch.exp(log).float().unsqueeze(-1) * (q @ states[:, :, :-1])
    out = o.permute(0, 2, 3, 1, 4).reshape(n, pieces * c, h, d)[:, :t]
    S = _matrix(s["buf"], d)
    S.copy_(states[:, :, -1].reshape(-1, d, d))
    return out, S


def _qk_norm(s, case):
    scale = case["d"] ** -0.5
    if own:
        from linear_attention_recurrent_lq_b200 import binding as B
        if "cfg" not in s:
            s["cfg"] = _config(case, 1)
        B.lq_qk_norm(s["cfg"], s["q"], s["k"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["q_out"], s["k_out"],
                     s["decay"], s["beta"], q_scale=scale, eps=_EPS, qk_heads=case["hk"])
        return s["q_out"], s["k_out"], s["decay"], s["beta"]
    q, k, a = s["q"].float(), s["k"].float(), s["a"].float()
    q = scale * q / (q.square().sum(-1, keepdim=True) + _EPS).sqrt()
    k = k / (k.square().sum(-1, keepdim=True) + _EPS).sqrt()
    a = a + s["dt_bias"]
    soft = a.clamp(min=0) + torch.log1p(torch.exp(-a.abs()))
    rate = torch.exp(s["a_log"])
    decay = torch.exp(-soft * (rate[:, None] if case["kda"] else rate))
    beta = 1 / (1 + torch.exp(-s["b"].float()))
    return q.to(_dtype(case)), k.to(_dtype(case)), decay, beta


def _out_norm(s, case):
    if own:
        from linear_attention_recurrent_lq_b200 import binding as B
        if "cfg" not in s:
            s["cfg"] = _config(case, 1)
        B.lq_out_norm(s["cfg"], s["o"], s["y"], weight=s["weight"], gate=s["gate"], gate_kind=case["gate"], eps=_EPS)
        return s["y"]
    o = s["o"]
    y = o / (o.square().mean(-1, keepdim=True) + _EPS).sqrt()
    if s["weight"] is not None:
        y = y * s["weight"]
    if s["gate"] is not None:
        g = s["gate"].float()
        y = y / (1 + torch.exp(-g)) * (g if case["gate"] == "silu" else 1.0)
    return y.to(_dtype(case))


def work(case):
    h, d, e = case["h"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "step":
        heads = (max(1, 3 * case["n"] // 4) if case["slots"] else case["n"]) * h
        return {"bytes": heads * (8 * d * d + d * e + 4 + 4 * d) + 2 * heads // h * case["hk"] * d * e, "flops": 4 * heads * d * d}
    if case["op"] == "prefill":
        tokens = case["n"] * case["t"] // (2 if case["lengths"] else 1)
        state = case["n"] * h * 4 * d * d * (1 if case["start"] == "zero" else 2)
        return {"bytes": tokens * (h * (d * e + 4) + 2 * case["hk"] * d * e) + case["n"] * case["t"] * h * 4 * d + state,
                "flops": 4 * tokens * h * d * d}
    if case["op"] == "qk_norm":
        logits = h * (d if case["kda"] else 1)
        return {"bytes": case["m"] * (4 * case["hk"] * d * e + (logits + h) * (e + 4)), "flops": case["m"] * (8 * case["hk"] * d + 8 * (logits + h))}
    return {"bytes": case["m"] * h * d * (4 + e + (0 if case["gate"] == "none" else e)), "flops": 8 * case["m"] * h * d}


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token."""
    s = prepare(case, seed)
    d, h = case["d"], case["h"]

    def wide(x):
        return s[x].double()

    if case["op"] in ("step", "prefill"):
        group = h // case["hk"]
        state = _matrix(s["buf"], d).double()
        if case.get("start") == "zero":
            state.zero_()
        if "S0" in s:
            state = wide("S0").reshape(-1, d, d)
        q, k, v, a = (wide(x) for x in ("q", "k", "v", "decay"))
        rows = q.shape[0]
        if case["op"] == "step":
            q, k, v, a = (x.unsqueeze(1) for x in (q, k, v, a))
        tokens = q.shape[1]
        index = torch.arange(state.shape[0], device="cuda") if s["heads"] is None else s["heads"]
        S = state[index].view(rows, case["hk"], group, d, d)
        out = torch.zeros(rows, tokens, h, d, dtype=torch.float64, device="cuda")
        lengths = s["lengths"].tolist() if "lengths" in s else None
        order = sorted(range(rows), key=lambda r: -lengths[r]) if lengths else list(range(rows))
        counts = [lengths[r] for r in order] if lengths else [tokens] * rows
        S = S[order] if lengths else S
        at = torch.tensor(order, device="cuda")
        for t in range(max(counts)):  # the longest rows come first
            n = sum(c > t for c in counts)
            r = at[:n]
            kt, vt, qt = k[r, t], v[r, t].view(n, -1, group, d), q[r, t]
            at_ = a[r, t].view(n, -1, group, 1, 1)
            S[:n] = S[:n] * at_ + kt[:, :, None, :, None] * vt[:, :, :, None, :]
            out[r, t] = torch.einsum("nki,nkgij->nkgj", qt, S[:n]).reshape(n, h, d)
        if lengths:
            back = torch.empty_like(S)
            back[at] = S
            S = back
        state[index] = S.reshape(-1, d, d)
        return (out.squeeze(1) if case["op"] == "step" else out), state
    if case["op"] == "qk_norm":
        q, k, a, b = (wide(x) for x in ("q", "k", "a", "b"))
        q = q * (case["d"] ** -0.5 / torch.sqrt(torch.einsum("mhd,mhd->mh", q, q) + _EPS))[..., None]
        k = k / torch.sqrt(torch.einsum("mhd,mhd->mh", k, k) + _EPS)[..., None]
        soft = torch.logaddexp(a + wide("dt_bias"), torch.zeros((), dtype=torch.float64, device="cuda"))
        rate = wide("a_log").exp().view((-1, 1) if case["kda"] else (-1,))
        return q, k, torch.exp(-rate * soft), torch.sigmoid(b)
    o = wide("o")
    y = o * torch.rsqrt(torch.einsum("mhd,mhd->mh", o, o) / d + _EPS)[..., None]
    if s["weight"] is not None:
        y = y * wide("weight")
    if s["gate"] is not None:
        g = wide("gate")
        y = y * (g * torch.sigmoid(g) if case["gate"] == "silu" else torch.sigmoid(g))
    return y
