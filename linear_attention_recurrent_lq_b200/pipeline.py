"""Decode windows fed from, and read back to, pinned host memory, with the
transfers overlapped with the kernels.

Each layer-state of a step has device input buffers (q, k, v, beta, decay
for W tokens), a device output buffer, and pinned host copies of both.  Per
layer l, the upload stream copies l's inputs host->device, the compute
stream runs l's window (W decode calls and the window flush, captured as one
CUDA graph per layer) once they have landed, and the download stream copies
l's outputs back once the window has written them.  So layer l+1's upload
and layer l-1's download run while layer l computes, on the GPU's separate
copy engines.  Buffers are reused from step to step, ordered by events: an
upload waits for the previous step's window to be done with that layer's
input buffers, a window for the previous step's download of its output
buffer.

A layer with `Projections` takes the raw projections instead (q, k, v, the decay
logits a, the write-strength logits b and, with an output gate, gate): its
window starts with lq_qk_norm over all W tokens and ends with lq_out_norm, so
that normalised keys and gates never cross the host link and the rows that come
back are in the input type, half the bytes of the FP32 rows with bf16.
"""
from __future__ import annotations

from dataclasses import dataclass, field

NAMES = ("q", "k", "v", "beta", "decay")


@dataclass
class Projections:
    """What turns a layer's raw projections into the recurrence's inputs, and
    its FP32 rows into the layer's: parameters of lq_qk_norm and lq_out_norm
    (device tensors a_log [H], dt_bias [H] or [H, dk], weight [dv] or None)."""
    a_log: object
    dt_bias: object
    weight: object = None
    gate_kind: str = "silu"
    q_scale: float = 1.0
    eps: float = 1e-6
    linear: bool = False   # plain decayed heads (lq_linear_step) instead of the delta rule


@dataclass
class Layer:
    state: object          # an LQState
    dev_in: dict           # name -> device tensor [W, ...]: q, k, v, beta, decay; with proj q, k, v, a, b (, gate)
    dev_out: object        # device tensor [W, rows, H, dv]: FP32 rows; with proj in the input type
    host_in: dict          # name -> pinned host tensor, same shapes
    host_out: object       # pinned host tensor, same shape as dev_out
    graph: object = field(default=None)
    proj: object = field(default=None)   # Projections, or None
    scratch: dict = field(default=None)  # with proj: normalised q and k, gates, FP32 rows


class HostIOPipeline:
    def __init__(self, layers: list[Layer], window: int, flush: bool = True):
        import torch
        self.torch = torch
        self.layers = layers
        self.window = window
        self.flush = flush
        for lay in layers:
            if lay.proj is not None:
                self._make_scratch(lay)
        self.up = torch.cuda.Stream()
        self.comp = torch.cuda.Stream()
        self.down = torch.cuda.Stream()
        n = len(layers)
        self.up_done = [torch.cuda.Event() for _ in range(n)]
        self.comp_done = [torch.cuda.Event() for _ in range(n)]
        self.down_done = [torch.cuda.Event() for _ in range(n)]

    def _make_scratch(self, lay: Layer):
        """The layer's scratch tensors.  They belong to the layer, as a graph that
        was captured from it holds their addresses: another pipeline over the layer
        uses the same ones, and a graph whose scratch no longer fits is dropped."""
        torch = self.torch
        x, c = lay.dev_in, lay.state.cfg
        heads = (*x["v"].shape[:-1],)  # [W, rows, H]
        want = dict(q=(x["q"].shape, x["q"].dtype), k=(x["k"].shape, x["k"].dtype), beta=(heads, torch.float32),
                    decay=(heads + ((c.dk,) if c.decay_kind == 1 else ()), torch.float32),
                    rows=(x["v"].shape, torch.float32))
        dev, have = x["v"].device, lay.scratch
        if have is not None and all(n in have and have[n].device == dev and have[n].dtype == t
                                    and tuple(have[n].shape) == tuple(s) for n, (s, t) in want.items()):
            have["v"] = x["v"]
            return
        lay.graph = None
        lay.scratch = dict({n: torch.empty(tuple(s), dtype=t, device=dev) for n, (s, t) in want.items()}, v=x["v"])

    def _window(self, lay: Layer):
        x, p, rows = lay.dev_in, lay.proj, lay.dev_out
        if p is not None:
            from . import binding as B
            s, rows = lay.scratch, lay.scratch["rows"]
            hk = x["q"].shape[-2]
            B.lq_qk_norm(lay.state.cfg, x["q"], x["k"], x["a"], x["b"], p.a_log, p.dt_bias, s["q"], s["k"], s["decay"],
                         s["beta"], q_scale=p.q_scale, eps=p.eps, qk_heads=hk)
            raw, x = x, s
        for t in range(self.window):
            if p is not None and p.linear:
                lay.state.linear_step(x["q"][t], x["k"][t], x["v"][t], x["decay"][t], rows[t], qk_heads=hk)
            else:
                lay.state.step(x["q"][t], x["k"][t], x["v"][t], x["beta"][t], x["decay"][t], rows[t])
        if self.flush:
            lay.state.flush()
        if p is not None:
            B.lq_out_norm(lay.state.cfg, rows, lay.dev_out, weight=p.weight, gate=raw.get("gate"),
                          gate_kind=p.gate_kind, eps=p.eps)

    def capture(self):
        """One graph per layer (run once eagerly first, which also sets the
        kernels' launch attributes outside the capture)."""
        torch = self.torch
        with torch.cuda.stream(self.comp):
            for lay in self.layers:
                self._window(lay)
        torch.cuda.synchronize()
        for lay in self.layers:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=self.comp):
                self._window(lay)
            lay.graph = g
        torch.cuda.synchronize()

    def bytes_per_step(self) -> tuple[int, int]:
        h2d = sum(t.numel() * t.element_size() for lay in self.layers for t in lay.host_in.values())
        d2h = sum(lay.host_out.numel() * lay.host_out.element_size() for lay in self.layers)
        return h2d, d2h

    def step(self):
        """Enqueue one step: every layer's upload, window and download."""
        torch = self.torch
        for i, lay in enumerate(self.layers):
            with torch.cuda.stream(self.up):
                self.up.wait_event(self.comp_done[i])
                for name in NAMES if lay.proj is None else lay.host_in:
                    lay.dev_in[name].copy_(lay.host_in[name], non_blocking=True)
                self.up_done[i].record(self.up)
            with torch.cuda.stream(self.comp):
                self.comp.wait_event(self.up_done[i])
                self.comp.wait_event(self.down_done[i])
                lay.graph.replay()
                self.comp_done[i].record(self.comp)
            with torch.cuda.stream(self.down):
                self.down.wait_event(self.comp_done[i])
                lay.host_out.copy_(lay.dev_out, non_blocking=True)
                self.down_done[i].record(self.down)

    def join(self, stream=None):
        """Make `stream` (default: the current one) wait for all enqueued work."""
        torch = self.torch
        s = stream or torch.cuda.current_stream()
        for ev in (self.up_done[-1], self.comp_done[-1], self.down_done[-1]):
            s.wait_event(ev)

    def fork(self, stream=None):
        """Make the three streams wait for the work enqueued so far on `stream`."""
        torch = self.torch
        s = stream or torch.cuda.current_stream()
        ev = torch.cuda.Event()
        ev.record(s)
        for st in (self.up, self.comp, self.down):
            st.wait_event(ev)
