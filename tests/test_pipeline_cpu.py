"""The host pipeline's scratch tensors, without a GPU: they stay where a captured
graph has them."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def pipeline(monkeypatch):
    from linear_attention_recurrent_lq_b200 import pipeline as p
    monkeypatch.setattr(torch.cuda, "Stream", lambda: object())
    monkeypatch.setattr(torch.cuda, "Event", lambda: object())
    return p


def layer(p, W=4, rows=3, H=4, hk=2, d=64, kda=False):
    ch = (d,) if kda else ()
    x = dict(q=torch.zeros(W, rows, hk, d, dtype=torch.bfloat16), k=torch.zeros(W, rows, hk, d, dtype=torch.bfloat16),
             v=torch.zeros(W, rows, H, d, dtype=torch.bfloat16), a=torch.zeros(W, rows, H, *ch), b=torch.zeros(W, rows, H))
    state = SimpleNamespace(cfg=SimpleNamespace(dk=d, decay_kind=int(kda)))
    proj = p.Projections(torch.zeros(H), torch.zeros(H, *ch))
    return p.Layer(state, x, torch.zeros(W, rows, H, d, dtype=torch.bfloat16), {}, None, proj=proj)


@pytest.mark.parametrize("kda", [False, True])
def test_a_second_pipeline_keeps_the_scratch_of_a_captured_layer(pipeline, kda):
    lay = layer(pipeline, kda=kda)
    pipeline.HostIOPipeline([lay], 4)
    assert lay.scratch["decay"].shape == (4, 3, 4, *((64,) if kda else ()))
    first, lay.graph = dict(lay.scratch), object()   # as capture() leaves it
    graph = lay.graph
    pipeline.HostIOPipeline([lay], 4)
    assert lay.graph is graph
    assert lay.scratch.keys() == first.keys() and all(lay.scratch[n] is first[n] for n in first)


def test_scratch_that_no_longer_fits_drops_the_graph(pipeline):
    lay = layer(pipeline)
    pipeline.HostIOPipeline([lay], 4)
    first, lay.graph = dict(lay.scratch), object()
    other = layer(pipeline, W=8)
    lay.dev_in, lay.dev_out = other.dev_in, other.dev_out
    pipeline.HostIOPipeline([lay], 8)
    assert lay.graph is None
    assert lay.scratch["rows"].shape == (8, 3, 4, 64) and lay.scratch["q"] is not first["q"]
    assert lay.scratch["v"] is lay.dev_in["v"]


def test_layers_without_projections_have_none(pipeline):
    lay = layer(pipeline)
    lay.proj = None
    pipeline.HostIOPipeline([lay], 4)
    assert lay.scratch is None
