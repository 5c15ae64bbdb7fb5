"""SpecEngine.export_kv8 without a GPU: what it checks and on which streams it works, over stand-ins for the engine's
library calls and for the cache."""

import types

import pytest
import torch

from speculative_decoding_06_b200 import engine as E

HEADS, LAYERS, BATCH, MAX_SEQ = 2, 3, 4, 8


class Cache:
    n_layers, n_kv_heads = LAYERS, HEADS

    def __init__(self, device="cpu"):
        self.device, self.calls = torch.device(device), []

    def plan_buffers(self, batch, n_seqs, rows):
        return Plan()

    def plan(self, *a, **kw):
        self.calls.append("plan")
        return Plan()

    def append(self, layer, k, v, slots, src_rows=None):
        self.calls.append(("append", layer, k, v, src_rows))


class Plan:
    status, slots = 0, None

    def _replace(self, **kw):
        return self


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append((self.name, other.name))


@pytest.fixture
def engine(monkeypatch):
    e = E.SpecEngine.__new__(E.SpecEngine)
    e.dims = types.SimpleNamespace(dtype="bf16", n_layers=LAYERS, n_kv_heads=HEADS, head_dim=128)
    e.log, e.asked = [], []
    e.stream = Stream("engine", e.log)
    e.kv = torch.zeros(LAYERS, 3, BATCH, HEADS, MAX_SEQ, 128, dtype=torch.float16)
    for i, x in enumerate(e.kv.view(-1, 128)):
        x.fill_(i)
    e.kv_view = lambda: e.kv
    e.seq_len = lambda s: (s + 2, 0)

    def current(device=None):
        e.asked.append(device)
        return Stream("current", e.log)

    monkeypatch.setattr(torch.cuda, "current_stream", current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: e.log.append(("kv", s.name)))
    return e


def pages():
    return types.SimpleNamespace(lengths=torch.zeros(5, dtype=torch.int32), tables=None, ring=None, state=None)


def test_rows_and_streams(engine):
    cache = Cache()
    assert engine.export_kv8([3, 1], cache, pages()) == [5, 3]
    assert cache.calls[0] == "plan" and [c[1] for c in cache.calls[1:]] == list(range(LAYERS))
    for _, layer, k, v, src in cache.calls[1:]:
        for plane, x in ((0, k), (1, v)):
            want = torch.cat([engine.kv[layer, plane, s, :, :n].transpose(0, 1) for s, n in ((3, 5), (1, 3))])
            assert torch.equal(x[src.long()], want)
    # the appends go between the engine's work before and after, on the stream that is current on the cache's device,
    # which the engine's memory is not given away before
    assert engine.log.index(("current", "engine")) < engine.log.index(("engine", "current"))
    assert ("kv", "current") in engine.log
    assert engine.asked and all(d == cache.device for d in engine.asked)


def test_refused_before_anything_is_planned(engine):
    for cache in (Cache("cuda:1"), Cache("meta")):  # not the engine's device
        with pytest.raises(ValueError):
            engine.export_kv8([0], cache, pages())
        assert cache.calls == []
    cache = Cache()
    cache.n_kv_heads = 1
    with pytest.raises(ValueError):
        engine.export_kv8([0], cache, pages())
    engine.dims.dtype = "f32"
    with pytest.raises(ValueError):
        engine.export_kv8([0], Cache(), pages())
    assert cache.calls == []
