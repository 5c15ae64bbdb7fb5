"""The operators of the 8-bit paged cache as they are used together: a decoding loop over draft trees, the same captured
into a CUDA graph, and the export of an engine's cache."""

import numpy as np
import pytest
import torch

import synth
from oracle import kv8 as O

pytestmark = pytest.mark.gpu

HKV, HQ, PAGE, LAYERS = 2, 8, 16, 2


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Mirror:
    """The oracle's copy of a cache and its pages."""

    def __init__(self, n_pages, n_seqs, max_blocks):
        self.codes = [np.zeros((2, n_pages, HKV, PAGE, 128), np.uint8) for _ in range(LAYERS)]
        self.exps = [np.zeros((2, n_pages, HKV), np.uint8) for _ in range(LAYERS)]
        self.lengths = np.zeros(n_seqs, np.int32)
        self.tables = np.full((n_seqs, max_blocks), -1, np.int32)
        self.ring = np.arange(n_pages, dtype=np.int32)
        self.state = np.array([0, n_pages], np.int32)

    def plan(self, add, max_rows, ids):
        off, slots, self.lengths, self.state, status, self.tables, self.ring = O.plan(
            self.lengths, add, self.tables, self.ring, self.state, PAGE, max_rows, ids)
        return off, slots, status


def tolerance(dtype, ref_out, mass, size):
    """As derived for the attention tests: half a step of the output, the probabilities' rounding, the scores' error."""
    u = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -11
    d = 2 * 130 * 2.0 ** -24 * size + 2.0 ** -18
    return u * np.abs(ref_out) + (u + 2.0 ** -11 + d[..., None]) * mass + 1e-7


@pytest.mark.parametrize("nodes,dtype", [(3, torch.bfloat16), (20, torch.float16)])
def test_decoding_loop(nodes, dtype):
    """Prompts are appended; each step's trees attend (both layers), a part of every tree is accepted and appended from
    the step's rows, one sequence ends and another one begins, pages go round the ring.  Everything on a side stream."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    g = np.random.default_rng(nodes)
    n_pages, n_seqs, max_blocks = 30, 5, 12
    cache = KV8Cache(LAYERS, HKV, n_pages, PAGE)
    cache.codes.zero_(), cache.exps.zero_()
    M = Mirror(n_pages, n_seqs, max_blocks)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        pages = cache.page_state(n_seqs, max_blocks)

        def rows(n, heads):
            return torch.from_numpy(g.normal(size=(n, heads, 128))).to(dtype)

        def step_plan(add, ids):
            """In place on the GPU; the oracle beside it."""
            max_rows = int(np.clip(add, 0, None).sum()) + 2
            out = cache.plan_buffers(len(ids), n_seqs, max_rows)._replace(lengths=pages.lengths, state=pages.state)
            p = cache.plan(pages.lengths, i32(add), pages.tables, pages.ring, pages.state, max_rows, i32(ids), out=out)
            off, slots, status = M.plan(add, max_rows, ids)
            assert int(p.status) == status == 0
            assert np.array_equal(p.slots.cpu().numpy(), slots) and np.array_equal(p.offsets.cpu().numpy(), off)
            for a, b in ((pages.lengths, M.lengths), (pages.tables, M.tables), (pages.ring, M.ring), (pages.state, M.state)):
                assert np.array_equal(a.cpu().numpy(), b)
            return p.slots, slots

        def store(kv, slots, np_slots, src=None):
            for layer, (k, v) in enumerate(kv):
                cache.append(layer, k.cuda(), v.cuda(), slots, None if src is None else i32(src))
                O.append(M.codes[layer], M.exps[layer], PAGE, k.double().numpy(), v.double().numpy(), np_slots, src)

        live = [4, 0, 2]
        prompt = [37, 16, 5]
        slots, np_slots = step_plan(prompt, live)
        n = sum(prompt)
        store([(rows(n + 2, HKV), rows(n + 2, HKV)) for _ in range(LAYERS)], slots, np_slots)
        for step in range(6):
            count = [int(g.integers(1, nodes + 1)) for _ in live]
            off = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
            T = int(off[-1])
            parents = np.concatenate([[-1] + [int(g.integers(0, i)) for i in range(1, c)] for c in count]).astype(np.int32)
            kv = [(rows(T, HKV), rows(T, HKV)) for _ in range(LAYERS)]
            q = rows(T, HQ)
            for layer, (k, v) in enumerate(kv):
                out, lse = cache.attention(layer, q.cuda(), pages.tables, pages.lengths, i32(off), max_prefix=PAGE * max_blocks,
                                           max_nodes=nodes, k_new=k.cuda(), v_new=v.cuda(), parents=i32(parents),
                                           seq_ids=i32(live))
                ref, ref_lse, mass, size = O.attention(M.codes[layer], M.exps[layer], PAGE, q.double().numpy(), M.tables,
                                                       M.lengths, off, 128 ** -0.5, k.double().numpy(), v.double().numpy(),
                                                       parents, live)
                assert (np.abs(out.double().cpu().numpy() - ref) <= tolerance(dtype, ref, mass, size)).all()
                assert np.allclose(lse.cpu().numpy(), ref_lse, rtol=0, atol=1e-4)
            # a random root path of every tree is accepted
            src, add = [], []
            for b, c in enumerate(count):
                path, j = [], int(g.integers(0, c))
                while j >= 0:
                    path.append(int(off[b]) + j)
                    j = int(parents[off[b] + j])
                src += path[::-1]
                add.append(len(path))
            slots, np_slots = step_plan(add, live)
            store(kv, slots, np_slots, src + [0, 0])
            for layer in range(LAYERS):
                assert np.array_equal(cache.exps[layer].cpu().numpy(), M.exps[layer])
                assert np.array_equal(cache.codes[layer].cpu().numpy(), M.codes[layer])
            if step == 2:  # one ends, one begins with a longer prompt, one rolls back three tokens
                step_plan([-(1 << 30), -3], [live[0], live[1]])
                live = [3] + live[1:]
                slots, np_slots = step_plan([50], [3])
                store([(rows(60, HKV), rows(60, HKV)) for _ in range(LAYERS)], slots, np_slots)


@pytest.mark.parametrize("nodes", [1, 17])
def test_captured_step_replays(nodes):
    """Attention, plan (in place) and append captured once and replayed: the same as the eager steps, bit for bit, while
    an eager step of another stream and workspace runs between."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    g = torch.Generator(device="cuda").manual_seed(nodes)
    B, steps = 3, 4
    caches = [KV8Cache(1, HKV, 60, PAGE) for _ in range(2)]
    states = [c.page_state(B, 20) for c in caches]
    q, k, v = (torch.randn(B * nodes, h, 128, device="cuda", generator=g).to(torch.bfloat16) for h in (HQ, HKV, HKV))
    off, add = i32(np.arange(B + 1) * nodes), i32([nodes] * B)
    outs = []

    def step(c, s, out, lse, ws, buf):
        c.attention(0, q, s.tables, s.lengths, off, max_prefix=320, max_nodes=nodes, k_new=k, v_new=v, out=out, lse=lse,
                    workspace=ws)
        c.plan(s.lengths, add, s.tables, s.ring, s.state, B * nodes, out=buf)
        c.append(0, k, v, buf.slots)

    for c, s in zip(caches, states):
        c.codes.zero_(), c.exps.zero_()
        out, lse = torch.zeros_like(q), torch.zeros(B * nodes, HQ, device="cuda")
        ws = c.attention_workspace(B, HQ, nodes, 320)
        buf = c.plan_buffers(B, B, B * nodes)._replace(lengths=s.lengths, state=s.state)
        outs.append((c, s, out, lse, ws, buf))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step(*outs[1])  # before the capture: kernels are loaded; then back to the empty state
        stream.synchronize()
        states[1].lengths.zero_()
        states[1].state.copy_(i32([0, 60]))
        caches[1].codes.zero_(), caches[1].exps.zero_()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step(*outs[1])
        for i in range(steps):
            graph.replay()
    for i in range(steps):
        step(*outs[0])
    torch.cuda.synchronize()
    for a, b in zip(states[0], states[1]):
        assert torch.equal(a, b)
    assert int(outs[0][5].status) == 0 and int(states[0].lengths[0]) == steps * nodes
    assert torch.equal(caches[0].codes, caches[1].codes) and torch.equal(caches[0].exps, caches[1].exps)
    assert torch.equal(outs[0][2], outs[1][2]) and torch.equal(outs[0][3], outs[1][3])


def test_same_results_every_time():
    """Chunks are merged in order, whoever arrives first: a split prefix gives the same bits in every run."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = KV8Cache(1, 1, 200, 64)
    cache.codes.random_(0, 120, generator=g)
    cache.exps.fill_(118)
    lengths, tables = i32([12000]), torch.arange(200, dtype=torch.int32, device="cuda").view(1, 200)
    for nodes in (1, 12, 40):
        q = torch.randn(nodes, 4, 128, device="cuda", generator=g).half()
        first = None
        for _ in range(20):
            out, lse = cache.attention(0, q, tables, lengths, i32([0, nodes]), max_prefix=12000, max_nodes=nodes)
            if first is None:
                first = out.clone(), lse.clone()
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_export_from_the_engine():
    """An engine's fp16 cache stored in 8 bits: the codes are those of its K and V rows, for every layer, and attention
    over them is within e4m3's rounding of attention over the rows themselves."""
    from speculative_decoding_06_b200.engine import SpecEngine
    from speculative_decoding_06_b200.kv8 import KV8Cache
    d = synth.MINI_BF16
    w = synth.model_weights(d, seed=0, device="cuda")
    eng = SpecEngine(d, w, max_batch=3, max_seq=256, max_nodes=32)
    lens = {0: 70, 2: 33}
    for s, n in lens.items():
        eng.prefill(s, synth.prefix_tokens(d.vocab, n, stream=s))
    cache = KV8Cache(d.n_layers, d.n_kv_heads, 12, 16)
    pages = cache.page_state(4, 8)
    assert eng.export_kv8([2, 0], cache, pages, kv8_ids=[3, 1]) == [33, 70]
    assert pages.lengths.tolist() == [0, 70, 0, 33]
    kv, tables = eng.kv_view().float().cpu().numpy(), pages.tables.cpu().numpy()
    codes, exps = cache.codes.cpu().numpy(), cache.exps.cpu().numpy()
    for s, to in ((2, 3), (0, 1)):
        for layer in range(d.n_layers):
            rows = kv[layer, :2, s, :, :lens[s]].transpose(0, 2, 1, 3)
            want_c, want_e = np.zeros_like(codes[layer]), np.zeros_like(exps[layer])
            slots = [tables[to, j // 16] * 16 + j % 16 for j in range(lens[s])]
            O.append(want_c, want_e, 16, rows[0], rows[1], slots)
            for j, slot in enumerate(slots):
                assert np.array_equal(codes[layer][:, slot // 16, :, slot % 16], want_c[:, slot // 16, :, slot % 16])
                assert np.array_equal(exps[layer][:, slot // 16], want_e[:, slot // 16])
    q = torch.randn(2, d.n_q_heads, 128, device="cuda").to(torch.bfloat16)
    out, _ = cache.attention(d.n_layers - 1, q, pages.tables, pages.lengths, i32([0, 1, 2]), max_prefix=128, max_nodes=1,
                             seq_ids=i32([1, 3]))
    for b, s in ((0, 0), (1, 2)):
        k, v = (torch.from_numpy(kv[d.n_layers - 1, p, s, :, :lens[s]]).double() for p in (0, 1))
        group = d.n_q_heads // d.n_kv_heads
        for h in range(d.n_q_heads):
            p = torch.softmax(k[h // group] @ q[b, h].double().cpu() * 128 ** -0.5, 0)
            ref, mass = p @ v[h // group], p @ v[h // group].abs()
            # e4m3 is within 2^-4 of a value, of V here and of K in the scores (their effect taken at four times)
            assert ((out[b, h].double().cpu() - ref).abs() <= 5 * 2.0 ** -4 * mass + 1e-3).all()
    with pytest.raises(Exception):
        eng.export_kv8([0], cache, pages, kv8_ids=[1])  # 140 tokens do not fit eight blocks of 16
    assert pages.lengths.tolist() == [0, 70, 0, 33]
    eng.close()


@pytest.mark.parametrize("nodes", [(1, 2), (1, 30), (20, 30)])
def test_two_streams_at_once(nodes):
    """Calls of two streams over one cache, each with a workspace and outputs of its own (and one with new outputs whose
    last rows belong to no entry): the same bits as one after the other."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    g = torch.Generator(device="cuda").manual_seed(4)
    B, P = 3, 3000
    cache = KV8Cache(1, HKV, 3 * 47, 64)
    cache.codes.random_(0, 120, generator=g)
    cache.exps.random_(110, 124, generator=g)
    lengths, tables = i32([P, 70, 1500]), torch.arange(3 * 47, dtype=torch.int32, device="cuda").view(3, 47)
    calls = []
    for n in nodes:
        q, k, v = (torch.randn(B * n + 2, h, 128, device="cuda", generator=g).half() for h in (HQ, HKV, HKV))
        ws = cache.attention_workspace(B, HQ, n, P)
        off = i32(np.arange(B + 1) * n)
        calls.append(lambda q=q, k=k, v=v, n=n, ws=ws, off=off: cache.attention(
            0, q, tables, lengths, off, max_prefix=P, max_nodes=n, k_new=k, v_new=v, workspace=ws))
    want = [c() for c in calls]
    for (out, lse), n in zip(want, nodes):
        assert not out[B * n:].any() and (lse[B * n:] == -np.inf).all() and not torch.isnan(out).any()
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(40):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
