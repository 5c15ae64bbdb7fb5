"""The 8-bit paged cache on the GPU against its float64 oracle: page plan, append, attention, and the three in a loop."""

import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O
from speculative_decoding_06_b200 import spec as S

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def make_cache(n_pages, hkv, page, layers=1, garbage=None):
    """A cache whose memory holds `garbage` until it is written (0x7F: e4m3's NaN, and an exponent of 0)."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    cache = KV8Cache(layers, hkv, n_pages, page)
    if garbage is not None:
        cache.codes.fill_(garbage)
        cache.exps.fill_(garbage)
    return cache


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plan
def plan_inputs(g, batch, n_seqs, page, max_blocks, top, seed_ids=True):
    lengths = g.integers(0, top + 1, n_seqs).astype(np.int32)
    used = [-(-int(n) // page) for n in lengths]
    n_pages = sum(used) + batch * 6 + 3
    order = g.permutation(n_pages).astype(np.int32)
    tables, at = np.full((n_seqs, max_blocks), -1, np.int32), 0
    for s, n in enumerate(used):
        tables[s, :n] = order[at:at + n]
        at += n
    head = int(g.integers(0, n_pages))
    ring = np.full(n_pages, -7, np.int32)
    ring[(head + np.arange(n_pages - at)) % n_pages] = order[at:]
    ids = g.permutation(n_seqs)[:batch].astype(np.int32) if seed_ids else None
    return lengths, tables, ring, np.array([head, n_pages - at], np.int32), ids, n_pages


def check_plan(cache, lengths, add, tables, ring, state, page, max_rows, ids, in_place=False):
    want = O.plan(lengths, add, tables, ring, state, page, max_rows, ids)
    gl, gs = i32(lengths), i32(state)
    gt, gr = i32(tables), i32(ring)
    out = None
    if in_place:
        out = cache.plan_buffers(len(add), len(lengths), max_rows)._replace(lengths=gl, state=gs)
    p = cache.plan(gl, i32(add), gt, gr, gs, max_rows, None if ids is None else i32(ids), out=out)
    got = (p.offsets, p.slots, p.lengths, p.state, p.status, gt, gr)
    for name, g, w in zip(("offsets", "slots", "lengths", "state", "status", "tables", "ring"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    return want


@pytest.mark.parametrize("batch,n_seqs,page,max_blocks,top,ids", [
    (1, 1, 64, 8, 100, False), (5, 9, 16, 40, 300, True), (33, 33, 32, 12, 300, False), (300, 400, 16, 30, 400, True),
    (1500, 2000, 128, 4, 400, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(batch, n_seqs, page, max_blocks, top, ids, in_place):
    g = np.random.default_rng(batch)
    lengths, tables, ring, state, ids, n_pages = plan_inputs(g, batch, n_seqs, page, max_blocks, top, ids)
    cache = make_cache(n_pages, 1, page)
    add = g.integers(-40, 30, batch)
    add[g.random(batch) < 0.2] = 0
    add[g.random(batch) < 0.1] = -(1 << 30)
    want = check_plan(cache, lengths, add, tables, ring, state, page, 30 * batch, ids, in_place)
    assert want[4] == 0
    check_plan(cache, lengths, add * 0, tables, ring, state, page, 0, ids, in_place)


def test_plan_many_rows():
    """Rows enough for the second launch, their count not a multiple of anything; and none at all."""
    g = np.random.default_rng(7)
    lengths, tables, ring, state, ids, _ = plan_inputs(g, 37, 50, 16, 700, 500)
    ring = np.concatenate([ring, np.full(30000, -7, np.int32)])
    n_pages = len(ring)
    free = np.setdiff1d(np.arange(n_pages), tables[tables >= 0])
    state = np.array([n_pages - 5, len(free)], np.int32)
    ring[(state[0] + np.arange(len(free))) % n_pages] = g.permutation(free)
    cache = make_cache(n_pages, 1, 16)
    add = g.integers(0, 5000, 37)
    add[[3, 4, 20]] = [0, -(1 << 30), -33]
    want = check_plan(cache, lengths, add, tables, ring, state, 16, int(add.clip(0).sum()) + 11, ids)
    assert want[4] == 0
    check_plan(cache, lengths, add * 0 - 1, tables, ring, state, 16, 5001, ids)
    want = check_plan(cache, lengths, add, tables, ring, state, 16, int(add.clip(0).sum()) - 1, ids)
    assert want[4] == S.SPEC_KV8_ROWS


@pytest.mark.parametrize("what,bits", [("rows", 1), ("pages", 2), ("table", 4), ("twice", 8), ("id", 8), ("length", 8),
                                       ("negative", 8), ("state", 8), ("count", 8)])
def test_plan_refused_on_the_device(what, bits):
    g = np.random.default_rng(3)
    lengths, tables, ring, state, ids, n_pages = plan_inputs(g, 6, 8, 16, 20, 200)
    add, max_rows = np.full(6, 3), 40
    if what == "rows":
        max_rows = 17
    if what == "pages":
        state[1] = 0
        add[:] = 16
        max_rows = 200
    if what == "table":
        add[2] = 16 * 20 + 1 - lengths[ids[2]]
        state[1], max_rows = n_pages - sum(-(-int(x) // 16) for x in lengths), 1000
    if what == "twice":
        ids[3] = ids[0]
    if what == "id":
        ids[3] = 8
    if what == "length":
        lengths[ids[1]] = 16 * 20 + 1
    if what == "negative":
        lengths[ids[1]] = -1
    if what == "state":
        state[0] = n_pages
    if what == "count":
        state[1] = -1
        add[:] = 0
    cache = make_cache(n_pages, 1, 16)
    gt, gr, gl, gs = i32(tables), i32(ring), i32(lengths), i32(state)
    p = cache.plan(gl, i32(add), gt, gr, gs, max_rows, i32(ids))
    assert int(p.status) & bits
    assert not p.offsets.any() and (p.slots == -1).all()
    assert torch.equal(p.lengths, gl) and torch.equal(p.state, gs)
    assert np.array_equal(gt.cpu().numpy(), tables) and np.array_equal(gr.cpu().numpy(), ring)


# ---------------------------------------------------------------- append
def check_append(cache, k, v, slots, src=None):
    codes, exps = cache.codes.cpu().numpy().copy(), cache.exps.cpu().numpy().copy()
    with np.errstate(all="ignore"):
        O.append(codes[0], exps[0], cache.page, k.float().cpu().numpy(), v.float().cpu().numpy(), slots, src)
    cache.append(0, k, v, i32(slots), None if src is None else i32(src))
    got_e, got_c = cache.exps.cpu().numpy(), cache.codes.cpu().numpy()
    assert np.array_equal(got_e, exps)
    # the codes of a page that holds NaN are unspecified; nothing else of the cache may have changed
    assert np.array_equal(got_c[exps < 255], codes[exps < 255])
    touched = np.zeros(exps.shape[2], bool)
    touched[[s // cache.page for s in slots if 0 <= s < cache.page * cache.n_pages]] = True
    assert np.array_equal(got_c[:, :, ~touched], codes[:, :, ~touched])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_append_runs(dtype, page, hkv):
    """Whole pages, ends of pages, single rows, skipped rows, a second call that raises some scales."""
    g = torch.Generator(device="cuda").manual_seed(page + hkv)
    cache = make_cache(7, hkv, page, garbage=0x7F)
    slots = list(range(page, 2 * page)) + [3 * page, 3 * page + 1] + [-1] + list(range(5 * page, 5 * page + 9)) + \
        [2 * page] + [7 * page, 1 << 30] + [0]
    x = torch.randn(2, len(slots), hkv, 128, device="cuda", generator=g)
    x = (x * torch.exp2(torch.randint(-9, 9, (2, len(slots), 1, 1), device="cuda", generator=g).float())).to(DT[dtype])
    check_append(cache, x[0], x[1], slots)
    more = [3 * page + 2, 3 * page + 3, 5 * page + 9, 2 * page + 1, 1]
    y = torch.randn(2, 5, hkv, 128, device="cuda", generator=g) * torch.tensor([1e3, 1.0, 1e-3, 100.0, 0.0], device="cuda")[:, None, None]
    check_append(cache, y[0].to(DT[dtype]), y[1].to(DT[dtype]), more)


def test_append_gathers_strided_rows_and_skips_bad_ones():
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = make_cache(6, 4, 16, garbage=0)
    wide = torch.randn(40, 3, 4, 136, device="cuda", generator=g).to(torch.float16)
    k, v = wide[:, 0, :, :128], wide[:, 2, :, 8:]
    slots = list(range(16, 29)) + [70, 71, 72]
    src = [39, 3, 3, 0, 1, 7, 40, 9, -1, 2, 2, 2, 5, 11, 38, 4]  # 40 and -1 store nothing and end their runs
    # a run behind a skipped row continues the page: its rows were opened by the first run of the same page, so
    # the runs are appended one after the other here
    for lo, hi in ((0, 6), (7, 8), (9, 16)):
        check_append(cache, k, v, slots[lo:hi], src[lo:hi])
    check_append(cache, k, v, slots[6:7], src[6:7])
    # planes swapped, heads as the outer dimension
    t = torch.randn(4, 40, 128, device="cuda", generator=g).to(torch.bfloat16).transpose(0, 1)
    check_append(cache, t, t, [80, 81, 82], [5, 6, 7])


def test_append_extremes():
    """Infinities, NaN, zeros, the smallest and the largest values, and a scale that leaves old codes subnormal."""
    cache = make_cache(4, 1, 16, garbage=0x7F)
    x = torch.zeros(6, 1, 128, device="cuda")
    x[0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 1.0, -2.5, 1e-9])
    x[1] = 3.4e38
    x[2] = 1e-42
    x[3, 0, ::2] = 2.0 ** -60
    x[4] = torch.linspace(-7, 7, 128, device="cuda")
    x[5] = 1e5
    check_append(cache, x, x.flip(0), [0, 16, 32, 48, 49, 50])
    check_append(cache, x[4:], x[:2], [51, 52])
    check_append(cache, x[1:2], x[1:2], [53])
    check_append(cache, torch.full((1, 1, 128), math.nan, device="cuda"), x[:1], [1])
    check_append(cache, x[:0], x[:0], [])


def test_append_writes_only_its_layer_and_rows():
    cache = make_cache(5, 2, 32, layers=3, garbage=0x55)
    cache.append(1, torch.ones(2, 2, 128, device="cuda"), torch.ones(2, 2, 128, device="cuda"), i32([64, 65]))
    c = cache.codes.clone()
    c[1, :, 2, :, :2] = 0x55
    assert (c == 0x55).all()
    e = cache.exps.clone()
    assert (e[1, :, 2] == 127 - 8).all()
    e[1, :, 2] = 0x55
    assert (e == 0x55).all()


# ---------------------------------------------------------------- attention
def attention_case(seed, prefixes, nodes, hq, hkv, page, dtype, tree="tree", extra_seqs=2, gain=1.0, garbage=0x7F):
    """Random cache, pages in random order, every slot behind a sequence's end holding `garbage`."""
    g = np.random.default_rng(seed)
    B, T = len(prefixes), sum(nodes)
    n_seqs = B + extra_seqs
    used = [-(-p // page) for p in prefixes]
    max_blocks = max(1, max(used)) + 1
    n_pages = sum(used) + 2
    order = g.permutation(n_pages)
    ids = g.permutation(n_seqs)[:B].astype(np.int32)
    tables, lengths, at = np.full((n_seqs, max_blocks), -1, np.int32), np.full(n_seqs, -5, np.int32), 0
    cache = make_cache(n_pages, hkv, page, garbage=garbage)
    codes = np.full(tuple(cache.codes.shape[1:]), garbage, np.uint8)
    exps = (127 - 8 + g.integers(-2, 3, tuple(cache.exps.shape[1:]))).astype(np.uint8)
    for b, s in enumerate(ids):
        tables[s, :used[b]] = order[at:at + used[b]]
        lengths[s] = prefixes[b]
        at += used[b]
        for j in range(prefixes[b]):
            codes[:, tables[s, j // page], :, j % page] = O.encode(g.normal(size=(2, hkv, 128)) * 120)
    cache.codes[0] = torch.from_numpy(codes)
    cache.exps[0] = torch.from_numpy(exps)
    q = torch.from_numpy(g.normal(size=(T, hq, 128)) * 1.5 * gain).to(DT[dtype])
    k = torch.from_numpy(g.normal(size=(T, hkv, 128))).to(DT[dtype])
    v = torch.from_numpy(g.normal(size=(T, hkv, 128))).to(DT[dtype])
    parents = None
    if tree == "tree":
        parents = np.concatenate([[-1] + [int(g.integers(0, i)) for i in range(1, n)] for n in nodes if n]).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return dict(cache=cache, codes=codes, exps=exps, page=page, q=q, k=k, v=v, tables=tables, lengths=lengths, ids=ids,
                parents=parents, offsets=offsets, dtype=dtype, prefix=max(prefixes), nodes=max(nodes), fresh=tree != "none")


def run_attention(c, scale=0.0, **kw):
    fresh = dict(k_new=c["k"].cuda(), v_new=c["v"].cuda(),
                 parents=None if c["parents"] is None else i32(c["parents"])) if c["fresh"] else {}
    args = dict(max_prefix=c["prefix"], max_nodes=c["nodes"], seq_ids=i32(c["ids"]), scale=scale, **fresh)
    args.update(kw)
    q = args.pop("q", c["q"].cuda())
    return c["cache"].attention(0, q, i32(c["tables"]), i32(c["lengths"]), i32(c["offsets"]), **args)


def reference(c, scale=0.0):
    n = lambda t: t.double().numpy()  # noqa: E731
    fresh = (n(c["k"]), n(c["v"]), c["parents"]) if c["fresh"] else (None, None, None)
    return O.attention(c["codes"], c["exps"], c["page"], n(c["q"]), c["tables"], c["lengths"], c["offsets"],
                       scale or 128 ** -0.5, *fresh, seq_ids=c["ids"])


def check_attention(c, got, ref):
    """|out - ref| <= u |ref| + (2^-11 + d) mass and |lse - ref| <= d + 2^-21 (1 + |ref|): u half a step of out's type;
    probabilities are rounded to fp16 at most (2^-11 each, so 2^-11 of sum p |v|), or to the row's own type for the
    step's own rows (u); d = 2 (the scores' error: products of exact values summed in 32 bits over 128 dimensions,
    at most 130 * 2^-24 of sum |q||k|, on both sides of the softmax) + 2^-18 (sums over up to 2^14 keys, exponentials)."""
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    ref_out, ref_lse, mass, size = ref
    u = 2.0 ** -8 if c["dtype"] == "bf16" else 2.0 ** -11
    d = 2 * 130 * 2.0 ** -24 * size + 2.0 ** -18
    dead = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), dead) and not out[dead].any()
    live = ~dead
    tol = u * np.abs(ref_out) + (u + 2.0 ** -11 + d[..., None]) * mass + 1e-7
    err = np.abs(out - ref_out)
    assert (err[live] <= tol[live]).all(), float((err / tol)[live].max())
    lse_err = np.abs(lse[live] - ref_lse[live])
    assert (lse_err <= d[live] + 2.0 ** -21 * (1 + np.abs(ref_lse[live]))).all(), float(lse_err.max())


CASES = [
    # prefixes, nodes, hq, hkv, page, dtype, mask
    ([1], [1], 1, 1, 16, "bf16", "tree"), ([0], [1], 4, 1, 64, "fp16", "tree"), ([64], [1], 8, 2, 64, "bf16", "none"),
    ([200, 0, 65, 64, 63], [1, 1, 1, 1, 1], 8, 2, 64, "bf16", "tree"),
    ([17, 0, 300], [1, 1, 1], 7, 1, 16, "fp16", "none"), ([700], [1], 6, 2, 32, "bf16", "chain"),
    ([130, 5], [3, 2], 4, 4, 128, "fp16", "tree"), ([257], [2], 16, 1, 128, "bf16", "none"),
    ([90, 33], [9, 4], 8, 2, 32, "bf16", "tree"), ([511], [5], 12, 2, 16, "fp16", "chain"),
    ([320, 100], [61, 17], 8, 2, 64, "bf16", "tree"), ([0, 40], [61, 0], 4, 1, 16, "fp16", "tree"),
    ([65], [128], 4, 2, 64, "fp16", "chain"), ([0, 129], [128, 127], 2, 1, 128, "bf16", "tree"),
    ([40], [33], 64, 1, 32, "bf16", "tree"), ([1000], [12], 5, 1, 64, "fp16", "none"),
    ([77, 600, 1], [1, 1, 1], 64, 1, 16, "bf16", "tree"), ([150], [70], 3, 3, 16, "bf16", "chain"),
    ([2500], [1], 4, 1, 64, "bf16", "tree"), ([3000, 20], [1, 1], 2, 1, 16, "fp16", "tree"),
    ([1500], [20], 8, 1, 128, "fp16", "tree"),
]


@pytest.mark.parametrize("prefixes,nodes,hq,hkv,page,dtype,tree", CASES)
def test_attention(prefixes, nodes, hq, hkv, page, dtype, tree):
    c = attention_case(len(prefixes) + sum(nodes) + hq, prefixes, nodes, hq, hkv, page, dtype, tree)
    check_attention(c, run_attention(c), reference(c))


@pytest.mark.parametrize("nodes,dtype", [([1, 1], "bf16"), ([20, 64], "fp16")])
def test_attention_scale_and_sharp_scores(nodes, dtype):
    """A given scale, and scores so large that one key takes nearly all of the weight."""
    c = attention_case(11, [190, 70], nodes, 4, 2, 32, dtype, gain=3.0)
    check_attention(c, run_attention(c, scale=0.31), reference(c, 0.31))


@pytest.mark.parametrize("nodes", [[1, 1], [30, 100]])
def test_attention_page_scales_far_apart(nodes):
    """Scales of neighbouring pages from 2^-30 to 2^7: keys and values of very unlike size in one tile."""
    c = attention_case(12, [150, 64], nodes, 4, 1, 16, "bf16")
    g = np.random.default_rng(4)
    c["exps"][0] = 127 + g.integers(-30, -5, c["exps"][0].shape)
    c["exps"][1] = 127 + g.integers(-30, 8, c["exps"][1].shape)
    c["cache"].exps[0] = torch.from_numpy(c["exps"])
    check_attention(c, run_attention(c), reference(c))


@pytest.mark.parametrize("nodes,hq,hkv", [([1, 1, 1], 8, 2), ([3, 40, 1], 8, 2), ([61, 61, 10], 4, 1)])
def test_attention_strides_and_untouched_rows(nodes, hq, hkv):
    """Columns of one wide activation as q, k and v; out with a wider row; rows behind the last entry stay."""
    c = attention_case(13, [100, 300, 7], nodes, hq, hkv, 64, "bf16")
    T = sum(nodes)
    wide = torch.zeros(T + 5, hq + 2 * hkv, 128, dtype=torch.bfloat16, device="cuda")
    wide[:T, :hq], wide[:T, hq:hq + hkv], wide[:T, hq + hkv:] = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    out = torch.full((T + 5, hq + 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 5, hq), 7.0, device="cuda")
    parents = i32(np.concatenate([c["parents"], [5, -1, 1 << 30, -9, 0]]))
    got = run_attention(c, q=wide[:, :hq], k_new=wide[:, hq:hq + hkv], v_new=wide[:, hq + hkv:], parents=parents,
                        out=out[:, :hq], lse=lse)
    assert got[0].data_ptr() == out.data_ptr()
    check_attention(c, (out[:T, :hq], lse[:T]), reference(c))
    assert (out[T:] == 7).all() and (out[:, hq:] == 7).all() and (lse[T:] == 7).all()


@pytest.mark.parametrize("nodes,hq", [([1, 1, 1, 1], 4), ([20, 30, 40, 50], 4)])
def test_attention_bad_descriptions_reach_no_other_entry(nodes, hq):
    """A page id outside the cache reads as NaN; entries out of range are left as they were."""
    c = attention_case(14, [100, 90, 80, 70], nodes, hq, 1, 32, "fp16")
    ref = reference(c)
    c["tables"][c["ids"][1], 1] = 1 << 30
    c["lengths"][c["ids"][2]] = 101  # above max_prefix
    ids = c["ids"].copy()
    ids[3] = 99
    T = sum(nodes)
    out = torch.full((T, hq, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, hq), 7.0, device="cuda")
    run_attention(c, seq_ids=i32(ids), out=out, lse=lse)
    o = c["offsets"]
    check_attention(c, (out[:o[1]], lse[:o[1]]), [x[:o[1]] for x in ref])
    assert torch.isnan(out[o[1]:o[2]]).all() and torch.isnan(lse[o[1]:o[2]]).all()
    assert (out[o[2]:] == 7).all() and (lse[o[2]:] == 7).all()


@pytest.mark.parametrize("n", [5, 61, 128])
def test_attention_nonfinite_values_reach_only_the_rows_that_see_them(n):
    c = attention_case(15, [70], [n], 4, 1, 64, "bf16")
    c["v"][3, 0, 5], c["v"][3, 0, 6], c["v"][4, 0, 7] = math.inf, math.nan, -math.inf
    c["k"][2, 0, 9] = math.nan
    got = run_attention(c)
    ref = reference(c)
    out, want = got[0].double().cpu().numpy(), ref[0]
    assert np.array_equal(np.isnan(out), np.isnan(want))
    assert np.array_equal(np.isinf(out), np.isinf(want)) and (out[np.isinf(want)] == want[np.isinf(want)]).all()
    fine = np.isfinite(want).all(axis=2)
    assert fine.any() and not fine.all()
    check_attention(c, (got[0].double().cpu()[torch.from_numpy(fine)][None], got[1].double().cpu()[torch.from_numpy(fine)][None]),
                    [x[fine][None] for x in ref])
    part = np.isfinite(want) & ~fine[..., None] & np.isfinite(ref[1])[..., None]  # the other dimensions of such rows
    assert np.allclose(out[part], want[part], rtol=0.02, atol=0.02)


@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("nodes", [[3, 2], [61, 30]])
def test_attention_nan_page_reaches_its_sequence_and_head_only(plane, nodes):
    c = attention_case(16, [70, 70], nodes, 4, 2, 16, "fp16")
    c["exps"][plane, c["tables"][c["ids"][0], 2], 1] = 255
    c["cache"].exps[0] = torch.from_numpy(c["exps"])
    got, ref = run_attention(c), reference(c)
    out, n = got[0].double().cpu().numpy(), nodes[0]
    assert np.isnan(ref[0][:n, 2:]).all() and np.isnan(out[:n, 2:]).all()
    assert not np.isnan(out[:n, :2]).any() and not np.isnan(out[n:]).any()
    check_attention(c, (got[0][n:], got[1][n:]), [x[n:] for x in ref])
    check_attention(c, (got[0][:n, :2], got[1][:n, :2]), [x[:n, :2] for x in ref])


@pytest.mark.parametrize("B,hkv", [(20, 8), (128, 2), (130, 2)])
def test_attention_of_more_row_tiles_than_sms(B, hkv):
    """Ragged batches whose tiles are started by length (up to 128 entries) or in order; equal lengths, no rows and no
    prefix among them; one entry out of range and one whose length is above max_prefix stay as they were."""
    g = np.random.default_rng(18)
    prefixes = [int(x) for x in g.choice([0, 1, 30, 64, 65, 130], B)]
    prefixes[7] = 131
    nodes = [int(x) for x in g.choice([0, 9, 17, 20], B)]
    nodes[3], nodes[7], nodes[9] = 20, 9, 17
    c = attention_case(19, prefixes, nodes, 2 * hkv, hkv, 32, "bf16")
    ref = reference(c)
    ids = c["ids"].copy()
    ids[9] = -1
    T, o = sum(nodes), c["offsets"]
    out = torch.full((T, 2 * hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 2 * hkv), 7.0, device="cuda")
    run_attention(c, seq_ids=i32(ids), out=out, lse=lse, max_prefix=130)
    left = np.zeros(T, bool)
    for b in (7, 9):
        left[o[b]:o[b + 1]] = True
    rest = torch.from_numpy(~left).cuda()
    assert (out[~rest] == 7).all() and (lse[~rest] == 7).all()
    check_attention(c, (out[rest], lse[rest]), [x[~left] for x in ref])


@pytest.mark.parametrize("nodes,prefix,dtype", [(17, 100, "fp16"), (34, 700, "bf16"), (9, 260, "bf16")])
def test_attention_with_idle_warps_repeats(nodes, prefix, dtype):
    """Tiles whose last rows are empty, so that some warps have nothing to do between the barriers: 300 calls in a row
    give the first one's results, which are right."""
    c = attention_case(20, [prefix] * 40, [nodes] * 40, 8, 2, 64, dtype)
    T = 40 * nodes
    first = run_attention(c)
    check_attention(c, first, reference(c))
    out, lse = torch.empty_like(first[0]), torch.empty(T, 8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    ws = c["cache"].attention_workspace(40, 8, c["nodes"], c["prefix"])
    for _ in range(300):
        run_attention(c, out=out, lse=lse, workspace=ws)
        wrong += (out != first[0]).any() | (lse != first[1]).any()
    assert int(wrong) == 0


@pytest.mark.parametrize("prefixes,nodes,bound", [([0, 0, 70], [20, 17, 30], 70), ([0], [40], 20000),
                                                  ([65, 0, 1], [33, 18, 17], 6000)])
def test_attention_of_tiles_without_units(prefixes, nodes, bound):
    """No prefix and no rows of its own, alone and beside tiles that have some; shares of a cluster's bound of which only
    the first holds keys.  Again and again, so that a CTA follows another one in the same shared memory."""
    c = attention_case(25, prefixes, nodes, 8, 2, 64, "bf16", "none")
    blocks = -(-bound // 64)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, max(0, blocks - c["tables"].shape[1]))), constant_values=-1)
    first, ref = run_attention(c, max_prefix=bound), reference(c)
    check_attention(c, first, ref)
    for _ in range(50):
        again = run_attention(c, max_prefix=bound)
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_refusals_of_the_torch_side():
    c = attention_case(17, [40], [2], 4, 2, 16, "bf16")
    cache, q = c["cache"], c["q"].cuda()
    with pytest.raises(ValueError):
        run_attention(c, q=q.float())
    with pytest.raises(ValueError):
        run_attention(c, q=q.cpu())
    with pytest.raises(ValueError):
        run_attention(c, v_new=None)
    with pytest.raises(ValueError):
        run_attention(c, k_new=c["k"].half().cuda())
    with pytest.raises(ValueError):
        run_attention(c, out=torch.empty(2, 4, 256, dtype=torch.bfloat16, device="cuda")[..., ::2])
    with pytest.raises(S.SpecError):
        run_attention(c, max_nodes=129)
    with pytest.raises(S.SpecError):
        run_attention(c, max_prefix=1 << 20)
    with pytest.raises(S.SpecError):
        run_attention(c, q=torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        cache.append(0, c["k"].cuda(), c["v"].cuda(), torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cache.append(0, c["k"].cuda(), c["v"].float().cuda(), i32([0, 1]))
    with pytest.raises(S.SpecError):
        cache.append(1, c["k"].cuda(), c["v"].cuda(), i32([0, 1]))
    with pytest.raises(S.SpecError):
        cache.append(0, c["k"].cuda(), c["v"].cuda(), i32([0, 1, 2]))
    with pytest.raises(ValueError):
        cache.plan(i32([0]), i32([1]), i32([[0]]), i32([0]), i32([0, 1]), 4)  # the ring holds every page


def test_workspace_serves_calls_of_other_bounds():
    """One workspace, used for many sequences, then for few, then for many: the counters are where every call looks."""
    big = attention_case(21, [700 + 5 * i for i in range(20)], [1] * 20, 4, 2, 32, "bf16")
    small = attention_case(22, [1500, 3], [2, 1], 4, 1, 64, "bf16")
    ws = big["cache"].attention_workspace(64, 8, 4, 4096)
    refs = [reference(c) for c in (big, small)]
    for _ in range(3):
        for c, ref in zip((big, small), refs):
            check_attention(c, run_attention(c, workspace=ws), ref)
    with pytest.raises(S.SpecError):
        run_attention(big, workspace=ws[:1000])


@pytest.mark.parametrize("nodes", [[20, 3], [128, 40]])
def test_many_rows_with_a_bound_beyond_the_tensor_core_kernel(nodes):
    """max_prefix above what the cluster kernel numbers: the streaming kernel takes the rows in tiles."""
    c = attention_case(23, [200, 90], nodes, 4, 1, 128, "fp16")
    wide = np.full((c["tables"].shape[0], 4000), -1, np.int32)
    wide[:, :c["tables"].shape[1]] = c["tables"]
    c["tables"] = wide
    check_attention(c, run_attention(c, max_prefix=500000), reference(c))


def test_more_groups_than_one_launch_takes():
    """2500 sequences of 8 kv heads, long and short ones on shared pages, in chunks: several launches, one workspace."""
    c = attention_case(24, [4600, 130], [1, 1], 8, 8, 64, "bf16", extra_seqs=0, tree="none")
    reps = 1250
    order = np.concatenate([np.arange(2)] * reps)
    tables, lengths = c["tables"][c["ids"]][order], c["lengths"][c["ids"]][order]
    lengths[2::2] = 70  # the first of them long, the last too
    lengths[-2] = 4600
    q = c["q"].cuda()[torch.from_numpy(order).cuda()]
    out, lse = c["cache"].attention(0, q, i32(tables), i32(lengths), i32(np.arange(2 * reps + 1)), max_prefix=4600,
                                    max_nodes=1)
    ref = reference(c)
    check_attention(c, (out[:2], lse[:2]), ref)
    check_attention(c, (out[-2:], lse[-2:]), ref)
    assert torch.equal(out[1::2], out[1:2].expand(reps, -1, -1)) and torch.equal(lse[1::2], lse[1:2].expand(reps, -1))
    assert torch.equal(out[2:-2:2], out[2:3].expand(reps - 2, -1, -1))


@pytest.mark.parametrize("nodes", [1, 40])
def test_pages_beyond_32_bit_offsets(nodes):
    """A cache of more than 2^32 bytes a plane: its last pages, written, read and attended to."""
    from speculative_decoding_06_b200.kv8 import KV8Cache
    hkv, page, n_pages = 8, 64, 66000
    cache = KV8Cache(1, hkv, n_pages, page)
    assert cache.codes[0, 0].numel() > 1 << 32
    g = np.random.default_rng(nodes)
    P = 100
    k, v = (torch.from_numpy(g.normal(size=(P, hkv, 128))).to(torch.bfloat16) for _ in range(2))
    used = [n_pages - 1, n_pages - 3]
    slots = [used[j // page] * page + j % page for j in range(P)]
    cache.append(0, k.cuda(), v.cuda(), i32(slots))
    codes, exps = np.zeros((2, 2, hkv, page, 128), np.uint8), np.zeros((2, 2, hkv), np.uint8)
    O.append(codes, exps, page, k.double().numpy(), v.double().numpy(), list(range(P)))
    got = cache.codes[0][:, used].cpu().numpy()
    assert np.array_equal(got[:, 0], codes[:, 0]) and np.array_equal(got[:, 1, :, :P - page], codes[:, 1, :, :P - page])
    c = dict(cache=cache, codes=codes, exps=exps, page=page, dtype="bf16",
             q=torch.from_numpy(g.normal(size=(nodes, hkv, 128))).to(torch.bfloat16))
    out = cache.attention(0, c["q"].cuda(), i32([used]), i32([P]), i32([0, nodes]), max_prefix=P, max_nodes=nodes)
    check_attention(c, out, O.attention(codes, exps, page, c["q"].double().numpy(), np.array([[0, 1]]), [P], [0, nodes],
                                        128 ** -0.5))


def test_workspace_of_the_largest_bounds_serves_a_draining_batch():
    """A batch that shrinks, trees between plain steps: one workspace, made for the most of each bound and full of
    something else behind its zeros, for all of them."""
    ws = None
    for B, n, top in ((40, 20, 900), (40, 1, 900), (39, 1, 700), (7, 3, 900), (1, 1, 900), (1, 20, 64), (12, 2, 300)):
        g = np.random.default_rng(B)
        prefixes = [int(x) for x in g.integers(1, top + 1, B)]
        prefixes[-1] = top
        c = attention_case(26, prefixes, [n] * B, 8, 2, 32, "bf16")
        if ws is None:
            ws = c["cache"].attention_workspace(40, 8, 20, 900)
            ws[S.SPEC_KV8_WORKSPACE_ZERO:] = 0x7F
        check_attention(c, run_attention(c, workspace=ws), reference(c))


@pytest.mark.parametrize("nodes,hq", [([1, 2, 1, 2], 4), ([20, 30, 40, 50], 4), ([2, 2, 3, 1], 12)])
@pytest.mark.parametrize("given", ["none", "out", "lse"])
def test_new_outputs_hold_no_old_memory(nodes, hq, given):
    """Rows before and behind the entries of a new output are those of rows that see nothing, an entry out of range is
    NaN; buffers that the caller gives keep what they had."""
    c = attention_case(27, [100, 1500, 80, 70], nodes, hq, 2, 32, "bf16")
    T, o = sum(nodes), c["offsets"] + 3
    c["offsets"], c["parents"] = o, np.concatenate([[-1] * 3, c["parents"], [-1] * 4])
    ref = reference(dict(c, offsets=o - 3, parents=c["parents"][3:-4]))
    for name in ("q", "k", "v"):
        c[name] = torch.cat([c[name][:3], c[name], c[name][:4]])
    c["lengths"][c["ids"][2]] = 1501  # above max_prefix
    ids = c["ids"].copy()
    ids[0] = -1
    old = [torch.full((T + 7, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T + 7, hq), 7.0, device="cuda")]
    kw = dict(out=old[0]) if given == "out" else dict(lse=old[1]) if given == "lse" else {}
    if given != "out":
        old[0] = None  # (the allocator's next block of this size)
    if given != "lse":
        old[1] = None
    out, lse = run_attention(c, seq_ids=i32(ids), **kw)
    want_out, want_lse = torch.zeros(T + 7, device="cuda"), torch.full((T + 7,), -math.inf, device="cuda")
    for b in (0, 2):
        want_out[o[b]:o[b + 1]] = want_lse[o[b]:o[b + 1]] = math.nan
    if given == "out":
        want_out[:] = 7
    if given == "lse":
        want_lse[:] = 7
    for x, want in ((out.float(), want_out[:, None, None]), (lse, want_lse[:, None])):
        for lo, hi in ((0, o[1]), (o[2], o[3]), (o[4], T + 7)):
            assert torch.equal(torch.nan_to_num(x[lo:hi], nan=99.0), torch.nan_to_num(want[lo:hi], nan=99.0).expand_as(x[lo:hi]))
    for b in (1, 3):
        sl, rs = slice(o[b], o[b + 1]), slice(o[b] - 3, o[b + 1] - 3)
        check_attention(c, (out[sl], lse[sl]), [x[rs] for x in ref])


def test_attention_after_a_plan_that_did_not_fit():
    """Its offsets are all 0: no entry has rows, and the new outputs say that nothing was seen."""
    c = attention_case(28, [40, 9], [2, 30], 4, 2, 16, "fp16")
    out, lse = c["cache"].attention(0, c["q"].cuda(), i32(c["tables"]), i32(c["lengths"]), i32([0, 0, 0]), max_prefix=40,
                                    max_nodes=30, seq_ids=i32(c["ids"]))
    assert not out.any() and (lse == -math.inf).all()
    out, lse = c["cache"].attention(0, c["q"].cuda(), i32(c["tables"]), i32(c["lengths"]), i32([0, 0, 0]), max_prefix=40,
                                    max_nodes=1, seq_ids=i32(c["ids"]))
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("nodes,hkv", [(1, 1), (3, 1), (1, 2)])
def test_strides_of_dimensions_of_one_do_not_matter(nodes, hkv):
    """One head, or one row: what stride that dimension has is never used."""
    c = attention_case(29, [70], [nodes], hkv, hkv, 32, "bf16")
    if hkv == 1:
        odd = lambda t: t.cuda().as_strided((nodes, 1, 128), (128, 3, 1))  # noqa: E731
        out = torch.empty(1, nodes, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        odd = lambda t: t.cuda().as_strided((1, hkv, 128), (5, 128, 1))  # noqa: E731
        out = torch.empty(hkv, 1, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got = run_attention(c, q=odd(c["q"]), k_new=odd(c["k"]), v_new=odd(c["v"]), out=out)
    assert got[0].data_ptr() == out.data_ptr()
    check_attention(c, got, reference(c))
    one = make_cache(4, hkv, 32, garbage=0)
    two = make_cache(4, hkv, 32, garbage=0)
    one.append(0, c["k"].cuda(), c["v"].cuda(), i32(np.arange(nodes) + 64))
    two.append(0, odd(c["k"]), odd(c["v"]), i32(np.arange(nodes) + 64))
    assert torch.equal(one.codes, two.codes) and torch.equal(one.exps, two.exps)


def plain64(cache, table, P, q, k, v):
    """Attention of a chain's rows over one kv head's prefix in 64 bits on the GPU: (out, lse, mass, score size)."""
    pages = table[:-(-P // cache.page)].long()
    kv = []
    for plane in (0, 1):
        x = cache.codes[0, plane, pages, 0].view(torch.float8_e4m3fn).double()
        x *= torch.exp2(cache.exps[0, plane, pages, 0].double() - 127)[:, None, None]
        kv.append(torch.cat([x.reshape(-1, 128)[:P], (k, v)[plane][:, 0].double()]))
    n, hq = q.shape[:2]
    s = torch.einsum("nhd,kd->nhk", q.double(), kv[0]) * 128 ** -0.5
    see = torch.arange(P + n, device="cuda")[None, :] <= P + torch.arange(n, device="cuda")[:, None]
    s.masked_fill_(~see[:, None, :], -math.inf)
    p = torch.softmax(s, 2)
    size = torch.einsum("nhd,kd->nhk", q.double().abs(), kv[0].abs()).amax(2) * 128 ** -0.5
    return [x.cpu().numpy() for x in (p @ kv[1], torch.logsumexp(s, 2), p @ kv[1].abs(), size)]


@pytest.mark.parametrize("P,bound,copies,n,hq,page", [
    (49100, 49152, 160, 9, 2, 64),     # a CTA per tile, as many units as a CTA takes
    (100, 100000, 1, 30, 4, 16), (100000, 100000, 2, 5, 4, 128),  # bounds that need a cluster
    (393206, 393216, 1, 9, 2, 64),     # shares as long as they can be
    (65, 393216, 3, 20, 1, 32), (70000, 393216, 1, 17, 1, 16)])
def test_long_prefixes_of_trees(P, bound, copies, n, hq, page):
    g = torch.Generator(device="cuda").manual_seed(P)
    blocks = -(-bound // page)
    used = -(-P // page)
    cache = make_cache(used + 3, 1, page, garbage=0x7F)
    table = torch.randperm(used + 3, generator=g, device="cuda")[:used].to(torch.int32)
    x = torch.randint(0, 118, (1, 2, used + 3, 1, page, 128), generator=g, device="cuda", dtype=torch.uint8)
    x += 128 * torch.randint(0, 2, x.shape, generator=g, device="cuda", dtype=torch.uint8)
    if P % page:
        x[0, :, table[-1].long(), :, P % page:] = 0x7F
    cache.codes.copy_(x)
    cache.exps.copy_(120 + torch.randint(-2, 3, cache.exps.shape, generator=g, device="cuda"))
    tables = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    tables[0, :used] = table
    q, k, v = (torch.randn(n, h, 128, device="cuda", generator=g).half() for h in (hq, 1, 1))
    many = lambda t: t.repeat(copies, 1, 1)  # noqa: E731
    out, lse = cache.attention(0, many(q), tables, i32([P]), i32(np.arange(copies + 1) * n), max_prefix=bound, max_nodes=n,
                               k_new=many(k), v_new=many(v), seq_ids=i32([0] * copies))
    ref = plain64(cache, table, P, q, k, v)
    # beyond the bound for 2^14 keys: sums in 32 bits, one after the other, of four products for each unit of 64 keys
    ref[3] = ref[3] + 4 * (P / 64) * 2.0 ** -23 / (2 * 130 * 2.0 ** -24)
    check_attention(dict(dtype="fp16"), (out[:n], lse[:n]), ref)
    assert torch.equal(out, many(out[:n])) and torch.equal(lse, lse[:n].repeat(copies, 1))
