"""Attention over the 8-bit paged cache where sizes lie far apart: pages, the step's own rows, rows of q.

The bounds are those of the attention tests: each score's error follows from that key's own products, the probabilities
are rounded once, and what a row does not see, or sees with a weight of 2^-60, has no part in its result."""

import numpy as np
import pytest
import torch

from oracle import kv8 as O
from test_gpu_kv8 import attention_case, check_attention, i32, reference, run_attention

pytestmark = pytest.mark.gpu


def set_exps(c, plane, table):
    """Exponent bytes of each sequence's pages, in the order of its tokens."""
    for b, s in enumerate(c["ids"]):
        for j in range(-(-int(c["lengths"][s]) // c["page"])):
            c["exps"][plane, c["tables"][s, j]] = table(b, j)
    c["cache"].exps[0] = torch.from_numpy(c["exps"])


def infinite_beyond_the_type(out, ref):
    """448 * 2^120 is above the largest bf16, 2^128 (1 - 2^-8): rounding to nearest gives that one up to 2^128 (1 - 2^-9)
    and infinity from there on.  A value beyond this border by more than its bound has to be infinite, one that the bound
    lets lie on either side may be; both are taken out of what is compared."""
    got, edge = out.double().cpu().numpy(), 2.0 ** 128 * (1 - 2.0 ** -9)
    off = (2.0 ** -8 + 2.0 ** -11 + 2 * 130 * 2.0 ** -24 * ref[3] + 2.0 ** -18)[..., None] * ref[2]  # before the last rounding
    inf = np.isinf(got) & (np.sign(got) == np.sign(ref[0])) & (np.abs(ref[0]) + off >= edge)
    assert inf[np.abs(ref[0]) - off > edge].all()
    out[torch.from_numpy(inf).cuda()], ref[0][inf] = 0, 0


@pytest.mark.parametrize("high", [150, 190, 247])
@pytest.mark.parametrize("order", ["small first", "large first", "in turn", "page by page"])
@pytest.mark.parametrize("prefixes,nodes,hq,page,dtype", [
    ([200, 77], [1, 1], 4, 16, "bf16"), ([3000], [1], 4, 64, "bf16"), ([900, 130], [3, 2], 4, 32, "bf16"),
    ([300, 190], [30, 100], 4, 64, "bf16"), ([3000], [40], 8, 64, "bf16"), ([500], [17], 2, 128, "bf16"),
    ([300, 61], [30, 100], 4, 16, "bf16"), ([1000], [40], 4, 32, "bf16")])
def test_weights_of_pages_whose_values_are_of_unlike_size(prefixes, nodes, hq, page, dtype, order, high):
    """V pages at the least scale (all zeros have it) beside very large ones: the weights do not depend on V."""
    c = attention_case(31, prefixes, nodes, hq, 1, page, dtype)
    blocks = [-(-p // page) for p in prefixes]
    # (in turn: no two scales within 64 keys)
    large = {"small first": lambda b, j: 2 * j >= blocks[b], "large first": lambda b, j: 2 * j < blocks[b],
             "in turn": lambda b, j: j * page // 64 % 2 == 1, "page by page": lambda b, j: j % 2 == 1}[order]
    if page < 64 and order != "page by page":  # whole units of 64 keys
        was = large
        large = lambda b, j: was(b, j // (64 // page) * (64 // page))  # noqa: E731
    set_exps(c, 1, lambda b, j: high if large(b, j) else 67)
    (out, lse), ref = run_attention(c), reference(c)
    infinite_beyond_the_type(out, ref)
    check_attention(c, (out, lse), ref)


def drop_pages(c, keep):
    """The same sequences without the pages for which keep(b, j) is false (their weights are below 2^-60)."""
    r = dict(c, tables=c["tables"].copy(), lengths=c["lengths"].copy())
    for b, s in enumerate(c["ids"]):
        P, page = int(c["lengths"][s]), c["page"]
        used = [j for j in range(-(-P // page)) if keep(b, j)]
        r["tables"][s, :len(used)] = c["tables"][s, used]
        r["lengths"][s] = sum(min(page, P - page * j) for j in used)
    return r


# prefixes of whole pages but for the last, which is kept
MIXED = [([64], [1], 4, 16, "bf16"), ([150, 64], [1, 3], 4, 16, "fp16"), ([150, 64], [30, 100], 4, 16, "bf16"),
         ([128, 331], [20, 17], 2, 32, "fp16"), ([1000], [40], 4, 16, "bf16")]


@pytest.mark.parametrize("gap", [9, 15, 16, 23, 25, 30, 60])
@pytest.mark.parametrize("prefixes,nodes,hq,page,dtype", MIXED)
def test_values_of_a_small_page_that_has_the_weight(prefixes, nodes, hq, page, dtype, gap):
    """Every other page holds V that is 2^gap larger, at keys whose scores are some 95 powers of two lower."""
    c = attention_case(32, prefixes, nodes, hq, 1, page, dtype, tree="none")
    keep = lambda b, j: j % 2 == (-(-prefixes[b] // page) - 1) % 2  # noqa: E731  (the last page is a small one)
    set_exps(c, 0, lambda b, j: 127 - 8)
    set_exps(c, 1, lambda b, j: 127 - 8 + (0 if keep(b, j) else gap))
    for b, s in enumerate(c["ids"]):
        for j in range(-(-prefixes[b] // page)):
            c["codes"][0, c["tables"][s, j], :, :, 0] = 0x77 if keep(b, j) else 0xF7  # K's first dimension: 240 or -240
    c["cache"].codes[0] = torch.from_numpy(c["codes"])
    c["q"][..., 0] = 400.0
    check_attention(c, run_attention(c), reference(drop_pages(c, keep)))


@pytest.mark.parametrize("gap", [9, 15, 16, 23, 25, 30, 60])
@pytest.mark.parametrize("prefixes,nodes,hq,page,dtype", MIXED)
def test_keys_of_a_small_page_beside_large_ones(prefixes, nodes, hq, page, dtype, gap):
    """Every other page holds K that is 2^gap larger, all of its scores far below the others'."""
    c = attention_case(33, prefixes, nodes, hq, 1, page, dtype, tree="none")
    keep = lambda b, j: j % 2 == (-(-prefixes[b] // page) - 1) % 2  # noqa: E731
    set_exps(c, 0, lambda b, j: 127 - 8 + (0 if keep(b, j) else gap))
    set_exps(c, 1, lambda b, j: 127 - 8)
    for b, s in enumerate(c["ids"]):
        for j in range(-(-prefixes[b] // page)):
            if not keep(b, j):
                c["codes"][0, c["tables"][s, j]] = 0
                c["codes"][0, c["tables"][s, j], :, :, 0] = 0xF7
    c["codes"][0, :, :, :, 0] = np.where(c["codes"][0, :, :, :, 0] == 0xF7, 0xF7, 0)  # else 0 where q is large
    c["cache"].codes[0] = torch.from_numpy(c["codes"])
    c["q"][..., 0] = 400.0
    check_attention(c, run_attention(c), reference(drop_pages(c, keep)))


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("size", [2.0 ** 13, 1e9, 1e30])
@pytest.mark.parametrize("prefixes,nodes,hq", [([70], [4], 4), ([70, 0], [61, 20], 4), ([33], [128], 2), ([0], [17], 2)])
def test_large_rows_reach_only_the_rows_that_see_them(prefixes, nodes, hq, size, which):
    """One of the step's own rows, which no other row sees, is very large but finite: the others' results stay."""
    c = attention_case(34, prefixes, nodes, hq, 1, 32, "bf16")
    off, big = c["offsets"], []
    for b, n in enumerate(nodes):
        for leaf in (1, n - 1):  # no row's parent any more
            at = off[b] + leaf
            for j in range(off[b], off[b + 1]):
                if c["parents"][j] == leaf:
                    c["parents"][j] = 0
            big.append(at)
    fine = np.ones(sum(nodes), bool)
    fine[big] = False
    ref = reference(c)  # (the rows that do not see them have the same result without)
    for at in big:
        for name in ("k", "v"):
            if which in (name, "both"):
                c[name][at] = (c[name][at].float() * size).to(c[name].dtype)
    out, lse = run_attention(c)
    rows = torch.from_numpy(fine).cuda()
    check_attention(c, (out[rows], lse[rows]), [x[fine] for x in ref])


@pytest.mark.parametrize("nodes", [[3], [61], [128]])
def test_rows_of_every_size(nodes):
    """K and V of each node of its own size, 2^-40 to 2^40: every row is right to within its own weights."""
    c = attention_case(35, [90], nodes, 4, 1, 64, "bf16")
    g = np.random.default_rng(5)
    c["v"] = (c["v"].float() * torch.exp2(torch.from_numpy(g.integers(-40, 41, (nodes[0], 1, 1)))).float()).to(torch.bfloat16)
    c["k"] = (c["k"].float() * torch.exp2(torch.from_numpy(g.integers(-40, 1, (nodes[0], 1, 1)))).float()).to(torch.bfloat16)
    check_attention(c, run_attention(c), reference(c))


@pytest.mark.parametrize("prefixes,nodes,tree", [([70, 5], [2, 1], "tree"), ([70, 5], [61, 20], "tree"),
                                                 ([70, 3], [40, 33], "none"), ([0], [100], "chain")])
def test_scores_that_vanish(prefixes, nodes, tree):
    """q near 2^-100 and keys of the least scale: every score is 0, what a row does not see stays out of it."""
    c = attention_case(36, prefixes, nodes, 4, 1, 16, "bf16", tree)
    c["q"] = (c["q"].float() * 2.0 ** -100).to(torch.bfloat16)
    set_exps(c, 0, lambda b, j: 67)
    check_attention(c, run_attention(c), reference(c))
    check_attention(c, run_attention(c, scale=1e-38), reference(c, 1e-38))


@pytest.mark.parametrize("nodes", [1, 3, 40])
def test_small_rows_of_q_over_keys_near_the_largest_float(nodes):
    """Scores of ordinary size whose factors are far from it, in the step's own rows and in the prefix."""
    c = attention_case(37, [40], [nodes], 4, 1, 16, "bf16", "chain")
    c["k"] = (c["k"].float() * 2.0 ** 120).to(torch.bfloat16)
    set_exps(c, 0, lambda b, j: 127 + 112)
    c["q"] = (c["q"].float() * 2.0 ** -120).to(torch.bfloat16)
    check_attention(c, run_attention(c), reference(c))


@pytest.mark.parametrize("nodes", [1, 3, 40])
def test_the_largest_scores(nodes):
    """Scores up to 2^21, where those in 32 bits lie 2^-3 apart (in powers of two): the best key has the weight."""
    c = attention_case(38, [40], [nodes], 4, 1, 16, "bf16", "chain")
    ref = reference(c)
    gain = 2.0 ** np.floor(np.log2(2.0 ** 21 / ref[3].max()))
    c["q"] = (c["q"].float() * gain).to(torch.bfloat16)
    got, (out, lse, mass, size) = run_attention(c), reference(c)
    assert size.max() > 2.0 ** 20
    # a score is off by at most 2^-13 of its own size: keys further below the best one weigh nothing
    d = 2 * 130 * 2.0 ** -24 * size
    assert (np.abs(got[1].double().cpu().numpy() - lse) <= d + 1).all()
    sure = np.zeros(lse.shape, bool)
    for i in range(nodes):
        for h in range(4):
            codes = O.E4M3[c["codes"][0][c["tables"][c["ids"][0], :3], 0].reshape(-1, 128)[:40]]
            e = np.repeat(c["exps"][0][c["tables"][c["ids"][0], :3], 0].astype(float) - 127, 16)[:40]
            keys = np.concatenate([codes * 2.0 ** e[:, None], c["k"][:i + 1, 0].double().numpy()])
            s = np.sort(128 ** -0.5 * keys @ c["q"][i, h].double().numpy())
            sure[i, h] = s[-1] - s[-2] > 2 * d[i, h] + 30
    assert sure.any()
    o = got[0].double().cpu().numpy()
    assert (np.abs(o - out)[sure] <= 2.0 ** -8 * np.abs(out)[sure] + 2.0 ** -11 * mass[sure] + 1e-7).all()
    assert np.isfinite(o).all()


@pytest.mark.parametrize("nodes,hq", [([1] * 60, 64), ([40] * 3, 64)])
@pytest.mark.parametrize("k,v", [(106, 73), (108, 76), (106, 80), (119, 67), (108, 100), (108, 150)])
def test_log_sum_exp_of_small_scores(nodes, hq, k, v):
    """Scores near 0 over few keys, whatever V's scale: the log-sum-exp is right to a few steps of its own size."""
    c = attention_case(39, [2 + i % 9 for i in range(len(nodes))], nodes, hq, 1, 16, "bf16", "none")
    set_exps(c, 0, lambda b, j: k)
    set_exps(c, 1, lambda b, j: v)
    check_attention(c, run_attention(c), reference(c))
