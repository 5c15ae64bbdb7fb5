"""The 8-bit paged cache without a GPU: its oracle against closed forms, and every refusal of its entry points (all
arguments are checked before any work is queued; a call that passes them ends in SPEC_ERR_CUDA here)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8 as O
from speculative_decoding_06_b200 import spec as S


# ---------------------------------------------------------------- the oracle
def test_e4m3_codes_are_torch_float8():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.E4M3, want, equal_nan=True)


def test_encode_rounds_to_nearest_even_and_saturates():
    x = np.concatenate([np.linspace(-460, 460, 9001), 2.0 ** np.arange(-14, 9), [0.0, -0.0, 447.9, 2.0 ** -10]])
    want = torch.tensor(np.clip(x, -448, 448), dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.encode(np.float32(x)), want)
    assert O.encode([np.inf, -np.inf]).tolist() == [126, 254]
    assert O.E4M3[O.encode([np.nan])[0]] != O.E4M3[O.encode([np.nan])[0]]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (224.0, -1), (224.5, 0), (1.75, -8), (0.0, -60),
                                    (1e-30, -60), (3.4e38, 120), (65504.0, 8)])
def test_exponent(amax, e):
    assert O.exponent(amax) == e


def test_append_keeps_rescales_and_reopens():
    page = 16
    codes = np.full((2, 2, 1, page, 128), 0x7F, np.uint8)  # garbage: every code NaN
    exps = np.full((2, 2, 1), 255, np.uint8)
    one = np.ones((1, 1, 128))
    O.append(codes, exps, page, one * 448, one, [16])
    assert exps[0, 1, 0] == 127 and exps[1, 1, 0] == 127 - 8  # 448 = 448 * 2^0; 1 = 256 * 2^-8
    assert O.E4M3[codes[1, 1, 0, 0, 0]] == 256.0
    O.append(codes, exps, page, one * 4 * 448, one * 0.5, [17])
    assert exps[0, 1, 0] == 129 and O.E4M3[codes[0, 1, 0, 0, 0]] == 112.0  # the first token, in the larger scale
    assert exps[1, 1, 0] == 119 and O.E4M3[codes[1, 1, 0, 1, 0]] == 128.0  # a smaller one does not lower it
    O.append(codes, exps, page, one * 0, one * 0, [16])
    assert exps[0, 1, 0] == 127 - 60  # opened anew
    assert codes[0, 0].min() == 0x7F  # the other page stays


def test_plan_grow_shrink_and_transaction():
    tables = np.full((3, 4), -1, np.int32)
    ring = np.arange(8, dtype=np.int32)[::-1].copy()
    lengths, state = np.zeros(3, np.int32), np.array([6, 8], np.int32)
    off, slots, l2, st, status, t2, r2 = O.plan(lengths, [17, 0, 3], tables, ring, state, 16, 22)
    assert status == 0 and off.tolist() == [0, 17, 17, 20]
    assert t2[0, :2].tolist() == [1, 0] and t2[2, 0] == 7  # the ring from place 6, around its end
    assert slots[:17].tolist() == list(range(16, 32)) + [0] and slots[17:].tolist() == [112, 113, 114, -1, -1]
    assert l2.tolist() == [17, 0, 3] and st.tolist() == [1, 5]
    off, slots, l3, st3, status, t3, r3 = O.plan(l2, [-2, 40, -(1 << 30)], t2, r2, st, 16, 64)
    assert status == 0 and l3.tolist() == [15, 40, 0] and st3.tolist() == [4, 4]
    assert r3[6:8].tolist() == [0, 7]  # given back behind the five that were free
    for add, rows, bits in (([200, 0, 0], 300, 4 | 2), ([72, 0, 0], 300, 4), ([48, 48, 48], 300, 2), ([5, 0, 0], 4, 1)):
        out = O.plan(lengths, add, tables, ring, state, 16, rows)
        assert out[4] == bits and out[0].max() == 0 and out[1].max() == -1
        assert np.array_equal(out[2], lengths) and np.array_equal(out[5], tables) and np.array_equal(out[6], ring)
    assert O.plan(lengths, [1, 1], tables, ring, state, 16, 9, seq_ids=[1, 1])[4] == 8


def test_attention_is_softmax_over_the_ancestors():
    g = np.random.default_rng(1)
    page, codes = 16, g.integers(0, 120, (2, 3, 1, 16, 128), dtype=np.uint8)
    exps = np.full((2, 3, 1), 120, np.uint8)
    q, k, v = (g.normal(size=(4, h, 128)) for h in (2, 1, 1))
    out, lse, _, _ = O.attention(codes, exps, page, q, np.array([[2, 0]], np.int32), [20], [0, 4], 0.1, k, v,
                                 parents=[-1, 0, 0, 2])
    x = O.E4M3[codes[:, [2, 0], 0].reshape(2, 32, 128)[:, :20]] * 2.0 ** -7
    keys, vals = np.concatenate([x[0], k[[0, 2, 3], 0]]), np.concatenate([x[1], v[[0, 2, 3], 0]])
    s = torch.tensor(0.1 * keys @ q[3, 1])
    assert np.allclose(torch.softmax(s, 0).numpy() @ vals, out[3, 1], atol=1e-12)
    assert np.isclose(torch.logsumexp(s, 0).item(), lse[3, 1])
    out, lse, _, _ = O.attention(codes, exps, page, q, np.array([[2, 0]], np.int32), [0], [0, 4], 0.1)
    assert not out.any() and np.all(lse == -np.inf)


# ---------------------------------------------------------------- refusals
def config(**kw):
    c = dict(n_layers=2, n_kv_heads=4, head_dim=128, page=64, n_pages=10)
    c.update(kw)
    return S.spec_kv8_config(**c)


@pytest.mark.parametrize("kw", [dict(n_layers=0), dict(n_kv_heads=0), dict(head_dim=64), dict(page=8), dict(page=48),
                                dict(page=256), dict(n_pages=0), dict(n_pages=1 << 25)])
def test_bad_configurations(kw):
    c = config(**kw)
    assert S.spec_kv8_code_bytes(ctypes.byref(c)) == 0 and S.spec_kv8_exp_bytes(ctypes.byref(c)) == 0
    h = ctypes.c_void_p()
    assert S.spec_kv8_open(ctypes.byref(c), 1 << 20, 1 << 40, 1 << 21, 1 << 40, ctypes.byref(h)) == S.SPEC_ERR_ARG


def test_sizes_and_open():
    c = config()
    assert S.spec_kv8_code_bytes(ctypes.byref(c)) == 2 * 2 * 10 * 4 * 64 * 128
    assert S.spec_kv8_exp_bytes(ctypes.byref(c)) == 2 * 2 * 10 * 4
    h = ctypes.c_void_p()
    n, m = S.spec_kv8_code_bytes(ctypes.byref(c)), S.spec_kv8_exp_bytes(ctypes.byref(c))
    for codes, nb, exps, mb, rc in ((None, n, 1 << 21, m, S.SPEC_ERR_ARG), (1 << 20, n, None, m, S.SPEC_ERR_ARG),
                                    ((1 << 20) + 64, n, 1 << 21, m, S.SPEC_ERR_ARG),
                                    (1 << 20, n - 1, 1 << 21, m, S.SPEC_ERR_CAPACITY),
                                    (1 << 20, n, 1 << 21, m - 1, S.SPEC_ERR_CAPACITY)):
        assert S.spec_kv8_open(ctypes.byref(c), codes, nb, exps, mb, ctypes.byref(h)) == rc
        assert not h.value
    assert S.spec_kv8_open(ctypes.byref(c), 1 << 20, n, 1 << 21, m, None) == S.SPEC_ERR_ARG
    assert S.spec_kv8_plan(None, None, None) == S.SPEC_ERR_ARG
    assert S.spec_kv8_append(None, 0, None, None) == S.SPEC_ERR_ARG
    assert S.spec_kv8_attention(None, 0, None, None) == S.SPEC_ERR_ARG
    assert S.spec_kv8_last_error(None) == b""


@pytest.fixture
def handle():
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: this one runs where no GPU could be reached")
    c, h = config(), ctypes.c_void_p()
    assert S.spec_kv8_open(ctypes.byref(c), 1 << 20, 1 << 40, 1 << 21, 1 << 40, ctypes.byref(h)) == S.SPEC_OK
    yield h
    S.spec_kv8_close(h)


def ptrs(*names):
    return {n: 4096 * (i + 1) for i, n in enumerate(names)}


PLAN = dict(ptrs("lengths", "add", "seq_ids", "tables", "ring", "state", "offsets", "slots", "lengths_out", "state_out",
                 "status"), batch=4, n_seqs=6, max_blocks=8, max_rows=100)
APPEND = dict(ptrs("k", "v", "slots", "src_rows"), k_row_stride=512, k_head_stride=128, v_row_stride=512,
              v_head_stride=128, dtype=S.SPEC_DTYPE_BF16, rows=5, n_src=9)
ATTN = dict(ptrs("q", "k_new", "v_new", "parents", "offsets", "tables", "lengths", "seq_ids", "out", "lse",
                 "workspace"), workspace_bytes=1 << 40, q_row_stride=1024, q_head_stride=128, k_row_stride=512,
            k_head_stride=128, v_row_stride=512, v_head_stride=128, out_row_stride=1024, dtype=S.SPEC_DTYPE_BF16,
            batch=4, n_seqs=6, max_blocks=8, n_q_heads=8, rows=20, max_nodes=16, max_prefix=512, scale=0.0)


@pytest.mark.parametrize("kw,rc", [
    ({}, S.SPEC_ERR_CUDA), (dict(seq_ids=None), S.SPEC_ERR_CUDA), (dict(max_rows=0, slots=None), S.SPEC_ERR_CUDA),
    *[({n: None}, S.SPEC_ERR_ARG) for n in ("lengths", "add", "tables", "ring", "state", "offsets", "slots",
                                            "lengths_out", "state_out", "status")],
    (dict(batch=0), S.SPEC_ERR_ARG), (dict(n_seqs=0), S.SPEC_ERR_ARG), (dict(max_blocks=0), S.SPEC_ERR_ARG),
    (dict(max_rows=-1), S.SPEC_ERR_ARG), (dict(seq_ids=None, batch=7), S.SPEC_ERR_ARG),
    (dict(batch=8193), S.SPEC_ERR_CAPACITY), (dict(n_seqs=65537), S.SPEC_ERR_CAPACITY),
    (dict(max_blocks=1 << 25), S.SPEC_ERR_CAPACITY)])
def test_plan_refusals(handle, kw, rc):
    a = S.spec_kv8_plan_args(**{**PLAN, **kw})
    assert S.spec_kv8_plan(handle, ctypes.byref(a), None) == rc
    assert S.spec_kv8_last_error(handle)
    assert S.spec_kv8_plan(handle, None, None) == S.SPEC_ERR_ARG


@pytest.mark.parametrize("layer,kw,rc", [
    (0, {}, S.SPEC_ERR_CUDA), (1, dict(dtype=S.SPEC_DTYPE_F32), S.SPEC_ERR_CUDA),
    (0, dict(rows=0, k=None, v=None, slots=None), S.SPEC_OK), (2, {}, S.SPEC_ERR_ARG), (-1, {}, S.SPEC_ERR_ARG),
    (0, dict(rows=-1), S.SPEC_ERR_ARG), (0, dict(n_src=-1), S.SPEC_ERR_ARG),
    (0, dict(src_rows=None, n_src=4), S.SPEC_ERR_ARG), (0, dict(src_rows=None, n_src=5), S.SPEC_ERR_CUDA),
    (0, dict(dtype=3), S.SPEC_ERR_ARG), (0, dict(k=4098), S.SPEC_ERR_ARG), (0, dict(v=8200), S.SPEC_ERR_ARG),
    (0, dict(k=None), S.SPEC_ERR_ARG), (0, dict(v=None), S.SPEC_ERR_ARG), (0, dict(slots=None), S.SPEC_ERR_ARG),
    (0, dict(k_row_stride=513), S.SPEC_ERR_ARG), (0, dict(v_head_stride=4), S.SPEC_ERR_ARG),
    (0, dict(dtype=S.SPEC_DTYPE_F32, v_head_stride=4), S.SPEC_ERR_CUDA), (0, dict(k_row_stride=-512), S.SPEC_ERR_ARG)])
def test_append_refusals(handle, layer, kw, rc):
    a = S.spec_kv8_append_args(**{**APPEND, **kw})
    assert S.spec_kv8_append(handle, layer, ctypes.byref(a), None) == rc
    assert S.spec_kv8_append(handle, layer, None, None) == S.SPEC_ERR_ARG


@pytest.mark.parametrize("layer,kw,rc", [
    (0, {}, S.SPEC_ERR_CUDA), (1, dict(scale=0.3, dtype=S.SPEC_DTYPE_F16), S.SPEC_ERR_CUDA),
    (0, dict(k_new=None, v_new=None, parents=None), S.SPEC_ERR_CUDA), (0, dict(lse=None), S.SPEC_ERR_CUDA),
    (0, dict(seq_ids=None), S.SPEC_ERR_CUDA), (0, dict(rows=0, q=None, out=None), S.SPEC_OK),
    (0, dict(max_prefix=0), S.SPEC_ERR_CUDA),
    (2, {}, S.SPEC_ERR_ARG), (0, dict(dtype=S.SPEC_DTYPE_F32), S.SPEC_ERR_ARG),
    *[(0, {n: None}, S.SPEC_ERR_ARG) for n in ("q", "out", "offsets", "tables", "lengths", "workspace")],
    (0, dict(k_new=None, parents=None), S.SPEC_ERR_ARG), (0, dict(v_new=None, parents=None), S.SPEC_ERR_ARG),
    (0, dict(k_new=None, v_new=None), S.SPEC_ERR_ARG),
    (0, dict(batch=0), S.SPEC_ERR_ARG), (0, dict(n_seqs=0), S.SPEC_ERR_ARG), (0, dict(rows=-1), S.SPEC_ERR_ARG),
    (0, dict(seq_ids=None, batch=7), S.SPEC_ERR_ARG), (0, dict(n_q_heads=6), S.SPEC_ERR_ARG),
    (0, dict(n_q_heads=4 * 65, out_row_stride=1 << 16), S.SPEC_ERR_CAPACITY),
    (0, dict(max_nodes=0), S.SPEC_ERR_CAPACITY), (0, dict(max_nodes=129), S.SPEC_ERR_CAPACITY),
    (0, dict(max_prefix=513), S.SPEC_ERR_CAPACITY), (0, dict(max_prefix=-1), S.SPEC_ERR_CAPACITY),
    (0, dict(max_blocks=1 << 25), S.SPEC_ERR_CAPACITY),
    (0, dict(scale=-1.0), S.SPEC_ERR_ARG), (0, dict(scale=float("nan")), S.SPEC_ERR_ARG),
    (0, dict(scale=float("inf")), S.SPEC_ERR_ARG),
    (0, dict(q=4100), S.SPEC_ERR_ARG), (0, dict(out=4104), S.SPEC_ERR_ARG), (0, dict(k_new=8200), S.SPEC_ERR_ARG),
    (0, dict(q_row_stride=1025), S.SPEC_ERR_ARG), (0, dict(q_head_stride=-128), S.SPEC_ERR_ARG),
    (0, dict(v_row_stride=4), S.SPEC_ERR_ARG), (0, dict(out_row_stride=1016), S.SPEC_ERR_ARG),
    (0, dict(workspace=4104), S.SPEC_ERR_ARG), (0, dict(workspace_bytes=0), S.SPEC_ERR_CAPACITY)])
def test_attention_refusals(handle, layer, kw, rc):
    a = S.spec_kv8_attention_args(**{**ATTN, **kw})
    assert S.spec_kv8_attention(handle, layer, ctypes.byref(a), None) == rc
    assert S.spec_kv8_attention(handle, layer, None, None) == S.SPEC_ERR_ARG


# ---------------------------------------------------------------- workspaces
def workspace(h, batch, n_q_heads, max_nodes, max_prefix):
    return S.spec_kv8_attention_workspace(h, batch, n_q_heads, max_nodes, max_prefix)


def test_workspace_grows_with_every_bound(handle):
    """A workspace made for a program's largest bounds is large enough for every call below them: fewer sequences, fewer
    nodes (the other kernel too), shorter prefixes (one chunk or many)."""
    g = np.random.default_rng(1)
    batches = sorted({1, 2, 46, 47, 64, 128, 255, 256, 512, 4096, 65535, *np.exp(g.uniform(0, 11, 20)).astype(int).tolist()})
    prefixes = sorted({0, 1, 128, 129, 1024, 2048, 2049, 4096, 4097, 131072, 393216, 393217,
                       *np.exp(g.uniform(0, 14, 40)).astype(int).tolist()})
    nodes = [1, 2, 3, 4, 5, 8, 9, 61, 128]
    size = np.array([[[workspace(handle, b, 8, n, p) for p in prefixes] for n in nodes] for b in batches], dtype=np.float64)
    assert size.min() >= 16
    for axis in range(3):
        assert (np.diff(size, axis=axis) >= 0).all()


@pytest.mark.parametrize("large,small", [
    ((47, 1, 4096), (46, 1, 4096)), ((64, 61, 4096), (64, 1, 4096)), ((256, 1, 2048), (128, 1, 2048)),
    ((512, 1, 1024), (8, 1, 1024)), ((1, 128, 200000), (1, 4, 131072)), ((2000, 1, 9000), (300, 2, 4100)),
    ((9000, 128, 393217), (9000, 8, 393216)), ((64, 16, 4096), (64, 15, 4000))])
def test_workspace_of_larger_bounds_serves_smaller_calls(handle, large, small):
    args = {**ATTN, "seq_ids": 4096, "max_blocks": 8192}
    for batch, nodes, prefix in (large, small):
        a = S.spec_kv8_attention_args(**{**args, "batch": batch, "max_nodes": nodes, "max_prefix": prefix,
                                         "workspace_bytes": workspace(handle, large[0], 8, large[1], large[2])})
        assert S.spec_kv8_attention(handle, 0, ctypes.byref(a), None) == S.SPEC_ERR_CUDA, S.spec_kv8_last_error(handle)


def test_workspace_of_random_bounds_serves_all_below_them(handle):
    g = np.random.default_rng(2)
    for _ in range(3000):
        large = [int(np.exp(g.uniform(0, np.log(top + 1)))) for top in (65535, 128, 500000)]
        small = [max(1, int(x * g.choice([1.0, 0.999, g.random(), np.exp(-8 * g.random())]))) for x in large]
        for hq in (4, 16, 64):
            a = S.spec_kv8_attention_args(**{**ATTN, "seq_ids": 4096, "max_blocks": 8192, "batch": small[0], "n_q_heads": hq,
                                             "max_nodes": small[1], "max_prefix": small[2], "out_row_stride": 8192,
                                             "workspace_bytes": workspace(handle, large[0], 64, large[1], large[2])})
            assert S.spec_kv8_attention(handle, 0, ctypes.byref(a), None) == S.SPEC_ERR_CUDA, (large, small, hq)


@pytest.mark.parametrize("fill,rc", [(0, S.SPEC_ERR_CUDA), (3, S.SPEC_ERR_CUDA), (4, S.SPEC_ERR_ARG), (-1, S.SPEC_ERR_ARG)])
def test_attention_fill_bits(handle, fill, rc):
    assert S.spec_kv8_attention(handle, 0, ctypes.byref(S.spec_kv8_attention_args(**{**ATTN, "fill": fill})), None) == rc


# ---------------------------------------------------------------- counts near 2^31
@pytest.mark.parametrize("rows,rc", [(1 << 30, S.SPEC_ERR_CUDA), ((1 << 30) + 1, S.SPEC_ERR_CAPACITY),
                                     ((1 << 31) - 100, S.SPEC_ERR_CAPACITY)])
def test_rows_that_32_bits_do_not_number(handle, rows, rc):
    """The kernels number rows in 32 bits, up to a grid's stride behind the last one."""
    a = S.spec_kv8_append_args(**{**APPEND, "rows": rows, "n_src": 9})
    assert S.spec_kv8_append(handle, 0, ctypes.byref(a), None) == rc
    a = S.spec_kv8_plan_args(**{**PLAN, "max_rows": rows})
    assert S.spec_kv8_plan(handle, ctypes.byref(a), None) == rc


def test_more_groups_than_32_bits_number():
    """65535 entries times 65535 kv heads: refused, where the number of row groups wrapped around and nothing was done."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    c, h = config(n_layers=1, n_kv_heads=65535, page=16, n_pages=1), ctypes.c_void_p()
    assert S.spec_kv8_open(ctypes.byref(c), 1 << 20, 1 << 40, 1 << 21, 1 << 40, ctypes.byref(h)) == S.SPEC_OK
    try:
        for batch, nodes, rc in ((16384, 1, S.SPEC_ERR_CUDA), (16385, 1, S.SPEC_ERR_CAPACITY), (65535, 1, S.SPEC_ERR_CAPACITY),
                                 (65535, 17, S.SPEC_ERR_CUDA)):  # (17 rows: the kernel of another grid)
            a = S.spec_kv8_attention_args(**{**ATTN, "n_q_heads": 65535, "out_row_stride": 65535 * 128, "batch": batch,
                                             "n_seqs": batch, "max_nodes": nodes, "max_blocks": 64, "max_prefix": 1000})
            assert S.spec_kv8_attention(h, 0, ctypes.byref(a), None) == rc
            assert (workspace(h, batch, 65535, nodes, 1000) == 0) == (rc == S.SPEC_ERR_CAPACITY)
    finally:
        S.spec_kv8_close(h)
