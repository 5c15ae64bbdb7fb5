"""Float64 / whole-number oracle of the 8-bit paged K/V cache: page plan, quantising append, attention.

Plain numpy over small cases, one sequence, run or row at a time; test infrastructure only, no code shared with the
library."""

from __future__ import annotations

import numpy as np

HD = 128
E_MIN, E_MAX, BIAS = -60, 120, 127

# what each of the 256 e4m3 codes stands for
_MAG = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(128)])
_MAG[127] = np.nan
E4M3 = np.concatenate([_MAG, -_MAG])


def encode(x):
    """Nearest e4m3 code, ties to the even code, saturating at 448; NaN to the NaN code."""
    x = np.asarray(x, np.float64)
    grid = _MAG[:127]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(amax):
    """The least e of [-60, 120] with amax <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def append(codes, exps, page, k, v, slots, src_rows=None):
    """Stores rows into codes [K, V][n_pages][hkv][page][128] and exps [K, V][n_pages][hkv], in place."""
    n_pages = codes.shape[1]
    rows = []
    for i, s in enumerate(slots):
        r = int(src_rows[i]) if src_rows is not None else i
        rows.append((int(s), r) if 0 <= s < n_pages * page and 0 <= r < len(k) else None)
    i = 0
    while i < len(rows):
        if rows[i] is None:
            i += 1
            continue
        j = i + 1
        while j < len(rows) and rows[j] is not None and rows[j][0] == rows[j - 1][0] + 1 and rows[j][0] % page:
            j += 1
        pg, place = divmod(rows[i][0], page)
        for plane, x in ((0, k), (1, v)):
            for h in range(codes.shape[2]):
                new = np.stack([np.asarray(x[r][h], np.float64) for _, r in rows[i:j]])
                if np.isnan(new).any() or (place and exps[plane, pg, h] == 255):
                    exps[plane, pg, h] = 255  # NaN: the codes are unspecified
                    continue
                e = exponent(np.max(np.abs(new), where=np.isfinite(new), initial=0.0))
                if place:
                    old = int(exps[plane, pg, h]) - BIAS
                    if e > old:
                        codes[plane, pg, h, :place] = encode(E4M3[codes[plane, pg, h, :place]] * 2.0 ** (old - e))
                    e = max(e, old)
                codes[plane, pg, h, place:place + j - i] = encode(new * 2.0 ** -e)
                exps[plane, pg, h] = e + BIAS
        i = j


def plan(lengths, add, tables, ring, state, page, max_rows, seq_ids=None):
    """Returns (offsets, slots, lengths, state, status, tables, ring); the inputs stay as they were."""
    n_seqs, max_blocks = tables.shape
    n_pages = len(ring)
    ids = list(range(len(add))) if seq_ids is None else [int(s) for s in seq_ids]
    lengths2, tables2, ring2 = lengths.copy(), tables.copy(), ring.copy()
    head, count = int(state[0]), int(state[1])
    status = 0
    if not (0 <= head < n_pages and 0 <= count <= n_pages):
        status |= 8
    offsets, slots, taken, given = [0], [], 0, []
    for b, s in enumerate(ids):
        if not 0 <= s < n_seqs or s in ids[:b] or not 0 <= lengths[s] <= max_blocks * page:
            status |= 8
            offsets.append(len(slots))
            continue
        cur = int(lengths[s])
        new = max(0, cur + int(add[b]))
        if new > max_blocks * page:
            status |= 4
        for pos in range(cur, new):
            if pos // page >= max_blocks:
                slots.append(0)
                taken += pos % page == 0
                continue
            if pos % page == 0:
                pg = int(ring[(head + taken) % n_pages]) if 0 <= head < n_pages else 0
                taken += 1
                tables2[s, pos // page] = pg
            slots.append(int(tables2[s, pos // page]) * page + pos % page)
        given += [int(tables[s, j]) for j in range(-(-new // page), -(-cur // page))]
        lengths2[s] = new
        offsets.append(len(slots))
    status |= (len(slots) > max_rows) * 1 | (taken > count) * 2 | (count + len(given) > n_pages) * 8
    if status:
        return (np.zeros(len(ids) + 1, np.int32), np.full(max_rows, -1, np.int32), lengths.copy(), state.copy(), status,
                tables.copy(), ring.copy())
    for j, pg in enumerate(given):
        ring2[(head + count + j) % n_pages] = pg
    slots = slots + [-1] * (max_rows - len(slots))
    return (np.array(offsets, np.int32), np.array(slots, np.int32), lengths2,
            np.array([(head + taken) % n_pages, count - taken + len(given)], np.int32), status, tables2, ring2)


def attention_row(q, keys, values, scale):
    """One row and head: (out, lse, sum of softmax |v|, largest scale * sum |q||k|) over the keys it sees."""
    if len(keys) == 0:
        return np.zeros(HD), -np.inf, np.zeros(HD), 0.0
    with np.errstate(all="ignore"):
        s = scale * (keys @ q)
        m = np.max(s)
        p = np.exp(s - m)
        w = p / p.sum()
        return (w @ values, m + np.log(p.sum()), w @ np.abs(values), scale * float(np.max(np.abs(keys) @ np.abs(q))))


def attention(codes, exps, page, q, tables, lengths, offsets, scale, k_new=None, v_new=None, parents=None,
              seq_ids=None):
    """All rows: (out, lse, sum of softmax |v|, score size), float64; codes [K, V][n_pages][hkv][page][128]."""
    rows, hq = q.shape[:2]
    hkv = codes.shape[2]
    out, mass = np.zeros((rows, hq, HD)), np.zeros((rows, hq, HD))
    lse, size = np.zeros((rows, hq)), np.zeros((rows, hq))
    for b in range(len(offsets) - 1):
        s = b if seq_ids is None else int(seq_ids[b])
        P, lo, hi = int(lengths[s]), int(offsets[b]), int(offsets[b + 1])
        n_pages = codes.shape[1]
        cached = []
        for plane in (0, 1):
            x = np.full((P, hkv, HD), np.nan)
            for j in range(P):
                pg = int(tables[s, j // page])
                if 0 <= pg < n_pages:
                    e = np.where(exps[plane, pg] == 255, np.nan, exps[plane, pg].astype(np.float64) - BIAS)
                    x[j] = E4M3[codes[plane, pg, :, j % page]] * (2.0 ** e)[:, None]
            cached.append(x)
        for i in range(hi - lo):
            seen, j = [], i
            while k_new is not None and j >= 0:
                seen.append(lo + j)
                up = j - 1 if parents is None else int(parents[lo + j])
                j = up if 0 <= up < j else -1
            for h in range(hq):
                g = h // (hq // hkv)
                keys, vals = cached[0][:, g], cached[1][:, g]
                if seen:
                    keys = np.concatenate([keys, k_new[seen, g].astype(np.float64)])
                    vals = np.concatenate([vals, v_new[seen, g].astype(np.float64)])
                out[lo + i, h], lse[lo + i, h], mass[lo + i, h], size[lo + i, h] = attention_row(
                    q[lo + i, h].astype(np.float64), keys, vals, scale)
    return out, lse, mass, size
