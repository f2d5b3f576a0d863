"""Plain implementations of the page operators, in 64 bits and Python integers: key bounds, page scores,
page selection, attention over selected pages, remapping and compaction.  Built on the oracle's own cache
layout (oracle/kvq3_oracle.py); they share no code with the CUDA path."""
from __future__ import annotations

import numpy as np

from oracle import kvq3_oracle as O


def num_pages_of(layout, n):
    return -(-int(n) // layout.page_size)


def page_keys(pool, layout, page, kv_head, which=0):
    """Dequantised rotated vectors of one physical page, fp64 [P][d], as the attention reads them (a stored
    -2^(b-1) as its own value)."""
    P, d, nb = layout.page_size, layout.d, layout.nb
    o = layout.record_offset(page, kv_head, which)
    head = pool[o:o + P * nb * layout.sb].reshape(P, nb * layout.sb)
    body = pool[o + P * nb * layout.sb:o + layout.record_bytes].reshape(P, layout.code_bytes)
    sc = O.decode_scales(head, layout.scale)
    c = O.unpack_codes(body, d, layout.bits, signed=layout.scale != "e4m3zp").astype(np.float64).reshape(P, nb, -1)
    if layout.scale == "e4m3zp":
        return (c * sc[..., 0:1] + sc[..., 1:2]).reshape(P, d)
    return (c * sc[..., None]).reshape(P, d)


def round_bound(x, layout):
    """A bound's fp16 value: the exact product rounded once, or with fp32 scales its fp32 value rounded."""
    with np.errstate(over="ignore"):
        return (x.astype(np.float32) if layout.scale == "f32" else x).astype(np.float16)


def key_bounds(pool, layout, lens, table, bounds, first_pos=None):
    """Updates bounds (fp16 [num_pages][Hkv][2][d]) in place."""
    P = layout.page_size
    for b, n in enumerate(lens):
        f = 0 if first_pos is None else int(first_pos[b])
        if not 0 <= n <= layout.max_pages_per_seq * P or f < 0 or f >= n:
            continue
        for lp in range(f // P, num_pages_of(layout, n)):
            page = layout.page_id(table, b, lp)
            if not 0 <= page < layout.num_pages:
                continue
            held = min(P, int(n) - lp * P)
            for h in range(layout.num_kv_heads):
                x = page_keys(pool, layout, page, h)[:held]
                bounds[page, h, 0] = round_bound(x.min(0), layout)
                bounds[page, h, 1] = round_bound(x.max(0), layout)


def page_scores(bounds, layout, U, q, lens, table):
    """(scores fp64 [B][Hkv][maxp], -inf where there is no page, +inf where a bound is not finite; tol: an error bound of an fp32 computation).

    The bound: q1 by a fast transform in fp32, log2(d) additions, a scaling and up to two quaternion products
    (8 products and sums), each rounding at most 2^-24 of |q|: 2^-24 (log2 d + 10) |q| per element, against
    sum_j max|bound|.  Then a chain of 4d products (2d elements, hi and lo parts) accumulated with at most 2^-23
    of the running sum each, the split itself dropping 2^-22 of an element: (4d + 2) 2^-23 sum_j |q1_j| max|bound|."""
    B, hkv, maxp, d = len(lens), layout.num_kv_heads, layout.max_pages_per_seq, layout.d
    G = q.shape[1] // hkv
    q64 = q.astype(np.float64)
    q1 = (q64 @ U.T).reshape(B, hkv, G, d)
    norm = np.linalg.norm(q64, axis=-1).reshape(B, hkv, G)
    out = np.full((B, hkv, maxp), -np.inf)
    tol = np.zeros((B, hkv, maxp))
    for b, n in enumerate(lens):
        if not 0 <= n <= maxp * layout.page_size:
            continue
        for lp in range(num_pages_of(layout, n)):
            page = layout.page_id(table, b, lp)
            if not 0 <= page < layout.num_pages:
                continue
            for h in range(hkv):
                lo, hi = bounds[page, h].astype(np.float64)
                if not np.isfinite(lo).all() or not np.isfinite(hi).all():
                    out[b, h, lp] = np.inf      # a key past the fp16 range: attended
                    continue
                out[b, h, lp] = np.maximum(q1[b, h] * lo, q1[b, h] * hi).sum(-1).max()
                m = np.maximum(np.abs(lo), np.abs(hi))
                tol[b, h, lp] = ((4 * d + 2) * 2.0 ** -23 * (np.abs(q1[b, h]) * m).sum(-1)
                                 + 2.0 ** -24 * (np.log2(d) + 10) * norm[b, h] * m.sum()).max()
    return out, tol


def page_scores_size(bounds, layout, U, q, lens, table):
    """T fp64 [B][Hkv][maxp]: the largest over the heads of sum_j |q1_j| max(|lo_j|, |hi_j|), 0 where there is no page."""
    B, hkv, d = len(lens), layout.num_kv_heads, layout.d
    q1 = np.abs(q.astype(np.float64) @ U.T).reshape(B, hkv, -1, d)
    out = np.zeros((B, hkv, layout.max_pages_per_seq))
    for b, n in enumerate(lens):
        for lp in range(num_pages_of(layout, n)):
            m = np.abs(bounds[layout.page_id(table, b, lp)].astype(np.float64)).max(1)      # [hkv][d]
            out[b, :, lp] = np.einsum("hgd,hd->hg", q1[b], m).max(-1)
    return out


# What the root mean square over many pages of a score's error may be, of the root mean square of T (page_scores_size).
# The worst case of page_scores' tolerance charges every rounding in full and in the same direction, so at d = 128 and
# 256 it would let a score through whose query lost its low half.  In units of 2^-23, the step of fp32:
#   0.4  the split: hi + lo leave at most 2^-22 of each query element, of either sign: sqrt(d) of them add up to d
#        terms, 2 / (0.8 sqrt(d)) at d = 64;
#   2.3  chains of 8 steps in the tensor core's accumulator, each cutting half a step of the running sum on average and
#        towards zero; the sum grows to its last value over the chain: (1 + 2 + ... + 8) / 8 / 2;
#   0.8  the chains' sums added in fp32, and the scaling;
#   0.5  the rotation in fp32: log2(d) + 10 roundings of 2^-24 of an element, independent over d elements, so that
#        their sum is at most sqrt(16) 2^-24 / (0.8 sqrt(d)) of T at d = 64.
SCORE_RMS = 4 * 2.0 ** -23


def page_select(scores, layout, lens, budget, sinks, recent):
    """(pages int32 [B][Hkv][budget], counts int32 [B][Hkv]) by a Python sort."""
    B, hkv, _ = scores.shape
    pages = np.full((B, hkv, budget), -1, np.int32)
    counts = np.zeros((B, hkv), np.int32)
    for b, n_tok in enumerate(lens):
        if not 0 <= n_tok <= layout.max_pages_per_seq * layout.page_size:
            continue
        n = num_pages_of(layout, n_tok)
        for h in range(hkv):
            if n <= budget:
                chosen = list(range(n))
            else:
                mid = range(sinks, n - recent)
                key = {i: -float(scores[b, h, i]) for i in mid}
                mid = sorted(mid, key=lambda i: (bool(np.isnan(key[i])), 0.0 if np.isnan(key[i]) else key[i], i))
                chosen = sorted(list(range(sinks)) + list(range(n - recent, n)) + list(mid[:budget - sinks - recent]))
            pages[b, h, :len(chosen)] = chosen
            counts[b, h] = len(chosen)
    return pages, counts


def decode_pages(pool, layout, U, q, lens, table, pages, counts, sm_scale=0.0):
    """fp64 [B][Hq][d]: attention of each head over the listed pages (strictly ascending; others left out, and a
    part-filled page that another page of the sequence follows)."""
    B, hq, d = q.shape
    hkv, P = layout.num_kv_heads, layout.page_size
    G = hq // hkv
    alpha = sm_scale if sm_scale > 0 else 1.0 / np.sqrt(d)
    q1 = q.astype(np.float64) @ U.T
    out = np.zeros((B, hq, d))
    for b in range(B):
        n = int(lens[b])
        if not 0 <= n <= layout.max_pages_per_seq * P:
            continue
        for h in range(hkv):
            c = int(counts[b, h])
            if not 0 <= c <= pages.shape[2]:
                continue
            ks, vs = [], []
            for i in range(c):
                lp = int(pages[b, h, i])
                if lp < 0 or lp * P >= n or (i > 0 and lp <= int(pages[b, h, i - 1])):
                    continue
                if (lp + 1) * P > n and any(0 <= int(e) and int(e) * P < n for e in pages[b, h, i + 1:c]):
                    continue
                page = layout.page_id(table, b, lp)
                if not 0 <= page < layout.num_pages:
                    continue
                held = min(P, n - lp * P)
                ks.append(page_keys(pool, layout, page, h, 0)[:held])
                vs.append(page_keys(pool, layout, page, h, 1)[:held])
            if not ks:
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            for g in range(G):
                s = alpha * (k @ q1[b, h * G + g])
                w = np.exp(s - s.max())
                out[b, h * G + g] = ((w @ v) / w.sum()) @ U
    return out


def remap(pool, layout, table, lens, src, new_lens):
    """(table_out, lens_out, enough): the new table row by row; copies part-filled pages in pool (in place)
    when there are enough free pages."""
    B, maxp, P, N = len(lens), layout.max_pages_per_seq, layout.page_size, layout.num_pages
    cap = maxp * P
    out = np.full((B, maxp), -1, np.int32)
    held = np.zeros(B, np.int32)
    rows = []
    for b in range(B):
        s, want = int(src[b]), int(new_lens[b])
        bad = s < -1 or s >= B or not 0 <= want <= cap or (s >= 0 and not 0 <= int(lens[s]) <= cap)
        if bad:
            s, want = -1, 0
        held[b] = min(int(lens[s]), want) if s >= 0 else 0
        rows.append((s, want))
    whole, taken = set(), set()
    for b, (s, want) in enumerate(rows):
        for i in range(int(held[b]) // P):
            page = int(table[s, i])
            if 0 <= page < N:
                out[b, i] = page
                whole.add(page)
    owner = {}
    for b, (s, want) in enumerate(rows):
        if held[b] % P:
            page = int(table[s, held[b] // P])
            if 0 <= page < N:
                owner.setdefault(page, b)
    wanted, copies = [], []
    for b, (s, want) in enumerate(rows):
        i = int(held[b]) // P
        if held[b] % P:
            page = int(table[s, i])
            if not 0 <= page < N:
                i += 1
            elif owner[page] == b and page not in whole:
                out[b, i] = page
                taken.add(page)
                i += 1
            else:
                copies.append((b, i, page))
        wanted += [(b, j) for j in range(i, -(-want // P))]
    free = [p for p in range(N) if p not in whole and p not in taken]
    if len(wanted) > len(free):
        return out, held, False
    for (b, j), page in zip(wanted, free):
        out[b, j] = page
    view = pool.reshape(N, layout.num_kv_heads * 2, layout.record_bytes)
    hdr = P * layout.nb * layout.sb
    for b, i, page in copies:
        t = int(held[b]) % P
        a, z = t * layout.nb * layout.sb, hdr + t * layout.code_bytes
        view[out[b, i], :, :a] = view[page, :, :a]
        view[out[b, i], :, hdr:z] = view[page, :, hdr:z]
    return out, held, True


def compact(pool, layout, table, lens, src_seq, dst_seq, keep, n_keep):
    """Gathers kept tokens in pool (in place): records move as stored."""
    P, N, cap = layout.page_size, layout.num_pages, layout.max_pages_per_seq * layout.page_size
    before = pool.copy()
    for i in range(len(src_seq)):
        s, d, n = int(src_seq[i]), int(dst_seq[i]), int(n_keep[i])
        if not 0 <= s < layout.batch or not 0 <= d < layout.batch or s == d:
            continue
        if not 0 <= int(lens[s]) <= cap or not 0 <= n <= min(keep.shape[2], cap):
            continue
        for h in range(layout.num_kv_heads):
            for t in range(n):
                pos = int(keep[i, h, t])
                if not 0 <= pos < int(lens[s]):
                    continue
                ps, pd = layout.page_id(table, s, pos // P), layout.page_id(table, d, t // P)
                if not 0 <= ps < N or not 0 <= pd < N:
                    continue
                for which in (0, 1):
                    for at, size in ((layout.scale_offset, layout.nb * layout.sb), (layout.code_offset, layout.code_bytes)):
                        a, z = at(ps, h, which, pos % P), at(pd, h, which, t % P)
                        pool[z:z + size] = before[a:a + size]
