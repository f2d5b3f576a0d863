"""The plain page operators (oracle/pages_oracle.py) against what defines them, on small cases by hand: no GPU."""
import numpy as np
import pytest

from oracle import kvq3_oracle as O
from oracle import pages_oracle as PO


def _pool(layout, seed=0):
    return np.random.default_rng(seed).integers(0, 256, layout.pool_bytes).astype(np.uint8)


def _written(layout, lens, seed=1):
    """A cache written by the oracle: (pool, U, table)."""
    rng = np.random.default_rng(seed)
    signs, quats = O.rotation_params(layout.d, 42)
    U = O.rotation_matrix(signs, quats)
    table = rng.permutation(layout.num_pages)[:layout.batch * layout.max_pages_per_seq].reshape(layout.batch, -1).astype(np.int32)
    pool = np.zeros(layout.pool_bytes, np.uint8)
    si = np.concatenate([np.full(n, b, np.int32) for b, n in enumerate(lens)])
    ps = np.concatenate([np.arange(n, dtype=np.int32) for n in lens])
    k, v = (rng.standard_normal((len(si), layout.num_kv_heads, layout.d)).astype(np.float16) for _ in range(2))
    assert O.write(pool, layout, U, k, v, si, ps, table) == 0
    return pool, U, table


@pytest.mark.parametrize("scale,bits", [("f16", 3), ("f32", 2), ("e4m3", 4), ("e4m3zp", 3)])
def test_page_keys_are_the_oracles_read_back(scale, bits):
    L = O.Layout(64, 2, 32, scale, 16, 2, 3, 7, bits)
    lens = (33, 48)
    pool, U, table = _written(L, lens)
    for b, n in enumerate(lens):
        for lp in range(PO.num_pages_of(L, n)):
            held = min(16, n - 16 * lp)
            for which in (0, 1):
                want = O.read_rotated(pool, L, b, 1, which, 16 * lp, held, table)[0]
                got = PO.page_keys(pool, L, int(table[b, lp]), 1, which)[:held]
                assert np.array_equal(got, want)


@pytest.mark.parametrize("scale,bits", [("f16", 3), ("e4m3zp", 3), ("f32", 4)])
def test_scores_bound_every_logit_and_full_selection_is_decode(scale, bits):
    L = O.Layout(64, 2, 64, scale, 16, 2, 4, 9, bits)
    lens = np.array([50, 64], np.int32)
    pool, U, table = _written(L, lens)
    q = np.random.default_rng(3).standard_normal((2, 6, 64)).astype(np.float16)
    bounds = np.zeros((9, 2, 2, 64), np.float16)
    PO.key_bounds(pool, L, lens, table, bounds)
    scores, _ = PO.page_scores(bounds, L, U, q, lens, table)
    q1 = q.astype(np.float64) @ U.T
    for b in range(2):
        for h in range(2):
            k = O.read_rotated(pool, L, b, h, 0, 0, int(lens[b]), table)[0]
            for lp in range(PO.num_pages_of(L, lens[b])):
                top = (k[16 * lp:16 * lp + 16] @ q1[b, 3 * h:3 * h + 3].T).max()
                assert top <= scores[b, h, lp] + 2.0 ** -11 * np.abs(scores[b, h, lp])
    pages, counts = PO.page_select(scores, L, lens, 4, 0, 1)
    assert np.array_equal(counts, [[4, 4], [4, 4]])
    got = PO.decode_pages(pool, L, U, q, lens, table, pages, counts)
    want = O.decode(pool, L, U, q, lens, table)
    assert np.allclose(got, want, rtol=0, atol=1e-12 * np.abs(want).max())


def test_select_by_hand():
    L = O.Layout(64, 1, 64, "f16", 16, 1, 10, 10)
    s = np.array([[[9.0, 1.0, 5.0, 5.0, -np.inf, np.nan, 5.0, 7.0, 0.0, -1.0]]])
    sel = lambda n, *a: PO.page_select(s, L, [n], *a)[0][0, 0].tolist()  # noqa: E731
    assert sel(160, 4, 0, 1) == [0, 2, 7, 9]           # 9, 7, the first of the fives, the last page
    assert sel(160, 5, 1, 2) == [0, 2, 7, 8, 9]
    assert sel(145, 3, 1, 2) == [0, 8, 9]               # nothing left to choose
    assert sel(160, 8, 0, 1) == [0, 1, 2, 3, 6, 7, 8, 9]   # -inf before NaN, both out
    assert sel(48, 4, 1, 1) == [0, 1, 2, -1]
    assert sel(0, 2, 0, 1) == [-1, -1]


def test_remap_by_hand():
    L = O.Layout(64, 1, 64, "f16", 16, 4, 4, 10)
    pool = _pool(L)
    before = pool.copy()
    table = np.array([[3, 7, -1, -1], [5, -1, -1, -1], [-1] * 4, [-1] * 4], np.int32)
    # row 0 (20 tokens) goes on; row 2 forks it; row 3 shares its first 16 tokens; row 1 is freed
    out, held, ok = PO.remap(pool, L, table, [20, 9, 0, 0], [0, 1, 0, 0], [21, 0, 40, 16])
    assert ok and held.tolist() == [20, 0, 20, 16]
    assert out.tolist() == [[3, 7, -1, -1], [-1] * 4, [3, 0, 1, -1], [3, -1, -1, -1]]
    rec = L.record_bytes
    a, z = pool[0:rec], before[7 * L.page_bytes:7 * L.page_bytes + rec]
    assert np.array_equal(a[:4 * 2], z[:4 * 2]) and np.array_equal(a[32:32 + 4 * 24], z[32:32 + 4 * 24])
    assert np.array_equal(a[8:32], before[8:32])        # beyond the copied tokens: as it was
    # a page that another row shares whole is copied by the row that would append to it
    table = np.array([[3, 7, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4], np.int32)
    out, held, ok = PO.remap(pool, L, table, [32, 0, 0, 0], [0, 0, -1, -1], [20, 32, 0, 5])
    assert out.tolist() == [[3, 0, -1, -1], [3, 7, -1, -1], [-1] * 4, [1, -1, -1, -1]]
    # too few pages
    before = pool.copy()
    out, held, ok = PO.remap(pool, L, table, [20, 0, 0, 0], [0, 0, 0, 0], [64, 64, 64, 64])
    assert not ok and np.array_equal(pool, before) and out[0].tolist() == [3, 7, -1, -1]


def test_compact_moves_records():
    L = O.Layout(64, 2, 32, "e4m3", 16, 2, 2, 5)
    pool, U, table = _written(L, (30, 32))
    want = [O.read_rotated(pool, L, 0, h, w, 0, 30, table)[1] for h in (0, 1) for w in (0, 1)]
    keep = np.array([[[29, 3, 3, 17], [0, 16, 1, 99]]], np.int32)
    PO.compact(pool, L, table, [30, 32], [0], [1], keep, [4])
    for h in (0, 1):
        for w in (0, 1):
            got = O.read_rotated(pool, L, 1, h, w, 0, 4, table)[1]
            for t in range(4 if h == 0 else 3):
                assert np.array_equal(got[t], want[2 * h + w][keep[0, h, t]])
