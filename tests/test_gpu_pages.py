"""Page operators on the GPU against oracle/pages_oracle.py: key bounds (bit exact), page scores (within the
rounding of an fp32 computation), selections (exact), attention over selected pages (the decode's bar plus one
fp16 rounding), remapping and compaction (exact tables and bytes), alone and run together."""
from __future__ import annotations

import numpy as np
import pytest

from cases import CANARY, CANARY_BYTE, TOL_DECODE
from oracle import kvq3_oracle as O
from oracle import pages_oracle as PO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Pages:
    """A paged (or contiguous) cache of random records: codes any bits, scales near 0.2."""

    def __init__(self, d=128, hkv=2, block=64, scale="f16", bits=3, page=16, lens=(37, 100), maxp=None, spare=3,
                 paged=True, flags=3, seed=7, rows=None):
        import torch
        import hadamard_rotated_bit_kvq3_gb300 as K
        self.K, self.torch = K, torch
        self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        B = len(lens)
        self.B, self.d, self.hkv, self.page = B, d, hkv, page
        need = [-(-int(n) // page) for n in lens]
        self.maxp = maxp or max(1, max(need))
        N = sum(need) + spare if paged else B * self.maxp
        self.N = N
        self.layout = L = O.Layout(d, hkv, block, scale, page, B, self.maxp, N, bits)
        self.desc = K.CacheDesc(d, hkv, block, bits, K.SCALE_TYPES[scale], 1e-6, page, B, self.maxp, 0, N)
        self.table = None
        if paged:
            ids, at = self.rng.permutation(N), 0
            self.table = np.full((B, self.maxp), -1, np.int32)
            for b, n in enumerate(need):
                self.table[b, :n] = ids[at:at + n]
                at += n
        pool = self.rng.integers(0, 256, L.pool_bytes, dtype=np.uint8)
        view = pool.reshape(N, hkv, 2, L.record_bytes)
        hdr = page * L.nb * L.sb
        n_s = page * L.nb
        s = (0.2 * np.exp(0.3 * self.rng.standard_normal((N, hkv, 2, n_s)))).astype(np.float32)
        if scale == "e4m3zp":
            z = self.rng.standard_normal((N, hkv, 2, n_s)).astype(np.float32)
            raw = np.stack([O.encode_e4m3(O.round_e4m3(s.astype(np.float64))),
                            O.encode_e4m3_signed(O.round_e4m3_signed(z.astype(np.float64)))], -1).astype(np.uint8)
        else:
            raw = O.encode_scales(O.round_scale(s.astype(np.float64), scale), scale)
        view[..., :hdr] = raw.reshape(N, hkv, 2, hdr)
        self.pool = pool
        if flags & 4:
            sg, q, qr = O.rotation_params_pair(d, 42, bool(flags & 1))
            self.U = O.rotation_matrix(sg, q, qr)
        else:
            sg, q = O.rotation_params(d, 42, bool(flags & 1), bool(flags & 2))
            self.U = O.rotation_matrix(sg, q)
        self.rot = K.Rotation(d, 42, flags)
        self.pool_full = self.dev(np.concatenate([pool, np.full(CANARY, CANARY_BYTE, np.uint8)]))
        self.table_t = None if self.table is None else self.dev(self.table)
        self.lens_t = self.dev(self.lens)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = self.cache_of(self.table_t, self.lens_t)

    def dev(self, x):
        return self.torch.as_tensor(np.ascontiguousarray(x), device="cuda")

    def cache_of(self, table_t, lens_t):
        return self.K.Cache(self.pool_full.data_ptr(), None if table_t is None else table_t.data_ptr(), lens_t.data_ptr())

    def pool_now(self):
        p = self.pool_full.cpu().numpy()
        assert np.all(p[-CANARY:] == CANARY_BYTE), "a kernel wrote past the pool"
        return p[:-CANARY]

    def flags(self):
        return int(self.status.item())

    def guarded(self, shape, dtype, fill):
        """A device tensor of `shape` with a row of guard values behind it."""
        t = self.torch
        n = int(np.prod(shape))
        full = t.full((n + 64,), fill, dtype=dtype, device="cuda")
        return full, full[:n].view(*shape)

    def queries(self, G, seed=3):
        return np.random.default_rng(seed).standard_normal((self.B, self.hkv * G, self.d)).astype(np.float16)


# ------------------------------------------------------------ key bounds
def _bounds(c, first=None, start=None):
    t = c.torch
    full, out = c.guarded((c.N, c.hkv, 2, c.d), t.float16, 7.0)
    c.K.kvq3_key_bounds(c.desc, c.cache, None if first is None else c.dev(np.array(first, np.int32)), out, c.status)
    t.cuda.synchronize()
    assert bool((full[-64:] == 7.0).all())
    want = np.full((c.N, c.hkv, 2, c.d), 7.0, np.float16)
    PO.key_bounds(c.pool, c.layout, c.lens, c.table, want, first)
    return out.cpu().numpy(), want


BOUNDS = [
    dict(),
    dict(bits=2, scale="e4m3", page=48, lens=(1, 0, 47, 48, 49, 200)),
    dict(bits=4, scale="f32", block=32, page=32, lens=(90, 3)),
    dict(d=64, block=32, bits=3, scale="f16", page=16, lens=(16, 65)),
    dict(d=64, block=64, bits=2, scale="f32", page=16, lens=(16, 65)),
    dict(d=64, block=32, bits=4, scale="e4m3", page=64, lens=(130,)),
    dict(d=256, block=64, bits=3, scale="e4m3zp", page=16, lens=(100, 33)),
    dict(d=256, block=32, bits=4, scale="f16", page=128, lens=(300,), hkv=3),
    dict(d=128, block=32, bits=3, scale="e4m3zp", page=16, lens=(7,), hkv=1, paged=False),
    dict(d=128, block=32, bits=3, scale="f32", page=112, lens=(500, 17), paged=False),
    dict(d=128, bits=3, page=128, lens=(9000, 4097, 128), hkv=4, spare=0),       # many pages: no lanes shared
    dict(d=64, bits=3, block=64, scale="f16", page=16, lens=tuple(i % 40 for i in range(1500)), hkv=1),   # two segments
]


@pytest.mark.parametrize("kw", BOUNDS, ids=lambda k: "-".join(f"{a}{b if not isinstance(b, tuple) else len(b)}" for a, b in k.items()) or "base")
def test_key_bounds_bit_exact(kw):
    c = Pages(**kw)
    got, want = _bounds(c)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    # the newest page alone, and nothing from a start at or past the end
    first = np.maximum(c.lens - 1, 0)
    first[-1] = c.lens[-1] + 3
    got, want = _bounds(c, first)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    assert c.flags() == 0


def test_key_bounds_bad_lengths_and_pages():
    c = Pages(lens=(40, 64, 33, 20), maxp=5)
    c.table[0, 1], c.table[2, 0] = c.N, -7
    c.table_t.copy_(c.dev(c.table))
    c.lens = np.array([40, -1, 33, 5 * 16 + 1], np.int32)
    c.lens_t.copy_(c.dev(c.lens))
    got, want = _bounds(c)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    assert c.flags() == c.K.DEV_BITS["bad_len"] | c.K.DEV_BITS["bad_page"]
    # a negative start
    c = Pages(lens=(40, 64))
    got, want = _bounds(c, [-1, 17])
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16)) and c.flags() == c.K.DEV_BITS["bad_len"]


# ------------------------------------------------------------ page scores
def _scores(c, bounds, q):
    t = c.torch
    full, out = c.guarded((c.B, c.hkv, c.maxp), t.float32, 5.0)
    c.K.kvq3_page_scores(c.rot.handle, c.desc, c.cache, c.dev(bounds), c.dev(q), out, c.status)
    t.cuda.synchronize()
    assert bool((full[-64:] == 5.0).all())
    return out.cpu().numpy()


def _random_bounds(c, seed=5):
    rng = np.random.default_rng(seed)
    mid, half = rng.standard_normal((c.N, c.hkv, 1, c.d)), rng.random((c.N, c.hkv, 1, c.d)) * 2
    return np.concatenate([mid - half, mid + half], 2).astype(np.float16)


@pytest.mark.parametrize("d,G,page,lens,kw", [
    (128, 4, 16, (37, 2100), {}),
    (128, 1, 64, (1, 0, 64, 65, 8200), dict(hkv=1)),
    (128, 3, 128, (5000,), dict(paged=False)),
    (128, 8, 16, (300, 2049), dict(flags=7)),
    (128, 5, 16, (300,), dict(flags=0)),
    (128, 16, 32, (40, 4095), dict(flags=2)),
    (64, 2, 16, (2500, 3), dict(block=32, hkv=3)),
    (64, 12, 16, (700,), dict(flags=7)),
    (256, 4, 16, (2048, 15), dict(flags=1)),
    (256, 16, 16, (100,), dict(flags=7, hkv=1)),
    (256, 7, 48, (10000,), {}),
])
def test_page_scores(d, G, page, lens, kw):
    c = Pages(d=d, page=page, lens=lens, maxp=-(-max(lens) // page) + 5, **kw)
    q, bounds = c.queries(G), _random_bounds(c)
    q[0, 0] = 0                     # a query of zeros, one large, one small
    q[-1, -1] *= 1000
    q[-1, 0] *= 1e-3
    got = _scores(c, bounds, q).astype(np.float64)
    want, tol = PO.page_scores(bounds, c.layout, c.U, q, c.lens, c.table)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert np.all(np.abs(got[fin] - want[fin]) <= tol[fin])
    assert c.flags() == 0


def test_page_scores_bad_lengths_and_pages():
    c = Pages(lens=(40, 64, 33), maxp=4)
    c.table[0, 1] = c.N
    c.table_t.copy_(c.dev(c.table))
    c.lens = np.array([40, 65, -3], np.int32)
    c.lens_t.copy_(c.dev(c.lens))
    q, bounds = c.queries(4), _random_bounds(c)
    got = _scores(c, bounds, q).astype(np.float64)
    want, tol = PO.page_scores(bounds, c.layout, c.U, q, c.lens, c.table)
    assert np.isneginf(want[0, :, 1]).all() and np.isneginf(want[1:]).any()
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin]) and np.all(np.abs(got[fin] - want[fin]) <= tol[fin])
    assert c.flags() == c.K.DEV_BITS["bad_len"] | c.K.DEV_BITS["bad_page"]


# ------------------------------------------------------------ selection
def _select_case(lens, maxp, hkv, scores, budget, sinks, recent):
    import torch
    import hadamard_rotated_bit_kvq3_gb300 as K
    B = len(lens)
    desc = K.CacheDesc(64, hkv, 64, 3, 1, 1e-6, 16, B, maxp, 0, 1)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    full = torch.full((B * hkv * budget + 64,), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((B, hkv), 77, dtype=torch.int32, device="cuda")
    pages = full[:-64].view(B, hkv, budget)
    K.kvq3_page_select(desc, K.Cache(None, None, lens_t.data_ptr()), torch.as_tensor(scores, device="cuda"), budget,
                       sinks, recent, pages, counts, status)
    torch.cuda.synchronize()
    assert bool((full[-64:] == 77).all())
    L = O.Layout(64, hkv, 64, "f16", 16, B, maxp, 1)
    want = PO.page_select(scores, L, lens, budget, sinks, recent)
    assert np.array_equal(pages.cpu().numpy(), want[0])
    assert np.array_equal(counts.cpu().numpy(), want[1])
    return int(status.item())


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special", "narrow", "wide"])
@pytest.mark.parametrize("n,budget,sinks,recent", [
    (1, 1, 0, 1), (5, 1, 0, 1), (5, 8, 1, 2), (33, 7, 1, 2), (64, 64, 3, 3), (65, 64, 0, 1), (100, 4, 2, 2),
    (257, 31, 1, 4), (2000, 1999, 5, 9), (4097, 256, 2, 4), (9001, 300, 1, 1), (20011, 9000, 0, 3)])
def test_page_select_exact(kind, n, budget, sinks, recent):
    rng = np.random.default_rng(n + budget)
    maxp = n + 3
    lens = [16 * n, 16 * n - 15, 16 * max(1, n // 2), 16 * n - 5, 0]
    s = rng.standard_normal((len(lens), 2, maxp)).astype(np.float32)
    if kind == "ties":
        s = np.round(s * 2) / 2
        s[s == 0] *= np.where(rng.random((s == 0).sum()) < 0.5, -1, 1)     # zeros of both signs are equal
    elif kind == "equal":
        s[:] = 1.5
    elif kind == "special":
        r = rng.random(s.shape)
        s[r < 0.3] = -np.inf
        s[(r >= 0.3) & (r < 0.5)] = np.nan
        s[r > 0.97] = np.inf
        s[r > 0.99] = np.finfo(np.float32).min
    elif kind == "narrow":
        s = (1000 + 1e-3 * s).astype(np.float32)
    elif kind == "wide":
        s = (s * np.exp(8 * rng.standard_normal(s.shape))).astype(np.float32)
    s[:, :, n:] = np.nan                                                    # what lies past the sequence is not read
    assert _select_case(lens, maxp, 2, s, budget, sinks, recent) == 0


def test_page_select_bad_length():
    import hadamard_rotated_bit_kvq3_gb300 as K
    s = np.random.default_rng(1).standard_normal((3, 1, 6)).astype(np.float32)
    assert _select_case([97, -1, 60], 6, 1, s, 3, 1, 1) == K.DEV_BITS["bad_len"]


# ------------------------------------------------------------ attention over selected pages
def _attend(c, q, pages, counts, sm=0.0):
    t = c.torch
    full, out = c.guarded(q.shape, t.float16, 9.0)
    c.K.kvq3_decode_attn_pages(c.rot.handle, c.desc, c.cache, c.dev(q), c.dev(pages), c.dev(counts), out, sm, c.status)
    t.cuda.synchronize()
    assert bool((full[-64:] == 9.0).all())
    c.pool_now()
    return out.cpu().numpy().astype(np.float64)


def _near(got, want):
    """The decode's bar, and one rounding to fp16 (half a step: 2^-11 of the value, 2^-25 below the normal range)."""
    rms = np.sqrt(np.mean(want ** 2))
    err = np.abs(got - want)
    print(f"max|err|/rms = {err.max() / rms:.2e}")
    assert np.all(err <= TOL_DECODE * rms + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)


def _lists(c, row, seed=11, last=True):
    """A random ascending choice of up to `row` pages of each (sequence, kv head)."""
    rng = np.random.default_rng(seed)
    pages = np.full((c.B, c.hkv, row), -1, np.int32)
    counts = np.zeros((c.B, c.hkv), np.int32)
    for b in range(c.B):
        n = -(-int(c.lens[b]) // c.page)
        for h in range(c.hkv):
            k = min(row, n)
            pick = np.sort(rng.permutation(n)[:k])
            if last and k:
                pick[-1] = n - 1
            pages[b, h, :k], counts[b, h] = pick, k
    return pages, counts


ATTN = [
    (dict(lens=(37, 100, 0, 1)), 4, 3),
    (dict(lens=(700, 333), page=64, hkv=4), 1, 5),
    (dict(lens=(130, 1000), page=128, scale="e4m3"), 8, 4),
    (dict(lens=(500, 64, 65), scale="f32", block=32), 5, 9),
    (dict(lens=(90, 257), bits=2, flags=7), 16, 8),
    (dict(lens=(400,), bits=4, page=48, hkv=3), 3, 6),
    (dict(lens=(300, 77), d=64, block=32, scale="e4m3", hkv=1), 12, 7),
    (dict(lens=(310, 77), d=64, block=64, bits=2), 2, 64),                 # longer lists than there are pages
    (dict(lens=(300, 200), d=256, page=16), 4, 10),
    (dict(lens=(300, 200), d=256, block=32, bits=4, scale="f32"), 7, 10),
    (dict(lens=(333, 20), d=256, scale="e4m3zp"), 16, 12),
    (dict(lens=(333, 20, 64), scale="e4m3zp", paged=False), 4, 4),
    (dict(lens=(5000, 4999, 3), page=16, hkv=8), 4, 200),
    (dict(lens=tuple(5 + 7 * i for i in range(70)), page=16, hkv=4), 4, 4),   # many short units
    # few units with long lists: up to 16 CTAs a unit
    (dict(lens=(40000,), page=16, hkv=1), 4, 2600),
    (dict(lens=(60000, 300), page=64, hkv=1, scale="e4m3", flags=7), 8, 800),
    (dict(lens=(33000, 0, 17), page=16, hkv=1, scale="e4m3zp", d=64, block=32), 3, 2000),
    # long lists of several units: whole clusters, chunks in turn
    (dict(lens=(9000, 8000, 100, 0), page=32, hkv=4, bits=4), 6, 250),
    # more pages a CTA than it looks up ahead
    (dict(lens=(70000,), page=16, hkv=1, d=64, block=64, bits=2), 2, 4375),
    # pages larger than a chunk; as large as the copy stages take
    (dict(lens=(700, 300), page=256, hkv=2), 4, 3), (dict(lens=(2500, 1024), page=1024, hkv=1), 4, 2),
]


@pytest.mark.parametrize("kw,G,row", ATTN)
def test_decode_attn_pages(kw, G, row):
    c = Pages(**kw)
    q = c.queries(G)
    for last in (True, False):
        pages, counts = _lists(c, row, last=last)
        got = _attend(c, q, pages, counts)
        _near(got, PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts))
    assert c.flags() == 0


def test_all_pages_is_the_dense_decode():
    c = Pages(lens=(777, 64, 1), page=32, hkv=2)
    q = c.queries(4)
    pages, counts = _lists(c, 40)
    got = _attend(c, q, pages, counts, 0.11)
    t = c.torch
    out = t.empty(q.shape, dtype=t.float32, device="cuda")
    ws = t.empty(c.K.kvq3_decode_workspace_size(c.desc, q.shape[1]), dtype=t.uint8, device="cuda")
    c.K.kvq3_decode_attn(c.rot.handle, c.desc, c.cache, c.dev(q), out, ws, 0.11, c.status)
    _near(got, out.cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("row", [5, 40000])   # short lists, and short ones in long rows (16 CTAs a unit, most idle)
def test_decode_attn_pages_bad_lists(row):
    c = Pages(lens=(100, 100, 100, 100, 100, 50), hkv=1, page=16, maxp=8)
    q = c.queries(4)
    pages = np.full((6, 1, row), -1, np.int32)
    pages[0, 0, :5] = [0, 2, 2, 5, 6]            # a page twice
    pages[1, 0, :5] = [1, 6, 3, 7, -2]           # not ascending; the part-filled page before the end; past the end
    pages[2, 0, :5] = [6, 6, 6, 6, 6]            # the part-filled page again
    pages[3, 0, :5] = [0, 1, 2, 3, 4]
    pages[4, 0, :5] = [0, 1, 2, 1 << 30, 3]
    pages[5, 0, :5] = [0, 1, 2, 3, 4]
    counts = np.array([[5], [5], [5], [row + 1], [5], [2]], np.int32)   # row 3: more than the list holds
    c.table[5, 1] = c.N + 4
    c.table_t.copy_(c.dev(c.table))
    want = PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts)
    got = _attend(c, q, pages, counts)
    assert not got[2].any() and not got[3].any()
    _near(got, want)
    assert c.flags() == c.K.DEV_BITS["bad_len"] | c.K.DEV_BITS["bad_page"]
    c.lens_t.copy_(c.dev(np.array([100, -1, 129, 100, 100, 50], np.int32)))
    c.lens = np.array([100, -1, 129, 100, 100, 50], np.int32)
    want = PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts)
    _near(_attend(c, q, pages, counts), want)


@pytest.mark.parametrize("kw,G,row", [
    (dict(lens=(700, 1, 129, 64), page=64), 4, 9), (dict(lens=(300, 17, 1000), d=256, page=16), 4, 70),
    (dict(lens=(40000,), page=16, hkv=1), 4, 2600)])
def test_decode_attn_pages_wait_that_runs_out(kw, G, row):
    # with no poll allowed every CTA takes its time-out path: it flags, drains its copies and still meets the
    # others of its cluster; a normal call on the same buffers follows
    import ctypes
    c = Pages(**kw)
    K, t = c.K, c.torch
    fn = K.lib.kvq3_test_decode_pages_polls
    fn.restype, fn.argtypes = ctypes.c_int, K.lib.kvq3_decode_attn_pages.argtypes + [ctypes.c_uint32]
    q = c.queries(G)
    pages, counts = _lists(c, row)
    qd, pd, nd = c.dev(q), c.dev(pages), c.dev(counts)
    out = t.empty(q.shape, dtype=t.float16, device="cuda")
    for _ in range(2):
        assert fn(c.rot.handle, c.desc, c.cache, qd.data_ptr(), q.shape[1], 0.0, pd.data_ptr(), nd.data_ptr(), row,
                  out.data_ptr(), c.status.data_ptr(), K._raw_stream(None), 0) == 0
        t.cuda.synchronize()
        assert c.flags() & K.DEV_BITS["timeout"]
        c.status.zero_()
    _near(_attend(c, q, pages, counts), PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts))
    assert c.flags() == 0


def test_decode_attn_pages_refuses_pages_past_the_stages():
    c = Pages(lens=(100,), page=4096, hkv=1)
    q, (pages, counts) = c.queries(4), _lists(c, 1)
    with pytest.raises(c.K.Kvq3Error) as e:
        _attend(c, q, pages, counts)
    assert e.value.status == 2                   # as the dense decode: two stages of a page do not fit


def test_offsets_past_32_bits():
    # the same cache at the end of a 6.4 GB pool: every operator gives the same bits
    page, hkv, d, far = 128, 8, 128, 60000
    c = Pages(lens=(700, 333, 0, 0), page=page, hkv=hkv, maxp=7, spare=8, d=d)
    t, K, L = c.torch, c.K, c.layout
    free = t.cuda.mem_get_info()[0]
    assert far * L.page_bytes > 1 << 32
    if free < 2 * far * L.page_bytes:
        pytest.skip("not enough device memory")
    q, G = c.queries(4), 4
    pages, counts = _lists(c, 5)
    keep = c.rng.integers(0, 333, (1, hkv, 300)).astype(np.int32)

    def run(shift):
        n = c.N + shift
        pool = t.zeros(n * L.page_bytes, dtype=t.uint8, device="cuda")
        pool[shift * L.page_bytes:] = c.dev(c.pool)
        table = c.dev(np.where(c.table >= 0, c.table + shift, -1).astype(np.int32))
        lens = c.dev(c.lens)
        desc = K.CacheDesc(d, hkv, 64, 3, 1, 1e-6, page, c.B, c.maxp, 0, n)
        cache = K.Cache(pool.data_ptr(), table.data_ptr(), lens.data_ptr())
        bounds = t.zeros(n, hkv, 2, d, dtype=t.float16, device="cuda")
        scores = t.empty(c.B, hkv, c.maxp, device="cuda")
        out = t.empty(c.B, hkv * G, d, dtype=t.float16, device="cuda")
        K.kvq3_key_bounds(desc, cache, None, bounds, c.status)
        K.kvq3_page_scores(c.rot.handle, desc, cache, bounds, c.dev(q), scores, c.status)
        K.kvq3_decode_attn_pages(c.rot.handle, desc, cache, c.dev(q), c.dev(pages), c.dev(counts), out, 0.0, c.status)
        # row 2 gets pages for 300 tokens gathered from row 1 (by hand: the pages below `shift` are free too)
        table2 = table.clone()
        spare = np.setdiff1d(np.arange(c.N), c.table[c.table >= 0])
        table2[2, :3] = c.dev((spare[:3] + shift).astype(np.int32))
        cache2 = K.Cache(pool.data_ptr(), table2.data_ptr(), lens.data_ptr())
        i32 = lambda x: c.dev(np.array(x, np.int32))   # noqa: E731
        K.kvq3_compact(desc, cache2, i32([1]), i32([2]), c.dev(keep), i32([300]), c.status)
        t.cuda.synchronize()
        moved = pool[shift * L.page_bytes:].cpu().numpy()
        got = (bounds[shift:].cpu().numpy().view(np.uint16), scores.cpu().numpy(), out.cpu().numpy(), moved)
        # a fork whose part-filled page lies past 4 GB is copied into the lowest free page
        table3, lens3 = t.empty_like(table), t.empty_like(lens)
        ws = t.empty(K.kvq3_remap_workspace_size(desc), dtype=t.uint8, device="cuda")
        K.kvq3_remap(desc, cache, i32([0, 1, -1, 0]), i32([700, 333, 0, 700]), table3, lens3, ws, c.status)
        t.cuda.synchronize()
        a, z = int(table3[0, 5]), int(table3[3, 5])
        rec = pool.view(n, hkv * 2, L.record_bytes)
        hdr, tok = page * L.nb * L.sb, 700 % page
        assert a != z and bool((rec[a, :, :tok * L.nb * L.sb] == rec[z, :, :tok * L.nb * L.sb]).all())
        assert bool((rec[a, :, hdr:hdr + tok * L.code_bytes] == rec[z, :, hdr:hdr + tok * L.code_bytes]).all())
        return got

    near, past = run(0), run(far)
    assert c.flags() == 0
    for a, b in zip(near, past):
        assert np.array_equal(a, b)


def test_decode_attn_pages_is_deterministic():
    c = Pages(lens=(5000, 4000, 77), page=16, hkv=4)
    q = c.queries(4)
    pages, counts = _lists(c, 250)
    first = _attend(c, q, pages, counts)
    for _ in range(5):
        assert np.array_equal(first, _attend(c, q, pages, counts))


# ------------------------------------------------------------ remapping
def _remap(c, src, new, status=None):
    t = c.torch
    out = t.full((c.B, c.maxp), 77, dtype=t.int32, device="cuda")
    lens = t.full((c.B,), 77, dtype=t.int32, device="cuda")
    n_ws = c.K.kvq3_remap_workspace_size(c.desc)
    ws = t.randint(0, 256, (n_ws + CANARY,), dtype=t.uint8, device="cuda")
    ws[n_ws:] = CANARY_BYTE
    c.K.kvq3_remap(c.desc, c.cache, c.dev(np.array(src, np.int32)), c.dev(np.array(new, np.int32)), out, lens, ws[:n_ws],
                   c.status)
    t.cuda.synchronize()
    assert bool((ws[n_ws:] == CANARY_BYTE).all())
    want_pool = c.pool.copy()
    want = PO.remap(want_pool, c.layout, c.table, c.lens, src, new)
    assert np.array_equal(lens.cpu().numpy(), want[1])
    assert np.array_equal(out.cpu().numpy(), want[0])
    assert np.array_equal(c.pool_now(), want_pool)
    c.pool, c.table, c.lens = want_pool, want[0], want[1]
    c.table_t, c.lens_t = out, lens
    c.cache = c.cache_of(out, lens)
    return want[2]


@pytest.mark.parametrize("kw", [
    dict(), dict(scale="e4m3", block=64, bits=2, page=48), dict(d=64, bits=3, block=32, scale="f32", hkv=1),
    dict(d=64, block=64, scale="e4m3", hkv=3), dict(d=256, scale="e4m3zp", page=32)])
def test_remap_steps(kw):
    # a run of steps over one cache: grow, fork, reorder, truncate, free, each from the one before
    page = kw.get("page", 16)
    rng = np.random.default_rng(17)
    lens = [0, 1, page, page + 1, 5 * page - 1, 3 * page, 7 * page + 3, 2 * page + 5, 0, 4 * page + 9]
    c = Pages(lens=lens, maxp=9, spare=160, **kw)
    B, cap = c.B, 9 * page
    same = np.arange(B)
    assert _remap(c, same, np.minimum(c.lens + 1, cap))
    c.lens = np.minimum(np.array(lens, np.int32) + 1, cap)          # the step's tokens, written
    c.lens_t.copy_(c.dev(c.lens))
    assert _remap(c, rng.integers(-1, B, B), rng.integers(0, cap + 1, B))
    for _ in range(4):
        # sequences grown to some length within their pages, then remapped at random
        held = (c.table >= 0).sum(1) * page
        c.lens = np.minimum(held, c.lens + rng.integers(0, page, B)).astype(np.int32)
        c.lens_t.copy_(c.dev(c.lens))
        assert _remap(c, rng.integers(-1, B, B), rng.integers(0, cap + 1, B))
    assert _remap(c, np.zeros(B), np.full(B, cap - 3))               # everyone continues row 0
    assert _remap(c, same, np.zeros(B))                              # everything freed
    assert c.flags() == 0 and (c.table == -1).all()


@pytest.mark.parametrize("rows", [33, 300, 512])
def test_remap_copies_of_many_rows(rows):
    # beams of 5, most rows with a part-filled page to copy: every CTA has to take its own share of the same list
    rng = np.random.default_rng(rows)
    c = Pages(d=128, hkv=1, block=32, scale="e4m3zp", page=48, lens=rng.integers(1, 300, rows), maxp=8, spare=2 * rows)
    src = np.minimum(np.arange(rows) // 5 * 5 + rng.integers(0, 5, rows), rows - 1)
    assert _remap(c, src, c.lens[src] + 1) and c.flags() == 0
    assert _remap(c, np.zeros(rows), np.full(rows, c.lens[0] + 1)) and c.flags() == 0


@pytest.mark.parametrize("rows,maxp,spare", [(900, 80, 9000), (60, 1100, 3000), (20, 40, 66000), (513, 3, 600), (512, 128, 700)])
def test_remap_large(rows, maxp, spare):
    # past what one CTA takes: by rows, by entries, by pages, by one row; and just as much as one CTA takes
    rng = np.random.default_rng(23)
    top = 16 * min(maxp, 75)
    lens = rng.integers(0, top, rows)
    c = Pages(d=64, hkv=1, bits=2, scale="e4m3", page=16, lens=lens, maxp=maxp, spare=spare)
    assert _remap(c, rng.integers(-1, rows, rows), np.minimum(rng.integers(0, top, rows), 7 * top // 12))
    assert _remap(c, np.arange(rows), c.lens + 1) and c.flags() == 0


def test_remap_runs_out_of_pages():
    c = Pages(lens=(20, 40, 0), maxp=6, spare=1)
    before = c.pool.copy()
    cache, table, lens = c.cache, c.table, c.lens
    assert not _remap(c, [0, 1, 0], [60, 40, 25])
    assert c.flags() == c.K.DEV_BITS["no_page"] and np.array_equal(c.pool, before)
    # the old table still holds: a step from it that fits
    c.cache, c.table, c.lens = cache, table, lens
    c.status.zero_()
    c.table_t, c.lens_t = c.dev(table), c.dev(lens)
    c.cache = c.cache_of(c.table_t, c.lens_t)
    assert _remap(c, [0, 1, -1], [30, 30, 10]) and c.flags() == 0
    # exactly as many as there are
    c2 = Pages(lens=(16, 32, 0), maxp=6, spare=2)
    assert _remap(c2, [0, 1, 0], [17, 48, 16]) and c2.flags() == 0
    assert sorted(set(c2.table[c2.table >= 0].tolist())) == list(range(c2.N))


def test_remap_bad_arguments_on_the_device():
    c = Pages(lens=(20, 40, 30, 33, 10), maxp=4, spare=12)
    c.table[2, 1], c.table[3, 0] = -5, c.N           # an unreadable part-filled page, an unreadable whole one
    c.table_t.copy_(c.dev(c.table))
    c.lens = np.array([20, 65, 30, 33, 10], np.int32)
    c.lens_t.copy_(c.dev(c.lens))
    _remap(c, [5, 1, 2, 3, -2], [20, 40, 40, 60, 5])
    bits = c.K.DEV_BITS
    assert c.flags() == bits["bad_seq"] | bits["bad_len"] | bits["bad_page"]
    c = Pages(lens=(20, 40), maxp=4, spare=12)
    _remap(c, [0, 1], [65, -1])
    assert c.flags() == bits["bad_len"] and (c.table == -1).all()


# ------------------------------------------------------------ compaction
def _compact(c, src, dst, keep, n_keep):
    c.K.kvq3_compact(c.desc, c.cache, c.dev(np.array(src, np.int32)), c.dev(np.array(dst, np.int32)), c.dev(keep),
                     c.dev(np.array(n_keep, np.int32)), c.status)
    c.torch.cuda.synchronize()
    PO.compact(c.pool, c.layout, c.table, c.lens, src, dst, keep, n_keep)
    assert np.array_equal(c.pool_now(), c.pool)


@pytest.mark.parametrize("d,block,bits,scale,page,kw", [
    (128, 64, 3, "f16", 16, {}), (128, 32, 2, "f32", 48, {}), (128, 64, 4, "e4m3", 128, dict(hkv=3)),
    (64, 64, 3, "e4m3", 16, {}), (64, 32, 3, "f32", 16, {}), (64, 64, 2, "f16", 32, dict(hkv=1)), (64, 64, 4, "f32", 16, {}),
    (256, 32, 3, "f32", 16, {}), (256, 64, 3, "e4m3zp", 16, {}), (256, 64, 2, "e4m3", 64, {}),
    (128, 64, 3, "e4m3zp", 32, dict(paged=False)), (256, 32, 4, "f16", 16, dict(paged=False))])
def test_compact(d, block, bits, scale, page, kw):
    n = 5 * page + 3
    c = Pages(d=d, block=block, bits=bits, scale=scale, page=page, lens=(n, n, n, page, 1, n - 1), maxp=8, **kw)
    rng = np.random.default_rng(d + bits)
    keep = rng.integers(0, n, (3, c.hkv, n - 1)).astype(np.int32)      # any order, any repeats
    keep[1] = np.sort(keep[1], -1)
    keep[2] %= page
    _compact(c, [0, 2, 3], [1, 5, 4], keep, [n - 1, n - 1, 1])
    _compact(c, [5], [0], keep[:1, :, :1] * 0, [1])
    _compact(c, [5, 4], [0, 1], keep[:2], [0, 0])                       # nothing kept
    assert c.flags() == 0


def test_compact_bad_arguments_on_the_device():
    c = Pages(lens=(40, 64, 64, 64, 64, 30, 64), maxp=4)
    keep = np.tile(np.arange(40, dtype=np.int32), (6, c.hkv, 1))
    keep[0, 0, 3], keep[0, 1, 5], keep[0, 1, 6] = -1, 40, 1 << 30     # outside the source
    c.table[3, 1] = -2
    c.table[5, 0] = c.N
    c.table_t.copy_(c.dev(c.table))
    # a fair pair with bad entries; ids out of range; equal ids; too many kept; a bad destination page, a bad source page
    _compact(c, [0, -1, 2, 4, 0, 5], [1, 2, 2, 6, 3, 6], keep, [40, 4, 4, 41, 40, 30])
    bits = c.K.DEV_BITS
    assert c.flags() == bits["bad_pos"] | bits["bad_seq"] | bits["bad_len"] | bits["bad_page"]
    c.status.zero_()
    c.lens = np.array([-4, 64, 65, 64, 64, 30, 64], np.int32)
    c.lens_t.copy_(c.dev(c.lens))
    _compact(c, [0, 2, 4, 5], [1, 3, 6, 6], keep[:4], [4, 4, -1, 65])
    assert c.flags() == bits["bad_len"]


# ------------------------------------------------------------ together
def _step_buffers(c, G, budget):
    t = c.torch
    heads = (c.B, c.hkv)
    return dict(
        scores=t.empty(*heads, c.maxp, device="cuda"), pages=t.empty(*heads, budget, dtype=t.int32, device="cuda"),
        counts=t.empty(*heads, dtype=t.int32, device="cuda"),
        q=t.empty(c.B, c.hkv * G, c.d, dtype=t.float16, device="cuda"),
        out=t.empty(c.B, c.hkv * G, c.d, dtype=t.float16, device="cuda"))


def _step(c, cache, b, bounds, first, k, v, seq, pos, q, budget):
    """One decode step of a serving loop over the page operators, with a copy and a kernel of torch's among them."""
    K = c.K
    b["q"].copy_(q)
    K.kvq3_write(c.rot.handle, c.desc, cache, k, v, seq, pos, c.status)
    K.kvq3_key_bounds(c.desc, cache, first, bounds, c.status)
    K.kvq3_page_scores(c.rot.handle, c.desc, cache, bounds, b["q"], b["scores"], c.status)
    b["pages"].fill_(-5)
    K.kvq3_page_select(c.desc, cache, b["scores"], budget, 1, 1, b["pages"], b["counts"], c.status)
    K.kvq3_decode_attn_pages(c.rot.handle, c.desc, cache, b["q"], b["pages"], b["counts"], b["out"], 0.0, c.status)


@pytest.mark.parametrize("how", ["eager", "side stream", "graph"])
def test_serving_loop(how):
    # a beam of three over one prompt: fork, write, summarise, score, select, attend; then evict and compact
    G, budget, hkv, page = 4, 4, 2, 16
    c = Pages(lens=(0,) * 5, maxp=10, spare=40, hkv=hkv, page=page)
    K, t, rng = c.K, c.torch, np.random.default_rng(31)
    n0 = 90
    ws = t.empty(K.kvq3_remap_workspace_size(c.desc), dtype=t.uint8, device="cuda")
    tables = [t.full((5, 10), -1, dtype=t.int32, device="cuda") for _ in range(2)]
    lens = [t.zeros(5, dtype=t.int32, device="cuda") for _ in range(2)]
    i32 = lambda x: c.dev(np.array(x, np.int32))   # noqa: E731
    oracle_pool, L, U = c.pool.copy(), c.layout, c.U
    # the prompt in row 0
    K.kvq3_remap(c.desc, c.cache_of(tables[0], lens[0]), i32([-1] * 5), i32([n0, 0, 0, 0, 0]), tables[1], lens[1], ws, c.status)
    k, v = (rng.standard_normal((n0, hkv, c.d)).astype(np.float16) for _ in range(2))
    cache = c.cache_of(tables[1], lens[1])
    K.kvq3_write(c.rot.handle, c.desc, cache, c.dev(k), c.dev(v), i32([0] * n0), i32(range(n0)), c.status)
    lens[1].copy_(i32([n0, 0, 0, 0, 0]))
    # three beams of it, room for one more token each
    K.kvq3_remap(c.desc, cache, i32([0, 0, 0, -1, -1]), i32([n0 + 1] * 3 + [0, 0]), tables[0], lens[0], ws, c.status)
    cache = c.cache_of(tables[0], lens[0])
    bounds = t.zeros(c.N, hkv, 2, c.d, dtype=t.float16, device="cuda")
    K.kvq3_key_bounds(c.desc, cache, None, bounds, c.status)
    lens[0].copy_(i32([n0 + 1] * 3 + [0, 0]))
    table = tables[0].cpu().numpy()
    assert (table[:3, :5] == table[0, :5]).all() and len(set(table[:3, 5])) == 3
    kn, vn = (rng.standard_normal((3, hkv, c.d)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((5, hkv * G, c.d)).astype(np.float16)
    args = (bounds, i32([n0] * 3 + [0, 0]), c.dev(kn), c.dev(vn), i32([0, 1, 2]), i32([n0] * 3), c.dev(q), budget)
    buf = _step_buffers(c, G, budget)
    t.cuda.synchronize()
    if how == "eager":
        _step(c, cache, buf, *args)
    else:
        s = t.cuda.Stream()
        with t.cuda.stream(s):
            _step(c, cache, buf, *args)
            if how == "graph":
                buf["out"].zero_()
                t.cuda.synchronize()
                graph = t.cuda.CUDAGraph()
                with t.cuda.graph(graph, stream=s):
                    _step(c, cache, buf, *args)
                for _ in range(3):
                    graph.replay()
    t.cuda.synchronize()
    assert c.flags() == 0
    # the same with the oracle
    assert O.write(oracle_pool, L, U, k, v, np.zeros(n0, np.int32), np.arange(n0, dtype=np.int32), table) == 0
    live = np.array([n0 + 1] * 3 + [0, 0])
    pool = c.pool_now()
    got_pages, got_counts = buf["pages"].cpu().numpy(), buf["counts"].cpu().numpy()
    assert (got_counts[:3] == budget).all() and (got_counts[3:] == 0).all()
    want_b = bounds.cpu().numpy().copy()
    PO.key_bounds(pool, L, live, table, want_b)
    assert np.array_equal(want_b.view(np.uint16), bounds.cpu().numpy().view(np.uint16))
    scores, tol = PO.page_scores(want_b, L, U, q, live, table)
    assert np.all(np.abs(buf["scores"].cpu().numpy()[:3, :, :6] - scores[:3, :, :6]) <= tol[:3, :, :6])
    want_pages, _ = PO.page_select(buf["scores"].cpu().numpy(), L, live, budget, 1, 1)
    assert np.array_equal(got_pages, want_pages)
    _near(buf["out"].cpu().numpy().astype(np.float64)[:3],
          PO.decode_pages(pool, L, U, q, live, table, got_pages, got_counts)[:3])
    # evict: beam 1 keeps 40 tokens, moved into row 3; then only row 3 stays
    keep = np.sort(np.stack([rng.permutation(n0 + 1)[:40] for _ in range(hkv)]), -1)[None].astype(np.int32)
    K.kvq3_remap(c.desc, cache, i32([0, 1, 2, -1, -1]), i32([n0 + 1] * 3 + [40, 0]), tables[1], lens[1], ws, c.status)
    cache = c.cache_of(tables[1], lens[1])
    K.kvq3_compact(c.desc, cache, i32([1]), i32([3]), c.dev(keep), i32([40]), c.status)
    lens[1].copy_(i32([n0 + 1] * 3 + [40, 0]))
    K.kvq3_remap(c.desc, cache, i32([3, -1, -1, -1, -1]), i32([41, 0, 0, 0, 0]), tables[0], lens[0], ws, c.status)
    t.cuda.synchronize()
    assert c.flags() == 0
    assert lens[0].cpu().tolist() == [40, 0, 0, 0, 0]
    last = tables[0].cpu().numpy()
    after = c.pool_now()
    for h in range(hkv):
        for w in (0, 1):
            want = O.read_rotated(pool, L, 1, h, w, 0, n0 + 1, table)[1][keep[0, h]]
            assert np.array_equal(O.read_rotated(after, L, 0, h, w, 0, 40, last)[1], want)


def test_bad_data_without_a_status_word():
    # the status word may be left out: bad data is skipped all the same
    c = Pages(lens=(40, 64, 33), maxp=4)
    c.lens_t.copy_(c.dev(np.array([40, 65, -3], np.int32)))
    t, K = c.torch, c.K
    b = _step_buffers(c, 4, 2)
    bounds = t.zeros(c.N, c.hkv, 2, c.d, dtype=t.float16, device="cuda")
    q = c.dev(c.queries(4))
    K.kvq3_key_bounds(c.desc, c.cache, None, bounds)
    K.kvq3_page_scores(c.rot.handle, c.desc, c.cache, bounds, q, b["scores"])
    K.kvq3_page_select(c.desc, c.cache, b["scores"], 2, 0, 1, b["pages"], b["counts"])
    b["pages"][0, :, 1] = 99
    K.kvq3_decode_attn_pages(c.rot.handle, c.desc, c.cache, q, b["pages"], b["counts"], b["out"])
    i32 = lambda x: c.dev(np.array(x, np.int32))   # noqa: E731
    out, lens = t.empty_like(c.table_t), t.empty_like(c.lens_t)
    K.kvq3_remap(c.desc, c.cache, i32([0, 7, 1]), i32([41, 5, 3]), out, lens,
                 t.empty(K.kvq3_remap_workspace_size(c.desc), dtype=t.uint8, device="cuda"))
    K.kvq3_compact(c.desc, c.cache, i32([0, 0]), i32([0, 1]), t.full((2, c.hkv, 3), -1, dtype=t.int32, device="cuda"), i32([3, 3]))
    t.cuda.synchronize()
    assert b["counts"].cpu().tolist() == [[2, 2], [0, 0], [0, 0]] and not b["out"][1:].any()
    assert lens.cpu().tolist() == [40, 0, 0] and (out[1:] == -1).all()
    c.pool_now()


def test_two_streams():
    # the same cache read by two streams at once (the attention has no workspace to share)
    c = Pages(lens=(700, 333, 64), page=16, hkv=2)
    t, G, row = c.torch, 4, 12
    q1, q2 = c.queries(G, 1), c.queries(G, 2)
    p1, n1 = _lists(c, row, 1)
    p2, n2 = _lists(c, row, 2)
    run = []
    for q, p, n in ((q1, p1, n1), (q2, p2, n2)):
        run.append((t.cuda.Stream(), c.dev(q), c.dev(p), c.dev(n), _step_buffers(c, G, row)))
    t.cuda.synchronize()
    for _ in range(20):
        for s, q, p, n, b in run:
            c.K.kvq3_decode_attn_pages(c.rot.handle, c.desc, c.cache, q, p, n, b["out"], 0.0, c.status, stream=s)
    t.cuda.synchronize()
    assert c.flags() == 0
    for q, p, n, r in ((q1, p1, n1, run[0]), (q2, p2, n2, run[1])):
        _near(r[4]["out"].cpu().numpy().astype(np.float64),
              PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, p, n))
