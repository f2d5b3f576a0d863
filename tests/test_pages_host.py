"""Refusals and sizes of the page operators: argument checks on the host, nothing is launched.  No GPU needed."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
A, B, C = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)   # aligned, never read


@pytest.fixture(scope="module")
def K():
    lib = os.path.join(ROOT, "hadamard_rotated_bit_kvq3_gb300", "libkvq3.so")
    if not os.path.exists(lib):
        import __graft_entry__
        __graft_entry__.build()
    import hadamard_rotated_bit_kvq3_gb300 as K
    return K


def _desc(K, **kw):
    base = dict(head_dim=128, num_kv_heads=2, block=64, bits=3, scale_type=1, eps=1e-6, page_size=16, batch=3,
                max_pages_per_seq=4, reserved=0, num_pages=12)
    base.update(kw)
    return K.CacheDesc(**base)


def _cache(K, pool=4096, table=8192, lens=12288):
    return K.Cache(pool, table, lens)


def test_key_bounds_refusals(K):
    def call(desc, cache, bounds):
        return K.lib.kvq3_key_bounds(ctypes.byref(desc), ctypes.byref(cache), None, bounds, None, None)
    d = _desc(K)
    assert call(d, _cache(K), None) == INVALID
    assert call(d, _cache(K), ctypes.c_void_p(4104)) == INVALID
    assert call(d, _cache(K, lens=None), A) == INVALID
    assert call(d, _cache(K, pool=4100), A) == INVALID
    assert call(_desc(K, num_pages=11), _cache(K, table=None), A) == INVALID   # contiguous: batch * max_pages pages
    assert call(_desc(K, bits=5), _cache(K), A) == UNSUPPORTED


def test_page_scores_refusals(K):
    rot, rot64 = K.Rotation(128, 1), K.Rotation(64, 1)
    def call(desc, hq=8, r=rot.handle, bounds=A, q=B, scores=C, cache=None):   # noqa: E306
        return K.lib.kvq3_page_scores(r, ctypes.byref(desc), ctypes.byref(cache or _cache(K)), bounds, q, hq, scores,
                                      None, None)
    d = _desc(K)
    for kw in (dict(r=None), dict(r=rot64.handle), dict(bounds=None), dict(q=None), dict(scores=None), dict(hq=0),
               dict(hq=7), dict(bounds=ctypes.c_void_p(8)), dict(q=ctypes.c_void_p(24)), dict(scores=ctypes.c_void_p(2)),
               dict(cache=_cache(K, lens=None))):
        assert call(d, **kw) == INVALID, kw
    assert call(d, hq=34) == UNSUPPORTED                                        # 17 heads per kv head
    assert call(_desc(K, max_pages_per_seq=(1 << 31) - 1, batch=1 << 10)) == UNSUPPORTED   # more than 2^31 tiles


def test_page_select_refusals(K):
    def call(budget=4, sinks=1, recent=1, desc=None, cache=None, scores=A, pages=B, counts=C):
        return K.lib.kvq3_page_select(ctypes.byref(desc or _desc(K)), ctypes.byref(cache or _cache(K)), scores, budget,
                                      sinks, recent, pages, counts, None, None)
    for kw in (dict(budget=0), dict(budget=-1), dict(sinks=-1), dict(recent=0), dict(sinks=4), dict(recent=4),
               dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), dict(scores=None), dict(pages=None), dict(counts=None),
               dict(cache=_cache(K, lens=None))):
        assert call(**kw) == INVALID, kw
    assert call(desc=_desc(K, batch=(1 << 30), num_kv_heads=2)) == UNSUPPORTED


def test_decode_attn_pages_refusals(K):
    rot, rot64 = K.Rotation(128, 1), K.Rotation(64, 1)
    def call(desc=None, hq=8, n=4, r=rot.handle, q=A, pages=A, counts=B, out=C, sm=0.0, cache=None):   # noqa: E306
        return K.lib.kvq3_decode_attn_pages(r, ctypes.byref(desc or _desc(K)), ctypes.byref(cache or _cache(K)), q, hq, sm,
                                            pages, counts, n, out, None, None)
    for kw in (dict(r=None), dict(r=rot64.handle), dict(q=None), dict(pages=None), dict(counts=None), dict(out=None),
               dict(hq=0), dict(hq=9), dict(n=0), dict(n=-3), dict(sm=float("inf")), dict(cache=_cache(K, lens=None)),
               dict(q=ctypes.c_void_p(4104)), dict(out=ctypes.c_void_p(4098))):
        assert call(**kw) == INVALID, kw
    assert call(hq=34) == UNSUPPORTED
    assert call(n=(1 << 31) // 16) == UNSUPPORTED                               # a list of 2^31 tokens
    assert call(desc=_desc(K, batch=(1 << 28))) == UNSUPPORTED                  # 2^31 query rows


def test_remap_refusals_and_workspace(K):
    d = _desc(K)
    need = K.kvq3_remap_workspace_size(d)
    up = lambda n: (n + 255) // 256 * 256   # noqa: E731
    n, b = 12, 3
    assert need == up(4 * -(-n // 32)) + 2 * up(4 * n) + 2 * up(4 * b) + up(8 * b) + 2 * up(16 * b)
    table, lens = ctypes.c_void_p(8192), ctypes.c_void_p(12288)

    D, E = ctypes.c_void_p(1 << 23), ctypes.c_void_p(1 << 24)

    def call(src=A, new=B, table_out=C, lens_out=D, ws=E, n_ws=need, desc=d, cache=None):
        return K.lib.kvq3_remap(ctypes.byref(desc), ctypes.byref(cache or _cache(K)), src, new, table_out, lens_out, ws,
                                n_ws, None, None)
    for kw in (dict(src=None), dict(new=None), dict(table_out=None), dict(lens_out=None), dict(table_out=table),
               dict(table_out=ctypes.c_void_p(8192 + 44)), dict(table_out=ctypes.c_void_p(8192 - 4)),
               dict(lens_out=lens), dict(lens_out=ctypes.c_void_p(12288 + 8)),
               dict(lens_out=A), dict(lens_out=B), dict(table_out=A), dict(table_out=ctypes.c_void_p((1 << 21) - 4)),
               dict(lens_out=ctypes.c_void_p((1 << 22) + 40)), dict(lens_out=table), dict(cache=_cache(K, table=None)), dict(cache=_cache(K, lens=None))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(n_ws=need - 1), dict(ws=ctypes.c_void_p(264))):
        assert call(**kw) == WORKSPACE, kw
    with pytest.raises(K.Kvq3Error) as e:
        K.kvq3_remap_workspace_size(_desc(K, num_pages=1 << 31))
    assert e.value.status == UNSUPPORTED


def test_compact_refusals(K):
    def call(n=2, stride=4, src=A, dst=A, keep=B, n_keep=C, cache=None, desc=None):
        return K.lib.kvq3_compact(ctypes.byref(desc or _desc(K)), ctypes.byref(cache or _cache(K)), src, dst, n, keep,
                                  n_keep, stride, None, None)
    assert call(n=0) == OK and call(stride=0) == OK and call(n=0, src=None, keep=None) == OK   # nothing to do
    for kw in (dict(n=-1), dict(stride=-1), dict(src=None), dict(dst=None), dict(keep=None), dict(n_keep=None),
               dict(cache=_cache(K, lens=None))):
        assert call(**kw) == INVALID, kw
    assert call(n=(1 << 30), stride=1 << 20) == UNSUPPORTED


def test_binding_refuses_other_tensors(K):
    torch = pytest.importorskip("torch")
    d, c = _desc(K), _cache(K)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)   # noqa: E731  (CPU tensors: refused as such)
    with pytest.raises(ValueError):
        K.kvq3_key_bounds(d, c, None, z(12, 2, 2, 128, t=torch.float16))
    with pytest.raises(ValueError):
        K.kvq3_page_select(d, c, z(3, 2, 4, t=torch.float32), 4, 0, 1, z(3, 2, 4), z(3, 2))
    with pytest.raises(ValueError):
        K.kvq3_remap(d, c, z(3), z(3), z(3, 4), z(3), z(8, t=torch.uint8))
    with pytest.raises(ValueError):
        K.kvq3_compact(d, c, z(2), z(2), z(2, 2, 4), z(2))


def test_status_bit_is_in_the_header(K):
    header = open(os.path.join(ROOT, "include", "kvq3.h")).read()
    assert "KVQ3_DEV_NO_PAGE = 128" in header and K.DEV_BITS["no_page"] == 128
