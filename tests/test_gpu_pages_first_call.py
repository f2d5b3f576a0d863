"""The page operators' first calls in a host thread made under stream capture: what they look up once (occupancy, kernel
attributes) may be looked up there, and the replayed graph gives what later plain calls give."""
import threading

import numpy as np
import pytest

from oracle import pages_oracle as PO
from test_gpu_pages import Pages, _near, _step_buffers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("kw,G", [(dict(d=64, block=32, bits=4, scale="f32", page=48), 6),
                                  (dict(d=256, block=32, bits=2, scale="f16", page=80), 11)])
def test_first_calls_of_a_thread_under_capture(kw, G):
    c = Pages(lens=(700, 333, 0, 65), maxp=20, spare=9, **kw)
    K, t = c.K, c.torch
    b = _step_buffers(c, G, 5)
    bounds = t.zeros(c.N, c.hkv, 2, c.d, dtype=t.float16, device="cuda")
    q = c.queries(G)
    b["q"].copy_(c.dev(q))
    i32 = lambda x: c.dev(np.array(x, np.int32))   # noqa: E731
    src, new = i32([0, 1, -1, 0]), i32([701, 320, 50, 690])
    table, lens = t.empty_like(c.table_t), t.empty_like(c.lens_t)
    ws = t.empty(K.kvq3_remap_workspace_size(c.desc), dtype=t.uint8, device="cuda")
    keep = c.dev(np.sort(c.rng.integers(0, 333, (1, c.hkv, 60)), -1).astype(np.int32))
    one, three, sixty = i32([1]), i32([3]), i32([60])
    t.cuda.synchronize()
    failed = []

    def run():
        try:
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph, stream=t.cuda.Stream()):
                K.kvq3_key_bounds(c.desc, c.cache, None, bounds, c.status)
                K.kvq3_page_scores(c.rot.handle, c.desc, c.cache, bounds, b["q"], b["scores"], c.status)
                K.kvq3_page_select(c.desc, c.cache, b["scores"], 5, 1, 1, b["pages"], b["counts"], c.status)
                K.kvq3_decode_attn_pages(c.rot.handle, c.desc, c.cache, b["q"], b["pages"], b["counts"], b["out"], 0.0,
                                         c.status)
                K.kvq3_remap(c.desc, c.cache, src, new, table, lens, ws, c.status)
                K.kvq3_compact(c.desc, c.cache, one, three, keep, sixty, c.status)
            for _ in range(2):
                graph.replay()
            t.cuda.synchronize()
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    before = c.pool.copy()
    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    assert not failed, failed
    assert c.flags() == 0
    # the oracle on the cache as it was: the copies and the gather come behind the attention, and again with it
    pages, counts = b["pages"].cpu().numpy(), b["counts"].cpu().numpy()
    for _ in range(2):
        want_b = np.zeros(bounds.shape, np.float16)
        PO.key_bounds(before, c.layout, c.lens, c.table, want_b)
        want = PO.decode_pages(before, c.layout, c.U, q, c.lens, c.table, pages, counts)
        want_t, want_l, _ = PO.remap(before, c.layout, c.table, c.lens, [0, 1, -1, 0], [701, 320, 50, 690])
        PO.compact(before, c.layout, c.table, c.lens, [1], [3], keep.cpu().numpy(), [60])
    assert np.array_equal(want_b.view(np.uint16), bounds.cpu().numpy().view(np.uint16))
    _near(b["out"].cpu().numpy().astype(np.float64), want)
    assert np.array_equal(table.cpu().numpy(), want_t) and np.array_equal(lens.cpu().numpy(), want_l)
    assert np.array_equal(c.pool_now(), before)
