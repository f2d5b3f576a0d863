"""Pages with keys past the fp16 range of the key bounds: an infinite bound gives the page the highest score, whatever
the sign of the query there, and the page is selected."""
import numpy as np
import pytest

from oracle import pages_oracle as PO
from test_gpu_pages import Pages, _bounds, _random_bounds, _scores, _select_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("d,G", [(64, 4), (128, 1), (128, 8), (256, 16)])
def test_scores_of_bounds_that_are_not_finite(d, G):
    c = Pages(d=d, page=16, lens=(700, 33), maxp=46)
    q, bounds = c.queries(G), _random_bounds(c)
    q[1, : G // 2 + 1] = 0                     # a query of zeros meets them too
    at = c.table[0]
    inf = np.float16(np.inf)
    bounds[at[0], :, 1, 5] = inf               # the maximum of one channel
    bounds[at[3], :, 0, d - 1] = -inf          # the minimum of one
    bounds[at[7], :, 0, 0], bounds[at[7], :, 1, 0] = -inf, inf
    bounds[at[9], :, :, 17] = inf              # every token of a channel past the range
    bounds[at[9], :, :, 40] = -inf
    bounds[at[11], 0, 1, 2] = np.nan           # one kv head of a page
    bounds[c.table[1, 2], :, 1, 8:24] = inf
    got = _scores(c, bounds, q).astype(np.float64)
    want, tol = PO.page_scores(bounds, c.layout, c.U, q, c.lens, c.table)
    assert np.isposinf(want).sum() == 2 * 4 + 1 + 2
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert np.all(np.abs(got[fin] - want[fin]) <= tol[fin])
    assert c.flags() == 0


def test_a_page_past_the_range_is_selected():
    # fp32 scales of 1e5 in one page: its bounds are infinite, its score the highest, and it is attended
    c = Pages(d=128, block=32, scale="f32", page=16, lens=(40 * 16,), hkv=1)
    L, far = c.layout, 13
    o = L.record_offset(int(c.table[0, far]), 0, 0)
    c.pool[o:o + 16 * L.nb * 4] = np.full(16 * L.nb, 1e5, np.float32).view(np.uint8)
    c.pool_full[:c.pool.size].copy_(c.dev(c.pool))
    with np.errstate(over="ignore"):
        got, want = _bounds(c)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16)) and np.isinf(got[c.table[0, far]]).any()
    scores = _scores(c, got, c.queries(4))
    assert np.isposinf(scores[0, 0, far]) and np.isfinite(np.delete(scores[0, 0], far)).all()
    assert _select_case([40 * 16], 40, 1, scores, 3, 1, 1) == 0
    assert PO.page_select(scores, L, c.lens, 3, 1, 1)[0][0, 0].tolist() == [0, far, 39]
