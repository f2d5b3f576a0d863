"""Page scores' root mean square error over many pages against 64 bits: a bar that a lost or misplaced low half of the
query does not pass (tests/test_pages_accuracy.py shows that on the CPU)."""
import numpy as np
import pytest

from oracle import pages_oracle as PO
from test_gpu_pages import Pages, _random_bounds, _scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 16])
def test_rms_error_of_the_scores(d, G):
    c = Pages(d=d, page=16, lens=(4800, 2001), flags=7 if G == 3 else 3)
    q, bounds = c.queries(G), _random_bounds(c)
    got = _scores(c, bounds, q).astype(np.float64)
    want, _ = PO.page_scores(bounds, c.layout, c.U, q, c.lens, c.table)
    T = PO.page_scores_size(bounds, c.layout, c.U, q, c.lens, c.table)
    there = T > 0
    err = np.sqrt(np.mean((got[there] - want[there]) ** 2)) / np.sqrt(np.mean(T[there] ** 2))
    print(f"rms error {err:.2e} of T")
    assert err <= PO.SCORE_RMS
    assert c.flags() == 0
