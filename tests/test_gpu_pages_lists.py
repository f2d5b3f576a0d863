"""Attention over lists with entries behind the sequence's part-filled newest page that are no pages: padding inside
the count, page numbers past the end.  Those entries are left out and reported; the newest tokens are attended."""
import numpy as np
import pytest

from oracle import pages_oracle as PO
from test_gpu_pages import Pages, _attend, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("kw,G", [
    (dict(page=16), 4), (dict(page=64, scale="e4m3"), 8), (dict(page=16, d=256), 4), (dict(page=48, d=64, bits=2), 16),
    (dict(page=128, scale="e4m3zp"), 3), (dict(page=256), 1)])
def test_entries_behind_the_part_filled_page(kw, G):
    P = kw["page"]
    n = 3 * P + 2                                   # pages 0 .. 3, two tokens in the last
    for row in (5, 300, 4000):                      # CTAs of a cluster that hold nothing but padding
        c = Pages(lens=(n,) * 8, hkv=1, maxp=8, **kw)
        q = c.queries(G)
        lists = [[0, 3], [0, 3, 99], [0, 3, -1], [0, 1, 3] + [-1] * (row - 3), [3] + [7, 6, 5, 4], [2, 3, 1 << 30, -(1 << 31)],
                 [0, 1, 2, 3] + [4] * (row - 4), [-1, 3, 4]]
        pages = np.full((8, 1, row), -1, np.int32)
        counts = np.zeros((8, 1), np.int32)
        for b, x in enumerate(lists):
            pages[b, 0, :len(x)], counts[b, 0] = x, len(x)
        got = _attend(c, q, pages, counts)
        assert c.flags() == c.K.DEV_BITS["bad_page"]
        want = PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts)
        _near(got, want)
        # by hand: the same lists without the entries that are no pages
        for b, x in enumerate(lists):
            x = [e for e in x if 0 <= e <= 3]
            pages[b, 0, :len(x)], counts[b, 0] = x, len(x)
        c.status.zero_()
        plain = _attend(c, q, pages, counts)
        assert c.flags() == 0
        _near(plain, want)
        assert np.array_equal(got[0], plain[0])


def test_a_part_filled_page_with_pages_behind_it():
    # left out, as kvq3.h has it: a page of the sequence follows it
    c = Pages(lens=(50,) * 4, hkv=1, maxp=8, page=16)
    q = c.queries(4)
    pages = np.array([[[0, 3, 3, -1]], [[0, 3, 1, -1]], [[3, 0, 3, 8]], [[0, 3, 5, 2]]], np.int32)
    counts = np.array([[3], [3], [4], [4]], np.int32)
    got = _attend(c, q, pages, counts)
    assert c.flags() == c.K.DEV_BITS["bad_page"]
    _near(got, PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts))
    # third list: the first 3 has pages behind it, 0 is not above it, the second 3 is above 0 and has none
    same = np.array([[[0]], [[0]], [[3]], [[0]]], np.int32)
    c.status.zero_()
    _near(got, _attend(c, q, same, np.ones((4, 1), np.int32)))


@pytest.mark.parametrize("tail", [1, 3, 40, 700])
def test_padding_behind_long_lists(tail):
    # the part-filled page in a CTA's later chunks, past the pages that it looks up ahead, with padding in the same
    # chunk and in chunks of its own
    for kw, n in ((dict(d=64, block=64, bits=2, page=16), 70001), (dict(page=64), 30001)):
        c = Pages(lens=(n,), hkv=1, **kw)
        q = c.queries(2)
        k = -(-n // c.page)
        pages = np.concatenate([np.arange(k), np.where(np.arange(tail) % 2, -1, k + np.arange(tail))]).astype(np.int32)[None, None]
        got = _attend(c, q, pages, np.array([[k + tail]], np.int32))
        assert c.flags() == c.K.DEV_BITS["bad_page"]
        _near(got, PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, np.array([[k + tail]], np.int32)))
