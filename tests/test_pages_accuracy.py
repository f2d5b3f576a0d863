"""The bar on the page scores' root mean square error (oracle/pages_oracle.py: SCORE_RMS) on the CPU: the kernel's
scheme, computed here as it is written down, passes it; the same without the low half of the query, or with that half
in the wrong place, does not, at any head dimension."""
import numpy as np
import pytest

from oracle import kvq3_oracle as O
from oracle import pages_oracle as PO


def case(d, G, pages=300, seed=0):
    rng = np.random.default_rng(seed + d + G)
    L = O.Layout(d, 2, 64, "f16", 16, 1, pages, pages)
    mid, half = rng.standard_normal((pages, 2, 1, d)), rng.random((pages, 2, 1, d)) * 2
    bounds = np.concatenate([mid - half, mid + half], 2).astype(np.float16)
    U = O.rotation_matrix(*O.rotation_params(d, 42, True, True))
    q = rng.standard_normal((1, 2 * G, d)).astype(np.float16)
    return L, U, bounds, q, np.array([16 * pages], np.int32), np.arange(pages, dtype=np.int32)[None]


def cut(x):
    """fp64 cut to 24 bits towards zero."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24), e - 24)


def scheme(L, U, bounds, q, halves, chain):
    """Scores [1][2][pages]: the query's negative part against the minima and its positive part against the maxima, in
    fp16 halves, chains of `chain` steps of 16 products cut to 24 bits a step, the chains added in fp32."""
    d = L.d
    q1 = (q.astype(np.float64) @ U.T).astype(np.float32).reshape(2, -1, d)
    sc = np.exp2(8 - np.ceil(np.log2(np.abs(q1).max(-1, keepdims=True)))).astype(np.float32)
    x = (q1 * sc)
    w = np.concatenate([np.minimum(x, 0), np.maximum(x, 0)], -1)                    # [h][G][2d]
    hi = w.astype(np.float16)
    lo = (w - hi.astype(np.float32)).astype(np.float16)
    a = np.concatenate([bounds[:, :, 0], bounds[:, :, 1]], -1).astype(np.float64)   # [pages][h][2d]
    out = np.full((1, 2, len(bounds)), -np.inf)
    for h in range(2):
        for g in range(w.shape[1]):
            total = 0.0
            for part in halves(hi[h, g], lo[h, g]):
                prod = (a[:, h] * part.astype(np.float64)).reshape(len(bounds), -1, 16).sum(-1)
                s = np.zeros(len(bounds), np.float32)
                for c in range(0, prod.shape[1], chain):
                    acc = np.zeros(len(bounds))
                    for k in range(c, min(c + chain, prod.shape[1])):
                        acc = cut(acc + prod[:, k])
                    s = (s + acc.astype(np.float32)).astype(np.float32)
                total = s + total
            out[0, h] = np.maximum(out[0, h], total / sc[h, g])
    return out


def rms_error(L, U, bounds, q, lens, table, halves, chain=8):
    got = scheme(L, U, bounds, q, halves, chain)
    want, _ = PO.page_scores(bounds, L, U, q, lens, table)
    T = PO.page_scores_size(bounds, L, U, q, lens, table)
    return np.sqrt(np.mean((got - want) ** 2)) / np.sqrt(np.mean(T ** 2))


@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 4), (128, 16), (256, 4), (256, 16)])
def test_the_bar_tells_a_lost_half(d, G):
    c = case(d, G)
    assert rms_error(*c, lambda hi, lo: (hi, lo)) <= PO.SCORE_RMS
    assert rms_error(*c, lambda hi, lo: (hi,)) > PO.SCORE_RMS
    assert rms_error(*c, lambda hi, lo: (hi, np.roll(lo, 16))) > PO.SCORE_RMS        # a k-step off
    assert rms_error(*c, lambda hi, lo: (hi, np.roll(lo, 1))) > PO.SCORE_RMS


def test_long_chains_cost_more():
    # why the kernel adds up in fp32 after 8 steps: the cuts of one chain of 32 grow with its running sum (the bar
    # leaves room for the rest of the scheme and is not what tells them)
    c = case(256, 4)
    assert rms_error(*c, lambda hi, lo: (hi, lo), 32) > 2 * rms_error(*c, lambda hi, lo: (hi, lo), 8)


def test_the_size_is_an_upper_bound():
    c = case(64, 2, pages=20)
    want, _ = PO.page_scores(c[2], *c[:2], *c[3:])
    assert np.all(np.abs(want) <= PO.page_scores_size(c[2], *c[:2], *c[3:]) * (1 + 1e-12))
