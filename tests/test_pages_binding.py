"""What the page operators' binding refuses before anything is launched: a status word that is no int32 CUDA tensor, a
tensor of another number of dimensions, something that is no tensor.  No GPU needed: the library's functions are
replaced by one that fails the test when it is called."""
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def K():
    lib = os.path.join(ROOT, "hadamard_rotated_bit_kvq3_gb300", "libkvq3.so")
    if not os.path.exists(lib):
        import __graft_entry__
        __graft_entry__.build()
    import hadamard_rotated_bit_kvq3_gb300 as K
    return K


class _Library:
    def __getattr__(self, name):
        def called(*args):
            pytest.fail(f"{name} was called")
        return called


def _z(*shape, t=torch.int32):
    return torch.zeros(*shape, dtype=t)


def _calls(K, **other):
    """Each page operator's call as (name, function of the status word) with tensors of the right types and shapes, but
    for those named in `other`."""
    d = K.CacheDesc(128, 2, 64, 3, 1, 1e-6, 16, 3, 4, 0, 12)
    c = K.Cache(4096, 8192, 12288)
    f16, f32, u8 = torch.float16, torch.float32, torch.uint8
    a = dict(first=_z(3), bounds=_z(12, 2, 2, 128, t=f16), q=_z(3, 8, 128, t=f16), scores=_z(3, 2, 4, t=f32),
             pages=_z(3, 2, 4), counts=_z(3, 2), out=_z(3, 8, 128, t=f16), src=_z(3), new=_z(3), table=_z(3, 4), lens=_z(3),
             ws=_z(4096, t=u8), ids=_z(2), keep=_z(2, 2, 4), n_keep=_z(2))
    a.update(other)
    a = type("Args", (), a)
    return [
        ("key_bounds", lambda s: K.kvq3_key_bounds(d, c, a.first, a.bounds, s)),
        ("page_scores", lambda s: K.kvq3_page_scores(None, d, c, a.bounds, a.q, a.scores, s)),
        ("page_select", lambda s: K.kvq3_page_select(d, c, a.scores, 4, 0, 1, a.pages, a.counts, s)),
        ("decode_attn_pages", lambda s: K.kvq3_decode_attn_pages(None, d, c, a.q, a.pages, a.counts, a.out, 0.0, s)),
        ("remap", lambda s: K.kvq3_remap(d, c, a.src, a.new, a.table, a.lens, a.ws, s)),
        ("compact", lambda s: K.kvq3_compact(d, c, a.ids, a.ids, a.keep, a.n_keep, s)),
    ]


@pytest.mark.parametrize("status", [_z(1), _z(1, t=torch.int64), _z(0), np.zeros(1, np.int32), 4096],
                         ids=["cpu", "int64", "empty", "numpy", "address"])
def test_a_status_word_that_is_no_cuda_int32(K, monkeypatch, status):
    monkeypatch.setattr(K, "lib", _Library())
    monkeypatch.setattr(K, "_at", lambda t, *a: t.data_ptr())   # the other tensors pass
    for name, call in _calls(K):
        with pytest.raises(ValueError, match="dev_status"):
            call(status)


@pytest.mark.parametrize("name,bad", [
    ("bounds", _z(128, t=torch.float16)), ("bounds", torch.tensor(1.0, dtype=torch.float16)), ("q", _z(3, t=torch.float16)),
    ("q", _z(3, 8, 128, 1, t=torch.float16)), ("pages", _z(3, 2)), ("keep", _z(2, 2)), ("keep", torch.tensor(3, dtype=torch.int32)),
    ("ids", torch.tensor(1, dtype=torch.int32)), ("ws", torch.tensor(1, dtype=torch.uint8)),
    ("bounds", np.zeros((12, 2, 2, 128), np.float16)), ("q", None), ("pages", [0, 1]), ("first", np.zeros(3, np.int32)),
    ("scores", None), ("counts", 4096), ("src", [0, 1, 2]), ("table", None), ("ws", bytearray(4096)), ("keep", None), ("n_keep", None)])
def test_other_dimensions_and_no_tensors(K, monkeypatch, name, bad):
    # device and alignment aside, every tensor but the bad one is as it should be: only that one is refused
    monkeypatch.setattr(K, "lib", _Library())
    plain = K._at
    monkeypatch.setattr(K, "_at", lambda t, *a: plain(t, *a) if t is bad else 4096)
    found = 0
    for op, call in _calls(K, **{name: bad}):
        try:
            call(_z(0))                  # refused in any case: by its status word where the bad tensor plays no part
        except ValueError as e:
            found += "dev_status" not in str(e)
    assert found
