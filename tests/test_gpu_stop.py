"""Waits of the decode loop that run out at a later chunk than the first: with a few polls a wait some CTAs get through
several chunks before one does, and the warps of a CTA still leave together (tests/test_stop_protocol.py explores why).
Every call returns, reports what happened, leaves the buffers usable; a call that reports nothing gives the result."""
import ctypes

import numpy as np
import pytest

from cases import TOL_DECODE, Case, rel_err
from oracle import pages_oracle as PO
from test_gpu_pages import Pages, _attend, _lists, _near

pytestmark = pytest.mark.gpu

POLLS = (1, 2, 5, 12, 40, 150, 1000)
TIMEOUT = 32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("kw,G,row", [
    (dict(lens=(9000, 8000, 100, 1), page=32, hkv=4), 4, 250), (dict(lens=(9000, 40), page=16, d=256, hkv=2), 4, 500),
    (dict(lens=(20000,), page=128, hkv=1, scale="e4m3"), 8, 150), (dict(lens=(5000, 17), page=16, hkv=2), 16, 300)])
def test_selected_pages(kw, G, row):
    c = Pages(**kw)
    K, t = c.K, c.torch
    fn = K.lib.kvq3_test_decode_pages_polls
    fn.restype, fn.argtypes = ctypes.c_int, K.lib.kvq3_decode_attn_pages.argtypes + [ctypes.c_uint32]
    q = c.queries(G)
    pages, counts = _lists(c, row)
    want = PO.decode_pages(c.pool, c.layout, c.U, q, c.lens, c.table, pages, counts)
    qd, pd, nd = c.dev(q), c.dev(pages), c.dev(counts)
    full, out = c.guarded(q.shape, t.float16, 9.0)
    for polls in POLLS:
        assert fn(c.rot.handle, c.desc, c.cache, qd.data_ptr(), q.shape[1], 0.0, pd.data_ptr(), nd.data_ptr(), row,
                  out.data_ptr(), c.status.data_ptr(), K._raw_stream(None), polls) == 0
        t.cuda.synchronize()
        assert bool((full[-64:] == 9.0).all()) and c.flags() in (0, TIMEOUT)
        if c.flags() == 0:
            _near(out.cpu().numpy().astype(np.float64), want)
        c.status.zero_()
    _near(_attend(c, q, pages, counts), want)
    assert c.flags() == 0


@pytest.mark.parametrize("cfg", [
    dict(d=128, block=64, scale="f16", page=64, lens=(9000, 1, 129, 4000), hkv=2, hq=8),
    dict(d=256, block=64, scale="f16", page=16, lens=(3000, 17, 1000), hkv=2, hq=8, paged=True),
    dict(d=128, block=64, scale="e4m3", page=64, lens=(8000, 333), hkv=2, hq=32),
], ids=lambda c: f"d{c['d']}-{c['scale']}-G{c['hq'] // c['hkv']}")
def test_dense_decode(cfg):
    import torch
    import hadamard_rotated_bit_kvq3_gb300 as K
    fn = K.lib.kvq3_test_decode_attn_polls
    fn.restype, fn.argtypes = ctypes.c_int, K.lib.kvq3_decode_attn.argtypes + [ctypes.c_uint32]
    c = Case(**cfg)
    k, v, si, ps = c.tokens()
    c.oracle_write(k, v, si, ps)
    c.upload_oracle_pool()
    want = c.oracle_decode(c.queries())
    q = torch.as_tensor(c.queries(), device="cuda")
    ws = torch.empty(K.kvq3_decode_workspace_size(c.desc, c.hq), dtype=torch.uint8, device="cuda")
    out = torch.zeros((c.B, c.hq, c.d), dtype=torch.float32, device="cuda")
    for polls in POLLS:
        assert fn(c.rot.handle, ctypes.byref(c.desc), ctypes.byref(c.cache), q.data_ptr(), c.hq, 0.0, out.data_ptr(),
                  ws.data_ptr(), ws.numel(), c.status.data_ptr(), K._raw_stream(None), polls) == 0
        torch.cuda.synchronize()
        status = c.device_status()
        assert status in (0, TIMEOUT)
        if status == 0:
            assert rel_err(out.cpu().numpy().astype(np.float64), want) <= TOL_DECODE
        c.status.zero_()
    assert rel_err(c.gpu_decode(c.queries()), want) <= TOL_DECODE
    assert c.device_status() == 0
