"""Attention over caches whose scales take 32 bytes a token (d = 256 in blocks of 32 with fp32 scales): the
decode and the chunked prefill read the scales of two tokens, 64 bytes, at once."""
import numpy as np
import pytest

import kvq3_inputs as I
from cases import TOL_DECODE, Case, rel_err
from oracle import kvq3_oracle as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("hq", [2, 7, 16])
def test_decode_and_prefill(bits, hq):
    c = Case(d=256, block=32, scale="f32", page=16, lens=(150, 33), hkv=1, hq=hq, bits=bits)
    k, v, si, ps = c.tokens()
    c.oracle_write(k, v, si, ps)
    c.upload_oracle_pool()
    q = c.queries()
    assert rel_err(c.gpu_decode(q), c.oracle_decode(q)) <= TOL_DECODE
    t, n = c.torch, 20
    qp = I.q_np(c.spec, n, hq, 5)
    out = t.empty((n, hq, c.d), dtype=t.float32, device=c.dev)
    ws = t.empty(c.K.kvq3_prefill_workspace_size(c.desc, hq, n), dtype=t.uint8, device=c.dev)
    c.K.kvq3_prefill_attn(c.rot.handle, c.desc, c.cache, 0, 130, t.as_tensor(qp, device=c.dev), out, ws, 0.0, c.status)
    ref = O.prefill(c.pool_o, c.layout, c.U, qp, 0, 130, c.table)
    assert c.device_status() == 0
    assert rel_err(out.cpu().numpy().astype(np.float64), ref) <= TOL_DECODE
