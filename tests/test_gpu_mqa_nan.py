"""The tensor-core MQA on queries that are NaN: their rows of the output are
NaN, the other rows those of a call without them, bit for bit."""
import numpy as np
import pytest
import torch

import synth
from tests.gpu_util import code_rows, desc_for, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_sink", [False, True])
# queries, heads, sequences: keys split over CTAs, a CTA a query, two queries a CTA
@pytest.mark.parametrize("nq,H,B,sparse", [(6, 128, 3, False), (90, 128, 3, False),
                                           (256, 64, 1, False), (5, 64, 2, True),
                                           (200, 128, 2, True)])
def test_nan_queries_show(nq, H, B, sparse, with_sink):
    import long_context_compressed_kv_b200 as v
    rng = np.random.default_rng(nq)
    d, N, k = 512, 700, 96
    m = 4 if sparse else 128
    ldesc = desc_for(synth.Layer("csa" if sparse else "hca", m, H, d, 64, 128, 4, 32, k))
    kv, kv_sc = code_rows(ldesc, dev(rng.standard_normal((B, N, d)).astype(np.float32)),
                          v.E4M3_BF16ROPE, d_rope=64)
    swa, swa_sc = code_rows(ldesc, dev(rng.standard_normal((B, 256, d)).astype(np.float32)),
                            v.E4M3_BF16ROPE, d_rope=64)
    pos = rng.integers(300, m * N - 1, nq)
    pos[0] = -1                                                # a query without a key
    Q = rng.standard_normal((nq, H, d)).astype(np.float32)
    bad = rng.random((nq, H)) < 0.2
    bad[0] = False
    kw = dict(q_pos=dev(pos, torch.int64), q_seq=dev(np.sort(rng.integers(0, B, nq)), torch.int32),
              B=B, kv=kv, kv_scale=kv_sc, kv_rows=N, swa=swa, swa_scale=swa_sc, swa_rows=256,
              ws=v.workspace(ldesc, nq, N),
              sink=dev(rng.standard_normal(H).astype(np.float32)) if with_sink else None)
    if sparse:
        idx = np.stack([np.sort(rng.permutation(70)[:k % 70]) for _ in range(nq)])
        idx = np.pad(idx, ((0, 0), (0, k - idx.shape[1])), constant_values=-1)
        idx[0] = -1
        kw["idx"] = dev(idx, torch.int32)
        call = v.sparse_mqa
    else:
        kw["max_vis"] = N
        call = v.dense_mqa
    got = []
    for rows in (Q, np.where(bad[..., None], np.nan, Q)):
        out = torch.zeros(nq, H, d, device="cuda")
        call(ldesc, Q=dev(rows, torch.bfloat16), out=out, **kw)
        assert v.device_status(kw["ws"]) == 0
        got.append(out.cpu())
    clean, out = got
    bad = torch.from_numpy(bad)
    assert clean.isfinite().all() and (clean[0] == 0).all()
    assert out[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad])
