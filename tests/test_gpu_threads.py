"""Calls from host threads that have made no CUDA call before."""
import threading

import numpy as np
import pytest
import torch

from tests.kv_util import Case, check, reference
from tests.test_gpu_kv import desc_of, outputs, v4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def test_two_host_threads_at_once():
    """Two threads, each with a stream, a workspace and a layer of its own type."""
    v = v4()
    work = []
    for dtype, d in (("bf16", 128), ("fp16", 64)):
        c = Case([3, 1], [900, 700], 8, 2, d, dtype, seed=d)
        desc = desc_of(c)
        kw = c.args(v.kv_workspace(desc))
        work.append((c, desc, c.q.cuda(), *outputs(c), kw, torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def run(c, desc, q, out, lse, kw, stream):
        try:
            for _ in range(200):
                v.paged_attention(desc, q=q, out=out, lse=lse, stream=stream, **kw)
        except Exception as e:          # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for c, _, _, out, lse, _, _ in work:
        check(c, out, lse, reference(c))


def test_compressed_layers_in_a_new_thread():
    import synth
    from tests.gpu_util import code_rows, desc_for, dev
    v = v4()
    rng = np.random.default_rng(3)
    m, H, d, N, B, nq = 128, 128, 512, 700, 3, 6
    ldesc = desc_for(synth.Layer("hca", m, H, d, 64, 128, 4, 32, 96))
    kv, kv_sc = code_rows(ldesc, dev(rng.standard_normal((B, N, d)).astype(np.float32)),
                          v.E4M3_BF16ROPE, d_rope=64)
    swa, swa_sc = code_rows(ldesc, dev(rng.standard_normal((B, 256, d)).astype(np.float32)),
                            v.E4M3_BF16ROPE, d_rope=64)
    kw = dict(Q=dev(rng.standard_normal((nq, H, d)).astype(np.float32), torch.bfloat16),
              q_pos=dev(rng.integers(0, m * N, nq), torch.int64),
              q_seq=dev(rng.integers(0, B, nq), torch.int32), B=B, kv=kv, kv_scale=kv_sc,
              kv_rows=N, swa=swa, swa_scale=swa_sc, swa_rows=256, max_vis=N,
              ws=v.workspace(ldesc, nq, N))
    outs = [torch.zeros(nq, H, d, device="cuda") for _ in range(2)]
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            v.dense_mqa(ldesc, out=outs[1], stream=stream, **kw)
        except Exception as e:          # noqa: BLE001 (shown below)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not failed, failed
    v.dense_mqa(ldesc, out=outs[0], **kw)
    assert v.device_status(kw["ws"]) == 0
    assert torch.equal(*outs) and outs[0].abs().max() > 0
