"""Host-side checks of the 16-bit K/V layers' calls: every refusal is made
before a launch (fake pointers, never dereferenced; no GPU needed)."""
import ctypes

import pytest
import torch

from long_context_compressed_kv_b200 import _abi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only check with fake device pointers")
FAKE, WS = 1 << 20, 1 << 21
INVALID, UNSUPPORTED, WORKSPACE = _abi.ERR_INVALID_ARG, _abi.ERR_UNSUPPORTED, _abi.ERR_WORKSPACE


def desc(**kw):
    f = dict(Hq=8, Hkv=2, d=128, d_rope=64, rope_theta=1e4, rope_halves=0, softmax_scale=0.0,
             n_win=0, dtype=_abi.BF16)
    f.update(kw)
    return _abi.KvDesc(**f)


def batch(**kw):
    f = dict(T=4, B=2, k_cache=FAKE, v_cache=FAKE, n_blocks=8, q_start=FAKE, kv_len=FAKE,
             block_table=FAKE, blocks_per_seq=4)
    f.update(kw)
    return f


def append(d=None, ws_bytes=None, ws=WS, **kw):
    lib, d = _abi.load(), d or desc()
    f = batch(k=FAKE, k_token_stride=1024, k_head_stride=128, v=FAKE, v_token_stride=1024,
              v_head_stride=128)
    f.update(kw)
    n = lib.v4attn_kv_workspace_size(ctypes.byref(d)) if ws_bytes is None else ws_bytes
    return lib.v4attn_kv_append(ctypes.byref(d), ctypes.byref(_abi.KvAppendArgs(**f)), ws, n, None)


def attention(fn="v4attn_paged_attention", d=None, ws_bytes=None, ws=WS, **kw):
    lib, d = _abi.load(), d or desc()
    f = batch(q=FAKE, q_token_stride=1024, q_head_stride=128, out=FAKE, out_token_stride=1024,
              out_head_stride=128, n_lists=1)
    f.update(kw)
    n = lib.v4attn_kv_workspace_size(ctypes.byref(d)) if ws_bytes is None else ws_bytes
    return getattr(lib, fn)(ctypes.byref(d), ctypes.byref(_abi.KvAttnArgs(**f)), ws, n, None)


@pytest.mark.parametrize("bad,want", [
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID),
    (dict(Hq=2048, Hkv=16), UNSUPPORTED), (dict(Hq=129, Hkv=1), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dtype=_abi.F32), UNSUPPORTED),
    (dict(d_rope=-16), INVALID), (dict(d_rope=144), INVALID), (dict(d_rope=24), UNSUPPORTED),
    (dict(rope_theta=0.0), INVALID), (dict(rope_theta=float("nan")), INVALID),
    (dict(n_win=-1), INVALID), (dict(softmax_scale=float("inf")), INVALID)])
def test_layers_that_are_refused(bad, want):
    d = desc(**bad)
    assert _abi.load().v4attn_kv_workspace_size(ctypes.byref(d)) == 0
    assert append(d, ws_bytes=1 << 40) == want
    assert attention(d=d, ws_bytes=1 << 40) == want


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(T=(1 << 20) + 1), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 8), INVALID),
    (dict(n_blocks=0), INVALID), (dict(blocks_per_seq=0), INVALID), (dict(q_start=None), INVALID),
    (dict(kv_len=FAKE + 4), INVALID), (dict(block_table=FAKE + 2), INVALID),
    (dict(blocks_per_seq=(1 << 23) + 1), UNSUPPORTED), (dict(n_blocks=1 << 23), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE)])
def test_batches_that_are_refused(bad, want):
    assert append(**bad) == want
    assert attention(**bad) == want
    assert attention("v4attn_block_sparse_attention", **bad) == want


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=FAKE + 2), dict(k_token_stride=1020), dict(v_head_stride=120),
    dict(k_head_stride=0), dict(q=FAKE), dict(q_out=FAKE),
    dict(q=FAKE, q_out=FAKE, q_token_stride=1024, q_head_stride=128, q_out_token_stride=1024,
         q_out_head_stride=4)])
def test_append_rows_that_are_refused(bad):
    assert append(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(out=None), dict(q=FAKE + 8), dict(out_token_stride=1028),
    dict(q_head_stride=64), dict(sink=FAKE + 2), dict(lse=FAKE + 1)])
def test_attention_rows_that_are_refused(bad):
    assert attention(**bad) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(n_sel=-1), INVALID), (dict(n_sel=2049, idx=FAKE), UNSUPPORTED), (dict(n_sel=4), INVALID),
    (dict(n_sel=4, idx=FAKE, n_lists=3), INVALID), (dict(n_sel=4, idx=FAKE, n_local=-1), INVALID),
    (dict(n_sel=4, idx=FAKE + 2), INVALID), (dict(d=desc(n_win=64)), INVALID)])
def test_lists_that_are_refused(bad, want):
    assert attention("v4attn_block_sparse_attention", **bad) == want


def test_packed_arguments_lie_as_the_structures_do():
    for name, cls in (("v4attn_kv_append", _abi.KvAppendArgs),
                      ("v4attn_paged_attention", _abi.KvAttnArgs)):
        values = list(range(1, len(cls._fields_) + 1))
        raw = _abi.PACKED[name].pack(*values)
        assert len(raw) == ctypes.sizeof(cls)
        got = cls.from_buffer_copy(raw)
        assert [getattr(got, f) for f, _ in cls._fields_] == values


def test_nothing_to_do_is_no_error():
    assert append(T=0, k=None, v=None) == _abi.OK
    assert attention(T=0, q=None, out=None) == _abi.OK
    assert attention(B=0) == _abi.OK


def test_the_binding_refuses_wrong_tensors():
    import long_context_compressed_kv_b200 as v
    with pytest.raises(ValueError):
        v.kv_desc(8, 2, 128, dtype=torch.float32)
    with pytest.raises(v.V4AttnError):
        v.kv_workspace(v.kv_desc(9, 2, 128))
    d = v.kv_desc(8, 2, 128)
    pool = torch.zeros(4, 2, 128, 128, dtype=torch.bfloat16)
    good = dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16), k_cache=pool, v_cache=pool,
                q_start=torch.zeros(2, dtype=torch.int32), kv_len=torch.zeros(1, dtype=torch.int64),
                block_table=torch.zeros(1, 4, dtype=torch.int32), ws=torch.zeros(256, dtype=torch.uint8))
    good["v"] = good["k"]
    for bad in (dict(k=good["k"].half()), dict(k=good["k"][:, :1]), dict(v=good["v"][:2]),
                dict(k_cache=pool[:, :, :64]), dict(v_cache=pool.transpose(0, 2)),
                dict(q_start=torch.zeros(3, dtype=torch.int32)),
                dict(kv_len=torch.zeros(1, dtype=torch.int32)),
                dict(block_table=torch.zeros(4, dtype=torch.int32)), dict(q=good["k"]), {}):
        # the last: tensors that are not on a GPU
        with pytest.raises(ValueError):
            v.kv_append(d, **{**good, **bad})


def test_pools_of_a_layer():
    import long_context_compressed_kv_b200 as v
    from long_context_compressed_kv_b200.paging import kv_pools
    k, x = kv_pools(v.kv_desc(8, 2, 64, dtype=torch.float16), 5, device="cpu")
    assert k.shape == x.shape == (5, 2, 128, 64) and k.dtype == torch.float16
    assert k.data_ptr() != x.data_ptr() and not k.any()
