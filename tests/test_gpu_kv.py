"""16-bit K/V layers on the GPU: appending with rotation, attention over the
paged cache and over selected blocks, against float64 references.  Cache rows
that no sequence holds are NaN throughout, token rows of no sequence must keep
what they held."""
import math

import numpy as np
import pytest
import torch

from tests import kv_util as ku
from tests.kv_util import BLOCK, Case, check, reference, rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def v4():
    import long_context_compressed_kv_b200 as v
    return v


def desc_of(c, **kw):
    return v4().kv_desc(c.Hq, c.Hkv, c.d, dtype=c.dt, **kw)


def outputs(c):
    return (torch.full((c.T, c.Hq, c.d), 7.0, dtype=c.dt, device="cuda"),
            torch.full((c.T, c.Hq), 7.0, device="cuda"))


def attend(c, n_win=0, sink=None, scale=0.0, status=0, ws=None):
    v = v4()
    desc = desc_of(c, n_win=n_win, softmax_scale=scale)
    ws = v.kv_workspace(desc) if ws is None else ws
    out, lse = outputs(c)
    v.paged_attention(desc, q=c.q.cuda(), out=out, lse=lse,
                      sink=None if sink is None else sink.cuda(), **c.args(ws))
    torch.cuda.synchronize()
    assert v.device_status_code(ws)[1] == status
    return out, lse


def select(c, idx, n_local, sink=None, status=0):
    v = v4()
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    out, lse = outputs(c)
    v.block_sparse_attention(desc, q=c.q.cuda(), out=out, lse=lse, idx=idx.cuda(),
                             n_local=n_local, sink=None if sink is None else sink.cuda(),
                             **c.args(ws))
    torch.cuda.synchronize()
    assert v.device_status_code(ws)[1] == status
    return out, lse


# new tokens, positions, heads, dim, type, window
DENSE = [
    ([1], [1], 4, 1, 128, "bf16", 0),                       # the first token
    ([1, 1, 1], [128, 129, 1000], 16, 2, 128, "bf16", 0),   # around a block's end
    ([1, 1], [127, 700], 8, 8, 64, "fp16", 0),
    ([1] * 9, [0 + 1, 64, 128, 256, 257, 300, 511, 2000, 5], 64, 8, 128, "bf16", 0),
    ([5], [5], 8, 1, 64, "bf16", 0),                        # a prompt from nothing
    ([300], [300], 4, 4, 128, "bf16", 0),                   # one K/V head a query head
    ([150], [1030], 6, 2, 128, "fp16", 0),                  # three heads a K/V head
    ([33, 0, 1, 70], [200, 50, 513, 70], 16, 2, 128, "bf16", 0),   # a sequence without new tokens
    ([2, 17, 130], [300, 17, 260], 20, 4, 64, "bf16", 0),   # five heads
    ([3, 40], [900, 41], 128, 1, 128, "bf16", 0),           # 128 heads on one
    ([3, 9], [400, 260], 100, 1, 64, "fp16", 0),
    ([64], [777], 12, 1, 128, "bf16", 0),
    ([1, 1], [1000, 90], 8, 1, 128, "bf16", 1),             # windows
    ([70, 1, 1], [800, 1200, 100], 8, 2, 128, "bf16", 100),
    ([200], [600], 4, 2, 64, "fp16", 128),
    ([129], [1025], 2, 1, 128, "bf16", 129),
    ([260], [261], 8, 1, 128, "fp16", 5000),
]


@pytest.mark.parametrize("with_sink", [False, True])
@pytest.mark.parametrize("ns,ls,Hq,Hkv,d,dtype,n_win", DENSE)
def test_paged_attention(ns, ls, Hq, Hkv, d, dtype, n_win, with_sink):
    c = Case(ns, ls, Hq, Hkv, d, dtype, seed=len(ns) + Hq + n_win, front=2, behind=3)
    sink = torch.randn(Hq, generator=torch.Generator().manual_seed(5)) if with_sink else None
    out, lse = attend(c, n_win, sink)
    check(c, out, lse, reference(c, n_win, sink))


def test_long_histories_and_few_rows():
    """The keys of one sequence spread over every SM; the merged parts agree
    with the reference, and a second run gives the same bits."""
    c = Case([1, 2], [9001, 4097], 8, 2, 128, seed=3)
    ref = reference(c)
    first = attend(c)
    check(c, *first, ref)
    again = attend(c)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("scale,q_scale", [(0.9, 12.0), (1e-39, 1.0), (1e-6, 1.0)])
def test_softmax_scale_and_large_logits(scale, q_scale):
    """Large logits, and scales so small (one a denormal) that every key weighs the same."""
    c = Case([3, 40], [500, 300], 8, 2, 64, seed=8, q_scale=q_scale)
    out, lse = attend(c, scale=scale)
    check(c, out, lse, reference(c, scale=float(np.float32(scale))))


def test_growing_maximum():
    """Keys whose logits rise steadily: every block moves the running maximum."""
    c = Case([4], [2000], 8, 1, 128, "fp16", seed=2, spare=0)
    ramp = torch.linspace(0.0, 3.0, 2000)[:, None, None]
    c.hist_k[0] = (ramp * torch.ones(2000, 1, 128)).half()
    c.q = torch.ones_like(c.q)
    for i in range(0, 2000, BLOCK):
        m = min(BLOCK, 2000 - i)
        c.k_pool[c.table[0, i // BLOCK], :, :m] = c.hist_k[0][i:i + m].transpose(0, 1)
    out, lse = attend(c)
    check(c, out, lse, reference(c))


def test_queries_that_see_no_key():
    """No history at all, and a q_start that claims more tokens than kv_len
    holds (positions below 0): out 0, lse the sink's or -inf."""
    c = Case([3, 2], [200, 1], 8, 2, 128, seed=1)       # second sequence: positions -1, 0
    sink = torch.randn(8, generator=torch.Generator().manual_seed(2))
    for sk in (None, sink):
        out, lse = attend(c, sink=sk, status=ku.ST_BAD_POSITION)
        check(c, out, lse, reference(c, sink=sk))
        t = int(c.start[1])
        assert (out[t] == 0).all()
        assert torch.equal(lse[t].cpu(), torch.full((8,), -math.inf) if sk is None else sk)
    c = Case([1, 1], [0, 0], 4, 1, 64, seed=1)
    out, lse = attend(c, status=ku.ST_BAD_POSITION)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_bad_table_entries_are_not_seen():
    c = Case([2, 1], [700, 300], 8, 2, 128, seed=4)
    good = c.table.copy()
    c.table[0, 2], c.table[1, 1] = c.n_blocks, -5
    out, lse = attend(c, status=ku.ST_BAD_INDEX)
    check(c, out, lse, reference(c, bad={(0, 2), (1, 1)}))
    c.table = good
    check(c, *attend(c), reference(c))


def test_bad_starts_are_caught():
    """A q_start that decreases or passes T: the rows it names stay inside the
    tensors, and a later good call is right."""
    v = v4()
    c = Case([4, 4, 4], [140, 200, 12], 8, 2, 64, seed=4)
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    for bad in ([0, 8, 4, 12], [-3, 4, 8, 12], [0, 4, 8, 1000]):
        v.workspace_init(ws)
        out, lse = outputs(c)
        kw = c.args(ws)
        kw["q_start"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        v.paged_attention(desc, q=c.q.cuda(), out=out, lse=lse, **kw)
        kw["k"] = kw["v"] = torch.zeros(c.T, c.Hkv, c.d, dtype=c.dt, device="cuda")
        assert v.device_status_code(ws)[1] & ku.ST_BAD_SEQ, bad
        v.workspace_init(ws)
        v.kv_append(desc, **kw)
        assert v.device_status_code(ws)[1] & ku.ST_BAD_SEQ, bad
    v.workspace_init(ws)
    check(c, *attend(c, ws=ws), reference(c))


def test_window_needs_no_blocks_before_it():
    """Blocks wholly before every window may have been given back."""
    c = Case([3, 1], [900, 650], 8, 2, 128, seed=6)
    c.table[0, :(897 - 1 - 199) // BLOCK] = -1
    c.table[1, :(649 - 199) // BLOCK] = -1
    out, lse = attend(c, n_win=200)
    check(c, out, lse, reference(c, n_win=200))
    # rows before the first window inside its block hold anything
    lo = 897 - 199
    c.k_pool[c.table[0, lo // BLOCK], :, :lo % BLOCK] = math.inf
    c.v_pool[c.table[0, lo // BLOCK], :, :lo % BLOCK] = math.nan
    check(c, *attend(c, n_win=200), reference(c, n_win=200))


# new tokens, positions, heads, dim, type, lists a token, entries, last blocks
SPARSE = [
    ([1], [3000], 8, 1, 128, "bf16", 1, 8, 2),
    ([1, 1, 1, 1], [2000, 130, 128, 1], 64, 8, 128, "bf16", 1, 16, 2),
    ([1, 1, 1], [1500, 900, 40], 16, 4, 64, "fp16", 4, 5, 1),
    ([40], [1500], 16, 2, 128, "bf16", 1, 4, 1),
    ([40, 1, 150], [1400, 1000, 150], 8, 2, 64, "fp16", 2, 3, 2),
    ([37], [2900], 3, 3, 128, "bf16", 1, 6, 1),              # one head a K/V head
    ([5, 3], [1100, 800], 128, 1, 128, "bf16", 1, 40, 0),    # lists longer than the history
    ([20, 1], [700, 700], 20, 4, 64, "bf16", 4, 2, 0),
    ([9, 1], [600, 513], 8, 1, 128, "bf16", 1, 1, 7),
    ([2, 1], [600, 513], 8, 1, 128, "fp16", 1, 0, 3),        # the last blocks alone
]


def lists_for(c, n_lists, n_sel, seed=0, messy=False):
    """Ascending, -1-padded lists of the blocks at or before each token; messy:
    any order, repeats, entries past the token."""
    rng = np.random.default_rng(seed)
    idx = np.full((c.T, n_lists, n_sel), -1, np.int32)
    for t, _, p in c.tokens():
        for h in range(n_lists):
            if messy:
                idx[t, h] = rng.integers(-2, max(p, 0) // BLOCK + 3, n_sel)
            else:
                m = int(rng.integers(0, min(n_sel, p // BLOCK + 1) + 1))
                idx[t, h, :m] = np.sort(rng.permutation(p // BLOCK + 1)[:m])
    return torch.from_numpy(idx)


@pytest.mark.parametrize("messy", [False, True])
@pytest.mark.parametrize("ns,ls,Hq,Hkv,d,dtype,n_lists,n_sel,n_local", SPARSE)
def test_block_sparse_attention(ns, ls, Hq, Hkv, d, dtype, n_lists, n_sel, n_local, messy):
    c = Case(ns, ls, Hq, Hkv, d, dtype, seed=n_sel + Hq, front=1, behind=2)
    idx = lists_for(c, n_lists, n_sel, seed=n_sel, messy=messy)
    sink = torch.randn(Hq, generator=torch.Generator().manual_seed(9)) if messy else None
    out, lse = select(c, idx, n_local, sink)
    check(c, out, lse, reference(c, sink=sink, idx=idx, n_local=n_local))


def test_every_block_selected_is_dense_attention():
    c = Case([50, 1], [900, 1030], 8, 2, 128, seed=12)
    idx = torch.arange(9, dtype=torch.int32).expand(c.T, 1, 9).contiguous()
    check(c, *select(c, idx, 0), reference(c))
    check(c, *select(c, idx[..., :0], 100), reference(c))


def test_selected_blocks_with_bad_pages():
    c = Case([1, 20], [1300, 700], 8, 2, 128, seed=4)
    idx = lists_for(c, 1, 3, seed=1)
    idx[0, 0] = torch.tensor([1, 4, 6])
    idx[5, 0] = torch.tensor([0, 2, 3])
    c.table[0, 4], c.table[1, 2] = -1, c.n_blocks + 100
    out, lse = select(c, idx, 1, status=ku.ST_BAD_INDEX)
    check(c, out, lse, reference(c, idx=idx, n_local=1, bad={(0, 4), (1, 2)}))


def test_blocks_that_nobody_selects_hold_anything():
    c = Case([1, 12], [1100, 900], 8, 2, 128, seed=7)
    idx = torch.full((c.T, 1, 2), -1, dtype=torch.int32)
    idx[:, 0] = torch.tensor([1, 3])
    ref = reference(c, idx=idx, n_local=1)
    for b, gone in ((0, (0, 2, 5)), (1, (0, 2, 4, 5))):
        for blk in gone:
            c.k_pool[c.table[b, blk]] = math.nan
            c.v_pool[c.table[b, blk]] = math.inf
    check(c, *select(c, idx, 1), ref)


# ------------------------------------------------------------------ append

APPEND = [
    ([1], [1], 4, 1, 128, "bf16", 128, False, True),
    ([1, 1, 1], [128, 129, 1000], 16, 2, 128, "bf16", 128, True, True),
    ([5, 0, 200], [300, 50, 260], 6, 2, 64, "fp16", 64, False, True),
    ([140], [1 << 20], 8, 8, 64, "bf16", 32, True, False),
    ([130, 3], [131, 129], 24, 8, 128, "fp16", 16, False, True),
    ([7], [1000], 4, 4, 64, "bf16", 0, False, True),
    ([9], [300], 128, 1, 128, "bf16", 112, True, True),
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("ns,ls,Hq,Hkv,d,dtype,d_rope,halves,with_q", APPEND)
def test_kv_append(ns, ls, Hq, Hkv, d, dtype, d_rope, halves, with_q, fused):
    """New rows against R(p) in float64 within one rounding (u |x|) and fp32
    arithmetic on the pair (angle, sine and products: 2^-21 of its length);
    V bit for bit; every other row of the pools untouched."""
    v = v4()
    if max(ls) > 4096:      # a far position on a small pool: only its last blocks are listed
        c = Case(ns, [x % 1024 + 512 for x in ls], Hq, Hkv, d, dtype, seed=d_rope)
        shift = max(ls) - c.ls[0]
    else:
        c = Case(ns, ls, Hq, Hkv, d, dtype, seed=d_rope + Hq, front=1, behind=2)
        shift = 0
    theta = 10000.0
    desc = desc_of(c, d_rope=d_rope, rope_halves=halves, rope_theta=theta)
    ws = v.kv_workspace(desc)
    g = torch.Generator().manual_seed(11)
    if fused:
        qkv = torch.randn(c.T, Hq + 2 * Hkv, d, generator=g).to(c.dt)
        q, k, vv = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        dev = qkv.cuda()
        qd, kd, vd = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    else:
        q, k, vv = (torch.randn(c.T, h, d, generator=g).to(c.dt) for h in (Hq, Hkv, Hkv))
        qd, kd, vd = q.cuda(), k.cuda(), vv.cuda()
    args = c.args(ws)
    if shift:
        m = shift // BLOCK
        far = torch.full((1, m + c.bps), -1, dtype=torch.int32)
        far[:, m:] = torch.from_numpy(c.table)
        args["block_table"], args["kv_len"] = far.cuda(), args["kv_len"] + shift
    q_out = torch.full((c.T, Hq, d), 7.0, dtype=c.dt, device="cuda")
    if with_q and fused:
        q_out = qd          # in place
    v.kv_append(desc, k=kd, v=vd, q=qd if with_q else None, q_out=q_out if with_q else None,
                **args)
    torch.cuda.synchronize()
    assert v.device_status_code(ws)[1] == 0
    rows = [t for t, _, _ in c.tokens()]
    pos = [p + shift for _, _, p in c.tokens()]
    u = torch.finfo(c.dt).eps / 2
    off, half = d - d_rope, d_rope // 2

    def close(got, src):
        want = rotated(src[rows], pos, d_rope, theta, halves)
        r = src[rows].double()[..., off:]
        a, b = (r[..., :half], r[..., half:]) if halves else (r[..., 0::2], r[..., 1::2])
        length = (a * a + b * b).sqrt()
        length = torch.cat((length, length), -1) if halves else \
            torch.stack((length, length), -1).flatten(-2)
        tol = u * want.abs()
        tol[..., off:] += (1 + u) * 2.0 ** -21 * length
        assert ((got[rows].double().cpu() - want).abs() <= tol).all()
        assert torch.equal(got[rows].cpu()[..., :off], src[rows][..., :off])

    if with_q:
        close(q_out, q)
        others = [t for t in range(c.T) if t not in rows]
        assert torch.equal(q_out[others].cpu(), q[others] if fused else
                           torch.full_like(q[others], 7.0))
    want_k, want_v = c.k_pool.clone(), c.v_pool.clone()
    got_k = torch.zeros(c.T, Hkv, d, dtype=c.dt)
    for t, b, p in c.tokens():
        blk, r = c.table[b, p // BLOCK], p % BLOCK
        got_k[t] = args["k_cache"][blk, :, r].cpu()
        want_k[blk, :, r], want_v[blk, :, r] = got_k[t], vv[t]
    close(got_k, k)
    bits = torch.int16
    assert torch.equal(args["k_cache"].cpu().view(bits), want_k.view(bits))
    assert torch.equal(args["v_cache"].cpu().view(bits), want_v.view(bits))


def test_append_leaves_bad_rows_out():
    v = v4()
    c = Case([2, 3, 1], [1, 300, 140], 4, 2, 64, seed=3)     # first: positions -1, 0
    c.table[1, 2] = -1                                       # positions 256 .. of sequence 1
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    args = c.args(ws)
    x = torch.ones(c.T, 2, 64, dtype=c.dt, device="cuda")
    v.kv_append(desc, k=x, v=x, **args)
    assert v.device_status_code(ws)[1] == ku.ST_BAD_POSITION | ku.ST_BAD_INDEX
    want = c.v_pool.clone()
    want[c.table[0, 0], :, 0] = 1.0
    want[c.table[2, 1], :, 139 - 128] = 1.0
    assert torch.equal(args["v_cache"].cpu().view(torch.int16), want.view(torch.int16))
    # a position past the table
    v.workspace_init(ws)
    args["kv_len"] = args["kv_len"] + torch.tensor([1, 0, 10000], device="cuda")
    v.kv_append(desc, k=x, v=x, **args)
    assert v.device_status_code(ws)[1] & ku.ST_BAD_POSITION


# ------------------------------------------------------------------ as they are used

def _generate(c_seed, Hq, Hkv, d, dtype, chunks, sparse):
    """Chunks of new tokens of two sequences through append and attention on
    paging's block tables; returns every chunk's outputs and the whole history."""
    v = v4()
    from long_context_compressed_kv_b200.paging import BlockPool, BlockTable, kv_pools
    dt = ku.DT[dtype]
    g = torch.Generator().manual_seed(c_seed)
    pool = BlockPool(24)
    table = BlockTable(2, 10, pool)
    desc = v.kv_desc(Hq, Hkv, d, dtype=dt, rope_halves=True)
    ws = v.kv_workspace(desc)
    kc, vc = (x.fill_(math.nan) for x in kv_pools(desc, 24))
    lens = [0, 0]
    hist, res = [[], []], []
    for n in chunks:
        T = sum(n)
        lens = [a + b for a, b in zip(lens, n)]
        for b in range(2):
            table.ensure(b, lens[b])
        q, k, x = (torch.randn(T, h, d, generator=g).to(dt) for h in (Hq, Hkv, Hkv))
        q_rot = torch.empty_like(q, device="cuda")
        out = torch.empty_like(q_rot)
        kw = dict(k_cache=kc, v_cache=vc, block_table=table.tensor(), ws=ws,
                  q_start=torch.tensor([0, n[0], T], dtype=torch.int32, device="cuda"),
                  kv_len=torch.tensor(lens, dtype=torch.int64, device="cuda"))
        v.kv_append(desc, k=k.cuda(), v=x.cuda(), q=q.cuda(), q_out=q_rot, **kw)
        if sparse:
            idx = torch.zeros(T, 1, 1, dtype=torch.int32, device="cuda")   # the first block
            v.block_sparse_attention(desc, q=q_rot, out=out, idx=idx, n_local=2, **kw)
        else:
            v.paged_attention(desc, q=q_rot, out=out, **kw)
        at = 0
        for b in range(2):
            hist[b].append((q[at:at + n[b]], k[at:at + n[b]], x[at:at + n[b]]))
            at += n[b]
        res.append((n, out.cpu()))
    assert v.device_status(ws) == 0
    return hist, res


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(8, 2, 128, "bf16"), (6, 2, 64, "fp16")])
def test_prefill_and_decode_through_the_cache(Hq, Hkv, d, dtype, sparse):
    """Prompts in chunks, then decode steps: each chunk's outputs are those of
    one causal attention over the whole rotated sequence in float64.  K and q
    are rounded to their type after the rotation, each off by u, so a logit is
    off by 2 u scale |q||k| (pairs turned, lengths kept) next to the kernel's
    own errors."""
    chunks = [(150, 7), (131, 0), (1, 1), (1, 260), (1, 1), (1, 1)]
    hist, res = _generate(5, Hq, Hkv, d, dtype, chunks, sparse)
    g, dt = Hq // Hkv, ku.DT[dtype]
    u = torch.finfo(dt).eps / 2
    for b in range(2):
        q, k, x = (torch.cat([h[i] for h in hist[b]]) for i in range(3))
        pos = list(range(len(q)))
        q, k, x = rotated(q, pos, d, 160000.0, True), rotated(k, pos, d, 160000.0, True), x.double()
        got = torch.cat([o[:n[0]] if b == 0 else o[n[0]:] for n, o in res]).double()
        p, j = torch.arange(len(q))[:, None], torch.arange(len(q))
        see = j <= p
        if sparse:
            see = see & ((j // BLOCK == 0) | (j // BLOCK > p // BLOCK - 2))
        for h in range(Hq):
            kk, vv = k[:, h // g], x[:, h // g]
            s = (q[:, h] @ kk.T / math.sqrt(d)).masked_fill(~see, -math.inf)
            w = s.softmax(1)
            size = q[:, h].norm(dim=1)[:, None] * kk.norm(dim=1) / math.sqrt(d)
            e = (2 * u * size.masked_fill(~see, 0.0)).amax(1, keepdim=True)
            tol = u * (w @ vv).abs() + (u + 2 * (e + 2.0 ** -12)) * (w @ vv.abs()) * (1 + u)
            assert ((got[:, h] - w @ vv).abs() <= tol).all()


def test_selection_by_the_indexer():
    """index_topk with m = 128 scores one key a 128-token block and selects;
    block_sparse_attention takes its lists as they are."""
    import synth
    from tests.gpu_util import code_rows, desc_for, dev
    v = v4()
    c = Case([3, 1], [128 * 40 + 50, 128 * 33], 16, 2, 128, seed=20)
    rng = np.random.default_rng(1)
    k, H_I, rows = 6, 64, 48
    ly = synth.Layer("csa", 128, 16, 512, 64, 128, H_I, 128, k, idx_fp4=True)
    ldesc = desc_for(ly)
    keys = rng.standard_normal((2, rows, 128)).astype(np.float32)
    qI = rng.standard_normal((1, c.T * H_I, 128)).astype(np.float32)
    krows, ksf = code_rows(ldesc, dev(keys), v.MXFP4)
    qrows, qsf = code_rows(ldesc, dev(qI), v.MXFP4)
    seqs = np.array([b for _, b, _ in c.tokens()], np.int32)
    pos = np.array([p for _, _, p in c.tokens()], np.int64)
    idx = torch.full((c.T, k), -9, dtype=torch.int32, device="cuda")
    iws = v.workspace(ldesc, c.T, rows)
    v.index_topk(ldesc, qI=qrows.reshape(c.T, H_I, -1), qI_sf=qsf.reshape(c.T, H_I, -1),
                 w=dev(rng.uniform(0, 1, (c.T, H_I)).astype(np.float32)),
                 q_pos=dev(pos, torch.int64), q_seq=dev(seqs, torch.int32), B=2, keys=krows,
                 keys_sf=ksf, key_rows=rows, max_vis=rows, idx_out=idx, ws=iws)
    assert v.device_status(iws) == 0
    assert (idx.cpu() >= 0).all()
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    out, lse = outputs(c)
    v.block_sparse_attention(desc, q=c.q.cuda(), out=out, lse=lse, idx=idx, n_local=1, **c.args(ws))
    assert v.device_status(ws) == 0
    check(c, out, lse, reference(c, idx=idx.cpu()[:, None], n_local=1))


def test_graphs_that_share_a_workspace():
    """A dense and a sparse call captured apart on one workspace, replayed in
    turn with new inputs and lengths written into their tensors."""
    v = v4()
    cases = [Case([4, 1], [600, 1100], 8, 2, 128, seed=s, bps=9, spare=20 - 14) for s in (1, 2)]
    later = Case([4, 1], [500, 1050], 8, 2, 128, seed=3, bps=9, spare=20 - 13)
    idx = lists_for(cases[1], 1, 3, seed=4)
    desc = desc_of(cases[0])
    ws = v.kv_workspace(desc)
    state = []
    for i, c in enumerate(cases):
        kw = c.args(ws)
        kw.update(q=c.q.cuda())
        kw.update(zip(("out", "lse"), outputs(c)))
        if i:
            kw.update(idx=idx.cuda(), n_local=1)
        fn = v.block_sparse_attention if i else v.paged_attention
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fn(desc, **kw)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fn(desc, **kw)
        state.append((graph, kw))
    for _ in range(2):
        for (graph, kw), c in zip(state, cases):
            kw["out"].fill_(7.0)
            kw["lse"].fill_(7.0)
            graph.replay()
    check(cases[0], state[0][1]["out"], state[0][1]["lse"], reference(cases[0]))
    check(cases[1], state[1][1]["out"], state[1][1]["lse"], reference(cases[1], idx=idx, n_local=1))
    graph, kw = state[0]
    new = later.args(ws)
    for name in ("k_cache", "v_cache", "kv_len", "block_table"):
        kw[name].copy_(new[name])
    kw["q"].copy_(later.q)
    graph.replay()
    check(later, kw["out"], kw["lse"], reference(later))
    assert v.device_status(ws) == 0


def test_two_streams_at_once():
    v = v4()
    cases = [Case([3, 1], [900, 2500], 8, 2, 128, seed=s) for s in (1, 2)]
    refs = [reference(c) for c in cases]
    desc = desc_of(cases[0])
    got = []
    for c in cases:
        ws = v.kv_workspace(desc)
        kw = c.args(ws)
        kw.update(zip(("out", "lse"), outputs(c)))
        got.append((torch.cuda.Stream(), c.q.cuda(), kw))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, q, kw in got:
            v.paged_attention(desc, q=q, stream=st, **kw)
    torch.cuda.synchronize()
    for c, r, (_, _, kw) in zip(cases, refs, got):
        check(c, kw["out"], kw["lse"], r)


def test_strided_queries_and_outputs():
    """q as a view of a fused projection, out head-major: any strides that are
    multiples of 8."""
    v = v4()
    c = Case([20, 1], [300, 200], 8, 2, 64, seed=9)
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    fused = torch.full((c.T, 12, 64), 5.0, dtype=c.dt, device="cuda")
    fused[:, :8] = c.q.cuda()
    out = torch.full((8, c.T, 72), 7.0, dtype=c.dt, device="cuda")
    lse = torch.full((c.T, 8), 7.0, device="cuda")
    v.paged_attention(desc, q=fused[:, :8], out=out.transpose(0, 1)[..., :64], lse=lse,
                      **c.args(ws))
    check(c, out.transpose(0, 1)[..., :64], lse, reference(c))
    assert (out[..., 64:] == 7.0).all()


def test_rows_beyond_32_bit_offsets():
    """Pools of more than 2^31 values: the last blocks of a 5 GB pool."""
    v = v4()
    c = Case([2, 1], [400, 130], 8, 2, 128, seed=10)
    big = (1 << 31) // (2 * BLOCK * 128) + 40
    kc = torch.empty(big, 2, BLOCK, 128, dtype=c.dt, device="cuda")
    vc = torch.empty(big, 2, BLOCK, 128, dtype=c.dt, device="cuda")
    base = big - c.n_blocks
    kc[base:], vc[base:] = c.k_pool.cuda(), c.v_pool.cuda()
    desc = desc_of(c, d_rope=0)
    ws = v.kv_workspace(desc)
    out, lse = outputs(c)
    kw = c.args(ws)
    kw.update(k_cache=kc, v_cache=vc, block_table=kw["block_table"] + base)
    new = torch.cat([c.hist_k[b][L - n:] for b, (n, L) in enumerate(zip(c.ns, c.ls))])
    new_v = torch.cat([c.hist_v[b][L - n:] for b, (n, L) in enumerate(zip(c.ns, c.ls))])
    v.kv_append(desc, k=new.cuda(), v=new_v.cuda(), **kw)
    v.paged_attention(desc, q=c.q.cuda(), out=out, lse=lse, **kw)
    check(c, out, lse, reference(c))
    idx = torch.tensor([0, 2], dtype=torch.int32).expand(c.T, 1, 2).contiguous()
    out, lse = outputs(c)
    v.block_sparse_attention(desc, q=c.q.cuda(), out=out, lse=lse, idx=idx.cuda(), n_local=1, **kw)
    check(c, out, lse, reference(c, idx=idx, n_local=1))
    assert v.device_status(ws) == 0


def test_nothing_to_do():
    v = v4()
    c = Case([0, 0], [200, 0], 8, 2, 64, seed=1)
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    empty = torch.empty(0, 8, 64, dtype=c.dt, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=c.dt, device="cuda")
    args = c.args(ws)
    v.kv_append(desc, k=kv, v=kv, q=empty, q_out=empty.clone(), **args)
    v.paged_attention(desc, q=empty, out=empty.clone(), **args)
    # rows, but every one of them outside the sequences
    c = Case([0, 0], [200, 0], 8, 2, 64, seed=1, front=2, behind=3)
    out, lse = attend(c)
    assert (out == 7.0).all() and (lse == 7.0).all()


# ------------------------------------------------------------------ many sequences, many items


@pytest.mark.parametrize("B", [33, 100, 300])
def test_many_sequences(B):
    """More sequences than a warp looks at in one go, some without new tokens,
    some with several, of every length up to 400."""
    rng = np.random.default_rng(B)
    ns = rng.choice([0, 1, 1, 1, 2, 9], B).tolist()
    ls = [int(n + rng.integers(0, 400 - n)) for n in ns]
    c = Case(ns, ls, 4, 2, 64, seed=B)
    check(c, *attend(c), reference(c))
    idx = lists_for(c, 2, 2, seed=B)
    check(c, *select(c, idx, 1), reference(c, idx=idx, n_local=1))


def test_many_items_of_a_head():
    """128 query heads on one K/V head: two tokens an item, more items of a
    head than lanes; and the same for a sequence behind it."""
    c = Case([90, 70], [300, 75], 128, 1, 64, seed=2)
    check(c, *attend(c), reference(c))
    idx = lists_for(c, 1, 2, seed=1)
    check(c, *select(c, idx, 1), reference(c, idx=idx, n_local=1))


# at most 16 rows a sequence on average
STEPS = [
    ([1] * 5, [1, 129, 700, 128, 3000], 16, 1, 128, "bf16", 0),        # 16 rows each
    ([4, 3, 0, 1, 4], [4, 300, 50, 1, 1000], 8, 2, 128, "fp16", 0),    # several tokens
    ([16, 9, 16], [16, 140, 1000], 2, 2, 64, "bf16", 0),
    ([5, 5, 1], [5, 1285, 128], 6, 2, 128, "bf16", 7),                 # 15 rows, windows
    ([16, 16], [400, 261], 4, 4, 128, "fp16", 130),
    ([1, 2], [2000, 1500], 16, 2, 64, "fp16", 300),
    ([1] * 90 + [100] + [1] * 10, [200] * 90 + [333] + [150] * 10, 8, 1, 128, "bf16", 0),
    ([2] * 60 + [20, 70, 130], [150] * 60 + [20, 300, 260], 4, 2, 64, "fp16", 0),
    ([1] * 70 + [3, 20, 90], [130] * 70 + [700, 600, 900], 8, 1, 128, "bf16", 200),
]


@pytest.mark.parametrize("with_sink", [False, True])
@pytest.mark.parametrize("ns,ls,Hq,Hkv,d,dtype,n_win", STEPS)
def test_steps_of_few_rows(ns, ls, Hq, Hkv, d, dtype, n_win, with_sink):
    """Decode steps, of one token and of several, alone and with longer
    sequences among them; dense and over selected blocks."""
    c = Case(ns, ls, Hq, Hkv, d, dtype, seed=len(ns) + Hq + n_win, front=2, behind=3)
    sink = torch.randn(Hq, generator=torch.Generator().manual_seed(5)) if with_sink else None
    check(c, *attend(c, n_win, sink), reference(c, n_win, sink))
    idx = lists_for(c, Hkv, 3, seed=Hq, messy=with_sink)
    check(c, *select(c, idx, 1, sink), reference(c, sink=sink, idx=idx, n_local=1))


def test_maxima_that_grow_in_decode_steps():
    """Logits that rise from block to block, at other rates for other heads and in
    other warps' keys, so that maxima move in some rows of some blocks alone."""
    for dtype, d in (("fp16", 128), ("bf16", 64)):
        c = Case([1, 2], [2000, 1999], 16, 2, d, dtype, seed=3)
        c.q = (torch.arange(16.0)[None, :, None] / 8).expand(c.T, 16, d).to(c.dt).contiguous()
        for b in range(2):
            n = c.hist_k[b].shape[0]
            ramp = torch.linspace(0.0, 3.0, n) + (torch.arange(n) % 97 == 5) * 0.5
            c.hist_k[b] = ramp[:, None, None].expand(n, 2, d).to(c.dt).contiguous()
            for i in range(0, n, BLOCK):
                m = min(BLOCK, n - i)
                c.k_pool[c.table[b, i // BLOCK], :, :m] = c.hist_k[b][i:i + m].transpose(0, 1)
        check(c, *attend(c), reference(c))


@pytest.mark.parametrize("n_win", [0, 1, 128, 1280])
@pytest.mark.parametrize("ns,ls", [([16], [5128]), ([16], [1288]), ([16, 1, 40], [136, 4000, 3720])])
def test_tiles_that_end_a_block_apart(ns, ls, n_win):
    """Items of two tiles whose tokens lie on both sides of a block's end, as
    parts of a block or two: one tile sees the last block, and with a window
    the first, that the other does not, or nothing of its part."""
    c = Case(ns, ls, 16, 1, 128, seed=ls[0] + n_win)
    check(c, *attend(c, n_win), reference(c, n_win))


def test_one_row_over_every_sm():
    """A single query head on a long history: as many parts as CTAs."""
    c = Case([1], [40000], 1, 1, 128, seed=5)
    sink = torch.tensor([1.5])
    for sk in (None, sink):
        check(c, *attend(c, sink=sk), reference(c, sink=sk))


def test_longest_lists():
    """2048 entries a list, most of them of no block, and a long last range."""
    c = Case([1, 3], [5000, 2500], 2, 1, 64, seed=6)
    idx = torch.full((c.T, 1, 2048), -1, dtype=torch.int32)
    rng = np.random.default_rng(0)
    for t, _, p in c.tokens():
        m = p // BLOCK + 1
        at = np.sort(rng.permutation(2048)[:m // 2])
        idx[t, 0, at] = torch.from_numpy(np.sort(rng.permutation(m)[:m // 2]).astype(np.int32))
    check(c, *select(c, idx, 0), reference(c, idx=idx, n_local=0))
    check(c, *select(c, idx, 1 << 30), reference(c, idx=idx, n_local=1 << 30))


@pytest.mark.parametrize("ns", [[640], [2] * 20])
def test_selection_joined_in_windows(ns):
    """Histories of more than 2048 blocks and so many items that a CTA's range
    of blocks passes 2048: the joined selection goes on in a second window.
    One block's K and V serve every table entry, so that only positions and
    masks tell; sampled tokens against the reference."""
    v = v4()
    L, n, Hkv, d, n_sel = 2100 * BLOCK - 37, sum(ns), 8, 64, 5
    start = np.concatenate([[0], np.cumsum(ns)])
    nb = -(-L // BLOCK)
    g = torch.Generator().manual_seed(4)
    kb = torch.randn(7, Hkv, BLOCK, d, generator=g).to(torch.float16)
    vb = torch.randn(7, Hkv, BLOCK, d, generator=g).to(torch.float16)
    table = torch.randint(0, 7, (1, nb), generator=g, dtype=torch.int32)
    q = torch.randn(n, Hkv, d, generator=g).to(torch.float16)
    idx = torch.stack([torch.randperm(nb - 6, generator=g)[:n_sel].sort().values
                       for _ in range(n)]).to(torch.int32)
    desc = v.kv_desc(Hkv, Hkv, d, dtype=torch.float16)
    ws = v.kv_workspace(desc)
    out = torch.empty(n, Hkv, d, dtype=torch.float16, device="cuda")
    lse = torch.empty(n, Hkv, device="cuda")
    v.block_sparse_attention(
        desc, q=q.cuda(), k_cache=kb.cuda(), v_cache=vb.cuda(), out=out, lse=lse, ws=ws,
        q_start=torch.from_numpy(start).to(torch.int32).cuda(),
        kv_len=torch.full((len(ns),), L, dtype=torch.int64, device="cuda"),
        block_table=table.repeat(len(ns), 1).cuda(),
        idx=idx.cuda(), n_local=2)
    assert v.device_status(ws) == 0
    u = 2.0 ** -11
    for t in list(range(0, n, 37)) + [n - 1]:
        p = L - int(start[start > t][0]) + t
        last = p // BLOCK
        blocks = sorted(set(idx[t].tolist()) | {last - 1, last})
        k = torch.cat([kb[table[0, b]][:, :(p % BLOCK + 1 if b == last else BLOCK)]
                       for b in blocks], 1).double()
        x = torch.cat([vb[table[0, b]][:, :(p % BLOCK + 1 if b == last else BLOCK)]
                       for b in blocks], 1).double()
        s = (k @ q[t].double()[:, :, None])[..., 0] / math.sqrt(d)
        w = s.softmax(1)
        want = (w[:, None] @ x)[:, 0]
        e = d * 2.0 ** -23 * (k.abs() @ q[t].double().abs()[:, :, None]).amax(1) / math.sqrt(d)
        tol = u * want.abs() + (u + 2 * (e + 2.0 ** -18)) * (w[:, None] @ x.abs())[:, 0] * (1 + u)
        assert ((out[t].double().cpu() - want).abs() <= tol).all(), t
        z = s.logsumexp(1)
        assert ((lse[t].double().cpu() - z).abs() <= e[:, 0] + 2.0 ** -18 + 2.0 ** -21 * 10).all()


def test_head_major_queries():
    """q stored [Hq][T][d] and handed over transposed: head stride above token stride."""
    v = v4()
    c = Case([20, 3], [300, 200], 8, 2, 128, seed=9)
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    q = c.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    out, lse = outputs(c)
    v.paged_attention(desc, q=q, out=out, lse=lse, **c.args(ws))
    check(c, out, lse, reference(c))


def test_without_lse_and_with_shared_blocks():
    """Two sequences whose first blocks are the same pool blocks (a shared
    prefix); no lse asked for."""
    v = v4()
    c = Case([2, 1], [400, 300], 8, 2, 128, seed=13)
    for hist in (c.hist_k, c.hist_v):
        hist[1][:256] = hist[0][:256]
    c.table[1, :2] = c.table[0, :2]
    desc = desc_of(c)
    ws = v.kv_workspace(desc)
    out, lse = outputs(c)
    v.paged_attention(desc, q=c.q.cuda(), out=out, **c.args(ws))
    ref = reference(c)
    full = attend(c)
    check(c, *full, ref)
    assert torch.equal(out, full[0]) and (lse == 7.0).all()


def test_a_visible_nan_shows():
    """A NaN key or value that a query sees is not swallowed."""
    c = Case([1], [700], 8, 2, 128, seed=14)
    c.k_pool[c.table[0, 3], 1, 5] = math.nan
    out, lse = attend(c)
    assert out[:, 4:].isnan().all() and lse[:, 4:].isnan().all()
    assert out[:, :4].isfinite().all()
    c = Case([1], [700], 8, 2, 128, seed=14)
    c.v_pool[c.table[0, 3], 0, 5, 7] = math.nan
    out, lse = attend(c)
    assert out[:, :4, 7].isnan().all() and lse.isfinite().all()


def test_calls_in_a_row_on_one_stream():
    """Append, attend, select and again on one workspace without a pause: each
    reads what the one before wrote."""
    v = v4()
    c = Case([1, 1], [300, 1], 8, 2, 64, "fp16", seed=15, bps=4, spare=4)
    c.table = np.arange(8, dtype=np.int32).reshape(2, 4)
    c.n_blocks = 8
    desc = desc_of(c, d_rope=0)
    ws = v.kv_workspace(desc)
    steps, lens = 60, [100, 0]
    g = torch.Generator().manual_seed(1)
    qs, ks, xs = (torch.randn(steps, 2, h, 64, generator=g).half() for h in (8, 2, 2))
    first = torch.randn(2, 100, 2, 64, generator=g).half()
    kc = torch.full((8, 2, BLOCK, 64), math.nan, dtype=torch.float16)
    vc = kc.clone()
    kc[0, :, :100], vc[0, :, :100] = first[0].transpose(0, 1), first[1].transpose(0, 1)
    kc, vc = kc.cuda(), vc.cuda()
    dev = [t.cuda() for t in (qs, ks, xs)]
    kv_len = torch.tensor(lens, dtype=torch.int64, device="cuda")
    outs = torch.empty(steps, 2, 2, 8, 64, dtype=torch.float16, device="cuda")
    idx = torch.tensor([[0, -1], [0, -1]], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(c.table).cuda()
    for i in range(steps):
        kv_len += 1
        kw = dict(k_cache=kc, v_cache=vc, q_start=q_start, kv_len=kv_len, block_table=table, ws=ws)
        v.kv_append(desc, k=dev[1][i], v=dev[2][i], **kw)
        v.paged_attention(desc, q=dev[0][i], out=outs[i, 0], **kw)
        v.block_sparse_attention(desc, q=dev[0][i], out=outs[i, 1], idx=idx, n_local=1, **kw)
    assert v.device_status(ws) == 0
    got, u = outs.double().cpu(), 2.0 ** -11
    for b in range(2):
        k = torch.cat((first[0][:100 * (b == 0)], ks[:, b])).double()
        x = torch.cat((first[1][:100 * (b == 0)], xs[:, b])).double()
        for i in range(steps):
            m = (100 if b == 0 else 0) + i + 1
            for h in range(8):
                s = k[:m, h // 4] @ qs[i, b, h].double() / 8.0
                w = s.softmax(0)
                want = w @ x[:m, h // 4]
                tol = u * want.abs() + (u + 2.0 ** -14) * (w @ x[:m, h // 4].abs()) * (1 + u)
                # every block is the first or the last: both calls see all keys
                for j in range(2):
                    assert ((got[i, j, b, h] - want).abs() <= tol).all(), (i, j, b, h)


def test_compressed_layers_after_nan_in_tensor_memory():
    """Tensor memory keeps what a kernel leaves there, NaN here; a dense MQA
    whose queries see few entries (splits without a key, and in the form
    without splits queries of an empty history) does not take it up."""
    import synth
    from tests.gpu_util import code_rows, desc_for, dev
    v = v4()
    rng = np.random.default_rng(3)
    m, H, d, N, B = 128, 128, 512, 700, 3
    ldesc = desc_for(synth.Layer("hca", m, H, d, 64, 128, 4, 32, 96))
    kv, kv_sc = code_rows(ldesc, dev(rng.standard_normal((B, N, d)).astype(np.float32)),
                          v.E4M3_BF16ROPE, d_rope=64)
    swa, swa_sc = code_rows(ldesc, dev(rng.standard_normal((B, 256, d)).astype(np.float32)),
                            v.E4M3_BF16ROPE, d_rope=64)
    for nq in (6, 90):
        pos = rng.integers(0, 600, nq)
        pos[:3] = m * N - 1, 5, -1
        seq = rng.integers(0, B, nq)
        out = torch.zeros(nq, H, d, device="cuda")
        ws = v.workspace(ldesc, nq, N)
        q = dev(rng.standard_normal((nq, H, d)).astype(np.float32), torch.bfloat16)
        c = Case([1] * 40, [5000] + [130] * 39, 8, 8, 128, seed=1)
        c.k_pool.fill_(math.nan)
        c.v_pool.fill_(math.nan)
        nan_out, _ = attend(c)
        assert nan_out.isnan().all()
        v.dense_mqa(ldesc, Q=q, q_pos=dev(pos, torch.int64), q_seq=dev(seq, torch.int32), B=B,
                    kv=kv, kv_scale=kv_sc, kv_rows=N, swa=swa, swa_scale=swa_sc, swa_rows=256,
                    max_vis=N, out=out, ws=ws)
        assert v.device_status(ws) == 0
        assert out.isfinite().all()
        assert (out[2] == 0).all()
