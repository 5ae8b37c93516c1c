"""16-bit K/V layers on the GPU, calls at the edges of what they admit: long
histories with few blocks selected, values and starts out of the ordinary,
against float64 references."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.kv_util import BLOCK, ST_BAD_POSITION, ST_BAD_SEQ, Case, check, counted, reference
from tests.test_gpu_kv import attend, desc_of, outputs, select, v4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


@pytest.mark.parametrize("ns", [[1280], [2] * 40])
@pytest.mark.parametrize("early", ["none", "first", "one", "late"])
def test_windows_that_hold_few_blocks(ns, early):
    """More than a million positions, five windows of the joined selection, and
    several items a CTA: items whose first windows hold no block or one (the
    last blocks alone, the first and the last ones, one in the second window
    for some tokens, entries of the last window) as chunks and as pairs of
    tokens.  One pool block stands at every table entry but the last four, so
    that a query's answer is that of a few keys with their numbers."""
    v = v4()
    nb, n, Hkv, d, n_local = 8300, sum(ns), 8, 64, 2
    L = nb * BLOCK - 37
    start = np.concatenate([[0], np.cumsum(ns)])
    g = torch.Generator().manual_seed(len(early) + len(ns))
    kb = torch.randn(5, Hkv, BLOCK, d, generator=g).to(torch.float16)
    vb = torch.randn(5, Hkv, BLOCK, d, generator=g).to(torch.float16)
    table = torch.zeros(1, nb, dtype=torch.int32)
    table[0, -4:] = torch.arange(1, 5)
    q = torch.randn(n, Hkv, d, generator=g).to(torch.float16)
    idx = {"none": torch.empty(n, 1, 0), "first": torch.zeros(n, 1, 1),
           "one": torch.where(torch.arange(n) % 32 == 5, 2100, -1)[:, None, None],
           "late": torch.tensor([8195, nb - 4]).expand(n, 1, 2)}[early].to(torch.int32).contiguous()
    desc = v.kv_desc(Hkv, Hkv, d, dtype=torch.float16)
    ws = v.kv_workspace(desc)
    out = torch.full((n, Hkv, d), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((n, Hkv), 7.0, device="cuda")
    v.block_sparse_attention(
        desc, q=q.cuda(), k_cache=kb.cuda(), v_cache=vb.cuda(), out=out, lse=lse, ws=ws,
        q_start=torch.from_numpy(start).to(torch.int32).cuda(),
        kv_len=torch.full((len(ns),), L, dtype=torch.int64, device="cuda"),
        block_table=table.repeat(len(ns), 1).cuda(), idx=idx.cuda(), n_local=n_local)
    assert v.device_status(ws) == 0
    out, lse, u = out.double().cpu(), lse.double().cpu(), 2.0 ** -11
    for t in [*range(0, n, 7 if n < 100 else 37), 5, n - 1]:
        p = L - int(start[start > t][0]) + t
        last = p // BLOCK
        blocks = sorted(counted(idx[t, 0].tolist(), last) | {last - 1, last})
        k, x = (torch.cat([pool[table[0, b]][:, :(p % BLOCK + 1 if b == last else BLOCK)]
                           for b in blocks], 1).double() for pool in (kb, vb))
        s = (k @ q[t].double()[:, :, None])[..., 0] / math.sqrt(d)
        w, z = s.softmax(1), s.logsumexp(1)
        want = (w[:, None] @ x)[:, 0]
        e = d * 2.0 ** -23 * (k.abs() @ q[t].double().abs()[:, :, None]).amax(1) / math.sqrt(d)
        tol = u * want.abs() + (u + 2 * (e + 2.0 ** -18)) * (w[:, None] @ x.abs())[:, 0] * (1 + u)
        assert ((out[t] - want).abs() <= tol).all(), t
        assert ((lse[t] - z).abs() <= e[:, 0] + 2.0 ** -18 + 2.0 ** -21 * (1 + z.abs())).all(), t


@pytest.mark.parametrize("Hq,Hkv,d,dtype,n", [(16, 2, 128, "bf16", 1), (8, 2, 64, "fp16", 3)])
def test_many_short_steps_a_cta(Hq, Hkv, d, dtype, n):
    """Decode steps of one to three blocks, eight and more items a CTA one after
    the other: maxima and sums of one item are not taken for those of the next,
    and ten runs give the same bits."""
    rng = np.random.default_rng(d)
    c = Case([n] * 600, [int(x) for x in rng.integers(n, 300, 600)], Hq, Hkv, d, dtype, seed=d)
    first = attend(c)
    check(c, *first, reference(c))
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, attend(c)))


@pytest.mark.parametrize("n_win", [0, 50])
@pytest.mark.parametrize("ns,g,d", [([3], 8, 128), ([5, 2, 1], 6, 64), ([17, 18], 8, 128)])
def test_warps_without_rows_clear_their_values(ns, g, d, n_win):
    """Tiles whose rows leave some warps idle, on histories whose last block (and
    with a window the first) is NaN past its end in every length of it: the
    idle warps clear their share of V before the first products."""
    for L in (133, 160, 161, 190, 200, 223, 255):
        ls = [L + 7 * i for i in range(len(ns))]
        c = Case(ns, ls, 4 * g, 4, d, seed=L)
        for _ in range(5):
            out, lse = attend(c, n_win)
        check(c, out, lse, reference(c, n_win))


# new tokens, positions, heads, dim: items whole on a CTA (many sequences) and
# cut over CTAs (few), of few rows and of many
FORMS = [([1] * 400, [150] * 400, 16, 2, 128), ([30] * 200, [60] * 200, 8, 2, 64),
         ([1, 2], [3000, 1500], 16, 2, 64), ([40], [1500], 8, 2, 128)]


def forms(seed, dtype="bf16"):
    """Each form's case, with calls of it over all keys and over every block as a selection."""
    for ns, ls, Hq, Hkv, d in FORMS:
        c = Case(ns, ls, Hq, Hkv, d, dtype, seed=seed)
        m = max(ls) // BLOCK + 1
        idx = torch.arange(m, dtype=torch.int32).expand(c.T, 1, m).contiguous()
        yield c, (lambda sink=None, c=c: attend(c, sink=sink),
                  lambda sink=None, c=c, idx=idx: select(c, idx, 0, sink))


@pytest.mark.parametrize("value", [math.inf, -math.inf, 3.0e38, -3.0e38])
def test_sinks_without_bounds(value):
    """A sink of +inf takes all of a row's weight (out 0, lse inf), one of -inf
    or near the type's lowest none, one near its largest all but nothing; the
    other heads are as ever.  Rows without a key have the sink itself."""
    for c, calls in forms(4):
        sink = torch.randn(c.Hq, generator=torch.Generator().manual_seed(2))
        want = list(reference(c, sink=sink))
        sink[::3] = value
        none = reference(c)
        for call in calls:
            out, lse = (x.cpu() for x in call(sink))
            if value > 0:
                assert (out[:, ::3] == 0).all()
                # 2^-22: three roundings of fp32, to the base of the exponentials and back
                assert (lse[:, ::3] == value).all() if value == math.inf else \
                    ((lse[:, ::3] - value).abs() <= 2.0 ** -22 * value).all()
                out[:, ::3], lse[:, ::3] = want[0][:, ::3].to(out.dtype), want[1][:, ::3].float()
                check(c, out, lse, want)
            else:
                check(c, out, lse, [torch.where((torch.arange(c.Hq) % 3 > 0).view(
                    -1, *[1] * (w.dim() - 2)), w, x) for w, x in zip(want, none)])
    c = Case([3], [1], 8, 2, 64, seed=1)                     # positions -2, -1, 0
    sink = torch.full((8,), value)
    out, lse = attend(c, sink=sink, status=ST_BAD_POSITION)
    assert (out[:2] == 0).all() and (lse[:2] == value).all()


@pytest.mark.parametrize("with_sink", [False, True])
def test_nan_queries_show(with_sink):
    """A query that is NaN has NaN as its output and as its log denominator (not
    that of a query without keys); the others have their own."""
    for c, calls in forms(3):
        rng = np.random.default_rng(1)
        bad = torch.from_numpy(rng.random((c.T, c.Hq)) < 0.2)
        sink = torch.randn(c.Hq, generator=torch.Generator().manual_seed(2)) if with_sink else None
        ref = reference(c, sink=sink)
        c.q = torch.where(bad[..., None], math.nan, c.q)
        for call in calls:
            out, lse = (x.cpu() for x in call(sink))
            assert out[bad].isnan().all() and lse[bad].isnan().all()
            out[bad], lse[bad] = ref[0][bad].to(out.dtype), ref[1][bad].float()
            check(c, out, lse, ref)


def taken(start, T):
    """The sequences whose rows a call takes, by the header's rule."""
    return [b for b, (x, y) in enumerate(zip(start, start[1:]))
            if 0 <= x <= y <= T and x >= max(start[:b + 1])]


@pytest.mark.parametrize("start", [
    [0, 8, 4, 12], [0, 4, 8, 1000], [-3, 4, 8, 12], [0, 20, 8, 12], [5, 3, 4, 9], [2, 6, 6, 5],
    # more sequences than a warp looks at in one go, a fall in the second group
    # that the third is past of, and one to the end
    [*range(0, 40), 20, *range(21, 70)], [*range(0, 40), 3, *range(4, 70)]])
def test_sequences_beside_a_start_that_falls(start):
    """A q_start that decreases or leaves [0, T]: appends and attention take the
    rows of the same sequences, each row at most once, and leave the others."""
    v = v4()
    T, B = max(12, max(start) if len(start) > 4 else 0), len(start) - 1
    rows = [(t, b, t - start[b]) for b in taken(start, T) for t in range(start[b], start[b + 1])]
    assert len({t for t, _, _ in rows}) == len(rows)
    # a history of 130 positions before each sequence's tokens
    ls = [130 + max(0, y - x) for x, y in zip(start, start[1:])]
    c = Case([0] * B, ls, 8, 2, 64, seed=B, front=T)
    c.tokens = lambda: ((t, b, 130 + i) for t, b, i in rows)
    desc = desc_of(c, d_rope=0)
    ws = v.kv_workspace(desc)
    kw = c.args(ws)
    kw["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    x = torch.randn(T, 2, 64, generator=torch.Generator().manual_seed(1)).to(c.dt)
    want_k = c.k_pool.clone()
    for t, b, i in rows:
        p = 130 + i
        want_k[c.table[b, p // BLOCK], :, p % BLOCK] = x[t]
        c.hist_k[b][p] = c.hist_v[b][p] = x[t]
    v.kv_append(desc, k=x.cuda(), v=x.cuda(), **kw)
    assert v.device_status_code(ws)[1] & ST_BAD_SEQ
    assert torch.equal(kw["k_cache"].cpu().view(torch.int16), want_k.view(torch.int16))
    v.workspace_init(ws)
    out, lse = outputs(c)
    v.paged_attention(desc, q=c.q.cuda(), out=out, lse=lse, **kw)
    assert v.device_status_code(ws)[1] & ST_BAD_SEQ
    check(c, out, lse, reference(c))


def test_append_to_thousands_of_sequences():
    """More sequences than threads, some without tokens."""
    v = v4()
    rng = np.random.default_rng(0)
    ns = rng.choice([0, 0, 1, 3], 3000)
    start = np.concatenate([[2], 2 + np.cumsum(ns)]).astype(np.int32)
    T, d = int(start[-1]) + 3, 64
    table = torch.from_numpy(rng.permutation(3000).astype(np.int32))[:, None]
    ls = ns + rng.integers(0, 100, 3000)
    x = torch.randn(T, 1, d, generator=torch.Generator().manual_seed(1)).half()
    kc = torch.zeros(3000, 1, BLOCK, d, dtype=torch.float16)
    want = kc.clone()
    for b in range(3000):
        t = np.arange(start[b], start[b + 1])
        want[table[b, 0], 0, ls[b] - ns[b]:ls[b]] = x[t, 0]
    desc = v.kv_desc(1, 1, d, dtype=torch.float16, d_rope=0)
    ws = v.kv_workspace(desc)
    kc, vc = kc.cuda(), kc.cuda()
    v.kv_append(desc, k=x.cuda(), v=x.cuda(), k_cache=kc, v_cache=vc, ws=ws,
                q_start=torch.from_numpy(start).cuda(), kv_len=torch.from_numpy(ls).cuda(),
                block_table=table.cuda())
    assert v.device_status(ws) == 0
    assert torch.equal(kc.cpu(), want) and torch.equal(vc.cpu(), want)


@pytest.mark.parametrize("theta", [1.1450824737548828, 1.0380772352218628, 10000.0])
@pytest.mark.parametrize("halves", [False, True])
def test_angles_at_the_farthest_positions(theta, halves):
    """Rotations at the last positions that a table can hold, of pairs that their
    angle turns onto an axis: what is left of the first member shows the angle.
    The angle is off by two roundings of its turns in double, 2^-52 p <= 2^-22,
    and by 2^-21 with sine and products in fp32; the result by a rounding."""
    v = v4()
    d, bps, n = 128, 1 << 23, 3
    L = bps * BLOCK
    p = np.arange(L - n, L)[:, None].astype(np.longdouble)
    k = np.arange(d // 2).astype(np.longdouble)
    angle = p * np.longdouble(theta) ** (-2 * k / d)
    cos, sin = np.cos(angle), np.sin(angle)
    size = 8.0
    a = torch.from_numpy((size * sin).astype(np.float64)).half()
    b = torch.from_numpy((size * cos).astype(np.float64)).half()
    lay = (lambda x, y: torch.cat((x, y), -1)) if halves else \
        (lambda x, y: torch.stack((x, y), -1).flatten(-2))
    x = lay(a, b)[:, None].contiguous()
    A, B = a.double().numpy().astype(np.longdouble), b.double().numpy().astype(np.longdouble)
    want = lay(*(torch.from_numpy(w.astype(np.float64)) for w in (A * cos - B * sin,
                                                                  A * sin + B * cos)))
    desc = v.kv_desc(1, 1, d, dtype=torch.float16, rope_theta=theta, rope_halves=halves)
    ws = v.kv_workspace(desc)
    table = torch.zeros(1, bps, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(1, 1, BLOCK, d, dtype=torch.float16, device="cuda") for _ in range(2))
    q_out = torch.empty_like(x, device="cuda")
    v.kv_append(desc, k=x.cuda(), v=x.cuda(), q=x.cuda(), q_out=q_out, k_cache=kc, v_cache=vc,
                q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), ws=ws,
                kv_len=torch.tensor([L], device="cuda"), block_table=table)
    assert v.device_status(ws) == 0
    tol = 2.0 ** -11 * want.abs() + (2.0 ** -21 + 2.0 ** -22) * size * (1 + 2.0 ** -10)
    for got in (q_out[:, 0], kc[0, 0, -n:]):
        assert ((got.double().cpu() - want).abs() <= tol).all()


def first_keys_apart(c, n, logit, other_v):
    """Keys whose logits are 0 but for the first n of each sequence, at ``logit``,
    with values 0 there and ``other_v`` (1 + j / 512) elsewhere."""
    q = 1.0
    c.q = torch.full_like(c.q, q)
    for b, x in enumerate(c.ls):
        c.hist_k[b] = torch.zeros_like(c.hist_k[b])
        c.hist_k[b][:n] = logit / (q * math.sqrt(c.d))
        v = other_v * (1 + (torch.arange(x) % 512) / 512.0)
        v[:n] = 0.0
        c.hist_v[b] = v[:, None, None].expand(x, c.Hkv, c.d).to(c.dt).contiguous()
        for i in range(0, x, BLOCK):
            m = min(BLOCK, x - i)
            for pool, hist in ((c.k_pool, c.hist_k), (c.v_pool, c.hist_v)):
                pool[c.table[b, i // BLOCK], :, :m] = hist[b][i:i + m].transpose(0, 1)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ns,ls,Hq,Hkv,d", [([1] * 160, [900] * 160, 16, 2, 64),
                                            ([30] * 60, [700] * 60, 8, 2, 64),
                                            ([1], [20000], 8, 1, 128)])
def test_many_keys_far_below_one(ns, ls, Hq, Hkv, d, dtype):
    """One key e^17.7 = 2^25.5 above all others, whose values are what the output
    holds: weights that small still count."""
    c = Case(ns, ls, Hq, Hkv, d, dtype, seed=1, spare=0)
    first_keys_apart(c, 1, 17.7, 64.0)
    check(c, *attend(c), reference(c))
    idx = torch.arange(-(-max(ls) // BLOCK), dtype=torch.int32).expand(c.T, 1, -1).contiguous()
    check(c, *select(c, idx, 0), reference(c))


@pytest.mark.parametrize("ns,ls,Hq,Hkv,d", [([1] * 160, [300] * 160, 16, 2, 64),
                                            ([30] * 60, [300] * 60, 8, 2, 64)])
def test_large_values(ns, ls, Hq, Hkv, d):
    """bf16 values whose sum, weights up to 1, fits fp32, behind logits that rise
    by less than what moves the running maximum."""
    c = Case(ns, ls, Hq, Hkv, d, "bf16", seed=1, spare=0)
    first_keys_apart(c, BLOCK, -5.0, 5e35)
    check(c, *attend(c), reference(c))


def test_workspaces_that_are_no_memory():
    """An expanded tensor has a workspace's size in its shape alone: refused."""
    v = v4()
    c = Case([1], [300], 8, 2, 64, seed=1)
    desc = desc_of(c)
    n = v.kv_workspace(desc).numel()
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.zeros(2, n, dtype=torch.uint8, device="cuda")[:, ::2]):
        args = c.args(ws)
        out, lse = outputs(c)
        x = torch.zeros(1, 2, 64, dtype=c.dt, device="cuda")
        with pytest.raises(ValueError, match="contiguous"):
            v.paged_attention(desc, q=c.q.cuda(), out=out, lse=lse, **args)
        with pytest.raises(ValueError, match="contiguous"):
            v.kv_append(desc, k=x, v=x, **args)
        assert (out == 7.0).all() and (lse == 7.0).all()


FIRST_CALL = """
import torch
from tests.kv_util import Case, check, reference
import long_context_compressed_kv_b200 as v
c = Case([20, 1], [300, 200], 8, 2, 64, seed=9)
desc = v.kv_desc(8, 2, 64, d_rope=0)
ws = v.kv_workspace(desc)
kw = c.args(ws)
q, out, lse = c.q.cuda(), torch.empty(c.T, 8, 64, dtype=c.dt, device="cuda"), torch.empty(c.T, 8, device="cuda")
new = [torch.cat([h[b][L - n:] for b, (n, L) in enumerate(zip(c.ns, c.ls))]).cuda()
       for h in (c.hist_k, c.hist_v)]
lists = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").expand(c.T, 2).contiguous()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    # a copy and a kernel on two streams, both waited for by the first call
    start = torch.cuda.current_stream()
    side.wait_stream(start)
    with torch.cuda.stream(side):
        kv = [x.clone() for x in new]
    q2 = q + 0
    lens = kw["kv_len"] * 1
    start.wait_stream(side)
    kw["kv_len"] = lens
    v.kv_append(desc, k=kv[0], v=kv[1], **kw)
    if SPARSE:
        v.block_sparse_attention(desc, q=q2, out=out, lse=lse, idx=lists, n_local=1, **kw)
    else:
        v.paged_attention(desc, q=q2, out=out, lse=lse, **kw)
    again = out * 2
for _ in range(3):
    out.zero_()
    graph.replay()
assert v.device_status(ws) == 0
check(c, out, lse, reference(c, idx=lists.cpu()[:, None] if SPARSE else None, n_local=1))
assert torch.equal(again, out * 2)
"""


@pytest.mark.parametrize("sparse", [False, True])
def test_first_calls_of_a_process_captured(sparse):
    """The first calls of a process are captured, behind a copy and a kernel of two
    streams and in front of one."""
    p = subprocess.run([sys.executable, "-c", f"SPARSE = {sparse}\n" + FIRST_CALL],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_rows_far_apart():
    """Token rows 2^30 elements apart: the third begins past 2^31."""
    v = v4()
    c = Case([2, 1], [300, 140], 8, 2, 64, seed=2)
    new = [torch.cat([h[b][L - n:] for b, (n, L) in enumerate(zip(c.ns, c.ls))])
           for h in (c.hist_k, c.hist_v)]
    wide = torch.empty((2 << 30) + 20 * 64, dtype=c.dt, device="cuda")

    def heads(first, n):
        return wide[first * 64:].as_strided((3, n, 64), (1 << 30, 64, 1))

    q, k, x, out = heads(0, 8), heads(8, 2), heads(10, 2), heads(12, 8)
    for dst, src in ((q, c.q), (k, new[0]), (x, new[1])):
        dst.copy_(src)
    out.fill_(7.0)
    desc = desc_of(c, d_rope=0)
    ws = v.kv_workspace(desc)
    kw = c.args(ws)
    before = [kw[n].cpu().view(torch.int16) for n in ("k_cache", "v_cache")]
    v.kv_append(desc, k=k, v=x, q=q, q_out=q, **kw)
    lse = torch.empty(3, 8, device="cuda")
    v.paged_attention(desc, q=q, out=out, lse=lse, **kw)
    assert v.device_status(ws) == 0
    assert all(torch.equal(kw[n].cpu().view(torch.int16), b)
               for n, b in zip(("k_cache", "v_cache"), before))
    check(c, out, lse, reference(c))


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
# sequences, new tokens, positions, heads, dim: items of thousands of blocks on a
# CTA, of 8, 32 and 100 rows and of two tiles
@pytest.mark.parametrize("B,n,L,Hq,Hkv,d", [(160, 1, 1 << 19, 8, 1, 128), (150, 1, 1 << 19, 32, 1, 64),
                                            (75, 1, 1 << 19, 200, 2, 64), (80, 40, 1 << 19, 8, 1, 128)])
def test_sums_over_long_histories(B, n, L, Hq, Hkv, d, dtype, rising):
    """Values of one sign over thousands of blocks on one CTA: the tensor core cuts
    its sums off, by up to 2^-23 of them each 16 keys, for which the 256 blocks
    that it takes in one go allow 2^-12.  The table's entries are seven pool blocks,
    in an order in which logits rise or at random."""
    v = v4()
    nb, u = L // BLOCK, torch.finfo(dtype).eps / 2
    g = torch.Generator().manual_seed(Hq)
    kb = 0.3 * torch.randn(7, Hkv, BLOCK, d, generator=g)
    kb[..., 0] = torch.arange(7.0)[:, None, None] * (4.0 if rising else 0.0)
    kb, vb = kb.to(dtype), (1 + torch.rand(7, Hkv, BLOCK, d, generator=g)).to(dtype)
    q = torch.randn(B * n, Hq, d, generator=g)
    q[..., 0] = math.sqrt(d) / 2
    q = q.to(dtype)
    table = torch.randint(0, 7, (nb,), generator=g, dtype=torch.int32)
    if rising:
        table = table.sort().values
    desc = v.kv_desc(Hq, Hkv, d, dtype=dtype)
    ws = v.kv_workspace(desc)
    kw = dict(q=q.cuda(), k_cache=kb.cuda(), v_cache=vb.cuda(), ws=ws,
              q_start=torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"),
              kv_len=torch.full((B,), L, device="cuda"), block_table=table.expand(B, nb).contiguous().cuda())
    got = []
    for sparse in (False, True):
        out = torch.full((B * n, Hq, d), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((B * n, Hq), 7.0, device="cuda")
        if sparse:
            v.block_sparse_attention(desc, idx=None, n_local=nb, out=out, lse=lse, **kw)
        else:
            v.paged_attention(desc, out=out, lse=lse, **kw)
        assert v.device_status(ws) == 0
        got.append((out.double().cpu(), lse.double().cpu()))
    kd, vd, gr = kb.double(), vb.double(), Hq // Hkv
    for t in {0, B * n - 1, *range(3, B * n, max(1, B * n // 9))}:
        p = L - n + t % n
        last = p // BLOCK
        # how often the query sees each of the 7 x 128 keys
        often = torch.bincount(table[:last], minlength=7).double()[:, None].repeat(1, BLOCK)
        often[table[last], :p % BLOCK + 1] += 1
        for h in range(Hkv):
            hs = slice(h * gr, h * gr + gr)
            qq, k, x = q[t, hs].double(), kd[:, h].flatten(0, 1), vd[:, h].flatten(0, 1)
            s = qq @ k.T / math.sqrt(d) + often.flatten().log()
            e = d * 2.0 ** -23 * (qq.abs() @ k.abs().T).amax(1)[:, None] / math.sqrt(d) + 2.0 ** -18
            z = s.logsumexp(1)
            want = (s - z[:, None]).exp() @ x
            tol = u * want + (u + 2 * e + 2.0 ** -12) * want * (1 + u)
            for out, lse in got:
                assert ((out[t, hs] - want).abs() <= tol).all(), (t, h)
                assert ((lse[t, hs] - z).abs() <= e[:, 0] + 2.0 ** -20 * (1 + z.abs())).all(), (t, h)
