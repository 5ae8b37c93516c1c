"""Work for the paged 16-bit K/V cache: appending new tokens (with the position
rotation), attention of new tokens over the cache, and attention over the
blocks that a selector chose for each query.

``run`` computes one pass of an operator: in elementary torch operations with
float32 arithmetic where ``own`` is false, through the framework's entry points
where it is true.  ``exact`` states the same results in float64.

Shapes (see include/v4attn.h): q [T][Hq][d], k / v [T][Hkv][d]; pools
[blocks][Hkv][128][d]; sequence b owns the token rows q_start[b] ..
q_start[b+1]-1, which sit at positions kv_len[b] - n_b .. kv_len[b] - 1.
"""
import math

import torch

own = False

BLOCK = 128          # tokens a block of the pools holds
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(op, name=None, *, B, n, L, Hq, Hkv, d, dtype="bf16", ragged=False, **more):
    """B sequences of up to n new tokens at the end of up to L positions;
    ragged: the sequences' lengths spread over the range below."""
    c = dict(op=op, B=B, n=n, L=L, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, ragged=ragged)
    c.update({"append": dict(d_rope=d, halves=False), "attend": dict(n_win=0, sink=False),
              "select": dict(n_sel=16, n_local=2, per_head=False)}[op])
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's keys and values of a small batch: launch latency
        _case("append", "append_step", B=16, n=1, L=700, Hq=64, Hkv=8, d=128),
        # a ragged batch, three query heads a K/V head, rotation of half the dims, halves paired
        _case("append", "append_ragged", B=7, n=301, L=1500, Hq=24, Hkv=8, d=64, dtype="fp16",
              ragged=True, d_rope=32, halves=True),
        # a long prefill chunk behind a prefix of its own length
        _case("append", "append_chunk", B=1, n=8192, L=16384, Hq=64, Hkv=8, d=128),
        # one sequence's decode step on a short history: the smallest call
        _case("attend", "attend_step_short", B=1, n=1, L=1999, Hq=64, Hkv=8, d=128),
        # a serving batch's decode step, histories of many lengths
        _case("attend", "attend_step", B=32, n=1, L=16384, Hq=64, Hkv=8, d=128, ragged=True),
        # one very long sequence: few rows, all the work along the keys
        _case("attend", "attend_step_long", B=1, n=1, L=262144, Hq=16, Hkv=2, d=128),
        # prompts and decode steps in one batch, sliding window, sink logits
        _case("attend", "attend_mixed", B=9, n=257, L=6001, Hq=32, Hkv=4, d=64, dtype="fp16",
              ragged=True, n_win=1024, sink=True),
        # chunked prefill deep in a long prompt
        _case("attend", "attend_chunk", B=1, n=2048, L=32768, Hq=64, Hkv=8, d=128),
        # whole prompts, one K/V head per query head
        _case("attend", "attend_prompt", B=4, n=4096, L=4096, Hq=32, Hkv=32, d=128, ragged=True),
        # decode at 128K, 16 selected blocks and the last two
        _case("select", "select_step", B=16, n=1, L=131072, Hq=64, Hkv=8, d=128, ragged=True),
        # short ragged chunks, a selection for each K/V head
        _case("select", "select_ragged", B=5, n=61, L=9000, Hq=32, Hkv=4, d=64, dtype="fp16",
              ragged=True, n_sel=8, n_local=1, per_head=True),
        # chunked prefill at 64K on selected blocks
        _case("select", "select_chunk", B=1, n=1024, L=65536, Hq=64, Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "select"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    more = dict(dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.6)
    B = _log(rng, 1, 32)
    # half of the draws are decode steps
    n = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
    # bounds that keep a draw below the largest listed case: the padded
    # (query, key) pairs over all heads, and the cache's values
    if op == "append":
        L = n + _log(rng, 1, 4096)
        B = max(1, min(B, 16384 // n, (1 << 25) // (Hkv * d * L)))
        more.update(d_rope=rng.choice([d, d // 2, d // 4]), halves=rng.random() < 0.5)
    else:
        L = n + _log(rng, 1, 65536 if n > 1 else 131072)
        L = min(L, max(n, (1 << 32) // (n * Hkv * g)))
        B = max(1, min(B, (1 << 32) // (n * L * Hkv * g), (1 << 30) // (Hkv * d * L)))
    if op == "attend":
        more.update(n_win=rng.choice([0, 0, _log(rng, 1, 4096)]), sink=rng.random() < 0.5)
    if op == "select":
        more.update(n_sel=_log(rng, 1, 64), n_local=rng.choice([0, 1, 2, 3]),
                    per_head=rng.random() < 0.3)
    return _case(op, B=B, n=n, L=L, Hq=Hkv * g, Hkv=Hkv, d=d, **more)


def _lengths(c):
    """(new tokens, positions) of each sequence, the same for every seed: all
    at the case's n and L, or spread evenly down to 1 and to n, out of step
    with each other."""
    B, n, L = c["B"], c["n"], c["L"]
    if not c["ragged"]:
        return [n] * B, [L] * B
    ns = [max(1, round(n * ((i * 5 + 1) % B + 1) / B)) for i in range(B)]
    ls = [max(m, round(L * ((i * 3 + 2) % B + 1) / B)) for i, m in enumerate(ns)]
    return ns, ls


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, Hq, Hkv = DTYPES[c["dtype"]], c["d"], c["Hq"], c["Hkv"]
    ns, ls = _lengths(c)
    T, B, bps = sum(ns), c["B"], -(-max(ls) // BLOCK)
    need = [-(-x // BLOCK) for x in ls]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt)

    # the pool's blocks are dealt to the sequences in a shuffled order; a few are free
    n_blocks = sum(need) + 3
    ids = torch.randperm(n_blocks, generator=gen, device=dev)[:sum(need)].to(torch.int32)
    table = torch.full((B, bps), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    start = [0]
    for m in ns:
        start.append(start[-1] + m)
    n_t = torch.tensor(ns, device=dev)
    seq = torch.repeat_interleave(torch.arange(B, device=dev), n_t, output_size=T)
    kv_len = torch.tensor(ls, dtype=torch.int64, device=dev)
    q_start = torch.tensor(start, dtype=torch.int32, device=dev)
    local = torch.arange(T, device=dev) - q_start.long()[seq]
    s = dict(c=c, T=T, n_max=max(ns), table=table, q_start=q_start, kv_len=kv_len, seq=seq,
             local=local, pos=kv_len[seq] - n_t[seq] + local,
             k_cache=randn(n_blocks, Hkv, BLOCK, d), v_cache=randn(n_blocks, Hkv, BLOCK, d),
             out=torch.empty(T, Hq, d, dtype=dt, device=dev))
    if c["op"] == "append":
        # the projections' fused output: q, k and v are strided views of it
        qkv = randn(T, Hq + 2 * Hkv, d)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], theta=160000.0)
        return s
    # logits of standard deviation 2: a few hundred keys carry a row
    s.update(q=randn(T, Hq, d).mul_(2.0), lse=torch.empty(T, Hq, device=dev), sink=None)
    if c["op"] == "attend" and c["sink"]:
        s["sink"] = torch.randn(Hq, generator=gen, device=dev)
    if c["op"] == "select":
        # a selector's scores of the complete blocks before each query, alike
        # for neighbouring queries; its choice in ascending order, -1 behind it
        lists = Hkv if c["per_head"] else 1
        score = torch.randn(B, lists, bps, generator=gen, device=dev)[seq]
        score += 0.5 * torch.randn(T, lists, bps, generator=gen, device=dev)
        blk = torch.arange(bps, device=dev)
        score.masked_fill_(blk >= (s["pos"] // BLOCK)[:, None, None], -math.inf)
        k = min(c["n_sel"], bps)
        top = score.topk(k, dim=-1)
        ids = torch.where(top.values > -math.inf, top.indices, bps).sort(dim=-1).values
        idx = torch.full((T, lists, c["n_sel"]), -1, dtype=torch.int32, device=dev)
        idx[:, :, :k] = torch.where(ids < bps, ids, -1).to(torch.int32)
        s["idx"] = idx
    return s


# ------------------------------------------------------------------ plain forms


def _rotate(x, pos, theta, d_rope, halves):
    """R(pos) on the last d_rope dims of x [T][H][d], rounded to x's type."""
    half = d_rope // 2
    k = torch.arange(half, dtype=torch.float64, device=x.device)
    a = pos.double()[:, None] * theta ** (-2.0 * k / d_rope)
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    y = x.float()
    keep, r = y[..., :x.shape[-1] - d_rope], y[..., x.shape[-1] - d_rope:]
    u, v = (r[..., :half], r[..., half:]) if halves else (r[..., 0::2], r[..., 1::2])
    turned = (u * cos - v * sin, u * sin + v * cos)
    r = torch.cat(turned, -1) if halves else torch.stack(turned, -1).flatten(-2)
    return torch.cat((keep, r), -1).to(x.dtype)


def _plain_append(s):
    c = s["c"]
    turn = (s["pos"], s["theta"], c["d_rope"], c["halves"])
    block, slot = s["table"][s["seq"], s["pos"] // BLOCK].long(), s["pos"] % BLOCK
    s["k_cache"][block, :, slot] = _rotate(s["k"], *turn)
    s["v_cache"][block, :, slot] = s["v"]
    return {"q": _rotate(s["q"], *turn), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _selected(s):
    """[T][lists][blocks]: whether a query's list or its last blocks hold a block."""
    idx, own_block = s["idx"].long(), (s["pos"] // BLOCK)[:, None, None]
    before = torch.cat((torch.full_like(idx[..., :1], -1), idx.cummax(-1).values[..., :-1]), -1)
    good = (idx >= 0) & (idx > before) & (idx <= own_block)
    bps = s["table"].shape[1]
    hit = torch.zeros(*idx.shape[:2], bps, dtype=torch.int32, device=idx.device)
    hit.scatter_add_(2, idx.clamp(0, bps - 1), good.to(torch.int32))
    blk = torch.arange(bps, device=idx.device)
    return (hit > 0) | (blk > own_block - s["c"]["n_local"])


def _plain_attention(s):
    c, q = s["c"], s["q"]
    B, n, Hkv, d = c["B"], s["n_max"], c["Hkv"], c["d"]
    g = c["Hq"] // Hkv

    def rows(cache):     # [B][Hkv][L][d], zero past a sequence's end
        x = cache[s["table"].clamp(min=0).long()].float().transpose(1, 2).flatten(2, 3)
        past = torch.arange(x.shape[2], device=x.device) >= s["kv_len"][:, None]
        return x.masked_fill_(past[:, None, :, None], 0.0)

    # queries padded to [B][Hkv][n * g][d]
    qp = torch.zeros(B, n, c["Hq"], d, device=q.device)
    qp[s["seq"], s["local"]] = q.float() * d ** -0.5
    qp = qp.view(B, n, Hkv, g, d).transpose(1, 2).reshape(B, Hkv, n * g, d)
    w = torch.matmul(qp, rows(s["k_cache"]).transpose(2, 3))
    L = w.shape[3]
    j = torch.arange(L, device=q.device)
    pos = torch.full((B, n), -1, dtype=torch.int64, device=q.device)
    pos[s["seq"], s["local"]] = s["pos"]
    see = (j <= pos[:, :, None])[:, None]                       # [B][1][n][L]
    if c["op"] == "attend" and c["n_win"]:
        see = see & (j > pos[:, :, None] - c["n_win"])[:, None]
    if c["op"] == "select":
        hit = _selected(s)
        pad = torch.zeros(B, n, *hit.shape[1:], dtype=torch.bool, device=q.device)
        pad[s["seq"], s["local"]] = hit
        see = see & pad.transpose(1, 2)[..., j // BLOCK]
    w = w.view(B, Hkv, n, g, L).masked_fill_(~see[:, :, :, None], -math.inf)
    top = w.amax(-1)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, 1, g)
        top = torch.maximum(top, sink)
    top = torch.where(top > -math.inf, top, 0.0)
    w = w.sub_(top[..., None]).exp_()
    total = w.sum(-1)
    if s["sink"] is not None:
        total = total + (sink - top).exp()
    o = torch.matmul(w.view(B, Hkv, n * g, L), rows(s["v_cache"])).view(B, Hkv, n, g, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = top + total.log()
    o, lse = o.transpose(1, 2).flatten(2, 3), lse.transpose(1, 2).flatten(2, 3)
    return {"out": o[s["seq"], s["local"]].to(q.dtype), "lse": lse[s["seq"], s["local"]]}


# ------------------------------------------------------------------ the framework's calls


def _own_run(s):
    import long_context_compressed_kv_b200 as v4
    c = s["c"]
    if "desc" not in s:      # a program keeps its layer's description and workspace
        more = dict(d_rope=c["d_rope"], rope_halves=c["halves"], rope_theta=s["theta"]) \
            if c["op"] == "append" else dict(n_win=c.get("n_win", 0))
        s["desc"] = v4.kv_desc(c["Hq"], c["Hkv"], c["d"], dtype=DTYPES[c["dtype"]], **more)
        s["ws"] = v4.kv_workspace(s["desc"])
    cache = dict(k_cache=s["k_cache"], v_cache=s["v_cache"], q_start=s["q_start"],
                 kv_len=s["kv_len"], block_table=s["table"], ws=s["ws"])
    if c["op"] == "append":
        v4.kv_append(s["desc"], k=s["k"], v=s["v"], q=s["q"], q_out=s["out"], **cache)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    cache.update(q=s["q"], out=s["out"], lse=s["lse"], sink=s["sink"])
    if c["op"] == "select":
        v4.block_sparse_attention(s["desc"], idx=s["idx"], n_local=c["n_local"], **cache)
    else:
        v4.paged_attention(s["desc"], **cache)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_run(state)
    return _plain_append(state) if state["c"]["op"] == "append" else _plain_attention(state)


# ------------------------------------------------------------------ bounds and exact results


def work(case):
    c = case
    ns, ls = _lengths(c)
    T, e = sum(ns), 2
    if c["op"] == "append":
        values = T * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return {"bytes": 2 * values * e, "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["d_rope"]}
    total = 2 * T * c["Hq"] * c["d"] * e + 4 * T * c["Hq"]
    row = 2 * c["Hkv"] * c["d"] * e                    # a position's keys and values
    pairs = 0.0                                        # visible (query, key) pairs of a head
    for n, L in zip(ns, ls):
        first = L - n                                  # position of the first new token
        if c["op"] == "attend":
            w = c["n_win"] or L
            full = max(0, min(n, L - w))               # queries with a whole window before them
            rest = n - full
            pairs += full * w + rest * (min(first + 1, w) + min(first + rest, w)) / 2
            total += row * min(L, n - 1 + w)
        else:
            seen, before = c["n_local"] * BLOCK, max(0, first // BLOCK - c["n_local"] + 1)
            chosen = min(c["n_sel"], before)
            pairs += n * min(first + (n + 1) / 2, chosen * BLOCK + max(0, seen - BLOCK // 2))
            lists = c["Hkv"] if c["per_head"] else 1
            total += 4 * n * lists * c["n_sel"]
            union = before * (1 - (1 - chosen / before) ** min(n, 4)) if before else 0
            total += row * min(L, (union + c["n_local"]) * BLOCK + n)
    return {"bytes": total, "flops": 4 * c["Hq"] * c["d"] * pairs}


def _exact_append(s):
    c = s["c"]
    off, half = c["d"] - c["d_rope"], c["d_rope"] // 2
    inverse = [s["theta"] ** (-2.0 * k / c["d_rope"]) for k in range(half)]
    angle = s["pos"].double()[:, None] * torch.tensor(inverse, dtype=torch.float64, device="cuda")
    phase = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turn(x):
        x = x.double().clone()
        a = list(range(off, off + half)) if c["halves"] else list(range(off, c["d"], 2))
        b = [i + (half if c["halves"] else 1) for i in a]
        z = torch.complex(x[..., a], x[..., b]) * phase
        x[..., a], x[..., b] = z.real, z.imag
        return x

    k_cache, v_cache, k = s["k_cache"].double(), s["v_cache"].double(), turn(s["k"])
    where = s["table"].long().cpu()
    ns, ls = _lengths(c)
    t = 0
    for b, (n, L) in enumerate(zip(ns, ls)):
        p = L - n
        while p < L:                                   # up to the end of a block at a time
            m = min(L, (p // BLOCK + 1) * BLOCK) - p
            at = int(where[b, p // BLOCK]), slice(None), slice(p % BLOCK, p % BLOCK + m)
            k_cache[at] = k[t:t + m].transpose(0, 1)
            v_cache[at] = s["v"][t:t + m].double().transpose(0, 1)
            t, p = t + m, p + m
    return {"q": turn(s["q"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_keys(c, s, b, t, h, p, L):
    """The positions that query t at position p of sequence b sees, as a mask of L."""
    j = torch.arange(L, device="cuda")
    see = j <= p
    if c["op"] == "attend":
        return see & (j > p - c["n_win"]) if c["n_win"] else see
    chosen = torch.zeros(-(-L // BLOCK), dtype=torch.bool, device="cuda")
    ids = s["idx"][t, h if c["per_head"] else 0].long()
    chosen[ids[ids >= 0]] = True
    chosen[max(0, p // BLOCK - c["n_local"] + 1):p // BLOCK + 1] |= c["n_local"] > 0
    return see & chosen.repeat_interleave(BLOCK)[:L]


def _exact_attention(s):
    c = s["c"]
    g, d = c["Hq"] // c["Hkv"], c["d"]
    ns, ls = _lengths(c)
    out = torch.zeros(s["T"], c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], c["Hq"], dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, L) in enumerate(zip(ns, ls)):
        blocks = s["table"][b, :-(-L // BLOCK)].long()
        step = max(1, (1 << 28) // (L * g))
        for h in range(c["Hkv"]):
            k = s["k_cache"][blocks, h].double().reshape(-1, d)[:L]
            v = s["v_cache"][blocks, h].double().reshape(-1, d)[:L]
            for i in range(0, n, step):
                m = min(step, n - i)
                t, heads = slice(t0 + i, t0 + i + m), slice(h * g, h * g + g)
                x = torch.einsum("thd,jd->thj", s["q"][t, heads].double(), k) / math.sqrt(d)
                p = torch.arange(L - n + i, L - n + i + m, device="cuda")[:, None]
                j = torch.arange(L, device="cuda")
                if c["op"] == "attend":
                    see = (j <= p) & ((j > p - c["n_win"]) if c["n_win"] else (j >= 0))
                else:
                    see = torch.stack([_exact_keys(c, s, b, t0 + i + r, h, L - n + i + r, L)
                                       for r in range(m)])
                x = x.masked_fill(~see[:, None], -math.inf)
                if s["sink"] is not None:
                    sink = s["sink"][heads].double()[None, :, None].expand(m, g, 1)
                    x = torch.cat((x, sink), -1)
                z = torch.logsumexp(x, -1)
                lse[t, heads] = z
                weight = (x[..., :L] - z[..., None]).exp().nan_to_num(0.0)
                out[t, heads] = torch.einsum("thj,jd->thd", weight, v)
        t0 += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
