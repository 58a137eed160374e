"""Cases of the operators that serve an HSTU stack from a paged key/value cache.

Four operators: the plan of a step (block tables and slot maps from request
lengths), the append of new keys, values and timestamps to the cache, the
attention of new tokens (a chain, a tree of drafted ones, or candidates side by
side) over the cache, and the projections of a few rows with 4-bit weights.

`run` computes them in a plain form of elementary torch operations in 32 bits;
with `own` set it calls the library. Sequence lengths are fixed by the case
(evenly spread quantiles of its distribution) and only their order, the pages
they lie in and all values come from the seed, so every seed of a case has the
same work.
"""

import math

import torch

own = False

GAP_S = 3600.0            # mean time between two actions of a user, seconds
T0 = 1_700_000_000        # first timestamps lie in the year after this one
BIAS_STD = 0.02           # bias tables ~ N(0, 0.02^2)


# ------------------------------------------------------------------ cases

def _plan(name, B, lo, hi, dist, new, page):
    return dict(name=name, op="plan", B=B, lo=lo, hi=hi, dist=dist, new=new, page=page)


def _append(name, T, H, d, page, dtype):
    return dict(name=name, op="append", T=T, H=H, d=d, page=page, dtype=dtype)


def _attn(name, B, lo, hi, dist, new, kind, H, d, page, dtype, num_pos):
    return dict(name=name, op="attn", B=B, lo=lo, hi=hi, dist=dist, new=new, kind=kind, H=H, d=d,
                page=page, dtype=dtype, num_pos=num_pos)


def _w4(name, M, K, N, group, epilogue):
    return dict(name=name, op="w4", M=M, K=K, N=N, group=group, epilogue=epilogue)


def listed():
    return [
        # one new action for each of 128 short histories: a serving step's bookkeeping
        _plan("plan_step_b128", 128, 20, 200, "uniform", 1, 16),
        # sixteen long histories enter the cache whole (no context yet)
        _plan("plan_prompt_b16", 16, 1, 8192, "beta", 0, 64),
        # the new rows of that serving step
        _append("append_step_128", 128, 2, 64, 16, "bf16"),
        # the keys and values of a batch of whole histories
        _append("append_prompt_79913", 79913, 4, 128, 64, "bf16"),
        # plain decoding: one token over short histories
        _attn("attn_step_short", 128, 20, 200, "uniform", 1, "chain", 2, 64, 16, "bf16", 200),
        # plain decoding over long histories, ragged to 8192
        _attn("attn_step_long", 16, 1, 8192, "beta", 1, "chain", 4, 128, 64, "bf16", 8192),
        # drafted trees of 64 tokens over histories of 256 to 4096
        _attn("attn_tree_64", 32, 256, 4096, "uniform", 64, "tree", 4, 128, 32, "bf16", 8192),
        # one user, 128 candidates side by side over a full history
        _attn("attn_candidates_128", 1, 8063, 8063, "uniform", 128, "siblings", 4, 128, 128,
              "bf16", 8192),
        # fp32, five new actions in a row, heads of 32
        _attn("attn_chain_f32", 64, 200, 1100, "uniform", 5, "chain", 2, 32, 16, "f32", 64),
        # the layer's UVQK projection for one token
        _w4("w4_uvqk_1", 1, 512, 2048, 128, "silu"),
        # its output projection for a small batch, odd row count
        _w4("w4_out_33", 33, 512, 512, 64, "residual"),
        # a large projection for eight rows: the weights' bytes
        _w4("w4_large_8", 8, 8192, 16384, 128, "none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "w4"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log_int(rng, 1, 2048)
        hi = _log_int(rng, 8, max(8, min(8192, 130000 // B)))
        c = _plan("", B, rng.randint(1, hi), hi, rng.choice(["uniform", "beta"]),
                  rng.choice([0, 1, 3, 17, 64]), page)
    elif op == "append":
        d = rng.choice([32, 64, 128])
        H = rng.randint(1, 8)
        dtype = rng.choice(["bf16", "f32"])
        most = 79913 * 512 * 2 // (H * d * (2 if dtype == "bf16" else 4))
        c = _append("", _log_int(rng, 1, min(most, 131072)), H, d, page, dtype)
    elif op == "attn":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([32, 64, 128])
        H = rng.randint(1, 8)
        B = _log_int(rng, 1, 512)
        rows = 32 * 4096 * 4 * 128 // (H * d) // (1 if dtype == "bf16" else 8)
        hi = _log_int(rng, 8, max(8, min(8192, rows // B)))
        kind = rng.choice(["chain", "tree", "siblings"])
        pairs = 32 * 4096 * 4 * 64 // (1 if dtype == "bf16" else 16)
        new = _log_int(rng, 1, max(1, min(128, pairs // (B * hi * H))))
        c = _attn("", B, rng.randint(0, hi), hi, rng.choice(["uniform", "beta"]), new, kind, H, d,
                  page, dtype, rng.choice([64, 200, 8192]))
    else:
        group = rng.choice([32, 64, 128])
        K = 128 * _log_int(rng, 1, 64)
        N = _log_int(rng, 1, 16384)
        c = _w4("", rng.randint(1, 64), K, N, group, rng.choice(["none", "silu", "residual"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes of a case

def _lengths(c):
    """Evenly spread quantiles of the length distribution (beta: hi * Beta(2, 1))."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    u = [(i + 0.5) / B for i in range(B)]
    if c["dist"] == "beta":
        return [min(hi, max(lo, int(round(hi * math.sqrt(x))))) for x in u]
    return [lo + int(x * (hi - lo + 1)) if hi > lo else lo for x in u]


def _pages(n, page):
    return -(-n // page)


def _plan_lengths(c):
    """(context, new) lengths; new = 0 stands for whole prompts without context.
    Otherwise sequences get 1..new new tokens in turn."""
    n = _lengths(c)
    if c["new"] == 0:
        return [0] * len(n), n
    return n, [1 + i % c["new"] for i in range(len(n))]


def _attn_lengths(c):
    """Chains and trees: 1 to `new` new tokens, most sequences the full count."""
    n = _lengths(c)
    return n, [c["new"] if i % 4 != 3 else 1 + (7 * i) % c["new"] for i in range(len(n))]


def _elt(c):
    return 2 if c["dtype"] == "bf16" else 4


def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new = _plan_lengths(c)
        need = sum(_pages(a + b, c["page"]) - _pages(a, c["page"]) for a, b in zip(ctx, new))
        part = sum(1 for a in ctx if a % c["page"])
        return {"bytes": 4 * len(ctx) + 8 * (len(ctx) + 1) + 8 + 8 * need + 4 * part + 8 * sum(new),
                "flops": sum(new)}
    if c["op"] == "append":
        return {"bytes": c["T"] * (2 * (2 * c["H"] * c["d"] * _elt(c) + 8) + 8), "flops": 0}
    if c["op"] == "attn":
        ctx, new = _attn_lengths(c)
        tok, T = sum(ctx) + sum(new), sum(new)
        # pairs: every cached token, then itself and its ancestors (a chain's
        # count; trees and siblings are counted with themselves alone)
        pairs = sum(a * b + (b * (b + 1) // 2 if c["kind"] == "chain" else b)
                    for a, b in zip(ctx, new))
        hd = c["H"] * c["d"]
        return {"bytes": tok * (2 * hd * _elt(c) + 8) + T * (2 * hd * _elt(c) + 12)
                + 4 * sum(_pages(a + b, c["page"]) for a, b in zip(ctx, new))
                + 4 * c["H"] * (min(c["num_pos"], max(a + b for a, b in zip(ctx, new))) + 128),
                "flops": 4 * hd * pairs}
    M, K, N, G = c["M"], c["K"], c["N"], c["group"]
    return {"bytes": N * K // 2 + 2 * N * (K // G) + 2 * M * K + 2 * M * N + 4 * N
            + (2 * M * N if c["epilogue"] == "residual" else 0), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _offsets(lens, device):
    t = torch.zeros(len(lens) + 1, dtype=torch.int64)
    t[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    return t.to(device)


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = {"case": c}

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=dev, generator=g) * std).to(dtype)

    def order(n):
        return torch.randperm(n, generator=h)

    if c["op"] == "plan":
        ctx, new = _plan_lengths(c)
        perm = order(len(ctx)).tolist()
        ctx, new = [ctx[i] for i in perm], [new[i] for i in perm]
        page = c["page"]
        have = [_pages(a, page) for a in ctx]
        need = [_pages(a + b, page) - x for a, b, x in zip(ctx, new, have)]
        pool = order(sum(have) + sum(need) + 64).to(torch.int32)
        s["B"], s["T"], s["need"] = len(ctx), sum(new), sum(need)
        width = max(x + y for x, y in zip(have, need))
        # pages that the sequences hold already; -1 where there is none yet
        table = torch.full((len(ctx), width), -1, dtype=torch.int32)
        hv = torch.tensor(have)
        at = torch.arange(width)[None, :] < hv[:, None]
        table[at] = pool[: sum(have)]
        s["block_table"] = table.to(dev)
        # the list of free pages: seven of it were taken by earlier steps
        s["free_pages"] = torch.cat([pool[-7:], pool[sum(have):-7]]).to(dev)
        s["free_start"] = torch.full((1,), 7, dtype=torch.int32, device=dev)
        s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["new_offsets"] = _offsets(new, dev)
        return s
    if c["op"] == "append":
        T, H, d, page = c["T"], c["H"], c["d"], c["page"]
        pages = _pages(T, page) + 8
        s["k"], s["v"] = normal(T, H, d, dtype=_dt(c)), normal(T, H, d, dtype=_dt(c))
        s["timestamps"] = T0 + torch.randint(0, 1 << 25, (T,), device=dev, generator=g)
        s["k_cache"] = normal(pages, page, H, d, dtype=_dt(c))
        s["v_cache"] = normal(pages, page, H, d, dtype=_dt(c))
        s["ts_cache"] = torch.zeros(pages, page, dtype=torch.int64, device=dev)
        # runs of a page each, the pages in any order
        first = order(pages)[: _pages(T, page)].to(dev)
        s["slots"] = (first[:, None] * page + torch.arange(page, device=dev)).reshape(-1)[:T].contiguous()
        return s
    if c["op"] == "attn":
        ctx, new = _attn_lengths(c)
        perm = order(len(ctx)).tolist()
        ctx, new = [ctx[i] for i in perm], [new[i] for i in perm]
        B, H, d, page = c["B"], c["H"], c["d"], c["page"]
        T, total = sum(new), [a + b for a, b in zip(ctx, new)]
        held = [_pages(n, page) for n in total]
        pages = sum(held) + 8
        width = max(held)
        table = torch.zeros((B, width), dtype=torch.int32)
        table[torch.arange(width)[None, :] < torch.tensor(held)[:, None]] = order(pages)[: sum(held)].to(torch.int32)
        s["block_table"] = table.to(dev)
        s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["new_offsets"] = _offsets(new, dev)
        s["q"] = normal(T, H, d, dtype=_dt(c))
        s["k_cache"] = normal(pages, page, H, d, dtype=_dt(c))
        s["v_cache"] = normal(pages, page, H, d, dtype=_dt(c))
        s["pos_bias"] = normal(H, c["num_pos"], std=BIAS_STD)
        s["time_bias"] = normal(H, 128, std=BIAS_STD)
        # the history's actions, then the new ones after them
        n = max(total)
        gaps = torch.empty(B, n, dtype=torch.float64, device=dev).exponential_(1.0 / GAP_S, generator=g)
        start = T0 + (torch.rand(B, 1, device=dev, generator=g, dtype=torch.float64) * 31_500_000.0)
        ts = torch.floor(start + torch.cumsum(gaps, 1)).to(torch.int64)
        ctx_d, tot_d = s["ctx_lens"].long()[:, None], torch.tensor(total, device=dev)[:, None]
        j = torch.arange(n, device=dev)[None, :].expand(B, n)
        slot = s["block_table"].long().gather(1, j // page) * page + j % page
        s["ts_cache"] = torch.zeros(pages * page, dtype=torch.int64, device=dev)
        live = j < tot_d
        s["ts_cache"][slot[live]] = ts[live]
        s["ts_cache"] = s["ts_cache"].view(pages, page)
        fresh = live & (j >= ctx_d)
        s["timestamps"] = ts[fresh].contiguous()
        i = (j - ctx_d)[fresh]
        if c["kind"] == "chain":
            s["parents"] = None
        elif c["kind"] == "siblings":
            s["parents"] = torch.full((T,), -1, dtype=torch.int32, device=dev)
        else:       # a drafted tree: any earlier token, or the last cached one
            s["parents"] = (torch.floor(torch.rand(T, device=dev, generator=g, dtype=torch.float64) * (i + 1))
                            - 1).to(torch.int32)
        s["max_new"], s["max_seqlen"] = c["new"], max(n, c["hi"])
        return s
    M, K, N, G = c["M"], c["K"], c["N"], c["group"]
    s["x"] = normal(M, K, dtype=torch.bfloat16)
    # symmetric 4-bit codes of N(0, 1/K) weights, two codes a byte, the even one low
    W = torch.randn(N, K, device=dev, generator=g) / math.sqrt(K)
    Wg = W.view(N, K // G, G)
    scales = (Wg.abs().amax(2) / 7).to(torch.bfloat16)
    codes = (torch.round(Wg / scales.float()[:, :, None]).clamp(-8, 7) + 8).to(torch.uint8).view(N, K)
    s["codes"] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
    s["scales"] = scales.contiguous()
    s["bias"] = normal(N, std=BIAS_STD)
    s["residual"] = normal(M, N, dtype=torch.bfloat16) if c["epilogue"] == "residual" else None
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_plan(s):
    import jagged_pointwise_attention_b200 as hstu
    slots, free_end = hstu.hstu_cache_plan(
        s["ctx_lens"], s["new_offsets"], s["free_pages"], s["free_start"], s["block_table"],
        s["case"]["page"], s["T"])
    return {"block_table": s["block_table"], "slots": slots, "free_end": free_end}


def _own_append(s):
    import jagged_pointwise_attention_b200 as hstu
    hstu.hstu_cache_append(s["k"], s["v"], s["timestamps"], s["slots"], s["k_cache"], s["v_cache"],
                           s["ts_cache"])
    return {"k": s["k_cache"], "v": s["v_cache"], "ts": s["ts_cache"]}


def _own_attn(s):
    import jagged_pointwise_attention_b200 as hstu
    return hstu.hstu_attn_cached_fwd(
        s["q"], s["k_cache"], s["v_cache"], s["ts_cache"], s["block_table"], s["ctx_lens"],
        s["new_offsets"], s["timestamps"], s["parents"], s["pos_bias"], s["time_bias"],
        s["max_seqlen"], s["max_new"])


def _own_w4(s):
    import jagged_pointwise_attention_b200 as hstu
    return hstu.hstu_linear_w4_fwd(s["x"], s["codes"], s["scales"], s["bias"],
                                   s["case"]["epilogue"], s["residual"])


def _plain_plan(s):
    page, T, B = s["case"]["page"], s["T"], s["B"]
    dev = s["ctx_lens"].device
    ctx, off = s["ctx_lens"].long(), s["new_offsets"]
    have = (ctx + page - 1) // page
    need = (ctx + off[1:] - off[:-1] + page - 1) // page - have
    ends = torch.cumsum(need, 0)
    first = s["free_start"].long() + ends - need
    col = torch.arange(s["block_table"].shape[1], device=dev)[None, :]
    k = col - have[:, None]
    fresh = (k >= 0) & (k < need[:, None])
    at = torch.where(fresh, first[:, None] + k, 0)
    table = torch.where(fresh, s["free_pages"][at], s["block_table"])
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(off, t, right=True) - 1
    pos = ctx[b] + t - off[b]
    slots = table.view(-1)[b * table.shape[1] + pos // page].long() * page + pos % page
    free_end = s["free_start"] + ends[-1:].to(torch.int32)
    return {"block_table": table, "slots": slots, "free_end": free_end}


def _plain_append(s):
    kc, vc, tc = s["k_cache"], s["v_cache"], s["ts_cache"]
    kc.view(-1, *kc.shape[2:])[s["slots"]] = s["k"]
    vc.view(-1, *vc.shape[2:])[s["slots"]] = s["v"]
    tc.view(-1)[s["slots"]] = s["timestamps"]
    return {"k": kc, "v": vc, "ts": tc}


def _plain_attn(s):
    """Every sequence padded to the longest, dense scores in 32 bits."""
    c = s["case"]
    B, page, N, M = c["B"], c["page"], s["max_seqlen"], s["max_new"]
    dev = s["q"].device
    ctx, off = s["ctx_lens"].long(), s["new_offsets"]
    new = off[1:] - off[:-1]
    n = s["block_table"].shape[1] * page
    j = torch.arange(n, device=dev)
    slot = (s["block_table"].long() * page)[:, :, None] + torch.arange(page, device=dev)
    slot = slot.view(B, n)
    K = s["k_cache"].flatten(0, 1)[slot].float().transpose(1, 2)            # [B, H, n, d]
    V = s["v_cache"].flatten(0, 1)[slot].float().transpose(1, 2)
    tk = s["ts_cache"].view(-1)[slot]
    i = torch.arange(M, device=dev)
    row = torch.clamp(off[:-1, None] + i, max=s["q"].shape[0] - 1)          # [B, M]
    q = s["q"][row].float().transpose(1, 2)                                 # [B, H, M, d]
    tq = s["timestamps"][row]
    if s["parents"] is None:
        depth = i.expand(B, M)
        reach = (i[:, None] >= i[None, :]).expand(B, M, M)
    else:
        # ancestors-or-self: (I - P)^-1 = I + P + P^2 + ..., P the parent's row
        par = torch.where(i < new[:, None], s["parents"][row].long(), -1)
        P = (par[:, :, None] == i).float()
        eye = torch.eye(M, device=dev).expand(B, M, M)
        reach = torch.linalg.solve_triangular(eye - P, eye, upper=False, unitriangular=True) > 0.5
        depth = reach.sum(2) - 1
    # keys behind the context are the new tokens, in their order
    m = j - ctx[:, None]                                                    # [B, n]
    mc = torch.clamp(m, 0, M - 1)
    pk = torch.where(m < 0, j, ctx[:, None] + depth.gather(1, mc))
    seen = (m < 0)[:, None, :] | reach.gather(2, mc[:, None, :].expand(B, M, n))
    seen = seen & (m < new[:, None])[:, None, :]
    pq = ctx[:, None] + depth
    rel = torch.clamp(pq[:, :, None] - pk[:, None, :], 0, c["num_pos"] - 1)
    dt = torch.clamp(tq[:, :, None] - tk[:, None, :], min=1)
    bucket = torch.clamp(torch.frexp(dt.double())[1].long() - 1, max=s["time_bias"].shape[1] - 1)
    S = q @ K.transpose(2, 3)
    S = S + s["pos_bias"][:, rel].transpose(0, 1) + s["time_bias"][:, bucket].transpose(0, 1)
    p = torch.where(seen[:, None], S / (1 + torch.exp(-S)), 0.0)
    out = (p @ V / N).transpose(1, 2)                                       # [B, M, H, d]
    return out[i < new[:, None]].to(s["q"].dtype)


def _plain_w4(s):
    G = s["case"]["group"]
    lo, hi = s["codes"] & 15, s["codes"] >> 4
    W = torch.stack([lo, hi], 2).flatten(1).float() - 8
    W = (W.view(W.shape[0], -1, G) * s["scales"].float()[:, :, None]).view(W.shape[0], -1)
    y = s["x"].float() @ W.t() + s["bias"]
    if s["case"]["epilogue"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["case"]["epilogue"] == "residual":
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


_OWN = {"plan": _own_plan, "append": _own_append, "attn": _own_attn, "w4": _own_w4}
_PLAIN = {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn, "w4": _plain_w4}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and query by query group."""
    c = case
    if c["op"] in ("plan", "append"):
        return None        # whole numbers and copies
    s = prepare(case, seed)
    if c["op"] == "attn":
        outs = []
        off, ctx, page = s["new_offsets"].tolist(), s["ctx_lens"].tolist(), c["page"]
        for b in range(c["B"]):
            o, m, a = off[b], off[b + 1] - off[b], ctx[b]
            pages = s["block_table"][b, : _pages(a + m, page)].long()
            K = s["k_cache"][pages].flatten(0, 1)[: a + m].double()
            V = s["v_cache"][pages].flatten(0, 1)[: a + m].double()
            tk = s["ts_cache"][pages].flatten()[: a + m].cpu()
            par = [t - 1 for t in range(m)] if s["parents"] is None else s["parents"][o: o + m].tolist()
            depth, see = [0] * m, torch.zeros(m, a + m, dtype=torch.bool)
            for t in range(m):
                if par[t] >= 0:
                    depth[t] = depth[par[t]] + 1
                    see[t] = see[par[t]]
                else:
                    see[t, :a] = True
                see[t, a + t] = True
            pos = torch.tensor(list(range(a)) + [a + x for x in depth])
            rel = torch.clamp(pos[a:, None] - pos[None, :], 0, c["num_pos"] - 1)
            dt = torch.clamp(s["timestamps"][o: o + m].cpu()[:, None] - tk[None, :], min=1)
            bucket = torch.zeros_like(dt)
            for e in range(1, 63):
                bucket += dt >= (1 << e)
            bucket = torch.clamp(bucket, max=s["time_bias"].shape[1] - 1)
            dev = K.device
            S = torch.einsum("ihd,jhd->hij", s["q"][o: o + m].double(), K)
            S += s["pos_bias"].double()[:, rel.to(dev)] + s["time_bias"].double()[:, bucket.to(dev)]
            S = S * torch.sigmoid(S) * see.to(dev)
            outs.append(torch.einsum("hij,jhd->ihd", S, V) / s["max_seqlen"])
        return torch.cat(outs)
    G, N = c["group"], c["N"]
    W = torch.empty(N, c["K"], dtype=torch.float64, device=s["x"].device)
    W[:, 0::2] = (s["codes"] % 16).double() - 8
    W[:, 1::2] = torch.div(s["codes"], 16, rounding_mode="floor").double() - 8
    W *= s["scales"].double().repeat_interleave(G, 1)
    y = s["bias"].double() + s["x"].double() @ W.t()
    if c["epilogue"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["epilogue"] == "residual":
        y = y + s["residual"].double()
    return y
