"""Random problems for the paged-cache operators and their definitions in 64
bits, written from the formulas, sequence by sequence. No code is shared with
the library."""

from __future__ import annotations

import dataclasses
from typing import List, Optional

import numpy as np
import torch

U32 = 2.0 ** -24          # half a step of fp32, relative
UBF = 2.0 ** -8           # half a step of bf16, relative


@dataclasses.dataclass
class Step:
    """A serving step: contexts, new tokens, a cache that holds both."""
    ctx: List[int]
    new: List[int]
    parents: Optional[np.ndarray]       # int32 [T] or None (chains)
    q: torch.Tensor                     # [T, H, dqk]
    kc: torch.Tensor                    # [pages, page, H, dqk]
    vc: torch.Tensor
    tsc: Optional[torch.Tensor]         # int64 [pages, page]
    table: np.ndarray                   # int32 [B, max_pages]
    ts: Optional[np.ndarray]            # int64 [T]
    pos: Optional[torch.Tensor]
    tb: Optional[torch.Tensor]
    max_seqlen: int
    page: int

    @property
    def off(self):
        return np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)

    @property
    def T(self):
        return int(sum(self.new))


def random_parents(kind, new, rng):
    out = []
    for n in new:
        for i in range(n):
            if kind == "siblings":
                out.append(-1)
            elif kind == "path":
                out.append(i - 1)
            else:
                out.append(int(rng.integers(-1, i)) if i else -1)
    return np.array(out, dtype=np.int32)


def make_step(ctx, new, kind, H, dqk, dv, page, dtype, num_pos=64, num_buckets=128, seed=0,
              spare=3, junk=float("nan"), use_time=True, use_pos=True, max_seqlen=None,
              scale=1.0, gap=3600.0) -> Step:
    """Pages in random order; every cache row outside a sequence's tokens holds
    `junk`, every table entry behind a sequence's pages an impossible number."""
    rng = np.random.default_rng(seed)
    B, T = len(ctx), sum(new)
    held = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(held) + spare
    order = rng.permutation(pages)
    table = np.full((B, max(max(held), 1) + 1), 2 ** 31 - 1, dtype=np.int32)
    kc = torch.full((pages, page, H, dqk), junk, dtype=dtype)
    vc = torch.full((pages, page, H, dv), junk, dtype=dtype)
    tsc = torch.full((pages, page), -(2 ** 62), dtype=torch.int64)
    at, ts = 0, []
    for b in range(B):
        n = ctx[b] + new[b]
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
        t = 1_700_000_000 + np.cumsum(rng.exponential(gap, n)).astype(np.int64)
        ts.append(t[ctx[b]:])
        kv = torch.from_numpy(rng.standard_normal((2, n, H * (dqk + dv)))).float() * scale
        for p in range(held[b]):
            m = min(page, n - p * page)
            rows = slice(p * page, p * page + m)
            g = table[b, p]
            kc[g, :m] = kv[0, rows, : H * dqk].reshape(m, H, dqk).to(dtype)
            vc[g, :m] = kv[1, rows, : H * dv].reshape(m, H, dv).to(dtype)
            tsc[g, :m] = torch.from_numpy(t[rows])
    q = (torch.from_numpy(rng.standard_normal((T, H, dqk))).float() * scale).to(dtype)
    pos = torch.from_numpy(rng.standard_normal((H, num_pos)) * 0.5).float() if use_pos else None
    tb = torch.from_numpy(rng.standard_normal((H, num_buckets)) * 0.5).float() if use_time else None
    return Step(list(ctx), list(new), None if kind == "chain" else random_parents(kind, new, rng),
                q, kc, vc, tsc if use_time else None, table,
                np.concatenate(ts).astype(np.int64) if use_time and T else
                (np.zeros(0, np.int64) if use_time else None),
                pos, tb, max_seqlen or max(c + n for c, n in zip(ctx, new)), page)


def oracle(s: Step):
    """(out, A, E) in float64 [T, H, dv]: the definition; A = sum |p v| / N; E:
    what errors of the scores of (dqk + 4) roundings in 32 bits can do to out
    (|silu'| <= 1.1)."""
    H, dqk, dv = s.q.shape[1], s.q.shape[2], s.vc.shape[3]
    out = np.zeros((s.T, H, dv))
    A, E = np.zeros_like(out), np.zeros_like(out)
    off, page = s.off, s.page
    for b in range(len(s.ctx)):
        c, n = s.ctx[b], s.new[b]
        if n == 0:
            continue
        at = [(int(s.table[b, j // page]), j % page) for j in range(c + n)]
        g, r = [a[0] for a in at], [a[1] for a in at]
        K, V = s.kc[g, r].double().numpy(), s.vc[g, r].double().numpy()
        tk = s.tsc[g, r].numpy() if s.tsc is not None else None
        position = list(range(c + n))
        anc = []
        for i in range(n):
            par = i - 1 if s.parents is None else int(s.parents[off[b] + i])
            anc.append((anc[par] if par >= 0 else []) + [i])
            position[c + i] = c + len(anc[i]) - 1
        for i in range(n):
            t = int(off[b]) + i
            see = list(range(c)) + [c + m for m in sorted(anc[i])]
            Q = s.q[t].double().numpy()
            x = np.einsum("hd,jhd->jh", Q, K[see])
            e = np.einsum("hd,jhd->jh", np.abs(Q), np.abs(K[see]))
            if s.pos is not None:
                rel = [min(position[c + i] - position[j], s.pos.shape[1] - 1) for j in see]
                add = s.pos.double().numpy()[:, rel].T
                x, e = x + add, e + np.abs(add)
            if s.tb is not None:
                bk = [min(max(1, int(s.ts[t]) - int(tk[j])).bit_length() - 1, s.tb.shape[1] - 1)
                      for j in see]
                add = s.tb.double().numpy()[:, bk].T
                x, e = x + add, e + np.abs(add)
            with np.errstate(over="ignore", invalid="ignore"):
                p = x / (1 + np.exp(-x))
            out[t] = np.einsum("jh,jhd->hd", p, V[see]) / s.max_seqlen
            A[t] = np.einsum("jh,jhd->hd", np.abs(p), np.abs(V[see])) / s.max_seqlen
            E[t] = np.einsum("jh,jhd->hd", 1.1 * (dqk + 4) * 2 * U32 * e, np.abs(V[see])) / s.max_seqlen
    return out, A, E


def attn_tolerance(s: Step, want, A, E):
    """Element by element. fp32: the scores' errors (E), a few roundings of silu
    (exp, division, product: at most 8 half steps of p), a sum of at most n
    terms and the last rounding. bf16: the same, p rounded to bf16 (half a step
    of p) and the result rounded to bf16. Sums on tensor cores may cut off
    instead of rounding, hence two half steps a term."""
    n = max(c + m for c, m in zip(s.ctx, s.new))
    tol = E + (2 * n + 16) * U32 * A + 2 * U32 * np.abs(want) + 1e-30
    if s.q.dtype == torch.bfloat16:
        tol = tol + UBF * (A + E) + UBF * (np.abs(want) + UBF * A)
    return tol


def check_attn(s: Step, got, rows=None):
    want, A, E = oracle(s)
    tol = attn_tolerance(s, want, A, E)
    got = got.double().cpu().numpy()
    if rows is not None:
        got, want, tol = got[rows], want[rows], tol[rows]
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) - tol
    assert np.all(bad <= 0), "off by up to %.3g times the bound" % np.max(np.abs(got - want) / tol)


def call_attn(hstu, s: Step, **kw):
    """The call on a step's own arrays; what `kw` gives is used as it is (and
    nothing else is copied, so a call with every array given can be captured)."""
    def dev(x):
        return None if x is None else (x if torch.is_tensor(x) else torch.from_numpy(x)).cuda()
    arrays = dict(q=s.q, k_cache=s.kc, v_cache=s.vc, ts_cache=s.tsc, block_table=s.table,
                  ctx_lens=np.array(s.ctx, dtype=np.int32), new_offsets=s.off, timestamps=s.ts,
                  parents=s.parents, pos_bias=s.pos, time_bias=s.tb)
    args = {name: dev(x) for name, x in arrays.items() if name not in kw}
    args.update(max_seqlen=s.max_seqlen, max_new=max(max(s.new), 1))
    args.update(kw)
    return hstu.hstu_attn_cached_fwd(**args)


def plan_oracle(ctx, off, page, free, start, table):
    """(table, slots, free_end) by a plain loop over sequences and tokens."""
    table, slots, at = table.copy(), [], start
    for b in range(len(ctx)):
        n = int(off[b + 1] - off[b])
        have, end = -(-ctx[b] // page), -(-(ctx[b] + n) // page)
        for k in range(have, end):
            table[b, k] = free[at] if at < len(free) else -1
            at += 1
        for i in range(n):
            p = ctx[b] + i
            g = int(table[b, p // page])
            slots.append(g * page + p % page if g >= 0 else -1)
    return table, np.array(slots, dtype=np.int64), min(at, len(free))


def quant_w4_oracle(W, G):
    """codes [N, K/2] and scales [N, K/G] of float64 weights (exact bf16 values)."""
    N, K = W.shape
    W = W.reshape(N, K // G, G)
    amax = np.abs(W).max(2).astype(np.float32)
    scale = torch.from_numpy(amax / np.float32(7)).to(torch.bfloat16)
    sf = scale.double().numpy()
    zero = sf == 0
    sf = np.where(zero, 1.0, sf)
    q = np.rint((W.astype(np.float32) / sf[:, :, None].astype(np.float32)))
    c = (np.clip(q, -8, 7) + 8).astype(np.uint8)
    c[zero] = 8
    c = c.reshape(N, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), torch.from_numpy(sf).to(torch.bfloat16)


def w4_values(codes, scales, G):
    """float64 [N, K] weights that codes and scales stand for."""
    c = codes.astype(np.int64)
    W = np.empty((c.shape[0], c.shape[1] * 2))
    W[:, 0::2] = (c & 15) - 8
    W[:, 1::2] = (c >> 4) - 8
    return W * np.repeat(scales.double().numpy(), G, axis=1)
