"""hstu_cache_plan and hstu_cache_append against plain loops; a run of plan,
append and attention over several steps."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from jagged_pointwise_attention_b200 import _native
from serving_util import Step, check_attn, plan_oracle

pytestmark = pytest.mark.gpu


def ok():
    assert hstu.hstu_device_status() == _native.HSTU_OK


def run_plan(ctx, new, page, free, start, table, **kw):
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    t = torch.from_numpy(table.copy()).cuda()
    slots, end = hstu.hstu_cache_plan(
        torch.tensor(ctx, dtype=torch.int32).cuda(), torch.from_numpy(off).cuda(),
        torch.from_numpy(free).cuda(), torch.tensor([start], dtype=torch.int32).cuda(), t, page,
        int(off[-1]), **kw)
    return t, slots, end, off


PLANS = [
    ([0], [1], 16), ([16], [1], 16), ([15], [1], 16), ([5], [0], 16), ([0, 0, 0], [0, 0, 0], 32),
    ([31, 32, 33, 0], [1, 0, 95, 64], 32), ([0], [5000], 64), ([100] * 7, [1] * 7, 1024),
    (list(range(300)), [i % 5 for i in range(300)], 16),
    ([i % 50 for i in range(2048)], [1 + i % 3 for i in range(2048)], 16),
    ([0] * 5 + [1000] * 3, [700, 0, 0, 3000, 1, 40, 0, 2], 128),
    ([7] * 100000, [1] * 100000, 16),
]


@pytest.mark.parametrize("ctx,new,page", PLANS, ids=lambda x: str(len(x)) if isinstance(x, list) else str(x))
def test_plan(ctx, new, page):
    rng = np.random.default_rng(len(ctx) + page)
    B = len(ctx)
    have = [-(-c // page) for c in ctx]
    width = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 2
    need = sum(-(-(c + n) // page) - h for c, n, h in zip(ctx, new, have))
    pool = rng.permutation(sum(have) + need + 20).astype(np.int32)
    table = np.full((B, width), -99, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, : have[b]] = pool[at: at + have[b]]
        at += have[b]
    free = np.concatenate([pool[-11:], pool[at:-11]])
    t, slots, end, off = run_plan(ctx, new, page, free, 11, table)
    ok()
    wt, ws, we = plan_oracle(ctx, off, page, free, 11, table)
    assert np.array_equal(t.cpu().numpy(), wt)
    assert np.array_equal(slots.cpu().numpy(), ws)
    assert end.item() == we


def test_plan_short_list_and_impossible_sequences():
    page, table = 16, np.full((4, 4), -99, dtype=np.int32)
    table[1, 0] = 3
    ctx, new = [0, 10, 0, 0], [20, 30, 16, 5]
    free = np.array([7, 5, 9], dtype=np.int32)                 # six are wanted
    t, slots, end, off = run_plan(ctx, new, page, free, 0, table)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    wt, ws, we = plan_oracle(ctx, off, page, free, 0, table)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(slots.cpu().numpy(), ws)
    assert end.item() == we == 3 and (ws == -1).sum() > 0
    # a sequence longer than its table row, and a negative context: no pages, slots -1
    free = np.arange(50, 80, dtype=np.int32)
    t, slots, end, off = run_plan([0, -4, 10, 0], [20, 3, 55, 5], page, free, 2, table)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    s = slots.cpu().numpy()
    assert (s[20:78] == -1).all() and (s[:20] >= 0).all() and (s[78:] >= 0).all()
    assert t.cpu().numpy()[0, :2].tolist() == [52, 53] and t[3, 0].item() == 54
    assert end.item() == 5
    # a start outside the list
    for start in (-1, 31):
        run_plan([0], [20], page, free, start, table[:1])
        assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    # an existing page that is none
    t, slots, _, _ = run_plan([3], [1], page, free, 0, np.full((1, 2), -1, dtype=np.int32))
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT and slots.item() == -1
    ok()


def test_plan_wider_rows_and_given_outputs():
    page = 16
    wide = torch.full((3, 9), -5, dtype=torch.int32).cuda()
    tab = wide[:, 2:6]
    slots = torch.full((7,), 99, dtype=torch.int64).cuda()
    end = torch.zeros(1, dtype=torch.int32).cuda()
    got = hstu.hstu_cache_plan(torch.zeros(3, dtype=torch.int32).cuda(),
                               torch.tensor([0, 3, 3, 7]).cuda(),
                               torch.arange(30, 40, dtype=torch.int32).cuda(),
                               torch.zeros(1, dtype=torch.int32).cuda(), tab, page, 7, slots=slots,
                               free_end=end)
    ok()
    assert got[0] is slots and got[1] is end
    assert wide.cpu().tolist() == [[-5, -5, 30] + [-5] * 6, [-5] * 9, [-5, -5, 31] + [-5] * 6]
    assert slots.cpu().tolist() == [480, 481, 482, 496, 497, 498, 499] and end.item() == 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,H,dqk,dv,page", [(1, 1, 64, 64, 16), (129, 2, 64, 64, 16),
                                             (1000, 4, 128, 128, 64), (37, 3, 5, 7, 32),
                                             (50, 1, 2, 33, 16), (4000, 1, 32, 32, 1024)])
def test_append(dtype, T, H, dqk, dv, page):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // page) + 3
    k, v = (torch.randn(T, H, d, generator=g).to(dtype) for d in (dqk, dv))
    kc, vc = (torch.randn(pages, page, H, d, generator=g).to(dtype) for d in (dqk, dv))
    tsc = torch.zeros(pages, page, dtype=torch.int64)
    ts = torch.randint(0, 2 ** 62, (T,), generator=g)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 3:
        slots[2] = -1                                          # padding
    dev = [x.cuda() for x in (k, v, ts, slots, kc, vc, tsc)]
    hstu.hstu_cache_append(*dev)
    ok()
    live = slots >= 0
    for c, x in ((kc, k), (vc, v)):
        c.view(pages * page, H, -1)[slots[live]] = x[live]
    tsc.view(-1)[slots[live]] = ts[live]
    assert torch.equal(dev[4].cpu(), kc) and torch.equal(dev[5].cpu(), vc)
    assert torch.equal(dev[6].cpu(), tsc)


@pytest.mark.parametrize("dtype,step", [(torch.bfloat16, 8), (torch.bfloat16, 2), (torch.bfloat16, 1),
                                        (torch.float32, 4), (torch.float32, 1)])
def test_append_strided_and_unaligned(dtype, step):
    """Rows of a wider projection, pages of one allocation, without timestamps;
    `step` elements of offset: 16, 4 or 2 byte alignment."""
    T, H, d, page, pages = 70, 2, 32, 16, 7
    g = torch.Generator().manual_seed(step)
    base = torch.randn(T, 3 * H * d + 2 * step, generator=g).to(dtype).cuda()
    k = base[:, step: step + H * d].view(T, H, d)
    v = base[:, step + H * d: step + 2 * H * d].view(T, H, d)
    store = torch.zeros(pages, 2, page, H * d + step, dtype=dtype).cuda()
    kc = store[:, 0, :, :H * d].view(pages, page, H, d)
    vc = store[:, 1, :, :H * d].view(pages, page, H, d)
    slots = torch.randperm(pages * page, generator=g)[:T].cuda()
    want = store.clone()
    for i, x in ((0, k), (1, v)):
        for t in range(T):
            s = int(slots[t])
            want[s // page, i, s % page, : H * d] = x[t].reshape(-1)
    hstu.hstu_cache_append(k, v, None, slots, kc, vc, None)
    ok()
    assert torch.equal(store, want)


def test_append_slot_past_the_cache_is_skipped():
    z = torch.ones(3, 1, 64, dtype=torch.bfloat16).cuda()
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16).cuda() for _ in range(2))
    hstu.hstu_cache_append(z, z, None, torch.tensor([5, 32, 2 ** 60]).cuda(), kc, vc, None)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    assert kc.float().sum().item() == 64 and vc.float().sum().item() == 64
    hstu.hstu_cache_append(z[:0], z[:0], None, torch.empty(0, dtype=torch.int64).cuda(), kc, vc, None)
    ok()


@pytest.mark.parametrize("dtype,H,d,page", [(torch.bfloat16, 2, 64, 16), (torch.bfloat16, 2, 128, 64),
                                            (torch.float32, 2, 32, 16)])
def test_steps_together(dtype, H, d, page):
    """A prompt, single tokens, a drafted tree of which a path is kept, another
    token: plan, append and attention, no host copy of lengths in between
    other than what the caller counts itself. Every step against the
    definition over the tokens a plain list holds."""
    rng = np.random.default_rng(21)
    B, pages, maxp, N = 3, 64, 20, 300
    kc, vc = (torch.full((pages, page, H, d), float("nan"), dtype=dtype).cuda() for _ in range(2))
    tsc = torch.zeros(pages, page, dtype=torch.int64).cuda()
    table = torch.full((B, maxp), -1, dtype=torch.int32).cuda()
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    taken = torch.zeros(1, dtype=torch.int32).cuda()
    pos = torch.from_numpy(rng.standard_normal((H, 64)) * 0.5).float()
    tb = torch.from_numpy(rng.standard_normal((H, 128)) * 0.5).float()
    ctx = [0] * B
    clock = 1_700_000_000

    def rows(n):
        return torch.from_numpy(rng.standard_normal((n, H, d))).float().to(dtype)

    for new, kind in (([40, 0, 17], "chain"), ([1, 30, 1], "chain"), ([1, 1, 1], "chain"),
                      ([12, 9, 20], "tree"), ([1, 1, 1], "chain"), ([5, 5, 0], "siblings")):
        T = sum(new)
        q, k, v = rows(T), rows(T), rows(T)
        ts = clock + np.sort(rng.integers(0, 10 ** 5, T)).astype(np.int64)
        clock = int(ts.max()) + 1
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        parents = None
        if kind == "siblings":
            parents = np.full(T, -1, dtype=np.int32)
        elif kind == "tree":
            parents = np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(n)]
                                      for n in new]).astype(np.int32)
        ctx_d = torch.tensor(ctx, dtype=torch.int32).cuda()
        off_d = torch.from_numpy(off).cuda()
        slots, taken = hstu.hstu_cache_plan(ctx_d, off_d, free, taken, table, page, T)
        kd, vd, td = k.cuda(), v.cuda(), torch.from_numpy(ts).cuda()
        hstu.hstu_cache_append(kd, vd, td, slots, kc, vc, tsc)
        got = hstu.hstu_attn_cached_fwd(
            q.cuda(), kc, vc, tsc, table, ctx_d, off_d, td,
            None if parents is None else torch.from_numpy(parents).cuda(), pos.cuda(), tb.cuda(), N,
            max(new))
        ok()
        s = Step(list(ctx), list(new), parents, q, kc.cpu(), vc.cpu(), tsc.cpu(),
                 table.cpu().numpy(), ts, pos, tb, N, page)
        check_attn(s, got)
        if kind == "tree":
            # keep the path to the last token: its rows go to the first slots
            keep, lens = [], []
            for b in range(B):
                path, p = [], new[b] - 1
                while p >= 0:
                    path.append(p)
                    p = int(parents[off[b] + p])
                path.reverse()
                keep += [int(off[b]) + i for i in path]
                lens.append(len(path))
            at = [int(off[b]) + i for b in range(B) for i in range(lens[b])]
            kd, vd, td = kd[keep], vd[keep], td[keep]
            hstu.hstu_cache_append(kd, vd, td, slots[at], kc, vc, tsc)
            ctx = [c + n for c, n in zip(ctx, lens)]
            # pages beyond the kept tokens stay in the table: the plan takes new ones
            table[:, :] = torch.where(
                torch.arange(maxp).cuda()[None, :] < torch.tensor([-(-c // page) for c in ctx]).cuda()[:, None],
                table, -1)
        elif kind == "chain":
            ctx = [c + n for c, n in zip(ctx, new)]
    ok()


def plan_any_offsets(ctx, off, total, page, free, start, table):
    """(table, slots, free_end, possible) for any offsets: a sequence is possible
    when its lengths are not negative, its offsets lie in [0, total], begin at 0
    for the first, and no earlier offset is greater than its own."""
    table, slots, at, possible = table.copy(), np.full(total, -1, dtype=np.int64), start, []
    top = np.maximum.accumulate(off)
    for b in range(len(ctx)):
        o, e = int(off[b]), int(off[b + 1])
        fits = (ctx[b] >= 0 and 0 <= o <= e <= total and o >= top[b] and (b > 0 or o == 0)
                and -(-(ctx[b] + e - o) // page) <= table.shape[1])
        possible.append(bool(fits))
        if not fits:
            continue
        have, end = -(-ctx[b] // page), -(-(ctx[b] + e - o) // page)
        for k in range(have, end):
            table[b, k] = free[at] if at < len(free) else -1
            at += 1
        for i in range(e - o):
            g = int(table[b, (ctx[b] + i) // page])
            slots[o + i] = g * page + (ctx[b] + i) % page if g >= 0 else -1
    return table, slots, min(at, len(free)), possible


def fallen_offsets(B, T, falls, seed):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.sort(rng.integers(0, T + 1, B - 1)), [T]]).astype(np.int64)
    for b in rng.choice(np.arange(1, B), falls, replace=False):
        off[b] = rng.integers(-3, T + 4)
    return off


BAD_OFFSETS = [
    ([3, 8, 10], 10), ([-2, 3, 10], 10), ([0, -3, 5, 9], 9), ([0, 10, 4, 12, 20], 20),
    ([0, 4, 50, 12, 20], 20), ([7, 7], 7), ([5, 2], 6), ([0, 700, 300, 5000], 6000),
    ([9, 700, 4000], 4500),
    (fallen_offsets(290, 900, 5, 1), 900), (fallen_offsets(2500, 9000, 9, 2), 9000),
    (fallen_offsets(80000, 100000, 40, 3), 100000),
]


@pytest.mark.parametrize("off,total", BAD_OFFSETS, ids=[str(i) for i in range(len(BAD_OFFSETS))])
def test_plan_offsets_that_cannot_be(off, total):
    """Offsets that do not begin at 0, fall, or lie outside the rows: no row keeps
    what it held, none belongs to two sequences, the same result every time."""
    off, page = np.asarray(off, dtype=np.int64), 16
    B = len(off) - 1
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 40, B).astype(np.int32)
    have = -(-ctx // page)
    width = min(int((ctx.max() + np.abs(np.diff(off)).max()) // page + 2), 64)
    table = np.full((B, width), -99, dtype=np.int32)
    pool = rng.permutation(int(have.sum()) + B + total + 20).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(have)])
    for b in range(B):
        table[b, : have[b]] = pool[at[b]: at[b + 1]]
    free = pool[at[B]:]
    wt, ws, we, possible = plan_any_offsets(ctx.tolist(), off, total, page, free, 2, table)
    assert not all(possible)
    for _ in range(3):
        t = torch.from_numpy(table).cuda()
        slots = torch.arange(total).cuda()                      # numbers that would do as slots
        _, end = hstu.hstu_cache_plan(
            torch.from_numpy(ctx).cuda(), torch.from_numpy(off).cuda(), torch.from_numpy(free).cuda(),
            torch.tensor([2], dtype=torch.int32).cuda(), t, page, total, slots=slots)
        assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
        assert np.array_equal(slots.cpu().numpy(), ws)
        assert np.array_equal(t.cpu().numpy(), wt)
        assert end.item() == we
