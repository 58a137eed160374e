"""hstu_attn_cached_fwd where its kernels change over, at odd strides and over
random batches, against the definition in 64 bits."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from jagged_pointwise_attention_b200 import _native
from serving_util import attn_tolerance, call_attn, check_attn, make_step, oracle

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ok():
    assert hstu.hstu_device_status() == _native.HSTU_OK


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ctx,new,kind", [
    ([3000, 1, 77], [1, 1, 1], "chain"), ([3000, 1, 77], [8, 3, 1], "tree"),
    ([2900, 40], [9, 9], "tree"), ([2900, 40], [16, 2], "siblings"), ([2500, 0], [17, 40], "tree"),
    ([1800], [64], "tree"), ([1800, 9], [65, 3], "tree"), ([1500, 3], [128, 128], "siblings"),
    ([900, 60, 0], [200, 129, 256], "tree"), ([200], [700], "chain"), ([127, 128, 129], [130, 128, 1], "chain"),
    ([250, 255, 100], [5, 1, 8], "tree"), ([1000, 2, 300], [8, 8, 1], "chain"),
])
def test_kernels_change_over(ctx, new, kind, d):
    s = make_step(ctx, new, kind, 2, d, d, 32, BF, seed=d + len(new) + max(new))
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_many_short_sequences_and_the_same_ones_in_one_long_batch(d):
    """Enough items that sequences up to 1024 tokens are taken whole, and the
    same sequences with a longer bound, along the line."""
    rng = np.random.default_rng(d)
    ctx = [int(x) for x in rng.integers(0, 700, 160)]
    new = [int(x) for x in rng.integers(0, 5, 160)]
    s = make_step(ctx, new, "tree", 2, d, d, 16, BF, seed=d, max_seqlen=1024)
    a = call_attn(hstu, s)
    ok()
    check_attn(s, a)
    s.max_seqlen = 2048                  # 1 / N is half as large, exactly
    b = call_attn(hstu, s)
    ok()
    check_attn(s, b)


@pytest.mark.parametrize("d,n", [(32, 8), (32, 16), (32, 40), (64, 8), (64, 40), (64, 128), (128, 8),
                                 (128, 64), (128, 120)])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_values_that_a_query_does_not_see(d, n, long, kind):
    """NaN and infinities in keys and values of new tokens reach the queries that
    see them and no others; around tile and page borders, twice in one page."""
    s = make_step([1700 if long else 100, 30], [n, 3], kind, 2, d, d, 16, BF, seed=n + d)
    odd = {1: ("v", float("nan")), 2: ("v", float("inf")), n // 2: ("v", float("-inf")),
           n - 2: ("k", float("nan")), n - 3: ("v", float("inf"))}
    for i, (what, x) in odd.items():
        j = s.ctx[0] + i
        c = s.kc if what == "k" else s.vc
        c[int(s.table[0, j // 16]), j % 16, :, 3:9] = x
    got = call_attn(hstu, s)
    ok()
    want, _, _ = oracle(s)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(g), inf) and np.array_equal(g[inf], want[inf])
    # whole rows that see none of them
    par = s.parents if s.parents is not None else np.array([i - 1 for i in range(n)] + [-1, 0, 1])
    clean = []
    for i in range(n):
        p, hit = i, False
        while p >= 0:
            hit = hit or p in odd
            p = int(par[p])
        clean.append(not hit)
    check_attn(s, got, np.array(clean + [True] * 3))
    # the finite columns of the others: a value that is not finite leaves them alone
    fin = np.isfinite(want)
    rel = np.linalg.norm((g - want)[fin]) / np.linalg.norm(want[fin])
    assert rel <= 1e-2, rel


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 12, 70])
def test_page_stride_that_is_no_multiple_of_the_tokens(d, n):
    H, page = 2, 16
    s = make_step([600, 33], [n, 1], "tree", H, d, d, page, BF, seed=d + n)
    pages, row = s.kc.shape[0], H * d + 8
    store = torch.full((pages * (2 * page * row + 24),), float("nan"), dtype=BF).cuda()
    views = []
    for i, c in enumerate((s.kc, s.vc)):
        v = torch.as_strided(store, (pages, page, H, d), (2 * page * row + 24, row, d, 1), i * page * row + 8)
        v.copy_(c.cuda())
        views.append(v)
    got = call_attn(hstu, s, k_cache=views[0], v_cache=views[1])
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("n", [1, 20, 100])
def test_bad_pages_parents_and_sequences(n):
    """On the tcgen05 kernel: a bad page counts as no tokens, a bad parent as -1,
    a sequence that cannot be is left out, the others keep their bits."""
    s = make_step([1500, 700, 90], [n, n, 1], "tree", 2, 64, 64, 16, BF, seed=n)
    want = call_attn(hstu, s)
    ok()
    check_attn(s, want)
    tab = s.table.copy()
    tab[0, 3], tab[0, 20] = -1, 2 ** 30
    got = call_attn(hstu, s, block_table=torch.from_numpy(tab).cuda())
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    assert bool(torch.isfinite(got).all()) and torch.equal(got[2 * n:], want[2 * n:])
    out = torch.full_like(want, 3.0)
    call_attn(hstu, s, ctx_lens=torch.tensor([1500, 10 ** 9, 90], dtype=torch.int32).cuda(), out=out)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    assert bool((out[n: 2 * n] == 3.0).all())
    s.ctx, s.new = [1500, 90], [n, 1]
    keep = list(range(n)) + [2 * n]
    s.q, s.ts, s.parents, s.table = s.q[keep], s.ts[keep], s.parents[keep], s.table[[0, 2]]
    check_attn(s, out[keep])
    if n > 2:
        bad = s.parents.copy()
        bad[2] = 2
        s.parents[2] = -1
        got = call_attn(hstu, s, parents=torch.from_numpy(bad).cuda())
        assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
        check_attn(s, got)
    ok()


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 12))
    dtype = F32 if seed % 6 == 5 else BF
    d = int(rng.choice([32, 64, 128]))
    most = int(rng.choice([1, 3, 8, 16, 60, 130]))
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(1500), B)).astype(int) - 1]
    new = [int(x) for x in rng.integers(0, most + 1, B)]
    new[int(rng.integers(0, B))] = most
    s = make_step(ctx, new, str(rng.choice(["chain", "tree", "siblings", "path"])), int(rng.integers(1, 5)),
                  d, d, int(rng.choice([16, 32, 64, 128, 256])), dtype, num_pos=int(rng.choice([1, 50, 4000])),
                  num_buckets=int(rng.choice([3, 30, 128])), seed=seed, use_time=bool(rng.integers(0, 4)),
                  use_pos=bool(rng.integers(0, 4)), gap=float(rng.choice([0.4, 3600.0, 4e8])))
    a = call_attn(hstu, s)
    ok()
    check_attn(s, a)
    assert torch.equal(a, call_attn(hstu, s))


@pytest.mark.parametrize("d,most", [(32, 3), (64, 3), (64, 30), (128, 100)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_padded_batches_and_shared_pages(d, most, dtype):
    """Rows behind the last sequence and sequences without new tokens are
    padding: no error, slots of -1, rows left as they were. Two sequences share
    the pages of a common prefix."""
    page, pad = 16, 9
    s = make_step([700, 700, 0, 40], [most, 2, 0, 1], "tree", 2, d, d, page, dtype, seed=d + most)
    s.table[1, : 640 // page] = s.table[0, : 640 // page]       # a common prefix of 640 tokens
    T = s.T
    q = torch.cat([s.q, torch.full((pad, 2, d), float("nan"), dtype=dtype)]).cuda()
    ts = torch.from_numpy(np.concatenate([s.ts, np.zeros(pad, np.int64)])).cuda()
    par = torch.from_numpy(np.concatenate([s.parents, np.full(pad, 77, np.int32)])).cuda()
    out = torch.full((T + pad, 2, d), 4.0, dtype=dtype).cuda()
    got = call_attn(hstu, s, q=q, timestamps=ts, parents=par, out=out)
    ok()
    check_attn(s, got[:T])
    assert bool((out[T:] == 4.0).all())
    # the plan and the append of the same batch
    tab = torch.full((4, s.table.shape[1]), -1, dtype=torch.int32)
    for b, c in enumerate(s.ctx):
        tab[b, : -(-c // page)] = torch.from_numpy(s.table[b, : -(-c // page)])
    tab = tab.cuda()
    free = torch.arange(1000, 1100, dtype=torch.int32).cuda()
    slots, end = hstu.hstu_cache_plan(torch.tensor(s.ctx, dtype=torch.int32).cuda(),
                                      torch.from_numpy(s.off).cuda(), free,
                                      torch.zeros(1, dtype=torch.int32).cuda(), tab, page, T + pad)
    ok()
    assert bool((slots[T:] == -1).all()) and bool((slots[:T] >= 0).all())
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(s.ctx, s.new))
    assert end.item() == need
    kc, vc = (torch.zeros(1100, page, 2, d, dtype=dtype).cuda() for _ in range(2))
    ones = torch.ones_like(q)
    hstu.hstu_cache_append(ones, ones, None, slots, kc, vc, None)
    ok()
    assert kc.float().sum().item() == T * 2 * d == vc.float().sum().item()


@pytest.mark.parametrize("dtype,d,kind", [(BF, 32, "chain"), (BF, 64, "chain"), (BF, 128, "chain"),
                                          (torch.float32, 32, "chain"), (BF, 64, "tree")])
@pytest.mark.parametrize("ctx,new", [([100, 3], [5, 20]), ([900, 40], [6, 9])], ids=["short", "long"])
def test_max_new_above_what_a_sequence_can_bring(dtype, d, kind, ctx, new):
    """max_new is a bound: one above max_seqlen gives the bits that max_seqlen gives."""
    s = make_step(ctx, new, kind, 2, d, d, 16, dtype, seed=d, max_seqlen=max(ctx) + 30)
    N = s.max_seqlen
    for most in ((2 ** 31 - 1, 2 ** 31 - 9, N + 1) if kind == "chain" else (256,)):
        got = call_attn(hstu, s, max_new=most)
        ok()
        assert torch.equal(got, call_attn(hstu, s, max_new=min(most, N)))
        check_attn(s, got)


@pytest.mark.parametrize("dtype,d,kind", [(BF, 64, "tree"), (BF, 128, "chain"), (BF, 32, "tree"),
                                          (F32, 32, "chain")])
def test_thousands_of_sequences_along_the_line(dtype, d, kind):
    """Several sequences a thread in the search of the line; many without new
    tokens or without a context; a long one among them keeps all on the line."""
    rng = np.random.default_rng(d)
    ctx = [int(x) for x in rng.integers(0, 40, 5000)]
    new = [int(x) for x in rng.integers(0, 3, 5000)]
    ctx[3333], new[3333] = 1500, 5
    s = make_step(ctx, new, kind, 1, d, d, 16, dtype, seed=d)
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


def chain_oracle(s):
    """`oracle` for one sequence whose new tokens are a chain, all pairs at once."""
    c, n, H, N = s.ctx[0], s.new[0], s.q.shape[1], s.max_seqlen
    g = [int(s.table[0, j // s.page]) for j in range(c + n)]
    r = [j % s.page for j in range(c + n)]
    K, V = s.kc[g, r].double().numpy(), s.vc[g, r].double().numpy()
    Q, tk = s.q.double().numpy(), s.tsc[g, r].numpy()
    i, j = np.arange(c, c + n)[:, None], np.arange(c + n)[None, :]
    rel = np.clip(i - j, 0, s.pos.shape[1] - 1)
    dt = np.maximum(s.ts[:, None] - tk[None, :], 1)
    bucket = np.minimum(np.frexp(dt.astype(np.float64))[1] - 1, s.tb.shape[1] - 1)
    out, A, E = (np.zeros((n, H, V.shape[2])) for _ in range(3))
    for h in range(H):
        x, e = Q[:, h] @ K[:, h].T, np.abs(Q[:, h]) @ np.abs(K[:, h]).T
        for add in (s.pos.double().numpy()[h][rel], s.tb.double().numpy()[h][bucket]):
            x, e = x + add, e + np.abs(add)
        p = np.where(j <= i, x / (1 + np.exp(-x)), 0.0)
        e = np.where(j <= i, 1.1 * (Q.shape[2] + 4) * 2 * 2.0 ** -24 * e, 0.0)
        a = np.abs(V[:, h])
        out[:, h], A[:, h], E[:, h] = p @ V[:, h] / N, np.abs(p) @ a / N, e @ a / N
    return out, A, E


@pytest.mark.parametrize("dtype,d,H", [(BF, 64, 2), (BF, 128, 1), (BF, 32, 1), (F32, 64, 1)])
@pytest.mark.parametrize("ctx,new", [(700, 2311), (0, 3001)])
def test_thousands_of_new_tokens_in_a_row(dtype, d, H, ctx, new):
    """A piece of a prompt, and a whole one. (Time differences below 2^53, so frexp
    is exact.)"""
    s = make_step([ctx], [new], "chain", H, d, d, 64, dtype, seed=d + new)
    got = call_attn(hstu, s).double().cpu().numpy()
    ok()
    want, A, E = chain_oracle(s)
    few = make_step([50], [9], "chain", H, d, d, 16, dtype, seed=1)
    assert all(np.allclose(x, y, rtol=1e-12, atol=1e-15) for x, y in zip(chain_oracle(few), oracle(few)))
    tol = attn_tolerance(s, want, A, E)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol), \
        "off by up to %.3g times the bound" % np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("dtype,d", [(BF, 32), (BF, 64), (BF, 128), (F32, 32)])
@pytest.mark.parametrize("ctx", [[50, 40, 30], [1500, 1100, 300]], ids=["short", "long"])
@pytest.mark.parametrize("off", [[2, 12, 18, 26], [0, 10, 4, 12], [0, 10, 10, 40], [-3, 7, 13, 21]],
                         ids=["begin", "fall", "end", "negative"])
def test_offsets_that_cannot_be(dtype, d, ctx, off):
    """Reported; rows that no sequence names stay as they were, rows that one
    possible sequence names alone are its own."""
    s = make_step(ctx, [10, 6, 8], "chain", 2, d, d, 16, dtype, seed=d + ctx[0])
    T = 28
    q, ts = torch.zeros(T, 2, d, dtype=dtype), np.full(T, 1_800_000_000, dtype=np.int64)
    first = max(off[0], 0)
    q[first: first + s.T], ts[first: first + s.T] = s.q, s.ts
    out = torch.full((T, 2, d), 7.0, dtype=dtype).cuda()
    call_attn(hstu, s, q=q.cuda(), timestamps=torch.from_numpy(ts).cuda(), max_new=10,
              new_offsets=torch.tensor(off).cuda(), out=out)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    named = np.zeros(T, dtype=bool)
    for b in range(3):
        named[max(off[b], 0): max(off[b + 1], 0)] = True
    assert bool((out.cpu()[torch.from_numpy(~named)] == 7.0).all())
    if off[0] == 0:             # sequence 0's first rows, before any other's
        check_attn(s, out[: s.T], rows=slice(0, 4))
