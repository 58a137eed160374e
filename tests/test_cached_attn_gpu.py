"""hstu_attn_cached_fwd: new tokens (chains, trees, candidates) over a paged
cache, against the definition in 64 bits; its edge cases and its refusals on
the device. Tolerances are derived in serving_util.attn_tolerance."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from jagged_pointwise_attention_b200 import _native
from serving_util import call_attn, check_attn, make_step, oracle

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ok():
    st = hstu.hstu_device_status()
    assert st == _native.HSTU_OK, "device status %d" % st


CASES = [
    # ctx, new, kind, H, d, page
    ([0], [1], "chain", 1, 64, 16),                              # one token, no context
    ([5], [1], "chain", 2, 64, 16),
    ([0, 7, 0, 130], [3, 0, 1, 2], "chain", 2, 64, 16),          # a sequence without new tokens
    ([127, 128, 129, 1], [1, 1, 1, 1], "chain", 3, 128, 32),     # around a 128-key tile
    ([15, 16, 17], [17, 16, 15], "chain", 1, 32, 16),            # around a page
    ([63, 64, 65], [9, 8, 7], "chain", 4, 32, 64),
    ([300, 40, 0], [64, 33, 5], "tree", 2, 64, 16),
    ([250, 3], [65, 128], "tree", 2, 128, 128),
    ([100], [256], "tree", 1, 64, 32),                           # the largest tree
    ([100], [200], "path", 1, 64, 32),
    ([513, 0, 31], [100, 17, 1], "siblings", 2, 128, 64),
    ([70, 1000], [140, 31], "chain", 2, 128, 16),                # more than one query tile
    ([0], [300], "chain", 2, 64, 256),                           # a prompt
    ([2000, 10], [4, 2], "chain", 1, 128, 1024),                 # large pages
    ([9] * 40, [1, 2, 3, 4] * 10, "tree", 2, 64, 16),            # many short sequences
    ([3000], [16], "tree", 2, 64, 16),                           # one item over many blocks
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, (len(c[0]), max(c[0]), max(c[1]), c[2], c[3], c[4], c[5]))))
def test_against_definition(case, dtype):
    ctx, new, kind, H, d, page = case
    s = make_step(ctx, new, kind, H, d, d, page, dtype, seed=len(ctx) * 100 + max(ctx) + page)
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("pos,time,buckets,num_pos", [(True, False, 128, 1), (False, True, 1, 64),
                                                      (False, False, 128, 64), (True, True, 7, 4096),
                                                      (True, True, 1000, 3)])
def test_bias_terms(dtype, pos, time, buckets, num_pos):
    s = make_step([200, 40], [20, 7], "tree", 2, 64, 64, 16, dtype, num_pos=num_pos,
                  num_buckets=buckets, use_pos=pos, use_time=time, seed=3)
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_timestamps_far_apart_equal_and_backwards(dtype):
    """Differences beyond 32 bits, zero, negative (bucket 0) and at powers of two."""
    s = make_step([150, 20], [12, 5], "tree", 2, 64, 64, 16, dtype, seed=4)
    rng = np.random.default_rng(4)
    flat = s.tsc.view(-1)
    far = torch.from_numpy(rng.choice(np.array([0, 1, 2, 3, 4, 2 ** 31, 2 ** 32, 2 ** 33 - 1, 2 ** 40,
                                                -5, 1023, 1024, 2 ** 30 - 1, 2 ** 30]), flat.numel()))
    s.tsc = (2 ** 41 - far).view_as(s.tsc)
    s.ts = np.full(s.T, 2 ** 41, dtype=np.int64)
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("dqk,dv", [(5, 7), (32, 16), (33, 128), (128, 1), (100, 100), (4, 64)])
def test_f32_head_dimensions(dqk, dv):
    s = make_step([70, 3, 0], [9, 1, 20], "tree", 3, dqk, dv, 16, F32, seed=dqk)
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_strided_views(dtype):
    """q and out inside wider rows, k and v pages of one allocation, a wider table."""
    H, d, page = 2, 64, 16
    s = make_step([50, 7, 200], [5, 1, 40], "tree", H, d, d, page, dtype, seed=6)
    T, pages = s.T, s.kc.shape[0]
    row = torch.full((T, 4 * H * d), 7.0, dtype=dtype).cuda()
    q = row[:, H * d: 2 * H * d].view(T, H, d)
    q.copy_(s.q)
    both = torch.full((pages, 2, page, H, d + 0), float("nan"), dtype=dtype).cuda()
    both[:, 0].copy_(s.kc)
    both[:, 1].copy_(s.vc)
    tab = torch.full((3, s.table.shape[1] + 5), -7, dtype=torch.int32).cuda()
    tab[:, : s.table.shape[1]] = torch.from_numpy(s.table).cuda()
    tsw = torch.zeros((pages, 3 * page), dtype=torch.int64).cuda()
    tsw[:, :page] = s.tsc.cuda()
    out = row[:, 2 * H * d: 3 * H * d].view(T, H, d)
    before = row.clone()
    got = call_attn(hstu, s, q=q, k_cache=both[:, 0], v_cache=both[:, 1],
                    block_table=tab[:, : s.table.shape[1]], ts_cache=tsw[:, :page], out=out)
    ok()
    check_attn(s, got)
    row[:, 2 * H * d: 3 * H * d] = before[:, 2 * H * d: 3 * H * d]
    assert torch.equal(row, before)             # nothing else was written


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,n", [(64, 24), (128, 100)])
def test_values_that_a_query_does_not_see(dtype, d, n):
    """NaN and infinities in the keys and values of drafted tokens reach the
    tokens that see them and no others (the cache outside the sequences is NaN
    in every test)."""
    s = make_step([140, 30], [n, 5], "tree", 2, d, d, 16, dtype, seed=8)
    par = s.parents
    bad = {3: ("v", float("nan")), 7: ("v", float("inf")), 11: ("k", float("nan")),
           13: ("v", float("-inf"))}
    for i, (what, x) in bad.items():
        j = s.ctx[0] + i
        (s.kc if what == "k" else s.vc)[int(s.table[0, j // 16]), j % 16] = x
    sees = []
    for i in range(n):
        p, hit = i, False
        while p >= 0:
            hit = hit or p in bad
            p = int(par[p])
        sees.append(hit)
    rows = np.array([not h for h in sees] + [True] * 5)
    assert rows.sum() > 5 and (~rows).sum() >= 4
    got = call_attn(hstu, s)
    ok()
    check_attn(s, got, rows)
    want, _, _ = oracle(s)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    assert np.array_equal(g[np.isinf(g)], want[np.isinf(want)])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_chain_gives_the_rows_of_the_whole_sequence(dtype):
    """The rows of the last tokens, out of the cache and by hstu_attn_fwd: both
    within the bound of the same definition."""
    s = make_step([400, 90], [33, 12], "chain", 2, 64, 64, 32, dtype, seed=9)
    got = call_attn(hstu, s).double().cpu().numpy()
    ks, vs, ts, qs, offs, rows = [], [], [], [], [0], []
    for b in range(2):
        n = s.ctx[b] + s.new[b]
        at = ([int(s.table[b, j // 32]) for j in range(n)], [j % 32 for j in range(n)])
        ks.append(s.kc[at])
        vs.append(s.vc[at])
        ts.append(s.tsc[at])
        qb = torch.zeros((n, 2, 64), dtype=dtype)
        qb[s.ctx[b]:] = s.q[s.off[b]: s.off[b + 1]]
        qs.append(qb)
        rows += list(range(offs[-1] + s.ctx[b], offs[-1] + n))
        offs.append(offs[-1] + n)
    whole = hstu.hstu_attn_fwd(torch.cat(qs).cuda(), torch.cat(ks).cuda(), torch.cat(vs).cuda(),
                               torch.tensor(offs).cuda(), torch.cat(ts).cuda(), s.pos.cuda(),
                               s.tb.cuda(), s.max_seqlen)
    ok()
    whole = whole.double().cpu().numpy()[rows]
    rel = np.linalg.norm(got - whole) / np.linalg.norm(whole)
    # hstu_attn_fwd's own bar is 1e-2 (bf16) and 1e-4 (fp32) of the definition
    assert rel <= (1e-2 if dtype == BF else 1e-4), rel


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_same_bits_again_and_workspace_contents_do_not_matter(dtype):
    s = make_step([3000, 5, 700], [7, 3, 30], "tree", 4, 64, 64, 16, dtype, seed=10)
    n = hstu.hstu_attn_cached_workspace_bytes(dtype, 30, 64)
    a = call_attn(hstu, s, workspace=torch.full((n // 4,), float("nan")).cuda())
    b = call_attn(hstu, s, workspace=torch.full((n // 4,), -1e30).cuda())
    c = call_attn(hstu, s)
    ok()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_behind_the_last_sequence_and_left_out_sequences(dtype):
    """Sequences that cannot be are reported and left out; the rows of the others
    are right and the rest of `out` stays."""
    s = make_step([20, 30, 40, 50], [2, 3, 2, 2], "chain", 2, 64, 64, 16, dtype, seed=11)
    want = call_attn(hstu, s)
    ok()
    ctx = torch.tensor([20, -1, 40, 10 ** 6], dtype=torch.int32).cuda()
    out = torch.full((s.T, 2, 64), 5.0, dtype=dtype).cuda()
    call_attn(hstu, s, ctx_lens=ctx, out=out)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    for b, rows in enumerate(([0, 1], [2, 3, 4], [5, 6], [7, 8])):
        if b in (0, 2):
            assert torch.equal(out[rows], want[rows])
        else:
            assert bool((out[rows] == 5.0).all())
    # more new tokens than max_new says
    call_attn(hstu, s, max_new=2)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    # longer than max_seqlen
    call_attn(hstu, s, max_seqlen=40)
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    ok()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("page_number", [-1, 2 ** 30, -2 ** 31])
def test_pages_outside_the_cache_count_as_no_tokens(dtype, page_number):
    s = make_step([100, 64], [3, 2], "chain", 2, 64, 64, 16, dtype, seed=12)
    want = call_attn(hstu, s)
    ok()
    tab = s.table.copy()
    tab[0, 2] = page_number
    got = call_attn(hstu, s, block_table=torch.from_numpy(tab).cuda())
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    assert torch.equal(got[3:], want[3:]) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_parents_that_are_not_before_their_token(dtype):
    s = make_step([100, 20], [6, 4], "tree", 2, 64, 64, 16, dtype, seed=13)
    s.parents[:] = [-1, 0, 1, 2, 3, 4, -1, 0, 0, 2]
    bad = s.parents.copy()
    bad[2], bad[4], bad[9] = 2, 9, -3
    s.parents[[2, 4, 9]] = -1                       # what they count as
    got = call_attn(hstu, s, parents=torch.from_numpy(bad).cuda())
    assert hstu.hstu_device_status() == _native.HSTU_ERR_BAD_INPUT
    check_attn(s, got)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_empty_steps(dtype):
    s = make_step([10, 3], [2, 1], "chain", 2, 64, 64, 16, dtype, seed=14)
    none = torch.empty((0, 2, 64), dtype=dtype).cuda()
    off = torch.zeros(3, dtype=torch.int64).cuda()
    got = call_attn(hstu, s, q=none, new_offsets=off, timestamps=torch.empty(0, dtype=torch.int64).cuda())
    assert got.shape == (0, 2, 64)
    ok()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_captured_replayed_and_on_another_stream(dtype):
    """One graph, replayed after the inputs changed in place; an eager call on a
    stream of its own between; a second graph with a workspace of its own."""
    a = make_step([300, 20, 64], [5, 9, 1], "tree", 2, 64, 64, 16, dtype, seed=15)
    b = make_step([300, 20, 64], [5, 9, 1], "tree", 2, 64, 64, 16, dtype, seed=16)
    dev = dict(q=a.q.cuda(), k_cache=a.kc.cuda(), v_cache=a.vc.cuda(), ts_cache=a.tsc.cuda(),
               block_table=torch.from_numpy(a.table).cuda(),
               timestamps=torch.from_numpy(a.ts).cuda(), parents=torch.from_numpy(a.parents).cuda(),
               pos_bias=a.pos.cuda(), time_bias=a.tb.cuda(),
               ctx_lens=torch.tensor(a.ctx, dtype=torch.int32).cuda(),
               new_offsets=torch.from_numpy(a.off).cuda())
    n = hstu.hstu_attn_cached_workspace_bytes(dtype, 9, 64)
    ws = [torch.empty(n, dtype=torch.uint8).cuda() for _ in range(2)]
    outs = [torch.empty((15, 2, 64), dtype=dtype).cuda() for _ in range(2)]
    call_attn(hstu, a, **dev, workspace=ws[0], out=outs[0])
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call_attn(hstu, a, **dev, workspace=ws[i], out=outs[i])
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    check_attn(a, outs[0])
    assert torch.equal(outs[0], outs[1])
    for k, v in (("q", b.q), ("k_cache", b.kc), ("v_cache", b.vc), ("ts_cache", b.tsc),
                 ("pos_bias", b.pos), ("time_bias", b.tb)):
        dev[k].copy_(v)
    for k, v in (("block_table", b.table), ("timestamps", b.ts), ("parents", b.parents)):
        dev[k].copy_(torch.from_numpy(v))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs[0].replay()
    got = call_attn(hstu, b, **dev, stream=side)
    graphs[1].replay()
    torch.cuda.synchronize()
    ok()
    check_attn(b, outs[0])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], got)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_offsets_beyond_32_bits(dtype):
    """A cache of more than 2^32 elements whose last pages are in use."""
    H, d, page = 4, 128, 64
    pages = 2 ** 32 // (page * H * d) + 40
    s = make_step([130, 20], [3, 1], "chain", H, d, d, page, dtype, seed=17, spare=0)
    small = s.kc.shape[0]
    kc = torch.zeros((pages, page, H, d), dtype=dtype, device="cuda")
    vc = torch.zeros((pages, page, H, d), dtype=dtype, device="cuda")
    ts = torch.zeros((pages, page), dtype=torch.int64, device="cuda")
    kc[-small:], vc[-small:], ts[-small:] = s.kc.cuda(), s.vc.cuda(), s.tsc.cuda()
    tab = s.table.copy()
    for b in range(2):
        m = -(-(s.ctx[b] + s.new[b]) // page)
        tab[b, :m] += pages - small
    got = call_attn(hstu, s, k_cache=kc, v_cache=vc, ts_cache=ts,
                    block_table=torch.from_numpy(tab).cuda())
    ok()
    check_attn(s, got)
