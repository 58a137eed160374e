"""hstu_layer_step_fwd: the layer on new tokens over a paged cache, against the
64-bit oracle of the layer on whole sequences; its refusals (CPU)."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
import oracle
from gen import make_layer_inputs, round_to_bf16
from gpu_util import assert_bf16_close, dev
from jagged_pointwise_attention_b200 import _native
from jagged_pointwise_attention_b200.build import build
from serving_util import quant_w4_oracle, w4_values

BF = torch.bfloat16
INV, UNS, OK = _native.HSTU_ERR_INVALID_ARG, _native.HSTU_ERR_UNSUPPORTED, _native.HSTU_OK


def test_refusals():
    build()
    lib = _native.load()

    def call(x=16, T=4, D=512, W1=16, s1=16, W2=16, s2=16, group=0, norm=0, kc=16, tsc=16, slots=16, B=2,
             max_new=2, H=4, d=128, ts=16, out=16, ws=16, wsb=1 << 30):
        row = H * d
        return lib.hstu_layer_step_fwd(x, T, D, W1, s1, None, W2, s2, None, group, None, None, 1e-5, norm,
                                       None, None, kc, 16 * row, row, 16, 16 * row, row, tsc, 16, 4, 16,
                                       16, 8, 8, 16, 16, B, slots, max_new, H, d, ts, None, None, 0, None,
                                       0, 64, out, ws, wsb, None)
    for kw in (dict(x=None), dict(W1=None), dict(W2=None), dict(out=None), dict(slots=None),
               dict(ws=None), dict(ws=24), dict(wsb=1000), dict(T=-1), dict(D=0), dict(H=0), dict(B=-1),
               dict(max_new=0), dict(ts=None), dict(tsc=None), dict(group=64, s1=None),
               dict(group=64, s2=None)):
        assert call(**kw) == INV, kw
    for kw in (dict(D=500), dict(d=32), dict(d=96), dict(H=3, d=64), dict(H=32), dict(group=16),
               dict(D=640, norm=1), dict(H=70000)):
        assert call(**kw) == UNS, kw
    assert call(T=0) == OK and call(B=0) == OK
    size = lib.hstu_layer_step_workspace_bytes
    assert size(4, 512, 4, 128, 1) > 0 and size(0, 512, 4, 128, 1) > 0
    assert size(-1, 512, 4, 128, 1) == 0 and size(4, 512, 4, 96, 1) == 0 and size(4, 512, 4, 128, 0) == 0


class Server:
    """A cache of one layer and the book-keeping of a serving loop."""

    def __init__(self, li, page, pages, W1, W2, **kw):
        self.li, self.page, self.W1, self.W2, self.kw = li, page, W1, W2, kw
        H, d = li.H, li.d
        nan = float("nan")
        self.kc, self.vc = (torch.full((pages, page, H, d), nan, dtype=BF).cuda() for _ in range(2))
        self.tsc = torch.zeros(pages, page, dtype=torch.int64).cuda()
        B = len(li.seq_offsets) - 1
        self.table = torch.full((B, -(-li.max_seqlen // page) + 2), -1, dtype=torch.int32).cuda()
        self.free = torch.from_numpy(np.random.default_rng(1).permutation(pages).astype(np.int32)).cuda()
        self.taken = torch.zeros(1, dtype=torch.int32).cuda()
        self.pos, self.tb = dev(li.pos_bias), dev(li.time_bias)
        self.ctx = [0] * B

    def step(self, rows, ts, new, parents=None, keep=True):
        """rows: [T, D] of the new tokens, `new` a sequence."""
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int64)).cuda()
        ctx = torch.tensor(self.ctx, dtype=torch.int32).cuda()
        slots, self.taken = hstu.hstu_cache_plan(ctx, off, self.free, self.taken, self.table, self.page,
                                                 len(rows))
        y = hstu.hstu_layer_step_fwd(
            dev(rows, BF), self.W1, self.W2, self.kc, self.vc, self.tsc, self.table, ctx, off, slots,
            dev(ts), None if parents is None else dev(parents), self.pos, self.tb, self.li.max_seqlen,
            max(new), ln_eps=self.li.ln_eps, **self.kw)
        assert hstu.hstu_device_status() == 0
        if keep:
            self.ctx = [c + n for c, n in zip(self.ctx, new)]
        return y.float().cpu().numpy()


def weights(li, group):
    """(W1, W2) as the call takes them, and as float64 for the oracle."""
    if group == 0:
        return dev(li.W1, BF), dev(li.W2, BF), li.W1, li.W2
    out = []
    for W in (li.W1, li.W2):
        codes, scales = hstu.hstu_quant_groups_w4(dev(W, BF), group)
        wc, ws = quant_w4_oracle(W.astype(np.float64), group)
        assert np.array_equal(codes.cpu().numpy(), wc) and torch.equal(scales.cpu(), ws)
        out.append(((codes, scales), w4_values(wc, ws, group)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


@pytest.mark.gpu
@pytest.mark.parametrize("group,norm", [(0, False), (0, True), (64, False), (128, True)])
def test_steps_give_the_rows_of_the_whole_sequences(group, norm):
    """Prompts, single tokens, a few at once: every row against the oracle of the
    layer on the whole sequences (a chain sees what causal attention sees)."""
    lens = [150, 3, 260, 40]
    li = make_layer_inputs(5, lengths_override=lens)
    W1, W2, o1, o2 = weights(li, group)
    rng = np.random.default_rng(2)
    D = li.x.shape[1]
    kw, okw = {}, {}
    if norm:
        g = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
        kw, okw = dict(input_norm=True, in_gamma=dev(g)), dict(input_norm=True, in_gamma=g)
    want = oracle.layer(li.seq_offsets, li.x, o1, o2, li.H, li.d, li.timestamps, li.pos_bias,
                        li.time_bias, li.max_seqlen, ln_eps=li.ln_eps, **okw)
    srv = Server(li, 16, 64, W1, W2, **kw)
    off = li.seq_offsets
    for new in ([100, 0, 200, 30], [1, 1, 1, 1], [20, 2, 7, 0], [1, 0, 1, 1], [28, 0, 51, 8]):
        rows = np.concatenate([np.arange(off[b] + srv.ctx[b], off[b] + srv.ctx[b] + n)
                               for b, n in enumerate(new)]).astype(np.int64)
        got = srv.step(li.x[rows], li.timestamps[rows], new)
        assert_bf16_close(got, want[rows], "step %s" % (new,))
    assert srv.ctx == lens


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128])
def test_candidates_side_by_side(group):
    """Candidates of one step are independent: each is the last row of the
    oracle's layer on the history and that candidate alone."""
    n, cand = 140, 21
    li = make_layer_inputs(5, lengths_override=[n])
    W1, W2, o1, o2 = weights(li, group)
    rng = np.random.default_rng(3)
    x = round_to_bf16(rng.standard_normal((cand, li.x.shape[1])).astype(np.float32))
    ts = li.timestamps[-1] + rng.integers(1, 10 ** 5, cand)
    li.max_seqlen = n + cand
    srv = Server(li, 32, 16, W1, W2)
    srv.step(li.x, li.timestamps, [n])
    got = srv.step(x, ts.astype(np.int64), [cand], np.full(cand, -1, dtype=np.int32))
    for i in range(cand):
        want = oracle.layer(np.array([0, n + 1]), np.concatenate([li.x, x[i:i + 1]]), o1, o2, li.H, li.d,
                            np.concatenate([li.timestamps, ts[i:i + 1]]), li.pos_bias, li.time_bias,
                            li.max_seqlen, ln_eps=li.ln_eps, rows=[n])
        assert_bf16_close(got[i:i + 1], want, "candidate %d" % i)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    li = make_layer_inputs(5, lengths_override=[90, 17])
    W1, W2, _, _ = weights(li, 64)
    srv = Server(li, 16, 32, W1, W2)
    srv.step(li.x, li.timestamps, [90, 17])
    srv.ctx = [80, 10]                     # the last tokens once more, into their own pages
    rows = np.concatenate([np.arange(80, 90), 90 + np.arange(10, 17)])
    x, ts = dev(li.x[rows], BF), dev(li.timestamps[rows])
    ctx = torch.tensor(srv.ctx, dtype=torch.int32).cuda()
    off = torch.tensor([0, 10, 17]).cuda()
    pos = np.concatenate([np.arange(80, 90), np.arange(10, 17)])
    tab = srv.table.cpu().numpy()
    slots = dev(np.array([int(tab[b, p // 16]) * 16 + p % 16
                          for b, p in zip([0] * 10 + [1] * 7, pos)], dtype=np.int64))
    args = (x, W1, W2, srv.kc, srv.vc, srv.tsc, srv.table, ctx, off, slots, ts, None, srv.pos, srv.tb,
            li.max_seqlen, 10)
    want = hstu.hstu_layer_step_fwd(*args)
    out = torch.zeros_like(want)
    ws = torch.empty(hstu.hstu_layer_step_workspace_bytes(17, 512, li.H, li.d, 10), dtype=torch.uint8).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hstu.hstu_layer_step_fwd(*args, out=out, workspace=ws)
    g.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = hstu.hstu_layer_step_fwd(*args, stream=side)
    torch.cuda.synchronize()
    assert hstu.hstu_device_status() == 0
    assert torch.equal(out, want) and torch.equal(other, want)


@pytest.mark.gpu
def test_binding_refuses():
    li = make_layer_inputs(5, lengths_override=[20])
    W1, W2, _, _ = weights(li, 0)
    srv = Server(li, 16, 8, W1, W2)
    z = lambda n, t: torch.zeros(n, dtype=t).cuda()  # noqa: E731
    args = [dev(li.x, BF), W1, W2, srv.kc, srv.vc, srv.tsc, srv.table, z(1, torch.int32),
            torch.tensor([0, 20]).cuda(), torch.arange(20).cuda(), dev(li.timestamps), None, srv.pos,
            srv.tb, 64, 20]

    def with_(i, v):
        a = list(args)
        a[i] = v
        return a
    for a, e in ((with_(1, W1.float()), TypeError), (with_(2, (W2, W2)), TypeError),
                 (with_(7, z(1, torch.int64)), TypeError), (with_(9, z(19, torch.int64)), ValueError),
                 (with_(0, args[0].cpu()), ValueError), (with_(1, W1[:, :256]), ValueError),
                 (with_(10, None), hstu.HstuError), (with_(4, srv.vc.transpose(1, 2)), ValueError)):
        with pytest.raises(e):
            hstu.hstu_layer_step_fwd(*a)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64])
def test_padded_batches(group):
    """Rows behind the last sequence (not a number, times of zero) change no row
    and raise no error."""
    li = make_layer_inputs(5, lengths_override=[130, 1, 44])
    W1, W2, o1, o2 = weights(li, group)
    want = oracle.layer(li.seq_offsets, li.x, o1, o2, li.H, li.d, li.timestamps, li.pos_bias,
                        li.time_bias, li.max_seqlen, ln_eps=li.ln_eps)
    srv = Server(li, 16, 64, W1, W2)
    off = li.seq_offsets
    for new, pad in (([120, 0, 40], 3), ([4, 1, 0], 11), ([6, 0, 4], 1)):
        rows = np.concatenate([np.arange(off[b] + srv.ctx[b], off[b] + srv.ctx[b] + n)
                               for b, n in enumerate(new)]).astype(np.int64)
        x = np.concatenate([li.x[rows], np.full((pad, li.x.shape[1]), np.nan, li.x.dtype)])
        ts = np.concatenate([li.timestamps[rows], np.zeros(pad, li.timestamps.dtype)])
        got = srv.step(x, ts, new)
        assert_bf16_close(got[:len(rows)], want[rows], "step %s" % (new,))


def test_every_refusal_comes_before_any_launch():
    """Without a GPU a launch fails with a CUDA error: what the parts of the layer
    refuse (the projections, the append, the attention) is refused first."""
    build()
    lib = _native.load()

    def call(x=16, T=4, D=512, W1=16, s1=16, b1=None, W2=16, s2=16, b2=None, group=0, eps=1e-5, norm=0,
             kc=16, kp=None, kt=None, vc=16, vp=None, vt=None, tsc=16, tsp=16, n=4, page=16, table=16,
             tstride=8, maxp=8, ctx=16, off=16, B=2, slots=16, max_new=2, H=4, d=128, ts=16, par=None,
             pos=16, P=8, tb=16, NB=8, N=64, out=16, ws=16):
        row = H * d
        kt, vt = row if kt is None else kt, row if vt is None else vt
        kp, vp = 16 * kt if kp is None else kp, 16 * vt if vp is None else vp
        return lib.hstu_layer_step_fwd(x, T, D, W1, s1, b1, W2, s2, b2, group, None, None, eps, norm, None,
                                       None, kc, kp, kt, vc, vp, vt, tsc, tsp, n, page, table, tstride,
                                       maxp, ctx, off, B, slots, max_new, H, d, ts, par, pos, P, tb, NB, N,
                                       out, ws, 1 << 40, None)
    for kw in (dict(N=0), dict(N=131073), dict(maxp=0), dict(tstride=7), dict(table=None), dict(ctx=None),
               dict(off=None), dict(P=0), dict(NB=0), dict(NB=1025), dict(n=0), dict(n=1 << 28),
               dict(kc=None), dict(vc=None), dict(kc=24), dict(vc=24), dict(kt=511), dict(kt=516),
               dict(vt=516), dict(kp=16 * 512 - 1), dict(vp=16 * 512 - 8), dict(tsp=15), dict(tsc=20),
               dict(x=24), dict(W1=24), dict(W2=24), dict(out=24), dict(eps=-1.0), dict(eps=float("nan")),
               dict(group=64, W1=24), dict(group=64, W2=24), dict(group=64, s1=17), dict(group=64, s2=17),
               dict(group=64, b1=18), dict(group=64, b2=18), dict(group=64, x=24),
               dict(norm=1, eps=-1.0)):
        assert call(**kw) == INV, kw
    for kw in (dict(page=8), dict(page=24), dict(par=16, max_new=257), dict(group=64, T=65535 * 8 + 1)):
        assert call(**kw) == UNS, kw


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64])
def test_a_refused_call_leaves_the_cache_and_the_output(group):
    li = make_layer_inputs(5, lengths_override=[40])
    W1, W2, _, _ = weights(li, group)
    srv = Server(li, 16, 8, W1, W2)
    srv.step(li.x[:30], li.timestamps[:30], [30])
    pages = srv.table[0, :2].cpu().tolist()
    pos, tb = srv.pos, srv.tb
    wide = torch.zeros(li.H, 1025).cuda()
    x = dev(li.x[30:32], BF)
    odd = torch.zeros(x.numel() + 4, dtype=BF).cuda()[4:].view_as(x)
    out = torch.full_like(x, 3.0)

    def call(x=x, parents=None, tb=tb, N=64, max_new=2, out=out, eps=1e-5):
        return hstu.hstu_layer_step_fwd(
            x, W1, W2, srv.kc, srv.vc, srv.tsc, srv.table, torch.tensor([30], dtype=torch.int32).cuda(),
            torch.tensor([0, 2]).cuda(), torch.tensor([pages[1] * 16 + 14, pages[1] * 16 + 15]).cuda(),
            dev(li.timestamps[30:32]), parents, pos, tb, N, max_new, ln_eps=eps, out=out)
    before = [t.clone() for t in (srv.kc, srv.vc, srv.tsc)]
    none = torch.full((2,), -1, dtype=torch.int32).cuda()
    refused = [dict(N=0), dict(N=131073), dict(tb=wide), dict(parents=none, max_new=257), dict(eps=-1.0),
               dict(x=odd)]
    if group == 0:                  # (the 4-bit projection writes rows of any alignment)
        refused.append(dict(out=odd))
    for kw in refused:
        with pytest.raises(hstu.HstuError):
            call(**kw)
        torch.cuda.synchronize()
        for t, b in zip((srv.kc, srv.vc, srv.tsc), before):
            assert torch.equal(t.view(torch.int16 if t.dtype == BF else t.dtype),
                               b.view(torch.int16 if b.dtype == BF else b.dtype)), kw
        assert bool((out == 3.0).all())
    call()
    torch.cuda.synchronize()
    assert hstu.hstu_device_status() == 0 and not torch.equal(srv.tsc, before[2])


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("D,H", [(512, 8), (256, 4), (1024, 32)])
def test_heads_of_64(group, D, H):
    """Other widths of the layer and its heads: prompts, then a token or a few."""
    lens, d = [170, 33], 64
    li = make_layer_inputs(5, lengths_override=lens)
    rng = np.random.default_rng(D)
    F = H * d
    li.H, li.d = H, d

    def matrix(rows, cols):
        return round_to_bf16((rng.standard_normal((rows, cols)) / np.sqrt(cols)).astype(np.float32))
    li.x, li.W1, li.W2 = round_to_bf16(rng.standard_normal((sum(lens), D)).astype(np.float32)), \
        matrix(4 * F, D), matrix(D, F)
    li.pos_bias, li.time_bias = ((0.1 * rng.standard_normal((H, n))).astype(np.float32) for n in (64, 128))
    W1, W2, o1, o2 = weights(li, group)
    want = oracle.layer(li.seq_offsets, li.x, o1, o2, H, d, li.timestamps, li.pos_bias, li.time_bias,
                        li.max_seqlen, ln_eps=li.ln_eps)
    srv = Server(li, 16, 32, W1, W2)
    off = li.seq_offsets
    for new in ([140, 20], [1, 1], [20, 12], [9, 0]):
        rows = np.concatenate([np.arange(off[b] + srv.ctx[b], off[b] + srv.ctx[b] + n)
                               for b, n in enumerate(new)]).astype(np.int64)
        got = srv.step(li.x[rows], li.timestamps[rows], new)
        assert_bf16_close(got, want[rows], "step %s" % (new,))
    assert srv.ctx == lens
