"""Calls on a stream that is not the current one: what they allocate must not be
memory that work still queued on the current stream uses, and their results must
not be handed out again while the caller's stream reads them."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from gen import custom_attn_inputs, make_layer_inputs
from gpu_util import attn_tensors, dev
from serving_util import make_step

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SLEEP = 100_000_000             # clock cycles: tens of milliseconds


def queued(sizes):
    """Blocks of these sizes that Python has let go of, while the current stream
    has yet to write them."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for b in blocks:
        b.fill_(0x5a)


def plan_call(seed):
    rng = np.random.default_rng(seed)
    ctx = torch.from_numpy(rng.integers(0, 60, 40).astype(np.int32)).cuda()
    T = 40 * 5000
    off = torch.arange(0, T + 1, 5000).cuda()
    free = torch.from_numpy(rng.permutation(13000).astype(np.int32)).cuda()
    start = torch.zeros(1, dtype=torch.int32).cuda()
    table = torch.zeros((40, 320), dtype=torch.int32).cuda()
    return lambda **kw: hstu.hstu_cache_plan(ctx, off, free, start, table, 16, T, **kw), [T * 8, 4]


def quant_call(seed):
    W = torch.randn(640, 512, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()
    return lambda **kw: hstu.hstu_quant_groups_w4(W, 64, **kw), [640 * 256, 640 * 8 * 2]


def linear_call(seed):
    g = torch.Generator().manual_seed(seed)
    x, W = torch.randn(9, 512, generator=g).to(BF).cuda(), torch.randn(640, 512, generator=g).to(BF).cuda()
    codes, scales = hstu.hstu_quant_groups_w4(W, 128)
    return lambda **kw: hstu.hstu_linear_w4_fwd(x, codes, scales, **kw), [9 * 640 * 2]


def attn_call(seed):
    s = make_step([700, 90], [5, 9], "tree", 2, 64, 64, 16, BF, seed=seed)
    d = [dev(a) if isinstance(a, np.ndarray) else a.cuda() for a in
         (s.q, s.kc, s.vc, s.tsc, s.table, np.array(s.ctx, np.int32), s.off, s.ts, s.parents, s.pos, s.tb)]
    return (lambda **kw: hstu.hstu_attn_cached_fwd(*d, 2000, 9, **kw),
            [14 * 2 * 64 * 2, hstu.hstu_attn_cached_workspace_bytes(BF, 9, 64)])


def layer_call(seed):
    li = make_layer_inputs(5, lengths_override=[300])
    rng = np.random.default_rng(seed)
    kc, vc = (torch.from_numpy(rng.standard_normal((24, 16, li.H, li.d))).to(BF).cuda() for _ in range(2))
    tsc = torch.from_numpy(rng.integers(10 ** 9, 2 * 10 ** 9, (24, 16))).cuda()
    table = torch.arange(24, dtype=torch.int32).view(1, 24).cuda()
    D = li.x.shape[1]
    args = (dev(li.x[:20], BF), dev(li.W1, BF), dev(li.W2, BF), kc, vc, tsc, table,
            torch.tensor([300], dtype=torch.int32).cuda(), torch.tensor([0, 20]).cuda(),
            torch.arange(300, 320).cuda(), torch.arange(2 * 10 ** 9, 2 * 10 ** 9 + 20).cuda(), None,
            dev(li.pos_bias), dev(li.time_bias), 2000, 20)
    return (lambda **kw: hstu.hstu_layer_step_fwd(*args, **kw),
            [20 * D * 2, hstu.hstu_layer_step_workspace_bytes(20, D, li.H, li.d, 20)])


def dense_call(which):
    """The calls on whole batches: their inputs for a seed, the call, what it allocates."""
    def make(seed):
        inp = custom_attn_inputs([300, 17, 90], H=4, d=64, num_pos=64, num_buckets=64,
                                 dtype="f32" if which.endswith("f32") else "bf16", seed=seed)
        t = attn_tensors(inp)
        T, F = t["q"].shape[0], 256
        args = [t[n] for n in ("seq_offsets", "timestamps", "pos_bias", "time_bias", "max_seqlen")]
        qkv = [t[n] for n in "qkv"]
        g = torch.Generator().manual_seed(seed)
        x, u = (torch.randn(T, F, generator=g).to(BF).cuda() for _ in range(2))
        W, W2 = torch.randn(4 * F, F, generator=g).to(BF).cuda() / 16, torch.eye(F, dtype=BF).cuda()
        if which.startswith("attn_fwd"):
            bf = which == "attn_fwd"
            ws = hstu.hstu_attn_workspace_bytes(3, T, inp.max_seqlen, 4, 64) if bf else 16
            return lambda **kw: hstu.hstu_attn_fwd(*qkv, *args, **kw), [T * F * (2 if bf else 4), ws]
        if which == "attn_bwd":
            ws = hstu.hstu_attn_bwd_workspace_bytes(3, T, inp.max_seqlen)
            return lambda **kw: hstu.hstu_attn_bwd(*qkv, u.view(T, 4, 64), *args, **kw), [T * F * 4] * 3 + [ws]
        if which == "attn_bwd_f32":
            dout = u.float().view(T, 4, 64)
            return (lambda **kw: hstu.hstu_attn_bwd_f32(*qkv, dout, *args, **kw),
                    [T * F * 4] * 3)
        if which == "bias_indices":
            return (lambda **kw: hstu.hstu_debug_bias_indices(args[0], args[1], 64, 64, **kw),
                    [T * T * 2] * 2)
        if which == "linear":
            return lambda **kw: hstu.hstu_linear_fwd(x, W, **kw), [T * 4 * F * 2]
        if which == "layernorm":
            return lambda **kw: hstu.hstu_layernorm_fwd(x, **kw), [T * F * 2]
        if which == "layernorm_gate":
            return lambda **kw: hstu.hstu_layernorm_gate_fwd(x, u, **kw), [T * F * 2]
        if which == "layernorm_fp8":
            return lambda **kw: hstu.hstu_layernorm_fp8_fwd(x, **kw), [T * F, T * 4]
        if which == "layernorm_gate_fp8":
            return lambda **kw: hstu.hstu_layernorm_gate_fp8_fwd(x, u, **kw), [T * F, T * 4]
        if which == "quant_rows":
            return lambda **kw: hstu.hstu_quant_rows_e4m3(x, **kw), [T * F, T * 4]
        if which == "layer":
            ws = hstu.hstu_layer_workspace_bytes(T, 3, F, 4, 64, inp.max_seqlen)
            return lambda **kw: hstu.hstu_layer_fwd(x, W, W2, *args[:4], 4, 64, args[4], **kw), [T * F * 2, ws]
        q1, q2 = hstu.hstu_quant_rows_e4m3(W), hstu.hstu_quant_rows_e4m3(W2)
        if which == "linear_fp8":
            xq = hstu.hstu_quant_rows_e4m3(x)
            return lambda **kw: hstu.hstu_linear_fp8_fwd(*xq, *q1, **kw), [T * 4 * F * 2]
        ws = hstu.hstu_layer_fp8_workspace_bytes(T, 3, F, 4, 64, inp.max_seqlen)
        return lambda **kw: hstu.hstu_layer_fp8_fwd(x, *q1, *q2, *args[:4], 4, 64, args[4], **kw), [T * F * 2, ws]
    return make


CALLS = {"plan": plan_call, "quant": quant_call, "linear_w4": linear_call, "attn": attn_call,
         "layer_step": layer_call}
CALLS.update((name, dense_call(name)) for name in (
    "attn_fwd", "attn_fwd_f32", "attn_bwd", "attn_bwd_f32", "bias_indices", "linear", "layernorm",
    "layernorm_gate", "layernorm_fp8", "layernorm_gate_fp8", "quant_rows", "layer", "linear_fp8",
    "layer_fp8"))


def tensors(r):
    return [t.clone() for t in (r if isinstance(r, tuple) else (r,))]


def assert_same(name, got, want):
    for g, w in zip(got, want):
        if name.startswith("attn_bwd"):         # (sums by atomics, in any order)
            assert float((g - w).norm()) <= 1e-4 * float(w.norm())
        else:
            assert torch.equal(g, w)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_not_memory_that_queued_work_writes(name):
    call, sizes = CALLS[name](1)
    want = tensors(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    queued(sizes)
    got = call(stream=side)
    torch.cuda.synchronize()
    assert_same(name, tensors(got), want)
    assert hstu.hstu_device_status() == 0


@pytest.mark.parametrize("name", CALLS)
def test_results_outlive_their_readers_on_the_current_stream(name):
    (call, _), (other, _) = CALLS[name](1), CALLS[name](2)
    want = tensors(call())
    other()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    copies = tensors(got)                       # queued behind the wait
    del got
    for _ in range(3):
        other(stream=side)
    torch.cuda.synchronize()
    assert_same(name, copies, want)
    assert hstu.hstu_device_status() == 0


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [0, 1], ids=["null", "legacy"])
def test_the_default_stream_given_while_another_is_current(name, handle):
    call, sizes = CALLS[name](1)
    want = tensors(call())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(torch.cuda.Stream()):
        queued(sizes)
        got = call(stream=handle)
        same = call(stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        for r in (got, same):
            assert_same(name, tensors(r), want)
    assert hstu.hstu_device_status() == 0


@pytest.mark.parametrize("name", [n for n in CALLS if n != "bias_indices"])     # (that one reads offsets)
def test_a_side_stream_inside_a_capture(name):
    """Allocations of a call on a stream that joined a capture, results let go of
    inside it too; replayed twice."""
    call, _ = CALLS[name](1)
    want = tensors(call())
    side = torch.cuda.Stream()
    call(stream=side)                           # (first use outside)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copies = tensors(got)
    for _ in range(2):
        for t in copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert_same(name, copies, want)
    assert hstu.hstu_device_status() == 0
