"""Calls on a stream that is not the current one: what they allocate must not be
memory that work still queued on the current stream uses, and their results must
not be handed out again while the caller's stream reads them."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from gen import make_layer_inputs
from gpu_util import dev
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


CALLS = {"plan": plan_call, "quant": quant_call, "linear_w4": linear_call, "attn": attn_call,
         "layer_step": layer_call}


def tensors(r):
    return [t.clone() for t in (r if isinstance(r, tuple) else (r,))]


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
    for g, w in zip(tensors(got), want):
        assert torch.equal(g, w)
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
    for g, w in zip(copies, want):
        assert torch.equal(g, w)
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
            for g, w in zip(tensors(r), want):
                assert torch.equal(g, w)
    assert hstu.hstu_device_status() == 0
