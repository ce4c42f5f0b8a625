"""Calls on another stream than the tensors' own, with outputs that the call
allocates: memory that the current stream still reads is not written early,
memory of an output that is freed early is not handed out before the call
has run, and values are those of the call on the current stream. The host
side of this is in tests/test_output_streams.py."""
import numpy as np
import pytest
import torch

import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import workloads as wl
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

SLEEP = 40_000_000       # clock ticks, tens of milliseconds


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def bf16(rng, *shape):
    return to_dev(wl.randn_bf16(rng, shape, 0.02, 0.001, 8.0)).view(torch.bfloat16)


def calls():
    """The calls that take no output tensors, with the order of one launch and the
    ranked one, and three others."""
    rng = np.random.default_rng(21)
    x, w = bf16(rng, 18000, 72), bf16(rng, 3, 1040, 528)
    ids = to_dev(rng.integers(-1, 8, (18000, 2)).astype(np.int32))
    off, rows, slots, a, sa, xp = mgs.mgs_moe_dispatch(x, ids, 8, permuted=True)
    ends, ws = to_dev(np.array([640, 7008, 18000], np.int32)), mgs.dim0_workspace(18000, 72)
    torch.cuda.synchronize()
    return {
        "sort": lambda **kw: mgs.mgs_moe_sort(ids[:9000], 8, **kw),
        "sort_ranked": lambda **kw: mgs.mgs_moe_sort(ids, 8, **kw),
        "dispatch": lambda **kw: mgs.mgs_moe_dispatch(x[:9000], ids[:9000], 8, permuted=True, **kw),
        "dispatch_ranked": lambda **kw: mgs.mgs_moe_dispatch(x, ids, 8, permuted=True, **kw),
        "blocks128": lambda **kw: mgs.mgs_quant_blocks128(w, **kw),
        "rows128": lambda **kw: mgs.mgs_quant_rows128(x, **kw),
        "combine": lambda **kw: (mgs.mgs_moe_combine(xp, rows, **kw),),
        "dim0_t": lambda **kw: mgs.mgs_quant_groups_dim0_t(x, ends, workspace=ws, **kw),
    }


def same(a, b):
    return all(torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)) for u, v in zip(a, b))


@pytest.mark.parametrize("as_int", [False, True])
def test_memory_that_the_current_stream_still_reads(as_int):
    side = torch.cuda.Stream()
    for name, call in calls().items():
        print(name, flush=True)
        want = [t.clone() for t in call()]
        # tensors of the outputs' sizes, freed while a copy of them is queued
        held = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda") for t in want]
        kept = [torch.zeros_like(h) for h in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        for k, h in zip(kept, held):
            k.copy_(h)
        del h, held
        got = call(stream=side.cuda_stream if as_int else side)
        torch.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept), name
        assert same(got, want), name


def test_memory_of_outputs_freed_before_the_call_has_run():
    side = torch.cuda.Stream()
    for name, call in calls().items():
        print(name, flush=True)
        sizes = [t.numel() * t.element_size() for t in call()]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        call(stream=side)
        taken = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert all(bool((t == 9).all()) for t in taken), name


def test_a_chain_of_calls_whose_tensors_are_freed_at_once():
    """The intermediate tensors of a chain on another stream live no longer
    than the statement; the current stream allocates and writes meanwhile."""
    rng = np.random.default_rng(22)
    x, w = bf16(rng, 400, 528), bf16(rng, 1, 272, 528)
    want = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(x), *mgs.mgs_quant_blocks128(w, transposed=False))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(x, stream=side),
                              *mgs.mgs_quant_blocks128(w, transposed=False, stream=side), stream=side)
    taken = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in (x.numel(), w.numel(), 8000, 512, 64)]
    torch.cuda.current_stream().wait_stream(side)
    assert same([got], [want]) and all(bool((t == 3).all()) for t in taken)


def test_outputs_of_another_stream_inside_a_capture():
    """A call on a second stream that a capture has forked to."""
    rng = np.random.default_rng(23)
    x = bf16(rng, 300, 264)
    want = [[t.clone() for t in mgs.mgs_quant_rows128(v)] for v in (x, x * 2)]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = mgs.mgs_quant_rows128(x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    x0 = x.clone()
    for i in (0, 1, 0, 1):
        x.copy_(x0 * 2 if i else x0)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want[i]), i
        assert same(mgs.mgs_quant_rows128(x), want[i])
