"""A graph of the expert calls that order more slots than one launch does: a
histogram, a ranking that reads it from the workspace, copy and cast. Every
replay has new inputs and is compared with the eager calls."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def same(a, b):
    return all(torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)) for u, v in zip(a, b))


def replays(inputs, call, order=(1, 2, 0, 1)):
    """Captures call(**inputs(0)) and replays it on other inputs, with eager
    work on the same inputs between the replays."""
    v = inputs(0)
    want = [[t.clone() for t in call(**inputs(i))] for i in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(**v)
    for i in order:
        for name, t in inputs(i).items():
            v[name].copy_(t)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want[i]), i
        assert same(call(**inputs(i)), want[i]), i


@pytest.mark.parametrize("T,k,E,D", [(17000, 2, 6, 16), (33001, 1, 70, 1040), (9000, 5, 600, 136)])
def test_dispatch_of_ranked_slots(T, k, E, D):
    assert T * k > 32768      # the slots that one launch orders

    def inputs(seed):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        return {"ids": to_dev(rng.integers(-1, E, (T, k)).astype(np.int32)),
                "x": torch.randn((T, D), generator=gen, device="cuda", dtype=torch.bfloat16)}

    def call(ids, x):
        return mgs.mgs_moe_sort(ids, E) + mgs.mgs_moe_dispatch(x, ids, E, permuted=True)
    replays(inputs, call)
    v = inputs(1)
    out = call(**v)
    r_off, r_rows, r_slots = ref.order(v["ids"].cpu().numpy(), E, 16)
    for got, want in ((out[0], r_off), (out[1], r_rows), (out[2], r_slots), (out[3], r_off), (out[5], r_slots)):
        assert np.array_equal(got.cpu().numpy(), want)
