"""CPU checks of the gated feed-forward and 8-bit integer calls: refusals of
the C entry points before any GPU work, the Python front end, the form that
each tested size takes, and the 64-bit forms that the GPU tests compare with."""
import contextlib
import inspect
import subprocess

import numpy as np
import pytest
import torch

import experts_ref as ref
import feedforward_ref as ff
import group_scaling_fp8_amd as mgs
from feedforward_cases import GATED, ROWS
from group_scaling_fp8_amd import api, experts, feedforward
from test_experts_host import A, INVALID, OK, UNSUPPORTED, with_defaults
from test_mm_form import CSRC, CUS
from test_output_streams import CURRENT, SIDE, Library, Stream, taken  # noqa: F401  (a fixture)

CALLS = ("mgs_mm_gated_block128", "mgs_mm_gated_grad_block128", "mgs_quant_rows_i8", "mgs_mm_i8", "mgs_mm_gated_i8")


@pytest.fixture(scope="module")
def L():
    return mgs.lib()


OPERANDS = ("a", "sa", "M", "K", "b", "sb", "G", "N", "off")
BAD = (dict(M=-1), dict(N=-16), dict(K=-16), dict(N=24), dict(K=24), dict(G=0), dict(G=-3), dict(off=None),
       dict(off=A + 2), dict(a=None), dict(a=A + 8), dict(b=None), dict(b=A + 8), dict(sa=None), dict(sa=A + 2),
       dict(sb=None), dict(sb=A + 1))
LARGE = (dict(G=1025), dict(M=1 << 31), dict(M=(1 << 31) - 256, N=16), dict(N=1 << 31), dict(N=1 << 21),
         dict(K=1 << 23), dict(M=1 << 30, N=1 << 20))


def refusals(f, bad, large=LARGE):
    for kw in BAD + bad:
        assert f(**kw) == INVALID, kw
    for kw in large:
        assert f(**kw) == UNSUPPORTED, kw
    assert f(M=0) == OK and f(N=0) == OK


def sizes(**kw):
    return dict(dict(a=A, sa=A, M=64, K=64, b=A, sb=A, G=2, N=64, off=A, stream=None), **kw)


def test_gated_refusals(L):
    f = with_defaults(L.mgs_mm_gated_block128, OPERANDS + ("act", "flags", "h", "gu", "stream"),
                      **sizes(act=0, flags=0, h=A, gu=None))
    refusals(f, (dict(act=2), dict(act=-1), dict(flags=1), dict(flags=2), dict(flags=4), dict(flags=16), dict(h=None),
                 dict(h=A + 8), dict(gu=A + 8)))


def test_gated_grad_refusals(L):
    f = with_defaults(L.mgs_mm_gated_grad_block128, OPERANDS + ("act", "flags", "gu", "dgu", "h", "stream"),
                      **sizes(act=1, flags=8, gu=A, dgu=A, h=None))
    refusals(f, (dict(act=2), dict(act=-1), dict(flags=1), dict(flags=4), dict(gu=None), dict(gu=A + 8), dict(dgu=None),
                 dict(dgu=A + 8), dict(h=A + 4), dict(K=0)))


def test_integer_refusals(L):
    f = with_defaults(L.mgs_mm_i8, OPERANDS + ("out", "y", "stream"), **sizes(out=0, y=A))
    refusals(f, (dict(out=2), dict(out=-1), dict(y=None), dict(y=A + 8)), LARGE + (dict(K=131072),))
    f = with_defaults(L.mgs_mm_gated_i8, OPERANDS + ("act", "h", "stream"), **sizes(act=0, h=A))
    refusals(f, (dict(act=2), dict(act=-1), dict(h=None), dict(h=A + 8)), LARGE + (dict(K=131072),))
    f = with_defaults(L.mgs_quant_rows_i8, ("x", "M", "K", "q", "s", "stream"), x=A, M=4, K=64, q=A, s=A, stream=None)
    for bad in (dict(M=-1), dict(K=-8), dict(K=12), dict(x=None), dict(x=A + 8), dict(q=None), dict(q=A + 4), dict(s=None),
                dict(s=A + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(M=1 << 31), dict(K=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(M=0) == OK and f(K=0) == OK


def test_sums_of_the_longest_contraction_fit_32_bits():
    assert mgs.MGS_I8_MAX_K % 16 == 0 and 128 * 128 * mgs.MGS_I8_MAX_K < 2 ** 31 <= 128 * 128 * (mgs.MGS_I8_MAX_K + 16)
    header = open(mgs._lib.PKG + "/../include/mgs.h").read()
    assert "#define MGS_I8_MAX_K %d\n" % mgs.MGS_I8_MAX_K in header


def test_python_front_end():
    u8, i8, f32 = torch.zeros((16, 64), dtype=torch.uint8), torch.zeros((16, 64), dtype=torch.int8), torch.zeros((16, 1))
    for call in (lambda: feedforward.mgs_mm_gated_block128(u8, f32, u8[None], f32[None]),
                 lambda: feedforward.mgs_mm_gated_grad_block128(u8, f32, u8[None], f32[None], u8),
                 lambda: feedforward.mgs_quant_rows_i8(u8.to(torch.bfloat16)),
                 lambda: feedforward.mgs_mm_i8(i8, f32[:, 0], i8[None], f32[None, :, 0]),
                 lambda: feedforward.mgs_mm_gated_i8(i8, f32[:, 0], i8[None], f32[None, :, 0])):
        with pytest.raises(ValueError):
            call()
    names = {n for n, f in vars(feedforward).items()
             if inspect.isfunction(f) and "stream" in inspect.signature(f).parameters and n.startswith("mgs_")}
    assert names == set(CALLS) and all(hasattr(mgs.lib(), n) for n in CALLS)


U8, I8, F32 = torch.zeros((32, 64), dtype=torch.uint8), torch.zeros((32, 64), dtype=torch.int8), torch.zeros((32, 1))
OFF, X = torch.tensor([32], dtype=torch.int32), torch.zeros((32, 64), dtype=torch.bfloat16)
MEMORY = {
    "mgs_mm_gated_block128": (lambda **kw: feedforward.mgs_mm_gated_block128(
        U8, F32, torch.stack([U8, U8]), F32[None, :1].expand(2, 1, 1), OFF, keep=True, **kw), 2),
    "mgs_mm_gated_grad_block128": (lambda **kw: feedforward.mgs_mm_gated_grad_block128(
        U8, F32, U8[None], F32[None, :1], X, OFF, hidden=True, **kw), 2),
    "mgs_quant_rows_i8": (lambda **kw: feedforward.mgs_quant_rows_i8(X, **kw), 2),
    "mgs_mm_i8": (lambda **kw: feedforward.mgs_mm_i8(I8, F32[:, 0], I8[None], F32[None, :, 0], OFF, **kw), 1),
    "mgs_mm_gated_i8": (lambda **kw: feedforward.mgs_mm_gated_i8(
        I8, F32[:, 0], torch.stack([I8, I8]), F32[:, 0].expand(2, 32), OFF, **kw), 1),
}


@pytest.mark.parametrize("name", MEMORY)
@pytest.mark.parametrize("stream", [None, SIDE, "object"])
def test_memory_of_outputs(taken, monkeypatch, name, stream):  # noqa: F811
    """Outputs are taken from the stream that the call runs on."""
    monkeypatch.setattr(feedforward, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(feedforward, "lib", Library)
    monkeypatch.setattr(feedforward, "_given", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)        # where CPU tensors say they are
    call, outputs = MEMORY[name]
    call(stream=Stream(SIDE) if stream == "object" else stream)
    if stream is None:           # torch's own memory of the current stream, by any of its functions
        assert all(t.taken_on == CURRENT and not t.recorded for t in taken)
        return
    assert [t.taken_on for t in taken] == [SIDE] * outputs
    assert [t.recorded for t in taken] == [[CURRENT]] * outputs


@pytest.mark.parametrize("current", [-1, 3])
def test_tensors_of_another_device(monkeypatch, current):
    """A call makes its tensors' device the current one, and leaves it as it was."""
    now, seen = [current], []

    @contextlib.contextmanager
    def device(d):
        now.append(-1 if d == torch.device("cpu") else d)
        yield
        now.pop()

    class Noting:
        def __getattr__(self, name):
            return lambda *a: seen.append(now[-1]) or mgs.MGS_OK
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(feedforward, "lib", Noting)
    feedforward._run("mgs_mm_i8", U8)
    assert seen == [-1] and now == [current]


PROGRAM = r"""
#include <stdio.h>
#include "mgs_mm_form.hpp"
int main() {
    long long ints, eight, grouped, M, N, K, G, cus;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &ints, &eight, &grouped, &M, &N, &K, &G, &cus) == 8) {
        const mgs::MmForm f = mgs::mm_form_rows(ints, eight, grouped, M, N, K, G, (int)cus);
        printf("%d %d %d\n", f.few, f.tile, f.sets);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "form.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-o", str(d / "form"), str(d / "form.cpp")], check=True)

    def run(*args):
        r = subprocess.run([str(d / "form")], input=" ".join(str(int(a)) for a in args), capture_output=True, text=True,
                           check=True)
        return tuple(int(v) for v in r.stdout.split())
    return run


@pytest.mark.parametrize("gated,case", [(False, c) for c in ROWS] + [(True, c) for c in GATED])
def test_sizes_take_their_forms(form, gated, case):
    """So that a changed rule cannot take a form out of the GPU tests unseen."""
    M, N, K, G, kind, ints, fast, exact = case
    N *= 2 if gated else 1
    assert form(1, 1, kind != "none", M, N, K, G, CUS) == ints
    assert form(0, 1, kind != "none", M, N, K, G, CUS) == fast
    assert form(0, 0, kind != "none", M, N, K, G, CUS) == exact


def test_every_form_is_tested():
    few = {(rows, lines, 0) for rows in (16, 32) for lines in (32, 64)}
    tiles = {(0, 128, 1), (0, 128, 2), (0, 256, 1)}
    for cases in (ROWS, GATED):
        assert {c[5] for c in cases} == few | {(64, 64, 0)} | tiles
        assert {c[6] for c in cases} == few | tiles
        assert {c[7] for c in cases} == few | tiles - {(0, 256, 1)}


def test_limits_between_the_forms(form):
    for args, want in (
            ((1, 1, 0, 1, 8192, 1024, 1), (16, 32, 0)), ((1, 1, 0, 1, 16400, 5104, 1), (16, 32, 0)),
            ((1, 1, 0, 1, 16400, 5120, 1), (16, 64, 0)), ((0, 1, 0, 1, 16400, 1024, 1), (16, 64, 0)),
            ((1, 1, 0, 1, 16384, 1024, 1), (16, 64, 0)), ((1, 1, 0, 32, 16384, 1024, 1), (32, 64, 0)),
            ((1, 1, 0, 33, 16384, 1024, 1), (64, 64, 0)), ((0, 1, 0, 33, 16384, 1024, 1), (32, 64, 0)),
            ((0, 1, 0, 41, 16384, 1024, 1), (0, 128, 2)), ((0, 0, 0, 64, 16384, 1024, 1), (32, 64, 0)),
            ((0, 0, 0, 65, 16384, 1024, 1), (0, 128, 2)), ((0, 0, 0, 512, 2048, 1024, 1), (32, 64, 0)),
            ((0, 0, 0, 513, 2048, 1024, 1), (0, 128, 2)), ((1, 1, 0, 65, 16384, 1024, 1), (0, 128, 2)),
            ((1, 1, 1, 320, 16384, 1024, 16), (16, 32, 0)), ((0, 1, 1, 320, 16384, 1024, 16), (16, 64, 0)),
            ((0, 1, 1, 640, 16384, 1024, 16), (32, 64, 0)), ((1, 1, 1, 640, 16384, 1024, 16), (0, 128, 1)),
            ((0, 0, 1, 640, 16384, 1024, 16), (32, 64, 0)), ((0, 0, 1, 641, 16384, 1024, 16), (0, 128, 1)),
            ((1, 1, 0, 64, 4096, 1024, 1), (32, 32, 0)), ((1, 1, 0, 128, 4096, 1024, 1), (32, 64, 0)),
            ((1, 1, 0, 256, 16384, 1024, 1), (0, 128, 2)), ((0, 0, 0, 256, 16384, 1024, 1), (0, 128, 2)), ((0, 0, 0, 257, 16384, 1024, 1), (0, 128, 1)),
            ((0, 1, 1, 256, 1040, 1024, 4), (32, 64, 0)), ((1, 1, 0, 2048, 4096, 1024, 1), (0, 128, 1)),
            ((1, 1, 1, 2048, 4096, 1024, 8), (0, 256, 1)), ((1, 1, 0, 1003, 4176, 1024, 1), (0, 128, 1)),
            ((1, 1, 1, 16640, 16384, 1024, 16), (0, 256, 1)), ((1, 1, 0, 2147483391, 2097072, 1024, 1), (0, 256, 1)),
            ((1, 1, 1, 1, 16, 1024, 1024), (16, 32, 0))):
        assert form(*args, CUS) == want, args


# ---- the plain forms themselves -------------------------------------------------

def test_activations_by_hand():
    assert abs(ff.act_of(ff.SILU, np.float64(2.0)) - 2 / (1 + np.exp(-2.0))) < 1e-15
    g = np.array([-9.0, -1.5, -0.1, 0.0, 0.3, 1.0, 4.0, 20.0])
    tanh = 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    assert np.abs(ff.act_of(ff.GELU, g) - tanh).max() < 1e-15
    for act, most in ((ff.SILU, 1.1), (ff.GELU, 1.13)):
        wide = np.linspace(-30, 30, 60001)
        assert np.abs(ff.slope_of(act, wide)).max() < most


@pytest.mark.parametrize("act", [ff.SILU, ff.GELU])
def test_gradient_by_differences(act):
    """The formula of the gradient against central differences of a sum of the layer's outputs."""
    rng = np.random.default_rng(act)
    M, N, D = 3, 16, 16
    g, u, w, dy = (rng.standard_normal(s) for s in ((M, N), (M, N), (N, D), (M, D)))

    def loss(g, u):
        return float((ff.act_of(act, g) * u @ w * dy).sum())
    dh = dy @ w.T
    dg, du = dh * u * ff.slope_of(act, g), dh * ff.act_of(act, g)
    h = 1e-6
    for at in np.ndindex(M, N):
        e = np.zeros((M, N))
        e[at] = h
        assert abs((loss(g + e, u) - loss(g - e, u)) / (2 * h) - dg[at]) < 1e-7
        assert abs((loss(g, u + e) - loss(g, u - e)) / (2 * h) - du[at]) < 1e-7


def test_integer_forms_by_hand():
    x = np.zeros((2, 16), np.float32)
    x[0, 3], x[0, 4], x[0, 5], x[0, 6] = -2.0, 0.0078125, 1.0, 0.0234375
    from group_scaling_fp8_amd import workloads as wl
    q, s = ff.quant_rows_i8(wl.f32_to_bf16_bits(x))
    assert s[0] == 63.5 and s[1] == np.float32(127) / np.float32(1e-12)
    # 0.49609375 to 0, 63.5 to the even 64, 1.48828125 to 1
    assert q[0, 3:7].tolist() == [-127, 0, 64, 1] and not q[1].any()
    a, b = np.array([[3, -2] + [0] * 14], np.int8), np.array([[[5, 7] + [0] * 14] * 16], np.int8)
    y, whole = ff.mm_i8(a, np.array([2.0], np.float32), b, np.full((1, 16), 0.25, np.float32), [1])
    assert (whole == 1).all() and (y == 2).all()
