"""Every kernel of the 8-bit products with every output, format and epilogue, at sizes
that ask the library's rule for it (a changed rule asks for another size): references
in 64 bits on the GPU from the codes' values, bounds as in test_gpu_f8.py.
"""
import numpy as np
import pytest
import torch

import mixed_gemm_amd as mg
from tests.f8_forms import FORMS, GATED, PAIRS, fused, tile
from tests.f8_util import codes, scales
from tests.test_gpu_f8 import TYPES, assert_same, big_act, big_close, big_product, big_q, halves, interleaved, values_on_gpu

pytestmark = pytest.mark.gpu


class Random:
    """Heavy-tailed rows on the GPU from a seed."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda")

    def rows(self, M, K, dtype="bf16", ld=0, size=1.0):
        """[M][K], K + ld apart, whose gaps hold NaN."""
        x = size * self.normal(M, K) * torch.exp(self.normal(M, 1))
        x[:, torch.randperm(K, generator=self.gen, device="cuda")[: max(1, K // 50)]] *= 25.0
        base = torch.full((M, K + ld), float("nan"), dtype=TYPES[dtype], device="cuda")
        base[:, :K] = x.to(TYPES[dtype])
        return base[:, :K]

    def index(self, M, rows):
        """Modulation rows of the tokens, some outside them."""
        return torch.randint(-1, rows + 1, (M,), generator=self.gen, device="cuda", dtype=torch.int32)


def _forms(out):
    return [f for f in FORMS if f[1] == out]


def _output(M, N, out):
    """NaN, with a row behind the last one."""
    base = torch.full((M + 1, N), float("nan"), dtype=TYPES[out], device="cuda")
    base[M] = 7.0
    return base, base[:M]


def _activated(v, bound, act):
    """act(v) of fp32 sums within `bound` of v, and its bound."""
    a, d = big_act(v, act)
    return a, d.abs() * bound + 1.2 * bound ** 2 + 2.0 ** -20 * v.abs()


def _gated(res, gate, where, a, bound):
    """res + gate a, padding tokens (where outside the gate's rows) res alone."""
    on = (where >= 0) & (where < len(gate))
    g = torch.where(on[:, None], gate.double()[where.clamp(0, len(gate) - 1).long()], 0.0)
    ref = res + g * a
    return ref, g.abs() * bound + 2.0 ** -22 * (ref.abs() + (g * a).abs())


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("want,out,M,K,N", FORMS)
def test_product_with_every_epilogue(want, out, M, K, N, act):
    assert tile(M, K, N, out) == want
    r = Random(M + K + N)
    x, p = mg.f8_checkpoint(r.rows(M, K)), mg.f8_plan(r.rows(N, K, size=0.02))
    v, bound = big_product(values_on_gpu(x), values_on_gpu(p.w), out)
    base, y = _output(M, N, out)
    if act == "none":
        mg.mg_f8_gemm(x, p.w, None, y)
        big_close(y, v, bound, out)
        again = torch.empty_like(y)
        mg.mg_f8_gemm(x, p.w, None, again)
        assert torch.equal(again, y)
    for bt in ("f32", "bf16"):
        bias = r.normal(N).to(TYPES[bt])
        z = v + bias.double()
        a, ab = _activated(z, bound + 2.0 ** -23 * z.abs(), act)
        y.fill_(float("nan"))
        mg.mg_f8_gemm(x, p.w, mg.Epilogue(bias, act), y)
        big_close(y, a, ab, out)
        # gate rows per token, with padding tokens, and one for each run of tokens; residuals of both types, rows apart
        gate = r.normal(3, N).to(TYPES[bt])
        index, group = r.index(M, 3), -(-M // 3)
        runs = torch.arange(M, device="cuda", dtype=torch.int32) // group
        for rt, mod, where in ((None, mg.Mod(gate=gate, index=index), index), ("f32", mg.Mod(gate=gate, index=index), index),
                               ("bf16", mg.Mod(gate=gate, group=group), runs), ("f32", mg.Mod(gate=gate, group=group), runs)):
            res = r.rows(M, N, rt, 8) if rt else None
            ref, rb = _gated(res.double() if rt else torch.zeros_like(v), gate, where, a, ab)
            y.fill_(float("nan"))
            mg.mg_f8_gemm(x, p.w, mg.Epilogue(bias, act, mod, res), y)
            big_close(y, ref, rb, out)
    # onto itself
    y.copy_(r.rows(M, N, out))
    want_y = y.double() + _activated(v, bound, act)[0]
    mg.mg_f8_gemm(x, p.w, mg.Epilogue(act=act, residual=y), y)
    big_close(y, want_y, _activated(v, bound, act)[1] + 2.0 ** -22 * (want_y.abs() + v.abs()), out)
    assert (base[M] == 7.0).all()


@pytest.mark.parametrize("want,out,M,K,N", FORMS)
def test_product_of_gradients(want, out, M, K, N):
    """E5M2 rows: no activation, every other epilogue."""
    assert tile(M, K, N, out) == want
    r = Random(M + K + N + 1)
    x, p = mg.f8_checkpoint(r.rows(M, K, size=1e-3), "e5m2"), mg.f8_plan(r.rows(N, K, size=0.02))
    v, bound = big_product(values_on_gpu(x), values_on_gpu(p.w), out)
    base, y = _output(M, N, out)
    mg.mg_f8_gemm(x, p.w, None, y)
    big_close(y, v, bound, out)
    size = v.abs().mean()
    bias = r.normal(N) * size
    z = v + bias.double()
    mg.mg_f8_gemm(x, p.w, mg.Epilogue(bias), y)
    big_close(y, z, bound + 2.0 ** -23 * z.abs(), out)
    gate, index = r.normal(3, N), r.index(M, 3)
    for rt in ("f32", "bf16"):
        res = (r.rows(M, N, "f32") * size).to(TYPES[rt])
        want_y = res.double() + v
        mg.mg_f8_gemm(x, p.w, mg.Epilogue(residual=res), y)
        big_close(y, want_y, bound + 2.0 ** -22 * (want_y.abs() + v.abs()), out)
        ref, rb = _gated(res.double(), gate, index, z, bound + 2.0 ** -23 * z.abs())
        mg.mg_f8_gemm(x, p.w, mg.Epilogue(bias, "none", mg.Mod(gate=gate, index=index), res), y)
        big_close(y, ref, rb, out)
    assert (base[M] == 7.0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("want,out,F,T,K", PAIRS)
def test_weight_gradients_of_two_projections(want, out, F, T, K, fmt):
    """dWg and dWu: runs of 128 rows of two outputs in turn, a run's surplus rows left out."""
    up = -(-T // 32) * 32
    Fp = -(-F // 128) * 128
    assert tile(2 * Fp, up, K, out) == want
    r = Random(F + T + K)
    x, dgu = mg.f8_checkpoint(r.rows(T, K)), mg.f8_checkpoint(r.rows(T, 2 * Fp, size=1e-3), fmt)
    xt, dgut = mg.F8.empty(K, up), mg.F8.empty(2 * Fp, up, fmt)
    mg.mg_f8_transpose(x, xt)
    mg.mg_f8_transpose(dgu, dgut)
    ref, bound = big_product(values_on_gpu(dgut), values_on_gpu(xt), out)
    y = torch.full((2, F + 1, K), 7.0, dtype=TYPES[out], device="cuda")
    y[:, :F] = float("nan")
    mg.mg_gated_gemm_dw(dgut, xt, y[0, :F], y[1, :F])
    for o, (a, b) in enumerate(zip(halves(ref.t(), F), halves(bound.t(), F))):
        big_close(y[o, :F], a.t(), b.t(), out)
    assert (y[:, F] == 7.0).all()


def _poisoned(x):
    x.q.fill_(0x55), x.s.fill_(0x11111111)
    return x


def _transposed(x):
    t = mg.F8.empty(x.cols, -(-x.rows // 32) * 32, x.fmt)
    mg.mg_f8_transpose(x, t)
    return t


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("M,K,F,N", GATED)
def test_gated_block_formed_in_the_epilogue(M, K, F, N, act):
    """Forward, with and without what is kept, and backward; every 8-bit matrix that a step leaves is
    compared, with buffers that held something else before."""
    assert fused(M, F, K)[:2] == (True, True) and fused(M, F, N)[2]
    r = Random(M + F + len(act))
    X, Wg, Wu, Wd = r.rows(M, K), r.rows(F, K, size=0.05), r.rows(F, K, size=0.05), r.rows(N, F, size=0.05)
    ffn = mg.gated_ffn(Wg, Wu, Wd, act, backward=True)
    saved, work = mg.GatedSaved.empty(ffn, M), mg.GatedWork.empty(ffn, M, "e4m3")
    for x in (saved.x, saved.gu, saved.h, work.x, work.h):
        _poisoned(x)
    y = mg.gated_ffn_forward(ffn, X, saved, work=work)
    x8 = mg.f8_checkpoint(X)
    assert_same(saved.x, codes(x8), scales(x8))
    xv, w13, wd = values_on_gpu(x8), values_on_gpu(ffn.w13), values_on_gpu(ffn.wd)
    wg, wu = (v.t() for v in halves(w13.t(), F))

    def check(out, h, gu):
        (g, bg), (u, bu) = big_product(xv, wg, out), big_product(xv, wu, out)
        a, ba = _activated(g, bg, act)
        big_q(h, a * u, ba * u.abs() + a.abs() * bu + ba * bu + 2.0 ** -23 * (a * u).abs(), "hidden")
        codes(h)                                                     # (columns past F hold 0)
        if gu is not None:
            big_q(gu, interleaved(g, u), interleaved(bg, bu), "gate and up sums")

    check("f32", saved.h, saved.gu)
    big_close(y, *big_product(values_on_gpu(saved.h), wd, "bf16"), "bf16")
    y = mg.gated_ffn_forward(ffn, X, work=work)                       # without keeping: the 8-bit instructions
    check("bf16", work.h, None)
    big_close(y, *big_product(values_on_gpu(work.h), wd, "bf16"), "bf16")
    g, u = halves(values_on_gpu(saved.gu), F)
    a, d = big_act(g, act)
    for fmt in ("e4m3", "e5m2"):
        dY = r.rows(M, N, size=1e-4)
        work = mg.GatedWork.empty(ffn, M, fmt)
        for x in work.back.values():
            _poisoned(x)
        dX, dWg, dWu, dWd = mg.gated_ffn_backward(ffn, saved, dY, work=work)
        b = work.back
        for got, ref in ((b["dy"], mg.f8_checkpoint(dY, fmt)), (b["dyt"], _transposed(b["dy"])), (b["ht"], _transposed(saved.h)),
                         (b["xt"], _transposed(saved.x)), (b["dgut"], _transposed(b["dgu"]))):
            assert_same(got, codes(ref), scales(ref))
        dh, bdh = big_product(values_on_gpu(b["dy"]), wd.t())
        ea, ed = 2.0 ** -20 * g.abs() + 1e-30, 2.0 ** -20 * (1 + g.abs() + d.abs())
        dg, du = dh * u * d, dh * a
        bg = u.abs() * (bdh * (d.abs() + ed) + dh.abs() * ed) + 2.0 ** -22 * dg.abs()
        bu = bdh * (a.abs() + ea) + dh.abs() * ea + 2.0 ** -22 * du.abs()
        big_q(b["dgu"], interleaved(dg, du), interleaved(bg, bu), "dgu")
        big_close(dX, *big_product(values_on_gpu(b["dgu"]), w13.t(), "bf16"), "bf16")
        ref, bound = big_product(values_on_gpu(b["dgut"]), values_on_gpu(b["xt"]))
        for got, v, e in zip((dWg, dWu), halves(ref.t(), F), halves(bound.t(), F)):
            big_close(got, v.t(), e.t())
        big_close(dWd, *big_product(values_on_gpu(b["dyt"]), values_on_gpu(b["ht"])))
