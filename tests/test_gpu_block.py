"""The operators around the block (norm + modulation, gated residual + norm,
norm + quantize, the dual GEMM's epilogue) against the float64 oracle.

Bounds.  u = 2^-24.  A sum of K terms formed with at most D additions in a row
is off by at most D u sum|x|, so the mean by D u A (A = mean|x|), the variance
by a relative (D + 6) u plus (D u A)^2, and each further operation adds one u;
`norm_bound` adds these up per element.  An output rounded to bf16 may be
another 2^-8 of itself away.  D follows from the kernel's layout: 8 V values
per thread, 6 steps in the wave, W waves.
"""
import ctypes

import numpy as np
import pytest
import torch

import mixed_gemm_amd as mg
import synth
from oracle import block
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _depth(K):
    nw = -(-K // 512)
    V = -(-nw // 8)
    V = V if V <= 4 else 8
    return 8 * V + 6 + -(-nw // V)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def norm_bound(x, n, a, c, K, kind, eps):
    """Absolute error of a f32 evaluation of n a + c (n the norm of x in f64, a
    and c the folded weights, c already in absolute values)."""
    D = _depth(K)
    A = np.abs(x).mean(axis=1, keepdims=True)
    mean = x.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    off = D * U * A * rstd if kind == "layer" else 0.0
    dn = off + np.abs(n) * (U * (D / 2 + 12) + off ** 2)
    return np.abs(a) * dn + 6 * U * (np.abs(n * a) + c) + 1e-37


def assert_close(got, ref, bound, out, what):
    bound = np.asarray(bound) + (2.0 ** -8 * (np.abs(ref) + bound) if out == "bf16" else 0.0)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.max(np.abs(got - ref) / bound)} x the bound"


def rows(rng, M, K, dtype, ld=0, mean=0.3, fill=float("nan")):
    """[M][K] view of heavy-tailed rows `K + ld` apart whose gaps hold `fill`, and the base."""
    x = rng.standard_normal((M, K)) + mean * rng.standard_normal(K)
    x[:, rng.permutation(K)[: max(1, K // 50)]] *= 25.0
    base = torch.full((M, K + ld), fill, dtype=TYPES[dtype], device="cuda")
    base[:, :K] = torch.from_numpy(x).to("cuda").to(TYPES[dtype])
    return base[:, :K], base


def out_rows(M, K, dtype, ld):
    """An output [M][K] with guard elements around and between its rows."""
    base = torch.full((M * (K + ld) + 32,), 776.0, dtype=TYPES[dtype], device="cuda")
    return base[16:16 + M * (K + ld)].view(M, K + ld)[:, :K], base


def assert_guards(view, base, M, K, ld):
    full = host(base.float())
    inner = np.zeros(full.size, bool)
    inner[16:16 + M * (K + ld)] = (np.arange(M * (K + ld)) % (K + ld)) < K
    assert (full[~inner] == 776.0).all(), "written outside the rows"


def modulation(rng, R, K, dtype, ld=0):
    e = torch.from_numpy(0.3 * rng.standard_normal((R, 3 * K + ld))).to("cuda").to(TYPES[dtype])
    return e[:, :K], e[:, K:2 * K], e[:, 2 * K:3 * K]


def vec(rng, K, dtype, at=0.0):
    return torch.from_numpy(at + 0.2 * rng.standard_normal(K)).to("cuda").to(TYPES[dtype])


NORM_CASES = [
    # M, K, x, out, kind, affine, modulation, its type, ld
    (1, 1, "f32", "f32", "layer", None, None, "f32", 0),
    (3, 7, "bf16", "f32", "rms", "bf16", "token", "bf16", 0),
    (2, 8, "bf16", "bf16", "layer", "f32", "sample", "f32", 8),
    (300, 31, "f32", "bf16", "layer", None, "token", "f32", 1),
    (2050, 128, "bf16", "bf16", "rms", "bf16", None, "f32", 0),
    (1030, 121, "bf16", "f32", "layer", "f32", "token", "bf16", 7),
    (70, 129, "f32", "f32", "layer", None, "token", "f32", 2),
    (515, 256, "bf16", "bf16", "layer", "bf16", "sample", "f32", 0),
    (70, 257, "f32", "f32", "layer", None, "token", "f32", 2),
    (64, 512, "bf16", "f32", "layer", "bf16", "sample", "bf16", 0),
    (7, 513, "bf16", "f32", "rms", None, "sample", "f32", 3),
    (33, 1537, "bf16", "bf16", "rms", "bf16", "token", "bf16", 9),
    (9, 5120, "f32", "f32", "layer", None, "sample", "f32", 0),
    (530, 5120, "f32", "bf16", "layer", None, "token", "f32", 0),
    (3, 5119, "f32", "f32", "layer", "f32", "sample", "bf16", 0),
    (5, 13824, "bf16", "f32", "layer", "f32", "token", "f32", 8),
    (4, 13817, "f32", "f32", "rms", "bf16", "sample", "f32", 1),
    (2, 40001, "bf16", "f32", "layer", "bf16", "sample", "f32", 0),
    (2, 65536, "f32", "f32", "layer", None, "sample", "f32", 0),
]


def _where(rng, mod, M, R):
    if mod == "token":
        idx = rng.integers(-1, R + 1, M).astype(np.int32)        # -1 and R are padding
        return dict(index=torch.from_numpy(idx).cuda()), block.rows_of(M, R, idx)
    g = -(-M // R)
    return dict(group=g), block.rows_of(M, R, group=g)


@pytest.mark.parametrize("M,K,xt,ht,kind,affine,mod,mt,ld", NORM_CASES)
def test_norm_mod(M, K, xt, ht, kind, affine, mod, mt, ld):
    rng = np.random.default_rng(M * 1000 + K)
    X, _ = rows(rng, M, K, xt, ld)
    w, b = (vec(rng, K, affine, 1.0), vec(rng, K, affine)) if affine else (None, None)
    norm = mg.Norm(kind, w, b, 1e-6)
    m, i, sc, sh = None, np.zeros(M, int), None, None
    if mod:
        R = 3
        sc, sh, _ = modulation(rng, R, K, mt, ld)
        where, i = _where(rng, mod, M, R)
        m = mg.Mod(scale=sc, shift=sh, **where)
    H, base = out_rows(M, K, ht, ld)
    mg.mg_norm_mod(norm, m, X, H)
    torch.cuda.synchronize()
    x = f64(X)
    n0 = block.norm(x, kind)
    ref = block.modulate(block.norm(x, kind, f64(w), f64(b)), i, f64(sc), f64(sh))
    k = np.maximum(i, 0)
    s1 = 1.0 + (f64(sc)[k] if sc is not None else 0.0)
    a = (1.0 if w is None else f64(w)) * s1
    c = np.abs((0.0 if b is None else f64(b)) * s1) + (np.abs(f64(sh)[k]) if sh is not None else 0.0)
    bound = norm_bound(x, n0, a, c, K, kind, 1e-6)
    assert_close(f64(H), ref, bound, ht, "H")
    assert (f64(H)[i < 0] == 0).all()
    assert_guards(H, base, M, K, ld)


def test_norm_mod_only_scale_or_shift_and_in_place():
    rng = np.random.default_rng(5)
    X, _ = rows(rng, 40, 96, "f32")
    sc, sh, _ = modulation(rng, 1, 96, "f32")
    x = f64(X)
    for kw in (dict(scale=sc), dict(shift=sh)):
        H = X.clone()
        mg.mg_norm_mod(mg.Norm(), mg.Mod(**kw), H, H)
        ref = block.modulate(block.norm(x), np.zeros(40, int), f64(kw.get("scale")), f64(kw.get("shift")))
        a = 1.0 + (f64(sc)[0] if "scale" in kw else 0.0)
        c = np.abs(f64(sh)[0]) if "shift" in kw else 0.0
        assert_close(f64(H), ref, norm_bound(x, block.norm(x), a, c, 96, "layer", 1e-6), "f32", str(list(kw)))


@pytest.mark.parametrize("K", [96, 5120, 5121])
def test_norm_of_rows_far_from_zero(K):
    """Rows whose mean is 4096 times their spread: a sum of squares would lose the variance."""
    rng = np.random.default_rng(K)
    X = torch.from_numpy(4096.0 + rng.standard_normal((5, K))).float().cuda()
    H = torch.empty_like(X)
    mg.mg_norm_mod(mg.Norm(), None, X, H)
    x = f64(X)
    n = block.norm(x)
    assert_close(f64(H), n, norm_bound(x, n, 1.0, 0.0, K, "layer", 1e-6), "f32", "H")
    assert norm_bound(x, n, 1.0, 0.0, K, "layer", 1e-6).max() < 0.05


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [8, 100, 129, 255, 257, 513, 1536, 2049, 5120, 8200, 13824, 20000])
def test_constant_rows_are_centred_exactly(K, xt):
    """The sum of up to 2^16 equal values of 8 bits is exact in f32, and the mean is their quotient
    correctly rounded: the value itself.  So the norm is 0, and its output the shift."""
    v = torch.tensor([1.0, 3.0, -100.0, 240.0, 0.0625 * 37, -251.0], device="cuda")
    X = v[:, None].expand(-1, K).contiguous().to(TYPES[xt])
    H, O, Y = torch.empty(6, K, device="cuda"), torch.empty_like(X), torch.zeros_like(X)
    mg.mg_norm_mod(mg.Norm("layer"), None, X, H)
    assert (H == 0).all(), H.abs().amax(1)
    H.fill_(7.0)
    mg.mg_residual_norm(X, Y, O, None, None, mg.Norm("layer"), None, H)
    assert torch.equal(O, X) and (H == 0).all()
    mg.mg_residual_norm(Y, X, O, None, mg.Norm("layer"))
    assert (O == 0).all()
    sh = vec(np.random.default_rng(K), K, "f32")[None]
    mg.mg_norm_mod(mg.Norm("layer"), mg.Mod(scale=sh, shift=sh), X, H)
    assert torch.equal(H, sh.expand(6, K))


@pytest.mark.parametrize("K", [96, 250, 1536, 5120, 5121, 13824])
def test_rows_on_a_grid_far_from_zero(K):
    """bf16 values 99.5, 100, 100.5: the sum is exact, so the mean is off by its rounding alone (u of
    it), and x - mean is exact or off by u of itself."""
    rng = np.random.default_rng(K)
    X = torch.from_numpy(100.0 + 0.5 * rng.integers(-1, 2, (40, K))).cuda().bfloat16()
    H = torch.empty(40, K, device="cuda")
    mg.mg_norm_mod(mg.Norm(), None, X, H)
    x = f64(X)
    n, mean = block.norm(x), x.mean(axis=1, keepdims=True)
    rstd = 1 / np.sqrt(x.var(axis=1, keepdims=True) + 1e-6)
    # the variance: (D + 6) u relative, and the square of the means' errors
    bound = rstd * U * np.abs(mean) + np.abs(n) * (U * (_depth(K) / 2 + 12) + (4 * U * 100 * rstd) ** 2)
    assert_close(f64(H), n, bound, "f32", "H")


def test_constant_zero_and_extreme_rows():
    K = 200
    X = torch.zeros(5, K, device="cuda")
    X[1] = 3.0
    X[2] = torch.linspace(-1e-20, 1e-20, K)
    X[3] = torch.linspace(-1e15, 1e15, K)
    X[4, 7] = 1.0
    H = torch.empty_like(X)
    mg.mg_norm_mod(mg.Norm("layer"), None, X, H)
    x = f64(X)
    n = block.norm(x)
    assert_close(f64(H), n, norm_bound(x, n, 1.0, 0.0, K, "layer", 1e-6), "f32", "H")
    assert (f64(H)[0] == 0).all()


def test_nan_and_infinity_stay_in_their_row_and_out_of_padding():
    K, M = 600, 6
    rng = np.random.default_rng(3)
    X, _ = rows(rng, M, K, "f32")
    Y, _ = rows(rng, M, K, "bf16")
    X[1, 599] = float("nan")
    X[3, 0] = float("inf")
    X[4, 5] = float("nan")                     # padding
    Y[5, 7] = float("inf")                     # padding
    sc, sh, ga = modulation(rng, 2, K, "f32")
    idx = torch.tensor([0, 1, 0, 1, -1, 2], dtype=torch.int32, device="cuda")
    m = mg.Mod(scale=sc, shift=sh, gate=ga, index=idx)
    H = torch.empty(M, K, device="cuda")
    mg.mg_norm_mod(mg.Norm(), m, X, H)
    h = f64(H)
    assert np.isnan(h[1]).all() and not np.isfinite(h[3]).any()
    assert np.isfinite(h[[0, 2]]).all() and (h[[4, 5]] == 0).all()
    O = torch.empty_like(X)
    mg.mg_residual_norm(X, Y, O, m, None, mg.Norm(), m, H)
    o, h = f64(O), f64(H)
    assert np.array_equal(o[4:], f64(X)[4:], equal_nan=True) and (h[4:] == 0).all()
    assert np.isnan(h[1]).all() and np.isfinite(h[[0, 2]]).all()


RES_CASES = [
    # M, K, x, y, out, post, norm, modulation, its type, ld
    (1, 1, "f32", "f32", "f32", False, None, "sample", "f32", 0),
    (17, 5120, "bf16", "bf16", "bf16", False, "layer", "sample", "bf16", 0),
    (70, 5120, "f32", "bf16", "bf16", False, "layer", "token", "f32", 0),
    (29, 2049, "bf16", "bf16", "bf16", True, "rms", "token", "f32", 3),
    (5, 13824, "f32", "f32", "f32", True, "layer", "sample", "bf16", 8),
    (300, 77, "bf16", "f32", "f32", True, None, "token", "bf16", 1),
    (3, 30011, "f32", "bf16", "f32", False, "rms", "sample", "f32", 0),
    (40, 8, "f32", "bf16", "f32", True, "layer", "token", "f32", 0),
    (513, 64, "bf16", "f32", "bf16", True, "rms", "sample", "bf16", 0),
    (600, 103, "f32", "f32", "bf16", False, "layer", "token", "f32", 5),
    (300, 251, "bf16", "bf16", "f32", True, "layer", "token", "f32", 3),
    (2, 65536, "bf16", "bf16", "f32", True, "layer", "sample", "f32", 0),
]


@pytest.mark.parametrize("M,K,xt,yt,ht,post,kind,mod,mt,ld", RES_CASES)
def test_residual_norm(M, K, xt, yt, ht, post, kind, mod, mt, ld):
    rng = np.random.default_rng(M * 77 + K)
    X, _ = rows(rng, M, K, xt, ld)
    Y, _ = rows(rng, M, K, yt, ld)
    sc, sh, ga = modulation(rng, 3, K, mt, ld)
    where, i = _where(rng, mod, M, 3)
    pw = vec(rng, K, "bf16", 1.0) if post else None
    O, obase = out_rows(M, K, xt, ld)
    H, hbase = out_rows(M, K, ht, ld) if kind else (None, None)
    mg.mg_residual_norm(X, Y, O, mg.Mod(gate=ga, **where), mg.Norm("rms", pw) if post else None,
                        mg.Norm(kind) if kind else None, mg.Mod(scale=sc, shift=sh, **where) if kind else None, H)
    torch.cuda.synchronize()
    x, y, k = f64(X), f64(Y), np.maximum(i, 0)
    g = f64(ga)[k]
    p = block.norm(y, "rms", f64(pw)) if post else y
    o = block.gated(x, p, i, f64(ga))
    dp = norm_bound(y, block.norm(y, "rms"), f64(pw), 0.0, K, "rms", 1e-6) if post else 0.0
    do = np.where((i < 0)[:, None], 0.0, np.abs(g) * dp + 2 * U * (np.abs(x) + np.abs(g * p)))
    assert_close(f64(O), o, do + 1e-37, xt, "O")
    pad = i < 0
    assert np.array_equal(f64(O)[pad], x[pad])
    assert_guards(O, obase, M, K, ld)
    if kind:
        n = block.norm(o, kind)
        ref = block.modulate(n, i, f64(sc), f64(sh))
        a = 1.0 + f64(sc)[k]
        mean = o.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
        rstd = 1 / np.sqrt(((o - mean) ** 2).mean(axis=1, keepdims=True) + 1e-6)
        # the sum's own error passes through the norm: its own element's, and the mean's and spread's
        thru = np.abs(a) * rstd * (do + do.mean(axis=1, keepdims=True) + np.abs(n) * np.sqrt((do ** 2).mean(axis=1, keepdims=True)))
        bound = norm_bound(o, n, a, np.abs(f64(sh)[k]), K, kind, 1e-6) + thru
        assert_close(f64(H), ref, bound, ht, "H")
        assert (f64(H)[pad] == 0).all()
        assert_guards(H, hbase, M, K, ld)


def test_residual_in_place_and_plain_sum():
    rng = np.random.default_rng(8)
    X, _ = rows(rng, 50, 640, "bf16")
    Y, _ = rows(rng, 50, 640, "bf16")
    O, H = torch.empty_like(X), torch.empty_like(Y)
    mg.mg_residual_norm(X, Y, O, None, None, mg.Norm(), None, H)
    x, y = X.clone(), Y.clone()
    mg.mg_residual_norm(x, y, x, None, None, mg.Norm(), None, y)
    assert torch.equal(x, O) and torch.equal(y, H)
    assert torch.equal(O, (X.float() + Y.float()).bfloat16())


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(5, 9), (700, 65), (700, 203), (1500, 2049), (1100, 2550), (900, 5121), (700, 8197), (520, 13823)])
def test_partial_vectors_in_place(M, K, xt):
    """Rows that end inside a vector: the same bytes in place, where the row's end is stored apart, as into other memory."""
    rng = np.random.default_rng(K)
    X, _ = rows(rng, M, K, xt)
    Y, _ = rows(rng, M, K, xt)
    sc, sh, g = modulation(rng, 2, K, "f32")
    at = torch.arange(M, dtype=torch.int32, device="cuda") * 2 // M
    at[M // 2] = -1
    mod, gate = mg.Mod(scale=sc, shift=sh, index=at), mg.Mod(gate=g, index=at)
    post = mg.Norm("rms", (1 + 0.2 * torch.randn(K, device="cuda")).bfloat16())
    for p in (None, post):
        O, H = torch.empty_like(X), torch.empty_like(Y)
        mg.mg_residual_norm(X, Y, O, gate, p, mg.Norm(), mod, H)
        x, y = X.clone(), Y.clone()
        mg.mg_residual_norm(x, y, x, gate, p, mg.Norm(), mod, y)
        assert torch.equal(x, O) and torch.equal(y, H)
    x, y = X.clone(), Y.clone()
    mg.mg_residual_norm(x, y, x, gate)
    O = torch.empty_like(X)
    mg.mg_residual_norm(X, Y, O, gate)
    assert torch.equal(x, O)
    H = torch.empty_like(X)
    mg.mg_norm_mod(mg.Norm(), mod, X, H)
    mg.mg_norm_mod(mg.Norm(), mod, x.copy_(X), x)
    assert torch.equal(x, H)


@pytest.mark.parametrize("K", [8, 9, 63, 64, 100, 128, 129, 192, 256, 257, 700])
def test_rows_do_not_depend_on_their_number(K):
    """A row's bits are the same in a call of many rows and of few."""
    rng = np.random.default_rng(K)
    M = 40003 if K <= 257 else 9001
    X, _ = rows(rng, M, K, "bf16")
    Y, _ = rows(rng, M, K, "f32")
    sc, sh, g = modulation(rng, 3, K, "f32")
    at = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    post = mg.Norm("layer", vec(rng, K, "bf16", 1.0), vec(rng, K, "bf16"))

    def run(a, b):
        i = at[a:b].contiguous()
        mod, gate = mg.Mod(scale=sc, shift=sh, index=i), mg.Mod(gate=g, index=i)
        o, h, n = torch.empty_like(X[a:b]), torch.empty_like(Y[a:b]), torch.empty_like(X[a:b])
        mg.mg_residual_norm(X[a:b], Y[a:b], o, gate, post, mg.Norm("rms"), mod, h)
        mg.mg_norm_mod(mg.Norm(), mod, X[a:b], n)
        return o, h, n

    whole = run(0, M)
    for a, b in ((0, 1), (5, 22), (M - 331, M)):
        for w, t in zip(whole, run(a, b)):
            assert torch.equal(w[a:b], t)


QUANT_CASES = [
    # M, K, k, x, kind, affine, modulation, its type, ld
    (1, 5120, 64, "bf16", "layer", None, "sample", "f32", 0),
    (17, 32, 0, "f32", "rms", "bf16", "sample", "f32", 1),
    (33, 352, 5, "bf16", "layer", "f32", "token", "bf16", 3),
    (300, 1568, 40, "f32", "layer", None, "token", "f32", 0),
    (515, 5120, 64, "f32", "layer", None, "sample", "f32", 0),
    (70, 13824, 128, "bf16", "rms", "bf16", "sample", "bf16", 8),
    (9, 16416, 300, "f32", "layer", None, "sample", "f32", 0),
    (3, 65536, 17, "bf16", "layer", None, "token", "f32", 0),
    (40, 544, 544, "bf16", "layer", None, "sample", "f32", 0),
    # enough rows for the form with a row per wave, every number of windows
    (2101, 5120, 64, "f32", "layer", "bf16", "token", "f32", 0),
    (4099, 4640, 33, "bf16", "rms", None, "sample", "bf16", 8),
    (2100, 32, 3, "f32", "layer", "f32", "token", "f32", 1),
    (3333, 1024, 0, "bf16", "layer", None, "token", "bf16", 0),
    (2050, 1376, 300, "f32", "rms", "f32", "sample", "f32", 3),
    (2049, 2048, 17, "bf16", "layer", None, "sample", "f32", 0),
    (2600, 2336, 40, "f32", "layer", None, "sample", "f32", 0),
    (2300, 2592, 5, "bf16", "layer", "bf16", "token", "f32", 0),
    (2200, 3104, 64, "f32", "layer", None, "token", "bf16", 0),
    (2150, 3616, 64, "bf16", "rms", "bf16", "sample", "f32", 0),
    (2500, 4096, 4096, "bf16", "layer", None, "sample", "f32", 0),
]


def _quant_plan(rng, K, N, k, H):
    W = dev(synth.weights(N, K, sigma=0.02, clip=0.6, seed=K + k, bf16=True))
    act_max = H.abs().amax(0).float().clamp(min=1e-3) if H.shape[0] else torch.ones(K, device="cuda")
    return mg.plan(act_max.contiguous(), W, 0.6, k)


@pytest.mark.parametrize("M,K,k,xt,kind,affine,mod,mt,ld", QUANT_CASES)
def test_norm_quantize_is_norm_then_quantize(M, K, k, xt, kind, affine, mod, mt, ld):
    """Every byte, pads included, of mg_norm_mod into bf16 followed by mg_quantize_act."""
    rng = np.random.default_rng(M + K)
    X, _ = rows(rng, M, K, xt, ld)
    w, b = (vec(rng, K, affine, 1.0), vec(rng, K, affine)) if affine else (None, None)
    sc, sh, _ = modulation(rng, 3, K, mt, ld)
    where, _ = _where(rng, mod, M, 3)
    norm, m = mg.Norm(kind, w, b), mg.Mod(scale=sc, shift=sh, **where)
    H = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    mg.mg_norm_mod(norm, m, X, H)
    p = _quant_plan(rng, K, 32, k, H)
    a, f = mg.Act.empty(p.desc, M), mg.Act.empty(p.desc, M)
    for t in (a.Aq, a.As, a.XO, f.Aq, f.As, f.XO):
        t.fill_(0xA5)
    mg.mg_quantize_act(p, H, a)
    mg.mg_norm_quantize_act(p, norm, m, X, f)
    torch.cuda.synchronize()
    for n in ("Aq", "As", "XO"):
        x, y = host(getattr(a, n)), host(getattr(f, n))
        assert np.array_equal(x, y), f"{n}: {int((x != y).sum())} of {x.size} bytes differ"


@pytest.mark.parametrize("M,K", [(40, 1024), (2100, 1024), (300, 5120), (40, 13824)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_quantize_keeps_nan_and_infinity_in_their_rows(M, K, kind):
    """Rows whose norm is not finite have unspecified codes, as in mg_quantize_act; all others have the
    bytes of the two steps, padding rows 0 whatever their input holds."""
    from tests.gpu_util import aq_rows, outlier_cols, scale_rows
    rng = np.random.default_rng(K + M)
    X, _ = rows(rng, M, K, "f32")
    k = 40
    p = _quant_plan(rng, K, 32, k, X.bfloat16())
    X[3, K // 2] = float("nan")
    X[5, 7] = float("inf")
    X[6, K - 1] = -float("inf")
    X[M - 2, 11], X[M - 2, 12] = -float("nan"), float("inf")
    sc, sh, _ = modulation(rng, 4, K, "f32")
    sh[1, 5], sh[1, K - 9] = float("inf"), -float("inf")
    sh[2, p.O[0]], sh[2, 70] = float("nan"), -float("nan")
    at = torch.arange(M, dtype=torch.int32, device="cuda") % 5
    X[at == 4] = float("nan")                                             # padding
    norm, m = mg.Norm(kind), mg.Mod(scale=sc, shift=sh, index=at)
    H = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    mg.mg_norm_mod(norm, m, X, H)
    fine = host(torch.isfinite(H).all(1))
    assert 0 < fine.sum() < M and fine[host(at) == 4].all()
    a, f = mg.Act.empty(p.desc, M), mg.Act.empty(p.desc, M)
    mg.mg_quantize_act(p, H, a)
    mg.mg_norm_quantize_act(p, norm, m, X, f)
    for x, y in zip(*[(aq_rows(z.Aq, M, K), scale_rows(z.As, M, K), outlier_cols(z.XO, M, k)) for z in (a, f)]):
        assert np.array_equal(x[fine], y[fine])
        assert not y[host(at) == 4].any()


@pytest.mark.parametrize("M,K,k,xt", [(2500, 5120, 64, "f32"), (700, 4640, 33, "bf16"), (4099, 2048, 17, "bf16"),
                                      (1100, 32, 3, "f32")])
@pytest.mark.parametrize("where", ["first", "last", "all"])
def test_norm_quantize_of_long_runs_of_padding(M, K, k, xt, where):
    """Workgroups whose first rows are all padding: the bytes of the two steps.  A call with infinite
    scales goes ahead, so that constants left in LDS by it would show as codes other than 0."""
    rng = np.random.default_rng(M + K)
    X, _ = rows(rng, M, K, xt)
    sc, sh, _ = modulation(rng, 3, K, "f32")
    idx = rng.integers(0, 3, M).astype(np.int32)
    run = {"first": slice(0, M - M // 8), "last": slice(M // 8, M), "all": slice(0, M)}[where]
    idx[run] = np.where(rng.random(len(idx[run])) < 0.5, -1, 3)
    norm, m = mg.Norm(), mg.Mod(scale=sc, shift=sh, index=torch.from_numpy(idx).cuda())
    H = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    mg.mg_norm_mod(norm, m, X, H)
    p = _quant_plan(rng, K, 32, k, X.bfloat16())
    a, f = mg.Act.empty(p.desc, M), mg.Act.empty(p.desc, M)
    left = mg.Plan.from_state(p.state())
    left.s = torch.full_like(p.s, float("inf"))
    left.rcp = torch.full_like(p.rcp, float("inf"))
    mg.mg_norm_quantize_act(left, norm, mg.Mod(scale=sc[:1], shift=sh[:1]), X, f)
    for t in (f.Aq, f.As, f.XO):
        t.fill_(0xA5)
    mg.mg_quantize_act(p, H, a)
    mg.mg_norm_quantize_act(p, norm, m, X, f)
    torch.cuda.synchronize()
    for n in ("Aq", "As", "XO"):
        assert torch.equal(getattr(a, n), getattr(f, n)), n
    if where == "all":
        assert not any(t.any() for t in (f.Aq, f.As, f.XO))


@pytest.mark.parametrize("M", [40, 2100])
def test_norm_quantize_with_scales_out_of_the_fast_range(M):
    """Smoothing scales far from 1 and rows of tiny values: the exact division's codes."""
    rng = np.random.default_rng(12)
    K, k = 1024, 24
    X, _ = rows(rng, M, K, "f32")
    X[7] *= 1e-30
    p = _quant_plan(rng, K, 32, k, X.bfloat16())
    s = torch.from_numpy(np.exp2(rng.uniform(-30, 30, K)).astype(np.float32)).cuda()
    s[:512] = torch.from_numpy(np.exp2(rng.uniform(-3, 3, 512)).astype(np.float32)).cuda()
    p.s.copy_(s)
    p.rcp.copy_((1.0 / s.double()).float())
    w = torch.from_numpy(np.exp2(rng.uniform(-90, 0, K)).astype(np.float32)).cuda()
    norm, m = mg.Norm("layer", w), None
    H = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    mg.mg_norm_mod(norm, m, X, H)
    a, f = mg.Act.empty(p.desc, M), mg.Act.empty(p.desc, M)
    mg.mg_quantize_act(p, H, a)
    mg.mg_norm_quantize_act(p, norm, m, X, f)
    for n in ("Aq", "As", "XO"):
        assert np.array_equal(host(getattr(a, n)), host(getattr(f, n))), n


# ------------------------------------------------------------------ epilogue

def decoded(p, a, M):
    """The fp32 sums' float64 value and the sum of their terms' magnitudes, from
    the kernel's own operands (exact decode)."""
    from oracle import mxfp4
    from tests.gpu_util import aq_rows, outlier_cols, scale_rows
    d = p.desc
    A = mxfp4.decode_rows(aq_rows(a.Aq, M, d.K), scale_rows(a.As, M, d.K)).astype(np.float64)
    W = mxfp4.decode_rows(aq_rows(p.Wq, d.N, d.K), scale_rows(p.Ws, d.N, d.K)).astype(np.float64)
    if d.k:
        from tests.gpu_util import bf16_to_f64
        A = np.concatenate([A, bf16_to_f64(outlier_cols(a.XO, M, d.k))], axis=1)
        W = np.concatenate([W, bf16_to_f64(outlier_cols(p.WO, d.N, d.k))], axis=1)
    A, W = torch.from_numpy(A).cuda(), torch.from_numpy(W).cuda()
    return f64(A @ W.t()), f64(A.abs() @ W.abs().t())


EP_CASES = [
    # M, K, N, k, y, bias, act, gate, residual, modulation, its type
    (1, 32, 32, 0, "f32", None, "none", False, None, "sample", "f32"),
    (1, 5120, 1024, 64, "bf16", "bf16", "gelu", False, None, "sample", "f32"),
    (17, 1568, 544, 40, "f32", "f32", "none", True, "f32", "sample", "f32"),
    (31, 13824, 96, 128, "bf16", "bf16", "none", True, "bf16", "token", "bf16"),
    (32, 512, 64, 5, "f32", "bf16", "silu", True, "bf16", "token", "f32"),
    (33, 544, 1056, 544, "f32", "bf16", "gelu", False, None, "sample", "f32"),
    (65, 5120, 160, 0, "bf16", None, "none", True, "f32", "sample", "bf16"),
    (130, 2080, 320, 33, "f32", "f32", "gelu", True, "f32", "token", "f32"),
    (300, 1056, 1312, 64, "bf16", "bf16", "silu", True, "bf16", "sample", "f32"),
    (777, 1568, 1056, 40, "f32", "bf16", "none", True, "f32", "token", "f32"),
    (1100, 640, 288, 16, "f32", None, "gelu", False, "bf16", "sample", "f32"),
    # larger tiles of the few-token form, ragged in both directions, and the 256x256 tiles
    (100, 4128, 4000, 40, "bf16", "f32", "none", True, "bf16", "token", "f32"),
    (515, 4128, 4000, 40, "f32", "bf16", "silu", True, "f32", "sample", "bf16"),
    (1010, 4128, 4000, 96, "bf16", "f32", "gelu", True, "f32", "token", "f32"),
    (2100, 4128, 4000, 5, "bf16", "bf16", "gelu", False, None, "sample", "f32"),
    (2100, 2080, 4000, 33, "f32", "bf16", "none", True, "f32", "sample", "f32"),
    (2050, 2080, 4000, 0, "bf16", "f32", "silu", True, "bf16", "token", "bf16"),
    (2305, 1056, 4000, 17, "f32", None, "none", False, "f32", "sample", "f32"),
    (2560, 1056, 4000, 17, "bf16", "f32", "none", False, "f32", "token", "f32"),
]


@pytest.mark.parametrize("M,K,N,k,yt,bias,act,gate,res,mod,mt", EP_CASES)
def test_gemm_epilogue(M, K, N, k, yt, bias, act, gate, res, mod, mt):
    rng = np.random.default_rng(M + 3 * N + K)
    X, _ = rows(rng, M, K, "bf16")
    p = _quant_plan(rng, K, N, k, X)
    a = mg.Act.empty(p.desc, M)
    mg.mg_quantize_act(p, X, a)
    b = vec(rng, N, bias) if bias else None
    ga = modulation(rng, 3, N, mt, 8)[2] if gate else None
    where, i = _where(rng, mod, M, 3)
    g = mg.Mod(gate=ga, rows=3, **where) if gate or mod == "token" else None
    R = rows(rng, M, N, res, 16)[0] if res else None
    Y = torch.full((M + 1, N), float("nan"), dtype=TYPES[yt], device="cuda")
    Y[M] = 776.0
    mg.mg_dual_gemm_ep(p, a, mg.Epilogue(b, act, g, R), Y[:M])
    Y2 = torch.full((M, N), float("nan"), dtype=TYPES[yt], device="cuda")
    mg.mg_forward_ep(p, X, a, mg.Epilogue(b, act, g, R), Y2)
    torch.cuda.synchronize()
    v, t = decoded(p, a, M)
    ref = block.epilogue(v, i if g is not None else np.zeros(M, int), f64(b), act, f64(ga), f64(R))
    # K + k products summed in any order, then bias; GELU / SiLU: slope at most 1.13, their own
    # evaluation off by (12 + 4 |exponent|) u of the result
    dv = (K + k + 2) * U * t + U * (np.abs(v) + (0 if b is None else np.abs(f64(b))))
    z = v + (0 if b is None else f64(b))
    av = np.abs(block.activation(z, act))
    if act != "none":
        e = np.abs(z) * 1.4427 if act == "silu" else np.abs(2.3022 * z + 0.10295 * z ** 3)
        dv = 1.13 * dv + av * (12 + 4 * e) * U + 1e-37
    gg = 1.0 if ga is None else np.abs(f64(ga)[np.maximum(i, 0)])
    live = (i >= 0)[:, None] if g is not None else True
    dy = np.where(live, gg * dv + 3 * U * gg * av, 0.0) + U * np.abs(ref) + 1e-37
    assert_close(f64(Y[:M]), ref, dy, yt, "Y")
    assert (f64(Y[M]) == 776.0).all()
    assert torch.equal(Y[:M], Y2), "forward_ep is quantize + gemm_ep"
    for _ in range(3):
        Y2.fill_(float("nan"))
        mg.mg_dual_gemm_ep(p, a, mg.Epilogue(b, act, g, R), Y2)
        assert torch.equal(Y[:M], Y2), "the same call gives the same bits"


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_every_form_of_the_large_tiles_epilogue(act, yt, res):
    """A large output of few channels, most of it at memory's rate; each activation, output
    and residual type, with one gate row, one per token, and none."""
    _every_form(act, yt, res, 5000, 512, 2048)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_every_form_of_the_256_wide_tiles_epilogue(act, yt, res):
    """The same at a shape where every form takes the 256x256 tiles."""
    _every_form(act, yt, res, 8190, 1312, 2048)


def _every_form(act, yt, res, M, K, N):
    rng = np.random.default_rng(len(act) + 10 * len(yt))
    X, _ = rows(rng, M, K, "bf16")
    p = _quant_plan(rng, K, N, 7, X)
    a = mg.Act.empty(p.desc, M)
    mg.mg_quantize_act(p, X, a)
    v, t = decoded(p, a, M)
    b = vec(rng, N, "f32")
    ga = modulation(rng, 3, N, "f32")[2]
    R = rows(rng, M, N, res)[0] if res else None
    z = v + f64(b)
    dv = (K + 9) * U * t + U * (np.abs(v) + np.abs(f64(b)))
    av = block.activation(z, act)
    if act != "none":
        e = np.abs(z) * 1.4427 if act == "silu" else np.abs(2.3022 * z + 0.10295 * z ** 3)
        dv = 1.13 * dv + np.abs(av) * (12 + 4 * e) * U + 1e-37
    for mode in ("none", "sample", "token"):
        i, g = np.zeros(M, int), None
        if mode != "none":
            where, i = _where(rng, mode, M, 3)
            g = mg.Mod(gate=ga, **where)
        Y = torch.full((M, N), float("nan"), dtype=TYPES[yt], device="cuda")
        mg.mg_dual_gemm_ep(p, a, mg.Epilogue(b, act, g, R), Y)
        ref = block.gated(np.zeros_like(v) if R is None else f64(R), av, i, f64(ga) if g else None)
        gg = np.abs(f64(ga)[np.maximum(i, 0)]) if g else 1.0
        dy = np.where((i < 0)[:, None], 0.0, gg * dv + 3 * U * gg * np.abs(av)) + U * np.abs(ref) + 1e-37
        assert_close(f64(Y), ref, dy, yt, mode)


FEW_TILES = [(0, 33, 2080, 544), (1, 197, 544, 1312), (2, 515, 1056, 1056), (3, 515, 4128, 2080), (3, 777, 4128, 1312)]


@pytest.mark.parametrize("tile,M,K,N", FEW_TILES)
@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_every_form_of_the_few_token_tiles(tile, M, K, N, yt, res):
    """Each few-token tile, ragged in both directions, with each output and residual type; the size
    has to take the tile (a changed rule asks for another size)."""
    size = {None: 0, "bf16": 2, "f32": 4}
    assert _tile(M, N, K, 7, size[yt] + size[res]) == tile
    _every_form({None: "gelu", "bf16": "silu", "f32": "none"}[res], yt, res, M, K, N)


def test_epilogue_in_place_on_the_residual():
    rng = np.random.default_rng(4)
    for M, yt in ((9, "bf16"), (300, "f32"), (300, "bf16")):
        X, _ = rows(rng, M, 512, "bf16")
        p = _quant_plan(rng, 512, 320, 8, X)
        a = mg.Act.empty(p.desc, M)
        R, _ = rows(rng, M, 320, yt)
        Y = torch.empty_like(R)
        mg.mg_forward_ep(p, X, a, mg.Epilogue(residual=R), Y)
        Z = R.clone()
        mg.mg_forward_ep(p, X, a, mg.Epilogue(residual=Z), Z)
        assert torch.equal(Y, Z), (M, yt)


def test_no_epilogue_is_the_dual_gemm():
    rng = np.random.default_rng(6)
    X, _ = rows(rng, 2100, 1056, "bf16")
    p = _quant_plan(rng, 1056, 1312, 20, X)
    a = mg.Act.empty(p.desc, 2100)
    mg.mg_quantize_act(p, X, a)
    for dt in (torch.float32, torch.bfloat16):
        Y, Z = (torch.empty(2100, 1312, dtype=dt, device="cuda") for _ in range(2))
        mg.mg_dual_gemm(p, a, Y)
        mg.mg_dual_gemm_ep(p, a, None, Z)
        v, t = decoded(p, a, 2100)
        assert_close(f64(Z), v, (1056 + 20) * U * t + 1e-37, "f32" if dt == torch.float32 else "bf16", "Y")


def test_the_dual_gemm_and_its_form_with_an_epilogue():
    """mg_dual_gemm and mg_dual_gemm_ep without an epilogue: the same bits where both take the
    256x256 tiles, else sums of the same products in another order."""
    rng = np.random.default_rng(16)
    for M, K, N, big in ((8190, 1312, 2048, True), (2100, 1056, 1312, False), (33, 5120, 544, False)):
        X, _ = rows(rng, M, K, "bf16")
        p = _quant_plan(rng, K, N, 20, X)
        a = mg.Act.empty(p.desc, M)
        mg.mg_quantize_act(p, X, a)
        _, t = decoded(p, a, M)
        for dt in ("f32", "bf16"):
            Y, Z = (torch.full((M, N), float("nan"), dtype=TYPES[dt], device="cuda") for _ in range(2))
            mg.mg_dual_gemm(p, a, Y)
            mg.mg_dual_gemm_ep(p, a, None, Z)
            assert (_tile(M, N, K, 20, 4 if dt == "f32" else 2) < 0) == big
            if big:
                assert torch.equal(Y, Z)
            other = 2.0 ** -8 * np.abs(f64(Y)) if dt == "bf16" else 0.0      # Y's own rounding, beside Z's
            assert_close(f64(Z), f64(Y), 2 * (K + 20) * U * t + other + 1e-37, dt, "Y")


def test_bf16_results_are_the_f32_results_rounded_once():
    rng = np.random.default_rng(17)
    for M, K, N in ((70, 1536, 96), (700, 5121, 0), (5000, 512, 2048), (300, 200, 0)):
        X, _ = rows(rng, M, K, "bf16")
        m = mg.Mod(**dict(zip(("scale", "shift"), modulation(rng, 1, K, "f32")[:2])))
        H = {t: torch.empty(M, K, dtype=TYPES[t], device="cuda") for t in TYPES}
        for h in H.values():
            mg.mg_norm_mod(mg.Norm(), m, X, h)
        assert torch.equal(H["f32"].bfloat16(), H["bf16"])
        if N:
            p = _quant_plan(rng, K, N, 9, X)
            a = mg.Act.empty(p.desc, M)
            mg.mg_quantize_act(p, X, a)
            R, b = rows(rng, M, N, "f32")[0], vec(rng, N, "f32")
            Y = {t: torch.empty(M, N, dtype=TYPES[t], device="cuda") for t in TYPES}
            assert _tile(M, N, K, 9, 6) == _tile(M, N, K, 9, 8)          # the same order of sums
            for y in Y.values():
                mg.mg_dual_gemm_ep(p, a, mg.Epilogue(b, "gelu", None, R), y)
            assert torch.equal(Y["f32"].bfloat16(), Y["bf16"])


def _tile(M, N, K, k, nbytes):
    """The GEMM's form by the rule that chooses it: 0 ... 3 the few-token tiles (32 x 32, 32 x 64,
    64 x 64, 64 x 96), -1 the 256x256 tiles."""
    f = mg.lib()["_ZN2mg8few_tileEliiii"]
    f.argtypes, f.restype = [ctypes.c_int64] + 4 * [ctypes.c_int32], ctypes.c_int32
    return f(M, N, K, k, nbytes)


def test_zero_rows_launch_nothing():
    p = _quant_plan(np.random.default_rng(0), 64, 32, 4, torch.ones(1, 64, device="cuda"))
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    a = mg.Act.empty(p.desc, 0)
    mg.mg_norm_mod(mg.Norm(), None, X, X)
    mg.mg_residual_norm(X, X, X)
    mg.mg_norm_quantize_act(p, mg.Norm(), None, X, a)
    mg.mg_forward_ep(p, X, a, None, torch.empty(0, 32, device="cuda"))
    torch.cuda.synchronize()


def test_on_another_stream():
    rng = np.random.default_rng(9)
    X, _ = rows(rng, 64, 512, "bf16")
    p = _quant_plan(rng, 512, 64, 8, X)
    a = mg.Act.empty(p.desc, 64)
    Y, Z, H, H2 = (torch.empty(64, n, device="cuda") for n in (64, 64, 512, 512))
    mg.mg_norm_mod(mg.Norm(), None, X, H)
    mg.mg_forward_ep(p, X, a, mg.Epilogue(act="gelu"), Y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mg.mg_norm_mod(mg.Norm(), None, X, H2, stream=s)
    mg.mg_forward_ep(p, X, a, mg.Epilogue(act="gelu"), Z, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(H, H2) and torch.equal(Y, Z)


def test_replayed_in_a_graph():
    """norm + quantize -> GEMM with epilogue -> residual captured once and replayed on new inputs."""
    rng = np.random.default_rng(10)
    M, K, N = 70, 512, 512
    X, _ = rows(rng, M, K, "bf16")
    p = _quant_plan(rng, K, N, 8, X)
    a = mg.Act.empty(p.desc, M)
    sc, sh, ga = modulation(rng, 1, K, "f32")
    b = vec(rng, N, "bf16")
    Y, O = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(X)

    def step():
        mg.mg_norm_quantize_act(p, mg.Norm(), mg.Mod(scale=sc, shift=sh), X, a)
        mg.mg_dual_gemm_ep(p, a, mg.Epilogue(b, "silu"), Y)
        mg.mg_residual_norm(X, Y, O, mg.Mod(gate=ga))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(5):
        X.copy_(rows(np.random.default_rng(100 + seed), M, K, "bf16")[0])
        O.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = O.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, O), seed


# ------------------------------------------------------- the path end to end

@pytest.mark.parametrize("M,dt", [(1, "bf16"), (40, "f32"), (700, "bf16"), (2600, "f32")])
def test_ffn_sublayer_on_unquantized_plans(M, dt):
    """The whole path -- attention residual, norm, both projections with biases,
    gate and residual -- on plans that keep every channel in bf16, against
    float64.  Each rounding to bf16 on the way (h, ffn.0's output, its GELU) is
    at most 2^-8 of its value and passes through the weights in absolute value;
    a value's f32 error is far below one such rounding, which is counted twice."""
    rng = np.random.default_rng(M)
    K, N = 256, 512
    x, _ = rows(rng, M, K, dt)
    attn, _ = rows(rng, M, K, "bf16")
    W0, W2 = (torch.from_numpy(rng.standard_normal(s) * 0.05).cuda().bfloat16() for s in ((N, K), (K, N)))
    b0, b2 = vec(rng, N, "bf16"), vec(rng, K, "f32")
    sc, sh, ga = modulation(rng, 2, K, "f32")
    where, i = _where(rng, "token" if M > 40 else "sample", M, 2)
    m = mg.Mod(scale=sc, shift=sh, gate=ga, **where)
    sub = mg.FFNSublayer(mg.FFNBlock(mg.reference_plan(W0), mg.reference_plan(W2)), mg.Norm(), b0, b2)
    out = mg.ffn_sublayer_forward(sub, x, m, attn, m)
    r = 2.0 ** -8
    x1 = block.gated(f64(x), f64(attn), i, f64(ga))
    dx = np.abs(x1) * (r if dt == "bf16" else 4 * U) + 1e-37
    h = block.modulate(block.norm(x1), i, f64(sc), f64(sh))
    rstd = 1 / np.sqrt(x1.var(axis=1, keepdims=True) + 1e-6)
    k = np.maximum(i, 0)
    n = np.abs(block.norm(x1))
    dh = np.abs(1 + f64(sc)[k]) * rstd * (dx + dx.mean(axis=1, keepdims=True) + n * np.sqrt((dx ** 2).mean(axis=1, keepdims=True)))
    dh = np.where((i < 0)[:, None], 0.0, dh * (1 + 4 * r) + 2 * r * np.abs(h))
    y = h @ f64(W0).T + f64(b0)
    dy = dh @ np.abs(f64(W0)).T + 2 * r * np.abs(y) + 1e-6
    g = block.activation(y, "gelu")
    dg = 1.13 * dy + 2 * r * np.abs(g) + 2.0 ** -24
    v = g @ f64(W2).T + f64(b2)
    dv = dg @ np.abs(f64(W2)).T + 1e-6
    ref = block.gated(x1, v, i, f64(ga))
    bound = dx + np.where((i < 0)[:, None], 0.0, np.abs(f64(ga)[k]) * dv * (1 + r)) + 4 * U * np.abs(ref)
    assert_close(f64(out), ref, bound, dt, "out")
    assert out.dtype == x.dtype


def test_ffn_sublayer_quantized():
    """Calibrated W4A4 plans: the path is its public steps, bit for bit, and the statistics are the steps'."""
    rng = np.random.default_rng(77)
    K, N, M = 512, 1024, 300
    W0, W2 = (torch.from_numpy(rng.standard_normal(s) * 0.03).cuda().bfloat16() for s in ((N, K), (K, N)))
    b0, b2 = vec(rng, N, "f32"), vec(rng, K, "bf16")
    sc, sh, ga = modulation(rng, 1, K, "bf16")
    m, norm = mg.Mod(scale=sc, shift=sh, gate=ga), mg.Norm("rms", vec(rng, K, "bf16", 1.0))
    xs = [rows(rng, M, K, "f32")[0] for _ in range(3)]
    act0, act2 = mg.ffn_sublayer_stats([(x, m) for x in xs], W0, norm, b0)
    hs = [torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in xs]
    for x, h in zip(xs, hs):
        mg.mg_norm_mod(norm, m, x, h)
    assert torch.equal(act0, torch.stack([h.abs().amax(0) for h in hs]).amax(0).float())
    blk = mg.ffn_block_plans(act0, act2, W0, W2, 0.6, 8, 0.5, 16)
    out = mg.ffn_sublayer_forward(mg.FFNSublayer(blk, norm, b0, b2), xs[0], m)
    a0, a2 = mg.Act.empty(blk.plan0.desc, M), mg.Act.empty(blk.plan2.desc, M)
    y0, want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(xs[0])
    mg.mg_forward_ep(blk.plan0, hs[0], a0, mg.Epilogue(b0), y0)
    mg.mg_gelu_quantize_act(blk.plan2, y0, a2)
    mg.mg_dual_gemm_ep(blk.plan2, a2, mg.Epilogue(b2, gate=m, residual=xs[0]), want)
    assert torch.equal(out, want)
    y = torch.nn.functional.gelu(hs[0].double() @ W0.double().t() + b0.double(), approximate="tanh")
    ref = xs[0].double() + ga.double() * (y @ W2.double().t() + b2.double())
    assert ((out - ref).norm() / (ref - xs[0]).norm()).item() < 0.5     # 4 bits: a coarse check of the wiring


@pytest.mark.parametrize("M", [90, 2300])
def test_sublayer_statistics_leave_padding_out(M):
    """ffn.2's maxima are those of gelu(h W0^T + bias0) over the live tokens, where the hidden row of
    a padding token, gelu(bias0), would exceed them.  h's rounding to bf16 (2^-8 of its value, counted
    twice for the f32 error below it) passes through W0, the hidden value is rounded to bf16 once more."""
    rng = np.random.default_rng(M)
    K, N = 256, 512
    # W0 < 0 and h > 0 in the mean: every live token's hidden row lies below the bias alone
    W0 = torch.from_numpy(-np.abs(rng.standard_normal((N, K))) * 0.01).cuda().bfloat16()
    b0 = torch.from_numpy(8.0 + rng.random(N)).float().cuda()
    sc, sh, _ = modulation(rng, 2, K, "f32")
    sh.abs_().add_(2.0)
    x, _ = rows(rng, M, K, "f32")
    idx = rng.integers(-1, 3, M).astype(np.int32)
    i = block.rows_of(M, 2, idx)
    m = mg.Mod(scale=sc, shift=sh, index=torch.from_numpy(idx).cuda())
    act0, act2 = mg.ffn_sublayer_stats([(x, m)], W0, mg.Norm(), b0)
    h = block.modulate(block.norm(f64(x)), i, f64(sc), f64(sh))[i >= 0]
    v = h @ f64(W0).T + f64(b0)
    g = np.abs(block.activation(v, "gelu"))
    r = 2.0 ** -8
    dg = 1.13 * (2 * r * np.abs(h)) @ np.abs(f64(W0)).T + 1e-4
    top = g.max(axis=0)
    bound = dg.max(axis=0) * (1 + r) + r * top
    assert_close(f64(act2), top, bound, "f32", "act2")
    assert (block.activation(f64(b0), "gelu") > top + 2 * bound).all(), "the case would not show the padding"
    assert np.abs(f64(act0) - np.abs(h).max(axis=0)).max() <= 2 * r * np.abs(h).max()


# ------------------------------------------------------------------ refusals

def test_binding_refuses_what_does_not_fit():
    X = torch.zeros(4, 64, device="cuda")
    H = torch.zeros(4, 64, device="cuda")
    V = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    bad = pytest.raises((ValueError, mg.MGError))
    with bad:
        mg.mg_norm_mod(mg.Norm(weight=V(63)), None, X, H)
    with bad:
        mg.mg_norm_mod(mg.Norm(), mg.Mod(scale=torch.zeros(1, 32, device="cuda")), X, H)
    with bad:
        mg.mg_norm_mod(mg.Norm(), mg.Mod(scale=torch.zeros(1, 64, device="cuda"), index=V(3).int()), X, H)
    with bad:
        mg.mg_norm_mod(mg.Norm(), mg.Mod(scale=torch.zeros(1, 64, device="cuda"), group=2), X, H)   # 2 groups, 1 row
    with bad:
        mg.mg_norm_mod(mg.Norm(), None, X, H[:3])
    with bad:
        mg.mg_norm_mod(mg.Norm(), None, X.t(), X.t())                  # columns are not consecutive
    with bad:
        mg.mg_norm_mod(mg.Norm(), None, X, H.cpu())
    with bad:
        mg.mg_norm_mod(mg.Norm(), None, X, H.double())
    with bad:
        mg.mg_norm_mod(mg.Norm(), None, X, X[:1].expand(4, 64))        # overlapping rows
    with bad:
        mg.mg_residual_norm(X, H, H.bfloat16())                        # O of another type than X
    with bad:
        mg.mg_residual_norm(X, H, H, mod=mg.Mod(scale=torch.zeros(1, 64, device="cuda")))
    with bad:
        mg.Norm("batch")
    with bad:
        mg.Mod()
    with bad:
        mg.Epilogue(act="tanh")
    with bad:
        mg.Mod(scale=torch.zeros(2, 64, device="cuda"), shift=torch.zeros(3, 64, device="cuda"))
    p = _quant_plan(np.random.default_rng(0), 64, 32, 4, X + 1)
    a, Y = mg.Act.empty(p.desc, 4), torch.empty(4, 32, device="cuda")
    with bad:
        mg.mg_forward_ep(p, X, a, mg.Epilogue(bias=V(31)), Y)
    with bad:
        mg.mg_forward_ep(p, X, a, mg.Epilogue(residual=torch.zeros(5, 32, device="cuda")), Y)
    with bad:
        mg.mg_forward_ep(p, X, a, mg.Epilogue(residual=torch.zeros(4, 36, device="cuda")[:, :32]), Y)  # ldr % 8
    with bad:
        mg.mg_forward_ep(p, X, a, mg.Epilogue(bias=V(33)[1:]), Y)      # not 16-byte aligned
    with bad:
        mg.mg_norm_quantize_act(p, mg.Norm(), None, H[:3], a)
    torch.cuda.synchronize()
