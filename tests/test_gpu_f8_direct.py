"""The gated block of a few rows, which goes straight from its activations in two launches, against the
float64 oracle, launch by launch, and the sizes just beyond, which do not.

The first launch leaves the hidden activation in fp32 at the start of scratch, the
second rounds it to 8 bits on its way in; beyond, its codes are in the workspace's h.
"""
import functools

import numpy as np
import pytest
import torch

import mixed_gemm_amd as mg
from oracle import f8 as of8
from tests.f8_forms import gated_direct, linear_direct
from tests.f8_util import value
from tests.test_gpu_f8 import TYPES, assert_close, assert_q, f64, hidden, product, rows

# (rows, K, F, N, whether they go direct): F with and without a remainder, several blocks of K and of F
SIZES = [(1, 64, 32, 32, True), (1, 288, 416, 96, True), (2, 1056, 1056, 160, True), (4, 288, 1184, 544, True),
         (7, 1056, 544, 64, True), (16, 544, 1056, 160, True), (9, 4128, 2080, 96, True), (13, 4128, 2080, 96, False),
         (16, 2080, 2848, 64, False), (16, 288, 544, 32800, False), (3, 288, 544, 32800, True), (17, 288, 416, 96, False)]


def test_sizes_take_their_path():
    for M, K, F, N, direct in SIZES:
        assert gated_direct(M, K, F, N) == direct, (M, K, F, N)


def hidden_close(h, x, wg, wu, act):
    ref, bound = hidden(x, wg, wu, act)[2]
    assert_close(h, ref, bound)


@functools.lru_cache(maxsize=1)
def weights(K, F, N):
    """A block's weights, and the values of their codes."""
    rng = np.random.default_rng(K + F + N)
    W = rows(rng, F, K, size=0.05), rows(rng, F, K, size=0.05), rows(rng, N, F, size=0.05)
    return W, tuple(of8.qw(f64(w)) for w in W)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("dtype,ld", [("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 3)])
@pytest.mark.parametrize("M,K,F,N,direct", SIZES)
def test_gated_block_of_few_rows(M, K, F, N, direct, dtype, ld, act):
    rng = np.random.default_rng(M + K + F + ld)
    X = rows(rng, M, K, dtype, ld)
    W, (wg, wu, wd) = weights(K, F, N)
    ffn = mg.gated_ffn(*W, act)
    work = mg.GatedWork.empty(ffn, M)
    x = of8.q(f64(X))
    bias = torch.from_numpy(rng.standard_normal(N)).float().cuda()
    gate = torch.from_numpy(rng.standard_normal((2, N))).to(torch.bfloat16).cuda()
    index = torch.from_numpy(rng.integers(-1, 2, M).astype(np.int32)).cuda()
    i = index.cpu().numpy()
    gr = np.where(i[:, None] >= 0, f64(gate)[i], 0.0)

    def codes_of_h():
        if not direct:
            ref, bound = hidden(x, wg, wu, act)[2]
            assert_q(work.h, ref, bound, "hidden")
            return value(work.h)
        h = f64(work.scratch[: 4 * M * F].view(torch.float32).reshape(M, F))
        hidden_close(h, x, wg, wu, act)
        assert (work.scratch[4 * M * F:] == 0xFF).all() and (work.h.q == 0x55).all()
        return of8.q(h)

    for out in ("f32", "bf16"):
        work.scratch.fill_(0xFF), work.h.q.fill_(0x55)                # (NaN in either)
        base = torch.full((M + 1, N), 7.0, dtype=TYPES[out], device="cuda")
        mg.gated_ffn_forward(ffn, X, Y=base[:M], work=work)
        ref, bound = product(codes_of_h(), wd, out)
        assert_close(f64(base[:M]), ref, bound, out)
        assert (base[M] == 7.0).all()
        # bias, gate rows with padding tokens, and a residual whose rows are apart
        res = rows(rng, M, N, out, 8)
        y = mg.gated_ffn_forward(ffn, X, Y=torch.empty(M, N, dtype=TYPES[out], device="cuda"), work=work,
                                 ep=mg.Epilogue(bias, "none", mg.Mod(gate=gate, index=index), res))
        v = ref + f64(bias)
        b = bound + 2.0 ** -23 * np.abs(v)
        r = f64(res) + gr * v
        assert_close(f64(y), r, np.abs(gr) * b + 2.0 ** -22 * (np.abs(r) + np.abs(gr * v)), out)


def test_exchanged_groups_would_show():
    """Gate and up rows exchanged from the second tile of 32 channels on leave the bound of h."""
    rng = np.random.default_rng(1)
    x, wg, wu = (of8.q(rng.standard_normal(s)) for s in ((2, 1056), (416, 1056), (416, 1056)))
    right = hidden(x, wg, wu, "silu")[2][0]
    with pytest.raises(AssertionError, match="off"):
        hidden_close(right, x, np.concatenate([wg[:32], wu[32:]]), np.concatenate([wu[:32], wg[32:]]), "silu")
    hidden_close(right, x, wg, wu, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3])
def test_few_rows_replayed(M):
    """A layer and a block straight from their activations, captured: replays with new inputs, between eager
    calls of the same workspace, give the eager bits."""
    K, F, N = 1056, 544, 160
    W, _ = weights(K, F, N)
    plan, ffn = mg.f8_plan(W[0]), mg.gated_ffn(*W, "silu")
    assert linear_direct(M, K, F) and gated_direct(M, K, F, N)
    act, work = mg.F8.empty(M, K), mg.GatedWork.empty(ffn, M)
    rng = np.random.default_rng(M)
    x, xs = rows(rng, M, K).contiguous(), [rows(rng, M, K).contiguous() for _ in range(4)]
    y, z = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (F, N))

    def step(a, b):
        mg.f8_forward(plan, x, act=act, Y=a)
        mg.gated_ffn_forward(ffn, x, Y=b, work=work)

    step(y, z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(y, z)
    want = []
    for v in xs:
        x.copy_(v)
        a, b = torch.empty_like(y), torch.empty_like(z)
        step(a, b)
        want.append((v, a, b))
    for v, a, b in want + want[:2]:
        x.copy_(v)
        y.fill_(float("nan")), z.fill_(float("nan"))
        g.replay()
        step(torch.empty_like(y), torch.empty_like(z))
        torch.cuda.synchronize()
        assert torch.equal(y, a) and torch.equal(z, b)
