"""The sizes of the GPU tests take every kernel of the 8-bit products (on the CPU: the rule is host code)."""
from tests.f8_forms import FORMS, GATED, PAIRS, TILES, fused, tile


def up(n, to):
    return -(-n // to) * to


def test_sizes_take_their_kernels():
    for want, out, M, K, N in FORMS:
        assert tile(M, K, N, out) == want, (out, M, K, N)
    for want, out, F, T, K in PAIRS:
        assert tile(2 * up(F, 128), up(T, 32), K, out) == want, (out, F, T, K)
    for M, K, F, N in GATED:
        assert fused(M, F, K)[:2] == (True, True) and fused(M, F, N)[2], (M, K, F, N)


def test_every_kernel_has_a_size():
    assert {(t, out) for t, out, *_ in FORMS} == {(t, out) for t in TILES for out in ("bf16", "f32")} - {("192 x 256", "f32")}


def test_no_size_takes_the_192_row_tiles_into_f32():
    """They are not built for it."""
    sizes = [1, 33, 130, 515, 777, 1560, 2055, 4100, 8200, 32760]
    widths = [32, 160, 1056, 1568, 5120, 13824]
    assert all(tile(M, K, N, "f32") != "192 x 256" for M in sizes for K in widths for N in widths)
