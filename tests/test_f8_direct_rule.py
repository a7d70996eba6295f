"""Few rows go straight from their activations where that was measured to be faster (on the CPU: the
rule is host code; times in us on a device of 256 CUs, weights from memory, in a graph)."""
import pytest

from tests.f8_forms import gated_direct, linear_direct

# rows, K, N, direct, in two launches: more than 5 % apart
LINEAR = [
    (1, 5120, 13824, 15.1, 17.1), (2, 5120, 13824, 15.9, 17.5), (5, 5120, 13824, 18.8, 17.5), (8, 5120, 13824, 21.2, 17.5),
    (1, 13824, 5120, 17.5, 20.1), (2, 13824, 5120, 19.1, 20.3), (4, 5120, 5120, 10.1, 10.7), (8, 5120, 5120, 12.6, 10.8),
    (16, 1024, 1056, 5.2, 6.2), (16, 1024, 8192, 6.1, 6.8), (8, 1024, 13824, 7.1, 7.9), (8, 1024, 27648, 11.6, 10.1),
    (1, 1024, 55296, 16.0, 14.7), (16, 1024, 55296, 24.4, 15.8), (16, 1024, 131072, 49.6, 29.9), (10, 2048, 13824, 10.8, 10.3),
    (14, 2048, 13824, 12.1, 10.4), (2, 2048, 27648, 13.4, 14.9), (14, 2048, 131072, 77.5, 51.8), (5, 5120, 27648, 34.4, 29.7),
    (1, 5120, 55296, 51.8, 57.6), (5, 5120, 55296, 60.3, 56.4),
]
# rows, K, F, N
GATED = [
    (1, 5120, 13824, 5120, 47.0, 49.9), (1, 1024, 1024, 1024, 8.4, 12.7), (16, 1024, 1024, 1024, 11.8, 13.8),
    (13, 1024, 4096, 1024, 19.5, 17.4), (4, 1024, 13824, 1024, 27.9, 29.9), (16, 1024, 1024, 13824, 15.5, 16.6),
    (16, 1024, 1024, 55296, 32.4, 23.9), (16, 2048, 2048, 55296, 50.0, 36.0), (7, 5120, 5120, 5120, 30.0, 26.9),
    (11, 5120, 1024, 5120, 22.3, 18.7), (2, 5120, 13824, 55296, 165.9, 174.9),
]


@pytest.mark.parametrize("M,K,N,direct,two", LINEAR)
def test_layer(M, K, N, direct, two):
    assert linear_direct(M, K, N) == (direct < two)


@pytest.mark.parametrize("M,K,F,N,direct,apart", GATED)
def test_gated_block(M, K, F, N, direct, apart):
    assert gated_direct(M, K, F, N) == (direct < apart)


def test_what_does_not_fit():
    """More rows than the kernel takes, or whose codes do not fit its LDS."""
    assert linear_direct(16, 1024, 1024) and not linear_direct(17, 32, 32)
    assert not linear_direct(1, 1 << 20, 32) and not gated_direct(1, 32, 65536, 32)
