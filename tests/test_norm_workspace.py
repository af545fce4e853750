"""The norm gradient's workspace sizes (CPU): what a larger shape asks for holds the
partial rows that a smaller one cannot do without."""
import random

from quantized_int8_gemm_amd import _binding as b

size = b.lib.rms_norm_grad_workspace_bytes


def test_a_larger_shape_asks_for_enough():
    rng = random.Random(7)
    edge = [1, 2, 4, 16, 127, 128, 129, 255, 256, 257, 511, 512, 513, 767, 768, 769, 1023, 1024, 1025, 2047, 2048, 2049, 4096, 8191,
            8192, 8193, 16384, 16385, 30000, 65536]
    shapes = [(m, n) for m in edge for n in edge] + [(rng.randrange(1, 40000), rng.randrange(1, 65537)) for _ in range(1000)]
    shapes += [(rng.randrange(1, 40000), rng.randrange(1, 1200)) for _ in range(1000)]
    least = {}
    for m, n in shapes:
        assert size(m, n) % (4 * n) == 0 and 1 <= size(m, n) // (4 * n) <= min(m, 512)
        least[m, n] = min(size(m, n), 256 * 4 * n)
    for m, n in shapes:
        for _ in range(20):
            big_m, big_n = rng.choice(shapes)
            if big_m >= m and big_n >= n:
                assert size(big_m, big_n) >= least[m, n], (m, n, big_m, big_n)
        for big in ((m + 1, n), (2 * m, n), (m, min(65536, n + 1)), (m, min(65536, 2 * n))):
            assert size(*big) >= least[m, n], (m, n, big)
