"""Scales of the 8-bit product at the ends of their range, in every tiling."""
import pytest

from product_cases import OUT, TILINGS, block_sums, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E(cuda):
    import error_compensated_bit_echo_amd as E
    E.load_library()
    return E


def generator(cuda, seed):
    import torch
    g = torch.Generator(device=cuda)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("last", [True, False])
def test_infinite_fp32_scales(E, cuda, tiling, out, block, last):
    """A block of an infinite scale, or of scales whose product is beyond fp32, gives an infinity
    of the sign of its sum (NaN where that is 0) in its row or column, and nothing elsewhere:
    in the last block, behind which groups that share k may have steps left, as in the first."""
    import torch
    M, N, K, P = TILINGS[tiling]
    at = (K - 1) // 128 if last else 0
    g = generator(cuda, 3)
    A = [operand(g, M, K, "e4m3", "f32", 1) for _ in range(P)]
    W = [operand(g, N, K, "e4m3", "f32", block) for _ in range(P)]
    inf = float("inf")
    for r in range(P):
        A[r][1][0, at] = inf
        A[r][1][1, at] = 2.0 ** 100  # only with the scales of W that follow does its product overflow
        W[r][1][-1, at] = 2.0 ** 100
    got = [torch.zeros(M, N, dtype=OUT[out], device=cuda) for _ in range(P)]
    E.echo_gemm_fp8(A, W, got)
    for r in range(P):
        s = block_sums(A[r], W[r])
        sa, sw = A[r][1].float(), W[r][1].float()
        if block == 128:
            sw = sw.repeat_interleave(128, 0)[:N]
        want = torch.zeros(M, N, dtype=torch.float64, device=cuda)
        for b, x in enumerate(s):
            want += x * (sa[:, b, None] * sw[None, :, b]).double()
        # finite elements of the last rows of W are near 2^100 times a whole number: the rest is rounded away
        special = want.abs() > 2.0 ** 60
        finite = want.isfinite() & ~special
        assert torch.equal(got[r].isnan(), want.isnan())
        assert torch.equal(got[r].isinf(), want.isinf())
        assert torch.equal(got[r].sign()[want.isinf()].double(), want.sign()[want.isinf()])
        assert torch.equal(got[r][finite], want[finite].to(OUT[out]))
        assert bool(want.isinf().any()) and bool(finite.any())
