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


def pinned(cuda, seed, rows, k, values, exponent, scale, fmt="e4m3"):
    """Random codes out of `values` under one scale 2^exponent."""
    import torch
    from product_cases import codes_of
    g = generator(cuda, seed)
    v = torch.tensor(values, device=cuda)[torch.randint(len(values), (rows, k), generator=g, device=cuda)]
    kb = -(-k // 128)
    if scale == "e8m0":
        s = torch.full((kb, rows), exponent + 127, dtype=torch.uint8, device=cuda).view(torch.float8_e8m0fnu)
    else:
        s = torch.full((kb, rows), 2.0 ** exponent, device=cuda)
    return codes_of(v, fmt), s.t()


def assert_ends(E, cuda, tiling, scale, out, low, high, fmt="e4m3"):
    """Codes `low[0]` under 2^low[1] against codes `high[0]` under 2^high[1], on either side."""
    import torch
    from product_cases import exact
    M, N, K, P = TILINGS[tiling]
    for swap in (False, True):
        (va, ea), (vw, ew) = (high, low) if swap else (low, high)
        A = [pinned(cuda, 2 * r, M, K, va, ea, scale, fmt) for r in range(P)]
        W = [pinned(cuda, 2 * r + 1, N, K, vw, ew, scale) for r in range(P)]
        got = [torch.full((M, N), 7.0, dtype=OUT[out], device=cuda) for _ in range(P)]
        E.echo_gemm_fp8(A, W, got)
        for r in range(P):
            assert torch.equal(got[r], exact(A[r], W[r]).to(OUT[out])), (tiling, swap)


WHOLE = [-4.0, -3.0, -1.0, 0.0, 1.0, 2.0, 4.0]


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponent_scales_at_the_ends_of_their_range(E, cuda, tiling, out, fmt):
    """Where a code times its scale is a normal bfloat16 the result is that of the definition:
    exponent byte 0 (2^-127) under codes of at least 2, exponent byte 254 (2^127) under codes
    below 2."""
    assert_ends(E, cuda, tiling, "e8m0", out, ([-4.0, -2.0, 0.0, 2.0, 3.0], -127), (WHOLE, 100), fmt)
    assert_ends(E, cuda, tiling, "e8m0", out, (WHOLE, -100), ([-1.5, -1.0, 0.0, 1.0], 127), fmt)


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_fp32_scales_at_the_ends_of_their_range(E, cuda, tiling, out):
    """Where the product of two scales is a normal fp32 number the result is that of the
    definition: products of 2^-126 and, over sums that cancel or stay small, 2^104."""
    assert_ends(E, cuda, tiling, "f32", out, (WHOLE, -126), (WHOLE, 0))
    assert_ends(E, cuda, tiling, "f32", out, (WHOLE, -63), (WHOLE, -63))
    assert_ends(E, cuda, tiling, "f32", out, (WHOLE, 120), (WHOLE, -16))
    assert_ends(E, cuda, tiling, "f32", out, (WHOLE, 52), (WHOLE, 52))
    assert_ends(E, cuda, tiling, "f32", out, ([0.0], 64), (WHOLE, 63))
