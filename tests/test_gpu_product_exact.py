"""The 8-bit product in every tiling, with every pair of formats, type and height of scale blocks
and output type, on products that are exact up to the rounding to the output type
(product_cases.py): the results are compared for equality, so that a term that is lost, counted
twice or taken from another k, row, column, block or rank shows whatever its size."""
import pytest

from product_cases import OUT, TILINGS, exact, operand

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


FORMAT_PAIRS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")]


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("fa,fw", FORMAT_PAIRS)
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("block_a,block_w", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_every_tiling_is_exact(E, cuda, tiling, fa, fw, scale, block_a, block_w):
    import torch
    M, N, K, P = TILINGS[tiling]
    g = generator(cuda, 1)
    A = [operand(g, M, K, fa, scale, block_a) for _ in range(P)]
    W = [operand(g, N, K, fw, scale, block_w) for _ in range(P)]
    want = [exact(a, w) for a, w in zip(A, W)]
    for out in OUT:
        whole = [torch.full((M, N + 3), 7.0, dtype=OUT[out], device=cuda) for _ in range(P)]
        E.echo_gemm_fp8(A, W, [o[:, :N] for o in whole])
        for r in range(P):
            assert torch.equal(whole[r][:, :N], want[r].to(OUT[out])), (out, r)
            assert (whole[r][:, N:] == 7.0).all(), "columns behind the output were written"


# the products of a training step of the tensor-parallel stack: outputs in bfloat16 over e4m3 or
# e5m2 gradients with weights in blocks of 128 rows, and weight gradients in fp32 over both
# operands' own rows; k long enough that every slab of the ring is filled again
STEP = [("e4m3", "e4m3", 128, "bf16"), ("e5m2", "e4m3", 128, "bf16"), ("e4m3", "e5m2", 1, "f32")]


@pytest.mark.parametrize("fa,fw,block_w,out", STEP)
@pytest.mark.parametrize("M,N,K,P", [(1024, 1024, 2048, 12), (2048, 2040, 1200, 4), (4096, 4096, 1040, 1)])
def test_products_of_a_training_step_are_exact(E, cuda, fa, fw, block_w, out, M, N, K, P):
    import torch
    g = generator(cuda, 2)
    A = [operand(g, M, K, fa, "e8m0", 1) for _ in range(P)]
    W = [operand(g, N, K, fw, "e8m0", block_w) for _ in range(P)]
    got = [torch.full((M, N), float("nan"), dtype=OUT[out], device=cuda) for _ in range(P)]
    E.echo_gemm_fp8(A, W, got)
    for r in range(P):
        assert torch.equal(got[r], exact(A[r], W[r]).to(OUT[out]))


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("fa,fw", FORMAT_PAIRS)
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_codes_that_are_not_finite_stay_in_their_row_and_column(E, cuda, tiling, fa, fw, scale, out):
    """NaN of either format and e5m2's infinities, in the first and the last element along k."""
    import torch
    M, N, K, P = TILINGS[tiling]
    g = generator(cuda, 3)
    A = [operand(g, M, K, fa, scale, 1) for _ in range(P)]
    W = [operand(g, N, K, fw, scale, 128) for _ in range(P)]
    want = [exact(a, w).to(OUT[out]) for a, w in zip(A, W)]
    special = {"e4m3": (0x7F, 0xFF), "e5m2": (0x7C, 0x7F)}  # NaN and -NaN; infinity and NaN
    r = P - 1
    A[r][0].view(torch.uint8)[1, K - 1] = special[fa][0]
    A[r][0].view(torch.uint8)[M - 1, 0] = special[fa][1]
    W[r][0].view(torch.uint8)[N - 1, K - 1] = special[fw][0]
    W[r][0].view(torch.uint8)[2, 0] = special[fw][1]
    got = [torch.full((M, N), 7.0, dtype=OUT[out], device=cuda) for _ in range(P)]
    E.echo_gemm_fp8(A, W, got)
    hit = torch.zeros(M, N, dtype=torch.bool, device=cuda)
    hit[[1, M - 1]] = True
    hit[:, [2, N - 1]] = True
    for q in range(r):
        assert torch.equal(got[q], want[q])
    assert torch.equal(got[r][~hit], want[r][~hit])
    # a NaN spoils all of its row and column; an infinity gives infinities, or NaN with a zero
    assert not torch.isfinite(got[r][hit]).any()
    for row, code in ((1, special[fa][0]), (M - 1, special[fa][1])):
        if not (fa == "e5m2" and code == 0x7C):
            assert got[r][row].isnan().all()
    for col, code in ((N - 1, special[fw][0]), (2, special[fw][1])):
        if not (fw == "e5m2" and code == 0x7C):
            assert got[r][:, col].isnan().all()


# every kernel of at most 32 rows, which adds in fp32 whatever the output type
FEW = [t for t, (M, _, _, _) in TILINGS.items() if M <= 32]


@pytest.mark.parametrize("tiling", FEW)
@pytest.mark.parametrize("fa,fw", FORMAT_PAIRS)
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_few_rows_are_summed_in_fp32(E, cuda, tiling, fa, fw, scale, out):
    """General codes and scales, held to the bound of fp32 sums: at most one unit in the last
    place (2^-23 of the running magnitude) lost per addition and two per block for its scaling,
    so (K + 4 blocks) 2^-23 sum |a w|, plus half a step of the output type."""
    import torch
    from product_cases import codes_of, widened
    M, N, K, P = TILINGS[tiling]
    g = generator(cuda, 4)

    def general(rows, fmt):
        kb = -(-K // 128)
        s = torch.exp(0.7 * torch.randn(kb, rows, generator=g, device=cuda)) / 32
        if scale == "e8m0":
            s = (s.log2().round().to(torch.int32) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        return codes_of(4 * torch.randn(rows, K, generator=g, device=cuda), fmt), s.t()

    A, W = [general(M, fa) for _ in range(P)], [general(N, fw) for _ in range(P)]
    got = [torch.empty(M, N, dtype=OUT[out], device=cuda) for _ in range(P)]
    E.echo_gemm_fp8(A, W, got)
    blocks = -(-K // 128)
    half = 0.0 if out == "f32" else torch.finfo(OUT[out]).eps / 2
    small = 2.0 ** -25 if out == "f16" else 0.0  # half a step of fp16's subnormals
    for r in range(P):
        a, w = widened(A[r]), widened(W[r])
        want = a @ w.t().contiguous()
        tol = (K + 4 * blocks) * 2.0 ** -23 * (a.abs() @ w.abs().t().contiguous())
        tol = tol + half * (want.abs() + tol) + small
        assert ((got[r].double() - want).abs() <= tol).all()
