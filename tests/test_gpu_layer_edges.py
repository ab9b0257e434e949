"""Calls of the layer operators at the ends of what they take: k of one element and of 2^22,
sixteen ranks, tensors that start at any element, indices near 2^62, and more chunks of rows
than a 32-bit number counts."""
import numpy as np
import pytest

from fp8_helpers import dropout_ref, keep_mask, quantize_ref, to_np64
from product_cases import OUT, TILINGS, codes_of, exact, operand

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


SIZES = {t: (M, N, P) for t, (M, N, K, P) in TILINGS.items() if K <= 1024 or M <= 32}


@pytest.mark.parametrize("tiling", SIZES)
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("K", [1, 15, 16, 17, 112, 127, 128, 129, 255, 256, 257, 384, 399, 512, 513])
def test_short_k_is_exact(E, cuda, tiling, scale, K):
    """One K step to a few: fewer than there are slabs or groups, whole and cut off."""
    import torch
    M, N, P = SIZES[tiling]
    P = min(P, 2) if M <= 32 else P  # the other tilings are chosen by the number of ranks too
    g = generator(cuda, K)
    A = [operand(g, M, K, "e5m2", scale, 1) for _ in range(P)]
    W = [operand(g, N, K, "e4m3", scale, 128) for _ in range(P)]
    for out in OUT:
        got = [torch.full((M, N), float("nan"), dtype=OUT[out], device=cuda) for _ in range(P)]
        E.echo_gemm_fp8(A, W, got)
        for r in range(P):
            assert torch.equal(got[r], exact(A[r], W[r]).to(OUT[out])), (out, r)


@pytest.mark.parametrize("M,N", [(3, 70), (20, 40), (64, 64), (70, 130)])
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_longest_k_is_exact(E, cuda, M, N, scale, out):
    """k = 2^22 of codes -1, 0 and 1: sums of whole numbers below 2^22."""
    import torch
    K = 1 << 22
    g = generator(cuda, M)
    one = lambda rows: (codes_of(torch.randint(-1, 2, (rows, K), generator=g, device=cuda).float(), "e4m3"),
                        torch.ones(K // 128, rows, device=cuda).t() if scale == "f32" else
                        torch.full((K // 128, rows), 127, dtype=torch.uint8, device=cuda).view(torch.float8_e8m0fnu).t())
    A, W = one(M), one(N)
    got = torch.empty(M, N, dtype=OUT[out], device=cuda)
    E.echo_gemm_fp8([A], [W], [got])
    want = torch.zeros(M, N, dtype=torch.float64, device=cuda)
    for k in range(0, K, 1 << 19):
        want += A[0][:, k:k + (1 << 19)].double() @ W[0][:, k:k + (1 << 19)].double().t().contiguous()
    assert torch.equal(got, want.to(OUT[out]))


@pytest.mark.parametrize("M,N,K", [(5, 1 << 22, 33), (1 << 22, 3, 33)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_most_rows_and_columns_are_exact(E, cuda, M, N, K, out):
    import torch
    g = generator(cuda, 5)
    A, W = operand(g, M, K, "e4m3", "e8m0", 1), operand(g, N, K, "e4m3", "e8m0", 128)
    got = torch.full((M, N), float("nan"), dtype=OUT[out], device=cuda)
    E.echo_gemm_fp8([A], [W], [got])
    assert torch.equal(got, exact(A, W).to(OUT[out]))


def at_any_element(rows, cols, dtype, cuda, at, pad=5):
    """A matrix whose first element lies `at` elements into its buffer."""
    import torch
    whole = torch.full((rows * (cols + pad) + at,), 7.0, dtype=dtype, device=cuda)
    return whole, whole[at:].as_strided((rows, cols), (cols + pad, 1), at)


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("at", [1, 3])
def test_product_outputs_at_any_element(E, cuda, tiling, out, at):
    import torch
    M, N, K, P = TILINGS[tiling]
    g = generator(cuda, 6)
    A = [operand(g, M, K, "e4m3", "e8m0", 1) for _ in range(P)]
    W = [operand(g, N, K, "e4m3", "e8m0", 128) for _ in range(P)]
    got = [at_any_element(M, N, OUT[out], cuda, at) for _ in range(P)]
    E.echo_gemm_fp8(A, W, [o for _, o in got])
    for r, (whole, o) in enumerate(got):
        assert torch.equal(o, exact(A[r], W[r]).to(OUT[out]))
        o.fill_(7.0)
        assert (whole == 7.0).all(), "memory outside the output was written"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("R,C", [(130, 260), (33, 7), (1, 300), (256, 128)])
def test_quantizer_of_sixteen_ranks_at_any_element(E, cuda, dtype, block, R, C):
    import torch
    g = np.random.default_rng(R + C)
    X = []
    for r in range(16):
        _, x = at_any_element(R, C, OUT[dtype], cuda, r % 5, pad=3)
        x.copy_(torch.from_numpy(g.standard_normal((R, C)) * np.exp(g.standard_normal((1, C)))))
        X.append(x)
    rows = [E.EchoFp8.empty(R, C, "e4m3", "f32", block, cuda) for _ in X]
    # scales of the transposes row by row
    cols = [(E.EchoFp8.empty(C, R, "e4m3", "f32", block, cuda)[0],
             torch.zeros(-(-C // block), -(-R // 128), device=cuda)) for _ in X]
    E.echo_quantize_fp8(X, rows, cols)
    alone = [E.EchoFp8.empty(R, C, "e4m3", "f32", block, cuda) for _ in X]
    E.echo_quantize_fp8(X, alone)
    for r in (0, 7, 15):
        x = to_np64(X[r])
        for o, v in ((rows[r], x), (alone[r], x), (cols[r], x.T)):
            q, s = quantize_ref(v, "e4m3", block)
            np.testing.assert_array_equal(to_np64(o[1]), s)
            np.testing.assert_array_equal(to_np64(o[0]), q)


@pytest.mark.parametrize("R,C,pad", [(5, 9, 0), (5, 9, 3), (64, 512, 0), (7, 513, 1)])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_dropout_of_the_last_indices_at_any_element(E, cuda, R, C, pad, at):
    import torch
    key, step = -3, -1  # the wrapping step and a negative key are ordinary values
    rng = torch.tensor([key, step], dtype=torch.int64, device=cuda)
    first = (1 << 62) - R * C
    (_, x), (_, r), (whole, out) = (at_any_element(R, C, t, cuda, at, pad) for t in (torch.bfloat16, torch.float32, torch.float32))
    g = generator(cuda, 7)
    x.copy_(torch.randn(R, C, generator=g, device=cuda))
    r.copy_(torch.randn(R, C, generator=g, device=cuda))
    E.echo_dropout_add(x, out, 0.3, rng, residual=r, offset=2, first=first)
    want = dropout_ref(x.float().cpu().numpy(), r.cpu().numpy(), 0.3, first, (step + 2) % (1 << 64), key % (1 << 64))
    assert np.array_equal(out.cpu().numpy(), want)
    out.fill_(7.0)
    assert (whole == 7.0).all(), "memory outside the output was written"
    with pytest.raises(E.EchoError):
        E.echo_dropout_add(x, out, 0.3, rng, first=first + 1)


def test_dropout_of_more_chunks_than_32_bits_count(E, cuda):
    """2^31 - 1 rows of one element, apart from each other: two chunks a row."""
    import torch
    R = (1 << 31) - 1
    whole = torch.ones(R, 2, dtype=torch.bfloat16, device=cuda)
    x = whole[:, :1]
    rng = torch.tensor([5, 6], dtype=torch.int64, device=cuda)
    E.echo_dropout_add(x, x, 0.5, rng, first=3)
    for at in (0, 65535 * 100 - 7, (1 << 30) + 1, R - 4096):
        keep = keep_mask(3 + at, 4096, 6, 5, 0.5)
        assert np.array_equal(x[at:at + 4096, 0].float().cpu().numpy(), np.where(keep, np.float32(2), np.float32(0)))
    assert bool((whole[::4097, 1] == 1).all()) and bool((whole[-4096:, 1] == 1).all())
