"""The 8-bit quantizer and product and the residual dropout on the GPU, against
plain 64-bit references (fp8_helpers.py).

The quantizer and the dropout are compared bit for bit: the scaling by a power of two
is exact and the generator is integer arithmetic.  The tolerance of the products is
fp8_helpers.product_tolerance."""
import numpy as np
import pytest

from fp8_helpers import dropout_ref, keep_mask, product_tolerance, quantize_ref, to_np64, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E(cuda):
    import error_compensated_bit_echo_amd as E
    E.load_library()
    return E


def torch_():
    import torch
    return torch


DT = {"bf16": "bfloat16", "f16": "float16", "f32": "float32"}


def dt(name):
    return getattr(torch_(), DT[name])


def normal(seed, *shape, spread=1.0):
    g = np.random.default_rng(seed)
    return g.standard_normal(shape) * np.exp(spread * g.standard_normal((1,) * (len(shape) - 1) + shape[-1:]))


def on_gpu(a, dtype, cuda, pad=0):
    """A matrix on the GPU, its rows `pad` elements apart."""
    torch = torch_()
    t = torch.full((a.shape[0], a.shape[1] + pad), 7.0, dtype=torch.float32)
    t[:, :a.shape[1]] = torch.from_numpy(a)
    return t.to(dtype).to(cuda)[:, :a.shape[1]]


def raw(codes):
    """The whole padded buffer of an EchoFp8's codes as bytes."""
    torch = torch_()
    rows, k = codes.shape
    return codes.as_strided((rows, codes.stride(0)), (codes.stride(0), 1)).view(torch.uint8)


def assert_quantized(got, x, fmt, block_rows):
    """got (EchoFp8) against the reference of x (float64 [rows, k])."""
    q, s = quantize_ref(x, fmt, block_rows)
    gq, gs = to_np64(got[0]), to_np64(got[1])
    np.testing.assert_array_equal(gs, s)
    np.testing.assert_array_equal(gq, q)  # NaN compares equal to NaN here
    fine = np.isfinite(q)
    np.testing.assert_array_equal(np.signbit(gq[fine]), np.signbit(q[fine] + 0.0 * x[fine]))


SHAPES = [(1, 1), (1, 128), (3, 130), (16, 256), (127, 129), (128, 128), (129, 127), (200, 1000), (257, 513), (64, 7)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("want", ["rows", "cols", "both"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantizer(E, cuda, R, C, dtype, want, block):
    torch = torch_()
    fmt, scale = (("e4m3", "e8m0"), ("e5m2", "f32"))[(R + C + block) % 2]
    P = 1 + (R + C) % 3
    X = [on_gpu(normal(7 * r + R, R, C), dt(dtype), cuda, pad=(C % 3)) for r in range(P)]
    mk = lambda rows, k: [E.EchoFp8.empty(rows, k, fmt, scale, block, cuda) for _ in range(P)]
    rows = mk(R, C) if want != "cols" else None
    cols = mk(C, R) if want != "rows" else None
    for o in (rows or []) + (cols or []):
        raw(o.codes).fill_(0x5A)
    E.echo_quantize_fp8(X, rows, cols)
    for r in range(P):
        x = to_np64(X[r])
        for o, v in ((rows, x), (cols, x.T)):
            if o is not None:
                assert_quantized(o[r], v, fmt, block)
                assert (raw(o[r].codes)[:, v.shape[1]:] == 0x5A).all(), "bytes behind the rows were written"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("P,R,C", [(8, 1100, 1000), (1, 4096, 2048), (2, 33000, 130)])
def test_quantizer_of_many_rows(E, cuda, dtype, P, R, C):
    """Alone, the codes along the rows are those of the call that writes both orientations
    (which the other tests check), whatever kernel the number of rows chooses."""
    torch = torch_()
    X = [torch.randn(R, C, device=cuda).to(dt(dtype)) for _ in range(P)]
    X[0][R - 1, C - 1], X[0][5, 7] = float("inf"), float("nan")
    alone = [E.EchoFp8.empty(R, C, "e5m2", "f32", 1, cuda) for _ in range(P)]
    both = [E.EchoFp8.empty(R, C, "e5m2", "f32", 1, cuda) for _ in range(P)]
    cols = [E.EchoFp8.empty(C, R, "e5m2", "f32", 1, cuda) for _ in range(P)]
    E.echo_quantize_fp8(X, alone)
    E.echo_quantize_fp8(X, both, cols)
    for r in range(P):
        assert torch.equal(alone[r].scales, both[r].scales)
        assert torch.equal(alone[r].codes.view(torch.uint8), both[r].codes.view(torch.uint8))
    rows = np.r_[0:3, 5, R - 2:R]
    x = X[0][torch.from_numpy(rows).to(cuda)]
    sub = (alone[0].codes[torch.from_numpy(rows).to(cuda)], alone[0].scales[torch.from_numpy(rows).to(cuda)])
    assert_quantized(sub, to_np64(x), "e5m2", 1)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantizer_of_every_16_bit_value(E, cuda, fmt, dtype):
    """All bit patterns, each in a block whose scale another element sets."""
    torch = torch_()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt(dtype))
    x = torch.empty(1024, 128, dtype=dt(dtype))
    x[:, :64] = bits.view(1024, 64)
    x[:, 64:] = bits.view(1024, 64)[torch.randperm(1024, generator=torch.Generator().manual_seed(1))]
    x[::3, 64:] = 0  # and where nothing else does
    rows, cols = E.EchoFp8.empty(1024, 128, fmt, "e8m0", 1, cuda), E.EchoFp8.empty(128, 1024, fmt, "e8m0", 1, cuda)
    E.echo_quantize_fp8([x.to(cuda)], [rows], [cols])
    v = to_np64(x)
    assert_quantized(rows, v, fmt, 1)
    assert_quantized(cols, v.T, fmt, 1)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantizer_special_values(E, cuda, fmt, block):
    """Zeros, subnormals, the largest values, ties, infinities and NaN."""
    R, C = 140, 300
    x = normal(5, R, C).astype(np.float32)
    x[:, :128] = 0.0
    x[1, 130:200] = np.float32(1e-45)
    x[2, 128:256] = np.float32(3e-39)
    x[3, 140] = np.float32(3.4028234e38)
    x[4, 150] = np.inf
    x[5, 151:170] = np.nan
    x[6, 128:256] = np.nan
    x[7, 128:256] = -np.inf
    x[8, 256:] = np.arange(44) * 0.5 + 0.25
    x[9, 3] = -0.0
    x[130, 270:280] = [448, 449, 447, 464, 480, 57344, 57345, 61440, -448, -1]
    X = on_gpu(x, dt("f32"), cuda)
    rows, cols = E.EchoFp8.empty(R, C, fmt, "f32", block, cuda), E.EchoFp8.empty(C, R, fmt, "f32", block, cuda)
    E.echo_quantize_fp8([X], [rows], [cols])
    v = x.astype(np.float64)
    assert_quantized(rows, v, fmt, block)
    assert_quantized(cols, v.T, fmt, block)
    alone = E.EchoFp8.empty(R, C, fmt, "f32", block, cuda)
    E.echo_quantize_fp8([X], [alone])  # the path without a transpose
    assert_quantized(alone, v, fmt, block)


def test_quantizer_output_layouts(E, cuda):
    """Scales row by row, codes at a wider pitch, ranks beside each other in one buffer."""
    torch = torch_()
    R, C, P = 150, 260, 2
    X = [on_gpu(normal(r, R, C), torch.bfloat16, cuda) for r in range(P)]
    wide = torch.zeros(R, 2 * 288, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    sc = torch.zeros(R, 2 * 3, dtype=torch.uint8, device=cuda).view(torch.float8_e8m0fnu)
    rows = [(wide[:, 288 * r:288 * r + C], sc[:, 3 * r:3 * r + 3]) for r in range(P)]
    E.echo_quantize_fp8(X, rows)
    for r in range(P):
        assert_quantized(rows[r], to_np64(X[r]), "e4m3", 1)
    with pytest.raises(E.EchoError):  # shared columns
        E.echo_quantize_fp8(X, [(wide[:, 0:C], sc[:, 0:3]), (wide[:, 256:256 + C], sc[:, 3:6])])


# ---- product ---------------------------------------------------------------------


def operand(E, cuda, seed, rows, k, fmt, scale, block, spread=0.7):
    """A random matrix in 8 bits: every kind of code, general fp32 scales or exponent bytes."""
    torch = torch_()
    g = np.random.default_rng(seed)
    m = E.EchoFp8.empty(rows, k, fmt, scale, block, cuda)
    raw(m.codes).fill_(0x7F)  # NaN in the padding: it must not count
    m.codes.copy_(torch.from_numpy(g.standard_normal((rows, k)) * 8).float().to(m.codes.dtype))
    s = np.exp(spread * g.standard_normal(tuple(m.scales.shape)))
    if scale == "e8m0":
        b = torch.from_numpy((np.rint(np.log2(s)) + 127).astype(np.uint8))
        m.scales.copy_(b.view(torch.float8_e8m0fnu).to(cuda))
    else:
        m.scales.copy_(torch.from_numpy(s))
    return m


def assert_product(out, A, W, block_a=1, block_w=1, m=slice(None), n=slice(None)):
    """out (rows m, columns n of the result) against A W^T in 64 bits."""
    want = values(A, block_a)[m] @ values(W, block_w)[n].T
    tol = product_tolerance(A, W, out.dtype, block_a, block_w, m, n)
    err = np.abs(to_np64(out) - want)
    assert (err <= tol).all(), f"off by up to {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 64, 1000), (2, 17, 127), (7, 130, 129), (16, 512, 1024), (17, 96, 384),
            (33, 200, 640), (64, 256, 256), (65, 129, 255), (100, 300, 1111), (128, 128, 2048), (129, 257, 130),
            (256, 256, 512), (300, 520, 144), (512, 384, 128), (1000, 72, 260), (5, 2000, 16)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("block", [1, 128])
def test_product(E, cuda, M, N, K, scale, block):
    torch = torch_()
    i = M + N + K + block
    fa, fw = (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2"))[i % 4]
    out_dtype = dt(("bf16", "f32", "f16")[i % 3])
    P = (1, 2, 3)[i % 3]
    A = [operand(E, cuda, 10 + r, M, K, fa, scale, 1) for r in range(P)]
    W = [operand(E, cuda, 50 + r, N, K, fw, scale, block) for r in range(P)]
    out = [torch.full((M, N + 3), 7.0, dtype=out_dtype, device=cuda)[:, :N] for _ in range(P)]
    if out_dtype == torch.float16:  # keep the results in range
        for a in A:
            a.codes.copy_((a.codes.float() / 64).to(a.codes.dtype))
    E.echo_gemm_fp8(A, W, out)
    for r in range(P):
        assert_product(out[r], A[r], W[r], 1, block)
        assert (out[r].as_strided((M, 3), (N + 3, 1), N) == 7.0).all(), "columns behind the output were written"


SWEEP = [(m, n, k, p) for m, n, k, p in (
    (48, 1024, 896, 8), (96, 640, 512, 4), (160, 512, 2176, 1), (192, 768, 320, 2), (384, 1024, 256, 4),
    (640, 896, 384, 1), (768, 1280, 768, 2), (1024, 1024, 200, 1), (1280, 2048, 1152, 1), (2048, 2304, 272, 1),
    (2300, 2100, 400, 1), (4001, 3003, 333, 1), (2000, 3001, 208, 1), (1023, 1100, 140, 8), (32, 8192, 640, 1), (4, 256, 8192, 2), (8, 16, 4096, 1))]


@pytest.mark.parametrize("M,N,K,P", SWEEP)
@pytest.mark.parametrize("scale,block", [("e8m0", 128), ("f32", 1), ("f32", 128)])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_product_sizes(E, cuda, M, N, K, P, scale, block, out_dtype):
    """Sizes over the whole range of tilings, sampled rows and columns."""
    torch = torch_()
    A = [operand(E, cuda, 10 + r, M, K, "e4m3", scale, 1) for r in range(P)]
    W = [operand(E, cuda, 50 + r, N, K, "e4m3", scale, block) for r in range(P)]
    out = [torch.full((M, N), float("nan"), dtype=dt(out_dtype), device=cuda) for _ in range(P)]
    E.echo_gemm_fp8(A, W, out)
    g = np.random.default_rng(1)
    for r in range(P):
        assert torch.isfinite(out[r]).all()
        m = np.unique(np.r_[0, M - 1, g.integers(0, M, 40)])
        n = np.unique(np.r_[0, N - 1, g.integers(0, N, 40)])
        sub = out[r][torch.from_numpy(m).to(cuda)][:, torch.from_numpy(n).to(cuda)]
        assert_product(sub, A[r], W[r], 1, block, m, n)


# (M, N, K, P) of few rows for all the columns: two groups that share k, low tiles, and
# tiles of 128 rows at the most, each at its edges
FEW_ROWS = [(60, 4090, 130, 8), (128, 2048, 1408, 4), (420, 4100, 260, 1), (65, 1000, 127, 16), (50, 2080, 260, 16),
            (64, 33000, 144, 1), (600, 4100, 300, 1), (100, 4160, 384, 16), (128, 33000, 130, 2), (300, 520, 1500, 2)]


@pytest.mark.parametrize("M,N,K,P", FEW_ROWS)
@pytest.mark.parametrize("scale,block", [("e8m0", 128), ("f32", 1), ("f32", 128)])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_product_of_few_rows(E, cuda, M, N, K, P, scale, block, out_dtype):
    test_product_sizes(E, cuda, M, N, K, P, scale, block, out_dtype)


# tiles of 128 rows and columns, two groups that share k
PAIRS = [(600, 4100, 1300, 1), (200, 1100, 1171, 8), (128, 4090, 1090, 8), (1024, 4096, 1152, 1), (130, 2600, 1411, 4)]


@pytest.mark.parametrize("M,N,K,P", PAIRS)
@pytest.mark.parametrize("scale,block", [("e8m0", 128), ("f32", 1), ("f32", 128)])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_product_of_a_tile_per_cu(E, cuda, M, N, K, P, scale, block, out_dtype):
    test_product_sizes(E, cuda, M, N, K, P, scale, block, out_dtype)


@pytest.mark.parametrize("M,N,P", [(50, 2080, 16), (600, 4100, 1), (100, 4160, 16), (128, 2048, 4)])
@pytest.mark.parametrize("scale,out_dtype,block", [("e8m0", "f32", 1), ("e8m0", "bf16", 128), ("f32", "f32", 1),
                                                   ("f32", "bf16", 128), ("f32", "bf16", 1)])
def test_nan_of_few_rows_stays_in_its_row_and_column(E, cuda, M, N, P, scale, out_dtype, block):
    """NaN codes of a row of A and a column of W, behind K and in the last block too."""
    torch = torch_()
    K = 300
    A = [operand(E, cuda, 10 + r, M, K, "e4m3", scale, 1) for r in range(P)]
    W = [operand(E, cuda, 50 + r, N, K, "e4m3", scale, block) for r in range(P)]
    out = [torch.zeros(M, N, dtype=dt(out_dtype), device=cuda) for _ in range(P)]
    for m in A + W:  # what lies behind K in the rows' padding
        whole = m.codes.as_strided((m.codes.shape[0], 304), (304, 1)).view(torch.uint8)
        whole[:, K:] = 0x7F
    A[0].codes.view(torch.uint8)[M // 2, 299] = 0x7F
    W[P - 1].codes.view(torch.uint8)[N - 1, 7] = 0x7F
    E.echo_gemm_fp8(A, W, out)
    for r in range(P):
        want = torch.zeros(M, N, dtype=torch.bool, device=cuda)
        if r == 0:
            want[M // 2] = True
        if r == P - 1:
            want[:, N - 1] = True
        assert torch.equal(out[r].isnan(), want)


def test_product_block_rows_on_both_sides_and_broadcast_scales(E, cuda):
    torch = torch_()
    M, N, K = 200, 150, 300
    A = operand(E, cuda, 1, M, K, "e4m3", "f32", 128)
    W = operand(E, cuda, 2, N, K, "e4m3", "f32", 128)
    out = torch.empty(M, N, dtype=torch.float32, device=cuda)
    E.echo_gemm_fp8([A], [W], [out])
    assert_product(out, A, W, 128, 128)
    one = torch.tensor([[0.375]], device=cuda)
    E.echo_gemm_fp8([(A.codes, one.expand(M, 3))], [(W.codes, one.expand(2, 3))], [out])
    assert_product(out, (A.codes, one.expand(M, 3)), (W.codes, one.expand(2, 3)), 1, 128)


def test_product_over_nothing_gives_zeros(E, cuda):
    torch = torch_()
    A, W = E.EchoFp8.empty(5, 0, device=cuda), E.EchoFp8.empty(7, 0, device=cuda)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        out = torch.full((5, 9), 3.0, device=cuda, dtype=dtype)
        E.echo_gemm_fp8([A], [W], [out[:, :7]])
        assert (out[:, :7] == 0).all() and (out[:, 7:] == 3).all()


@pytest.mark.parametrize("M,N,K", [(4, 64, 300), (70, 140, 300), (130, 300, 1500), (2000, 3000, 300), (4000, 3000, 300)])
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
def test_nan_stays_in_its_row_and_column(E, cuda, M, N, K, scale, out_dtype, block):
    torch = torch_()
    A, W = operand(E, cuda, 1, M, K, "e4m3", scale, 1), operand(E, cuda, 2, N, K, "e4m3", scale, block)
    clean = torch.empty(M, N, device=cuda, dtype=dt(out_dtype))
    E.echo_gemm_fp8([A], [W], [clean])
    A.codes.view(torch.uint8)[1, 299] = 0x7F
    W.codes.view(torch.uint8)[3, 0] = 0xFF
    if scale == "f32":
        A.scales[2, 1] = float("inf")
    else:
        A.scales.view(torch.uint8)[2, 1] = 0xFF
    out = torch.empty_like(clean)
    E.echo_gemm_fp8([A], [W], [out])
    hit = torch.zeros(M, N, dtype=torch.bool, device=cuda)
    hit[1:3], hit[:, 3] = True, True
    assert not torch.isfinite(out[hit]).any()
    assert torch.equal(out[~hit], clean[~hit])


def test_product_into_columns_of_one_buffer(E, cuda):
    """Column-parallel outputs beside each other."""
    torch = torch_()
    P, M, N, K = 3, 70, 50, 256
    A = [operand(E, cuda, 1, M, K, "e4m3", "e8m0", 1)] * P
    W = [operand(E, cuda, 50 + r, N, K, "e4m3", "e8m0", 128) for r in range(P)]
    whole = torch.zeros(M, P * N, dtype=torch.bfloat16, device=cuda)
    E.echo_gemm_fp8(A, W, [whole[:, r * N:(r + 1) * N] for r in range(P)])
    for r in range(P):
        assert_product(whole[:, r * N:(r + 1) * N], A[r], W[r], 1, 128)
    with pytest.raises(E.EchoError):
        E.echo_gemm_fp8(A[:2], W[:2], [whole[:, 0:N], whole[:, 1:N + 1]])


# ---- dropout ---------------------------------------------------------------------


KEY, STEP = 0x1234567_89ABCDEF, (1 << 40) + 17


def rng_tensor(cuda, key=KEY, step=STEP):
    return torch_().tensor([key, step], dtype=torch_().int64, device=cuda)


def f32(t):
    return t.detach().float().cpu().numpy()


@pytest.mark.parametrize("R,C", [(1, 1), (1, 7), (3, 8), (5, 9), (2, 2049), (64, 512), (33, 77), (1, 100000)])
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                   ("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
def test_dropout(E, cuda, R, C, xt, ot, residual, pad):
    torch = torch_()
    first, p = ((0, 0.1), (8 * 12345678901, 0.5), (13, 0.25))[(R + C + pad) % 3]
    x = on_gpu(normal(1, R, C), dt(xt), cuda, pad)
    r = on_gpu(normal(2, R, C), dt(ot), cuda, pad) if residual else None
    out = on_gpu(np.zeros((R, C)), dt(ot), cuda, pad)
    E.echo_dropout_add(x, out, p, rng_tensor(cuda), residual=r, offset=3, first=first)
    want = dropout_ref(f32(x), None if r is None else f32(r), p, first, STEP + 3, KEY)
    want = torch.from_numpy(want).to(dt(ot))
    assert torch.equal(out.cpu(), want)
    if pad:
        assert (out.as_strided((R, pad), (C + pad, 1), C) == 7.0).all()


def test_dropout_drops_what_is_not_finite_and_keeps_p_zero_whole(E, cuda):
    torch = torch_()
    n = 4096
    x = torch.full((n,), float("nan"), device=cuda)
    out = torch.empty_like(x)
    E.echo_dropout_add(x, out, 0.5, rng_tensor(cuda))
    keep = keep_mask(0, n, STEP, KEY, 0.5)
    assert np.array_equal(np.isnan(f32(out)), keep) and (f32(out)[~keep] == 0).all()
    y, r = torch.randn(n, device=cuda), torch.randn(n, device=cuda)
    E.echo_dropout_add(y, out, 0.0, rng_tensor(cuda), residual=r)
    assert torch.equal(out, y + r)
    E.echo_dropout_add(y, out, 1 - 2.0 ** -16, rng_tensor(cuda))
    assert np.array_equal(f32(out) != 0, keep_mask(0, n, STEP, KEY, 1 - 2.0 ** -16))


def test_dropout_shards_agree_with_the_whole(E, cuda):
    """Ranks that hold parts of the rows draw the mask of the whole message."""
    torch = torch_()
    R, C = 37, 129
    x, r = torch.randn(R, C, device=cuda), torch.randn(R, C, device=cuda)
    whole, parts = torch.empty_like(x), torch.empty_like(x)
    rng = rng_tensor(cuda)
    E.echo_dropout_add(x, whole, 0.3, rng, residual=r)
    for a, b in ((0, 5), (5, 6), (6, 37)):
        E.echo_dropout_add(x[a:b], parts[a:b], 0.3, rng, residual=r[a:b], first=a * C)
    assert torch.equal(whole, parts)


def test_dropout_in_place_and_overlaps(E, cuda):
    torch = torch_()
    x, r, rng = torch.randn(100, 33, device=cuda), torch.randn(100, 33, device=cuda), rng_tensor(cuda)
    want = torch.empty_like(x)
    E.echo_dropout_add(x, want, 0.2, rng, residual=r)
    for into in ("x", "r"):
        a, b = x.clone(), r.clone()
        E.echo_dropout_add(a, a if into == "x" else b, 0.2, rng, residual=b)
        assert torch.equal(a if into == "x" else b, want)
    flat = torch.randn(200, device=cuda)
    with pytest.raises(E.EchoError):
        E.echo_dropout_add(flat[:100], flat[1:101], 0.2, rng)


# ---- streams, graphs, a run of them together ---------------------------------------


def test_another_stream_and_two_at_once(E, cuda):
    torch = torch_()
    M, N, K = 96, 384, 640
    A, W = operand(E, cuda, 1, M, K, "e4m3", "e8m0", 1), operand(E, cuda, 2, N, K, "e4m3", "e8m0", 128)
    want = torch.empty(M, N, device=cuda)
    E.echo_gemm_fp8([A], [W], [want])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty(M, N, device=cuda) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            E.echo_gemm_fp8([A], [W], [o], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_captured_calls_follow_their_inputs(E, cuda):
    """Quantizer, product and dropout in one graph, replayed over changed inputs with
    eager work between the replays."""
    torch = torch_()
    M, N, K = 40, 256, 512
    x = torch.randn(M, K, device=cuda).bfloat16()
    res = torch.randn(M, N, device=cuda)
    W = operand(E, cuda, 2, N, K, "e4m3", "e8m0", 128)
    rng = rng_tensor(cuda)

    def step(q, y, out):
        E.echo_quantize_fp8([x], [q])
        E.echo_gemm_fp8([q], [W], [y])
        E.echo_dropout_add(y, out, 0.1, rng, residual=res, offset=1)

    mk = lambda: (E.EchoFp8.empty(M, K, device=cuda), torch.empty(M, N, dtype=torch.bfloat16, device=cuda),
                  torch.empty(M, N, device=cuda))
    bufs, eager = mk(), mk()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*bufs)
    seen = []
    for i in range(4):
        x.copy_(torch.randn(M, K, device=cuda))
        rng[1] += 1
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        assert torch.equal(bufs[2], eager[2]) and torch.equal(bufs[0].codes.view(torch.uint8), eager[0].codes.view(torch.uint8))
        seen.append(bufs[2].clone())
    assert not torch.equal(seen[0], seen[1])


# ---- beyond 32-bit offsets -----------------------------------------------------------


def test_quantizer_and_product_beyond_4_gib(E, cuda):
    """Matrices of more than 2^32 elements: the last rows agree with those of a small call."""
    torch = torch_()
    R, C, N = (1 << 20) + 130, 4224, 48
    X = torch.empty(R, C, dtype=torch.bfloat16, device=cuda).normal_()
    rows, cols = E.EchoFp8.empty(R, C, device=cuda), E.EchoFp8.empty(C, R, device=cuda)
    E.echo_quantize_fp8([X], [rows], [cols])
    at = R - 258  # a multiple of 128: blocks along the columns start where the whole matrix's do
    tail = X[at:].contiguous()
    r, c = E.EchoFp8.empty(258, C, device=cuda), E.EchoFp8.empty(C, 258, device=cuda)
    E.echo_quantize_fp8([tail], [r], [c])
    assert at % 128 == 0
    assert torch.equal(rows.codes[at:].view(torch.uint8), r.codes.view(torch.uint8))
    assert torch.equal(cols.codes[:, at:].view(torch.uint8), c.codes.view(torch.uint8))
    assert torch.equal(rows.scales[at:].contiguous().view(torch.uint8), r.scales.contiguous().view(torch.uint8))
    del X, cols
    W = operand(E, cuda, 1, N, C, "e4m3", "e8m0", 128)
    out, small = torch.empty(R, N, dtype=torch.bfloat16, device=cuda), torch.empty(258, N, dtype=torch.bfloat16, device=cuda)
    E.echo_gemm_fp8([rows], [W], [out])
    E.echo_gemm_fp8([r], [W], [small])
    assert_product(small, r, W, 1, 128)
    assert_product(out[at:], r, W, 1, 128)


@pytest.mark.parametrize("dtype,block,C", [("f32", 1, 8192), ("f32", 128, 8200), ("f16", 1, 8184), ("bf16", 128, 8192)])
def test_quantizer_of_more_than_the_last_level_cache(E, cuda, dtype, block, C):
    """A call of more than 256 MB stores past the caches: each part of its rows agrees
    with a small call's."""
    torch = torch_()
    R, n = 8192 + 70, 1536
    X = torch.empty(R, C, dtype=getattr(torch, {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}[dtype]),
                    device=cuda).normal_()
    def run(x):
        rows = E.EchoFp8.empty(x.shape[0], C, block_rows=block, device=cuda)
        cols = E.EchoFp8.empty(C, x.shape[0], block_rows=block, device=cuda)
        E.echo_quantize_fp8([x], [rows], [cols])
        return [t.view(torch.uint8) for t in (rows.codes, cols.codes, rows.scales.contiguous(), cols.scales.contiguous())]
    whole = run(X)
    for at in range(0, R, n):
        end = min(R, at + n)
        part = run(X[at:end])
        s0, s1 = (at, end) if block == 1 else (at // 128, -(-end // 128))
        assert torch.equal(whole[0][at:end], part[0]) and torch.equal(whole[1][:, at:end], part[1])
        assert torch.equal(whole[2][s0:s1], part[2]) and torch.equal(whole[3][:, at // 128:-(-end // 128)], part[3])


def test_dropout_beyond_4_gib(E, cuda):
    torch = torch_()
    whole = torch.empty((1 << 32) + 72, dtype=torch.bfloat16, device=cuda)
    with pytest.raises(E.EchoError):  # more columns than a row may have; as eight rows it is in range
        E.echo_dropout_add(whole, whole, 0.5, rng_tensor(cuda))
    wide = torch.empty((1 << 20) + 3, 4104, dtype=torch.bfloat16, device=cuda)
    for x in (whole.view(8, -1), wide[:, :4099]):
        x.fill_(1.0)
        R, C = x.shape
        E.echo_dropout_add(x, x, 0.5, rng_tensor(cuda))
        tail = torch.ones(min(C, 4099), dtype=torch.bfloat16, device=cuda)
        want = torch.empty_like(tail)
        at = R * C - tail.numel()  # of the last row's end
        E.echo_dropout_add(tail, want, 0.5, rng_tensor(cuda), first=at)
        assert torch.equal(x[-1, C - tail.numel():], want)
        assert np.array_equal(f32(want) != 0, keep_mask(at, tail.numel(), STEP, KEY, 0.5))
