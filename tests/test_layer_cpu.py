"""CPU checks of the operators of the layer around the all-reduce: the published
vectors of the generator, the references' own identities, and every refusal of the
C ABI (the host code checks before anything is launched; pointers are fake)."""
import ctypes

import numpy as np
import pytest

from error_compensated_bit_echo_amd import binding as B
from fp8_helpers import FORMATS, dequantize, keep_mask, philox10, quantize_ref, round_to_format


def test_generator_gives_the_published_vectors():
    """Random123's known answers of philox4x32-10 (counter words 0, 1 are the chunk,
    2, 3 the step, in this framework)."""
    for chunk, step, key, want in (
            (0, 0, 0, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            (2 ** 64 - 1, 2 ** 64 - 1, 2 ** 64 - 1, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            (0x85A308D3243F6A88, 0x0370734413198A2E, 0x299F31D0A4093822,
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = [int(w[0]) for w in philox10(np.array([chunk], dtype=np.uint64), step, key)]
        assert tuple(got) == want


def test_keep_mask_has_the_probability_and_does_not_depend_on_the_split():
    n, p = 1 << 18, 0.25
    m = keep_mask(0, n, 5, 77, p)
    assert abs(m.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)
    assert np.array_equal(m[1000:3001], keep_mask(1000, 2001, 5, 77, p))
    assert not np.array_equal(m, keep_mask(0, n, 6, 77, p))
    assert keep_mask(3, 100, 1, 2, 0.0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_reference_rounding_agrees_with_every_code_and_tie(fmt):
    import torch
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    values = torch.arange(256, dtype=torch.uint8).view(dt).double().numpy()
    values = np.unique(values[np.isfinite(values)])
    assert np.array_equal(round_to_format(values, fmt), values)
    mid = (values[1:] + values[:-1]) / 2  # ties: exact in fp32, so torch's CPU cast is a second opinion
    assert np.array_equal(round_to_format(mid, fmt), torch.from_numpy(mid).float().to(dt).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_reference_scale_is_the_smallest_power_of_two(fmt, block_rows):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((130, 260)) * np.exp(rng.standard_normal((130, 1)) * 3)
    q, s = quantize_ref(x, fmt, block_rows)
    bits, low, limit = FORMATS[fmt]
    a = np.abs(dequantize(q, s, block_rows) - x)
    half = dequantize(np.maximum(np.abs(q), 2.0 ** low) * 2.0 ** -(bits + 1), s, block_rows)
    assert (a <= half).all()  # half a step of the value, or of the subnormals
    assert (np.abs(q).max() <= limit) and (np.log2(s) % 1 == 0).all()


# ---- refusals ------------------------------------------------------------------


def ptrs(*p):
    return (ctypes.c_void_p * len(p))(*p)


def fp8(codes, scales, ld=256, srs=1, sks=512, fmt=B.ECHO_E4M3, st=B.ECHO_SCALE_E8M0, block=1):
    f = B._Fp8Struct()
    f.codes, f.scales = codes, scales
    f.ld, f.scale_row_stride, f.scale_k_stride, f.format, f.scale_type, f.block_rows = ld, srs, sks, fmt, st, block
    return f


X, Q, S, QC, SC = 1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30


def quantize(x=None, P=1, R=64, C=256, ldx=256, dtype=B.ECHO_BF16, rows="default", cols=None):
    rows = fp8(ptrs(Q), ptrs(S)) if rows == "default" else rows
    ref = lambda f: None if f is None else ctypes.byref(f)
    return B.load_library().echo_quantize_fp8(ptrs(X) if x is None else x, P, R, C, ldx, dtype, ref(rows), ref(cols), None)


@pytest.mark.parametrize("want,kw", [
    (B.ECHO_ERR_DTYPE, dict(dtype=3)), (B.ECHO_ERR_DTYPE, dict(dtype=-1)),
    (B.ECHO_ERR_SHAPE, dict(P=0)), (B.ECHO_ERR_SHAPE, dict(P=17)), (B.ECHO_ERR_SHAPE, dict(R=-1)),
    (B.ECHO_ERR_SHAPE, dict(C=(1 << 22) + 1)), (B.ECHO_ERR_SHAPE, dict(ldx=255)),
    (B.ECHO_ERR_SHAPE, dict(R=1 << 22, C=1 << 14)),
    (B.ECHO_ERR_ARG, dict(rows=None)), (B.ECHO_ERR_ARG, dict(x=ptrs(None))), (B.ECHO_ERR_ARG, dict(x=ptrs(X + 1))),
    (B.ECHO_ERR_ARG, dict(x=ptrs(Q + 128))),  # the input under the codes
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q + 8), ptrs(S)))), (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(None), ptrs(S)))),
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(None)))), (B.ECHO_ERR_ARG, dict(rows=fp8(None, ptrs(S)))),
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(Q + 100)))),  # scales among the codes
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(S + 2), st=B.ECHO_SCALE_F32))),
    (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), ld=264))), (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), ld=240))),
    (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), srs=0))), (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), sks=63))),
    (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), sks=-1))), (B.ECHO_ERR_SHAPE, dict(rows=fp8(ptrs(Q), ptrs(S), srs=1, sks=0))),
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(S), fmt=2))), (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(S), st=2))),
    (B.ECHO_ERR_ARG, dict(rows=fp8(ptrs(Q), ptrs(S), block=64))),
    (B.ECHO_ERR_ARG, dict(cols=fp8(ptrs(QC), ptrs(SC), fmt=B.ECHO_E5M2))),
    (B.ECHO_ERR_ARG, dict(cols=fp8(ptrs(QC), ptrs(SC), block=128))),
    (B.ECHO_ERR_ARG, dict(cols=fp8(ptrs(Q + 256 * 63), ptrs(SC)))),  # the transposed codes over the last row
    (B.ECHO_ERR_ARG, dict(x=ptrs(X, X), P=2, rows=fp8(ptrs(Q, Q + 16), ptrs(S, S + 4096)))),  # two ranks' codes
])
def test_quantizer_refusals(want, kw):
    assert quantize(**kw) == want


def test_quantizer_of_nothing_is_a_no_op():
    assert quantize(R=0) == B.ECHO_OK and quantize(C=0, ldx=0) == B.ECHO_OK


def gemm(A=None, W=None, out=None, P=1, M=64, N=32, K=256, ldo=32, dtype=B.ECHO_BF16):
    A = fp8(ptrs(Q), ptrs(S)) if A is None else A
    W = fp8(ptrs(QC), ptrs(SC)) if W is None else W
    return B.load_library().echo_gemm_fp8(ctypes.byref(A), ctypes.byref(W), ptrs(X) if out is None else out, P, M, N, K,
                                          ldo, dtype, None)


@pytest.mark.parametrize("want,kw", [
    (B.ECHO_ERR_DTYPE, dict(dtype=5)), (B.ECHO_ERR_SHAPE, dict(P=0)), (B.ECHO_ERR_SHAPE, dict(P=17)),
    (B.ECHO_ERR_SHAPE, dict(M=-1)), (B.ECHO_ERR_SHAPE, dict(N=(1 << 22) + 1)), (B.ECHO_ERR_SHAPE, dict(K=(1 << 22) + 1)),
    (B.ECHO_ERR_SHAPE, dict(M=1 << 22, N=1 << 14, ldo=1 << 14)), (B.ECHO_ERR_SHAPE, dict(ldo=31)),
    (B.ECHO_ERR_ARG, dict(A=fp8(ptrs(Q), ptrs(S), st=B.ECHO_SCALE_F32))),  # scale types that differ
    (B.ECHO_ERR_ARG, dict(out=ptrs(None))), (B.ECHO_ERR_ARG, dict(out=ptrs(X + 1))),
    (B.ECHO_ERR_ARG, dict(out=ptrs(Q))), (B.ECHO_ERR_ARG, dict(out=ptrs(SC - 64))),
    (B.ECHO_ERR_ARG, dict(A=fp8(ptrs(Q + 4), ptrs(S)))), (B.ECHO_ERR_ARG, dict(W=fp8(ptrs(QC), ptrs(None)))),
    (B.ECHO_ERR_SHAPE, dict(W=fp8(ptrs(QC), ptrs(SC), ld=250))), (B.ECHO_ERR_SHAPE, dict(W=fp8(ptrs(QC), ptrs(SC), srs=-1))),
    (B.ECHO_ERR_ARG, dict(A=fp8(ptrs(Q), ptrs(S), block=2))), (B.ECHO_ERR_ARG, dict(A=fp8(ptrs(Q), ptrs(S), fmt=-1))),
    (B.ECHO_ERR_ARG, dict(P=2, A=fp8(ptrs(Q, Q), ptrs(S, S)), W=fp8(ptrs(QC, QC), ptrs(SC, SC)), out=ptrs(X, X + 62))),
])
def test_product_refusals(want, kw):
    assert gemm(**kw) == want


def test_product_of_nothing_is_a_no_op():
    assert gemm(M=0) == B.ECHO_OK and gemm(N=0, ldo=0) == B.ECHO_OK


RNG = 9 << 30


def dropout(x=X, residual=None, out=Q, R=64, C=256, ldx=256, ldr=256, ldo=256, xt=B.ECHO_BF16, ot=B.ECHO_BF16, p=0.1,
            rng=RNG, offset=0, first=0):
    return B.load_library().echo_dropout_add(x, residual, out, R, C, ldx, ldr, ldo, xt, ot, p, rng, offset, first, None)


@pytest.mark.parametrize("want,kw", [
    (B.ECHO_ERR_DTYPE, dict(xt=3)), (B.ECHO_ERR_DTYPE, dict(ot=-1)), (B.ECHO_ERR_SHAPE, dict(R=-1)),
    (B.ECHO_ERR_SHAPE, dict(C=1 << 31)), (B.ECHO_ERR_SHAPE, dict(R=1 << 30, C=1 << 30)),
    (B.ECHO_ERR_SHAPE, dict(ldx=255)), (B.ECHO_ERR_SHAPE, dict(ldo=255)), (B.ECHO_ERR_SHAPE, dict(residual=S, ldr=1)),
    (B.ECHO_ERR_ARG, dict(p=-0.1)), (B.ECHO_ERR_ARG, dict(p=1.0)), (B.ECHO_ERR_ARG, dict(p=float("nan"))),
    (B.ECHO_ERR_ARG, dict(first=-1)), (B.ECHO_ERR_ARG, dict(first=1 << 62)),
    (B.ECHO_ERR_ARG, dict(x=None)), (B.ECHO_ERR_ARG, dict(out=None)), (B.ECHO_ERR_ARG, dict(rng=None)),
    (B.ECHO_ERR_ARG, dict(x=X + 1)), (B.ECHO_ERR_ARG, dict(rng=RNG + 4)), (B.ECHO_ERR_ARG, dict(residual=S + 1)),
    (B.ECHO_ERR_ARG, dict(out=X + 2)), (B.ECHO_ERR_ARG, dict(out=X, ot=B.ECHO_F32)), (B.ECHO_ERR_ARG, dict(out=X, ldo=512)),
    (B.ECHO_ERR_ARG, dict(residual=Q + 16)), (B.ECHO_ERR_ARG, dict(rng=Q + 8)),
])
def test_dropout_refusals(want, kw):
    assert dropout(**kw) == want


def test_dropout_of_nothing_is_a_no_op():
    assert dropout(R=0) == B.ECHO_OK and dropout(C=0) == B.ECHO_OK


def test_binding_refuses_what_is_not_on_a_gpu_or_not_alike():
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q = B.EchoFp8.empty(4, 128, device="cpu")
    o = torch.zeros(4, 4)
    rng = torch.zeros(2, dtype=torch.int64)
    cases = [
        lambda: B.echo_quantize_fp8([x], rows=[q]), lambda: B.echo_quantize_fp8([x]),
        lambda: B.echo_quantize_fp8([x.double()], rows=[q]), lambda: B.echo_quantize_fp8([x, x], rows=[q]),
        lambda: B.echo_quantize_fp8([x.t()], rows=[q]), lambda: B.echo_quantize_fp8([], rows=[]),
        lambda: B.echo_gemm_fp8([q], [q], [o]), lambda: B.echo_gemm_fp8([q], [q, q], [o]),
        lambda: B.echo_gemm_fp8([q], [(q[0].float(), q[1])], [o]), lambda: B.echo_gemm_fp8([q], [q], [o[:, :3]]),
        lambda: B.echo_gemm_fp8([(q[0], q[1].expand(4, 1)[:3])], [q], [o]),
        lambda: B.echo_dropout_add(x, x.clone(), 0.1, rng), lambda: B.EchoFp8.empty(4, 4, fmt="e3m4", device="cpu"),
    ]
    for f in cases:
        with pytest.raises(B.EchoError):
            f()
