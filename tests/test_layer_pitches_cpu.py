"""Row pitches at the ends of their range, in the layer operators' C ABI (the host code checks
before anything is launched; pointers are fake)."""
import ctypes

import pytest

from error_compensated_bit_echo_amd import binding as B


def ptrs(*p):
    return (ctypes.c_void_p * len(p))(*p)


def fp8(codes, scales, ld=16, srs=1, sks=1 << 22):
    f = B._Fp8Struct()
    f.codes, f.scales = codes, scales
    f.ld, f.scale_row_stride, f.scale_k_stride, f.format, f.scale_type, f.block_rows = ld, srs, sks, B.ECHO_E4M3, B.ECHO_SCALE_E8M0, 1
    return f


X, Q, S, QC, SC, RNG = (i << 30 for i in range(1, 7))


# a pitch times the rows that wraps past 64 bits, so that the end of the matrix seems to lie
# before its start; the inputs lie within the outputs
@pytest.mark.parametrize("ld", [1 << 40, (1 << 40) - 1, 1 << 34])
def test_matrices_beyond_the_address_space_are_refused(ld):
    lib = B.load_library()
    R = 1 << 22
    assert lib.echo_quantize_fp8(ptrs(Q + 16), 1, R, 8, ld, B.ECHO_F32, ctypes.byref(fp8(ptrs(Q), ptrs(S))), None,
                                 None) == B.ECHO_ERR_SHAPE
    A, W = fp8(ptrs(Q), ptrs(S)), fp8(ptrs(QC), ptrs(SC))
    assert lib.echo_gemm_fp8(ctypes.byref(A), ctypes.byref(W), ptrs(Q + 16), 1, R, 8, 16, ld, B.ECHO_F32,
                             None) == B.ECHO_ERR_SHAPE
    for at in range(3):
        pitches = [8, 8, 8]
        pitches[at] = ld
        assert lib.echo_dropout_add(X, Q, S, 1 << 28, 8, *pitches, B.ECHO_F32, B.ECHO_F32, 0.1, RNG, 0, 0,
                                    None) == B.ECHO_ERR_SHAPE
