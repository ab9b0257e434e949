"""Products in 8-bit floating point whose every step is exact, for tests that ask for equality.

Codes are whole numbers of at most 4 in magnitude and scales are powers of two, 1/2, 1 or 2.
A product of two codes is then a whole number of at most 16, and the products of a run of 8
lie within 2^4 of each other, so the fixed-point sums of the 8-bit matrix instruction (unit
2^-13 of a run's largest product) lose nothing.  A scaled sum is a multiple of 1/4 below
16 * 4 * K, that is a whole number of quarters below 2^8 K, which fp32 holds exactly up to
K = 2^16 whatever the order and the grouping.  What is left is one rounding, to the output type.
"""
import torch

FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# (M, N, K, P) for every tiling of the product, named by what the launch rules take there for
# 16-bit outputs with exponent bytes; each has edge tiles in both directions and a last block
# of k that is cut off inside a 16-byte run.
TILINGS = {
    "few rows, 4 column tiles": (5, 2100, 1171, 8),
    "few rows, 2 column tiles": (16, 1100, 2203, 8),
    "few rows, 1 column tile": (3, 203, 4301, 2),
    "two row tiles": (29, 301, 2203, 2),
    "64 x 64, four groups": (65, 129, 1171, 2),
    "64 x 64, two groups": (65, 129, 301, 2),
    "128 x 128, two groups": (200, 1100, 1101, 8),
    "64 x 128": (200, 1100, 301, 8),
    "64 x 128, few rows": (50, 2100, 301, 16),
    "128 x 128": (300, 1100, 301, 8),
    "256 x 256": (1000, 1001, 301, 12),
    "256 x 128": (520, 1000, 301, 12),
}


def codes_of(values, fmt):
    """Codes [rows, k] of fp32 values that the format holds, on rows of a multiple of 16 bytes
    with NaN behind the values (which must not count)."""
    rows, k = values.shape
    whole = torch.full((rows, -(-k // 16) * 16), 0x7F, dtype=torch.uint8, device=values.device).view(FORMATS[fmt])
    whole[:, :k].copy_(values)
    return whole[:, :k]


def operand(gen, rows, k, fmt, scale, block_rows, top=4):
    """A random operand of the kind above: (codes, scales), scales laid out k block by k block."""
    dev = gen.device
    v = torch.randint(-top, top + 1, (rows, k), generator=gen, device=dev).float()
    n = rows if block_rows == 1 else -(-rows // 128)
    e = torch.randint(-1, 2, (-(-k // 128), n), generator=gen, device=dev)
    s = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return codes_of(v, fmt), (s if scale == "e8m0" else s.float()).t()


def block_sums(A, W):
    """The sums of A W^T over each block of 128 along k, without scales, in 64 bits: a list."""
    a, w = A[0].double(), W[0].double()
    return [a[:, k:k + 128].contiguous() @ w[:, k:k + 128].t().contiguous() for k in range(0, a.shape[1], 128)]


def widened(m):
    """The values an operand stands for, in 64 bits."""
    codes, scales = m
    rows, k = codes.shape
    s = scales.double()
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return codes.double() * s.repeat_interleave(128, 1)[:, :k]


def exact(A, W):
    return widened(A) @ widened(W).t().contiguous()
