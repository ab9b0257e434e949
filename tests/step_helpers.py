"""Plain references of the training step's operators in 64 bits (numpy), how far the kernels may
be off them, and inputs for both."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative to the value


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype, v):
    """What one rounding to the type may move a value by: half a step of the value, or of the
    type's subnormals."""
    import torch
    smallest = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[dtype]
    return torch.finfo(dtype).eps / 2 * np.abs(v) + smallest


def assert_close(got, want, off, dtype, what=""):
    """`off`: how far the value may be off before its rounding to the type."""
    got = np64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = off + half_step(dtype, np.abs(want) + off)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, up to {np.max(np.where(bad, err / tol, 0)):.3g} of the tolerance"


def depth(C):
    """Additions behind one another in a row's sum, at most: a thread adds 8 columns of each run in
    turn (up to 2 runs of 8), or, in rows of more than 16384 columns, one sum of 8 for each 8192
    columns; then 6 exchanges in a wavefront and 4 between wavefronts."""
    return 16 + C / 8192 + 10


def rs_error(C):
    """Relative error of 1 / sqrt(mean of squares + eps): each square is rounded and passes `depth`
    additions (all terms positive, so their errors are relative to the sum); 1 / C, the product with
    it and the addition of eps make three more roundings; the root halves all that, and its
    instruction is off by one unit in the last place at most, two half steps."""
    return ((depth(C) + 4) / 2 + 2) * U


def rs(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def factor(w, offset):
    return 1.0 if w is None else w + offset


def gates(gate, T):
    return 1.0 if gate is None else np.repeat(gate, T // gate.shape[0], axis=0)


def block_norm_ref(x, y, gate, w_post, post, alpha, offset, eps):
    """(out before its rounding, how far it may be off before it)."""
    n = y * rs(y, eps) * factor(w_post, offset) if post else y
    n = n * gates(gate, x.shape[0])
    # rs; the factor's addition, the products with rs, with it and with the gate; alpha x; the sum
    off = (rs_error(x.shape[1]) + 6 * U) * (np.abs(alpha * x) + np.abs(n))
    return alpha * x + n, off


def norm_ref(s, w_pre, offset, eps):
    a = s * rs(s, eps) * factor(w_pre, offset)
    return a, (rs_error(s.shape[1]) + 4 * U) * np.abs(a)


def block_norm_backward_ref(s, y, dout, da, gate, w_post, w_pre, post, alpha, offset, eps):
    """{name: (gradient, how far it may be off before its rounding)}.

    With D = depth(C) and E = rs_error(C): mean(u s) is off by (D + 5) U mean|u s| (the sum, three
    roundings in a term, the division), k = rs^2 mean(u s) by that and 2 E + 2 U; t = dout + rs (u
    - s k) by less than (D + 5 + 3 E / U + 8) U of T, the sum of its terms' magnitudes with mean|u s|
    for mean(u s).  dy repeats that on dn = gate t, so twice as much and what t is off.  A sum over R
    rows is off by at most R U of the magnitudes it adds, whatever its order."""
    T, C = s.shape
    D, E = depth(C), rs_error(C)
    K = (D + 13) * U + 3 * E
    r = rs(s, eps)
    t, mag, res = np.zeros_like(s), np.zeros_like(s), {}
    if dout is not None:
        t, mag = t + dout, mag + np.abs(dout)
    if da is not None:
        u = da * factor(w_pre, offset)
        t = t + r * (u - s * r * r * (u * s).mean(axis=1, keepdims=True))
        mag = mag + r * (np.abs(u) + np.abs(s) * r * r * np.abs(u * s).mean(axis=1, keepdims=True))
        res["dw_pre"] = ((da * s * r).sum(axis=0), ((T + 3) * U + E) * np.abs(da * s * r).sum(axis=0))
    res["dx"] = (alpha * t, (K + U) * np.abs(alpha) * mag)
    if y is not None:
        g = gates(gate, T)
        dn, mag_n = g * t, np.abs(g) * mag
        n, dy, mag_y = y, dn, mag_n
        if post:
            w, ry = factor(w_post, offset), rs(y, eps)
            n = y * ry * w
            v, mag_v = dn * w, mag_n * np.abs(w)
            dy = ry * (v - y * ry * ry * (v * y).mean(axis=1, keepdims=True))
            mag_y = ry * (mag_v + np.abs(y) * ry * ry * (mag_v * np.abs(y)).mean(axis=1, keepdims=True))
            res["dw_post"] = ((dn * y * ry).sum(axis=0), (K + (T + 4) * U + E) * (mag_n * np.abs(y) * ry).sum(axis=0))
        res["dy"] = (dy, (2 * K + 4 * U) * mag_y)
        if gate is not None:
            cut = (gate.shape[0], -1, C)
            res["dgate"] = ((t * n).reshape(cut).sum(axis=1), (K + (T + 5) * U + E) * (mag * np.abs(n)).reshape(cut).sum(axis=1))
    return res


def embed_backward_ref(dout, tokens, n, first, scale):
    """(gradient of all ranks' rows, how far it may be off before its rounding): a sum of m terms in
    any order is off by at most m - 1 roundings of their magnitudes, the scale is one more."""
    d, mag, count = np.zeros((n, dout.shape[1])), np.zeros((n, dout.shape[1])), np.zeros((n, 1))
    at = tokens - first
    here = (at >= 0) & (at < n)
    np.add.at(d, at[here], dout[here])
    np.add.at(mag, at[here], np.abs(dout[here]))
    np.add.at(count, at[here], 1.0)
    return d * scale, (count + 1) * U * mag * abs(scale)


def matrix(gen, shape, dtype, pad=0, at=0, size=1.0, device="cuda"):
    """A random matrix inside a wider buffer, `at` elements into it: rows of any alignment."""
    import torch
    T, C = shape
    buf = size * torch.randn(T * (C + pad) + at, generator=gen, device=device)
    return buf.to(dtype)[at:].view(T, C + pad)[:, :C]


class Guarded:
    """An output inside a wider buffer filled with a pattern; check() says whether anything but
    the output was written."""

    def __init__(self, shape, dtype, pad=0, at=0, device="cuda"):
        import torch
        T, C = shape
        self.buf = torch.full((T * (C + pad) + at + 16,), 7.25, dtype=dtype, device=device)
        self.t = self.buf[at:at + T * (C + pad)].view(T, C + pad)[:, :C]

    def check(self):
        self.t.fill_(7.25)
        return bool((self.buf == 7.25).all())
