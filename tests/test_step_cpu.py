"""CPU checks of the training step's operators: every refusal of the C ABI and of the binding (the
host code checks before anything is launched; pointers are fake), and what the references say."""
import ctypes

import numpy as np
import pytest

from error_compensated_bit_echo_amd import binding as B
from step_helpers import block_norm_backward_ref, block_norm_ref, norm_ref

G = 1 << 30
X, Y, OUT, A, GATE, WPOST, WPRE, DOUT, DA, DX, DY, DGATE, DWPOST, DWPRE, WS = (i * G for i in range(1, 16))


def block(y=True, **kw):
    f = dict(rows=64, cols=256, gate=GATE if y else None, ld_gate=256, gate_rows=1, w_post=WPOST if y else None, w_pre=WPRE,
             residual_scale=0.5 if y else 1.0, weight_offset=0.0, eps=1e-6, x_dtype=B.ECHO_BF16, y_dtype=B.ECHO_F32,
             a_dtype=B.ECHO_BF16, param_dtype=B.ECHO_F32, post_norm=int(y))
    f.update(kw)
    return B.EchoBlock(**f)


def norm(b=None, x=X, ldx=256, y=Y, ldy=256, out=OUT, ldo=256, a=A, lda=256, **kw):
    b = block(y is not None, **kw) if b is None else b
    return B.load_library().echo_block_norm(ctypes.byref(b), x, ldx, y, ldy, out, ldo, a, lda, None)


BAD_BLOCKS = [
    (B.ECHO_ERR_DTYPE, dict(x_dtype=3)), (B.ECHO_ERR_DTYPE, dict(y_dtype=-1)), (B.ECHO_ERR_DTYPE, dict(a_dtype=9)),
    (B.ECHO_ERR_DTYPE, dict(param_dtype=3)), (B.ECHO_ERR_DTYPE, dict(a_dtype=B.ECHO_F16)),
    (B.ECHO_ERR_DTYPE, dict(y_dtype=B.ECHO_F16)), (B.ECHO_ERR_DTYPE, dict(x_dtype=B.ECHO_F32, y_dtype=B.ECHO_F16)),
    (B.ECHO_ERR_SHAPE, dict(rows=-1)), (B.ECHO_ERR_SHAPE, dict(cols=-1)), (B.ECHO_ERR_SHAPE, dict(cols=(1 << 22) + 1)),
    (B.ECHO_ERR_SHAPE, dict(rows=1 << 31)), (B.ECHO_ERR_SHAPE, dict(rows=(1 << 31) - 1, cols=1 << 22)),
    (B.ECHO_ERR_SHAPE, dict(gate_rows=0)), (B.ECHO_ERR_SHAPE, dict(gate_rows=-1)), (B.ECHO_ERR_SHAPE, dict(gate_rows=3)),
    (B.ECHO_ERR_SHAPE, dict(gate_rows=128)), (B.ECHO_ERR_SHAPE, dict(gate_rows=2, ld_gate=255)),
    (B.ECHO_ERR_ARG, dict(post_norm=2)), (B.ECHO_ERR_ARG, dict(post_norm=0)),  # w_post without a post-norm
    (B.ECHO_ERR_ARG, dict(eps=0.0)), (B.ECHO_ERR_ARG, dict(eps=-1.0)), (B.ECHO_ERR_ARG, dict(eps=float("nan"))),
    (B.ECHO_ERR_ARG, dict(eps=1e39)), (B.ECHO_ERR_ARG, dict(residual_scale=float("inf"))),
    (B.ECHO_ERR_ARG, dict(residual_scale=1e39)), (B.ECHO_ERR_ARG, dict(weight_offset=float("nan"))),
    (B.ECHO_ERR_ARG, dict(gate=GATE + 2)), (B.ECHO_ERR_ARG, dict(w_post=WPOST + 1)), (B.ECHO_ERR_ARG, dict(w_pre=WPRE + 2)),
]


@pytest.mark.parametrize("want,kw", BAD_BLOCKS + [
    (B.ECHO_ERR_SHAPE, dict(ldx=255)), (B.ECHO_ERR_SHAPE, dict(ldy=1 << 46)), (B.ECHO_ERR_SHAPE, dict(ldo=0)),
    (B.ECHO_ERR_SHAPE, dict(lda=-256)),
    (B.ECHO_ERR_ARG, dict(x=None)), (B.ECHO_ERR_ARG, dict(out=None)), (B.ECHO_ERR_ARG, dict(x=X + 1)),
    (B.ECHO_ERR_ARG, dict(y=Y + 2)), (B.ECHO_ERR_ARG, dict(a=A + 1)), (B.ECHO_ERR_ARG, dict(out=OUT + 1)),
    (B.ECHO_ERR_ARG, dict(a=None)),  # a weight for a norm that is not wanted
    (B.ECHO_ERR_ARG, dict(out=X + 2)), (B.ECHO_ERR_ARG, dict(out=X, ldo=512)), (B.ECHO_ERR_ARG, dict(out=Y)),
    (B.ECHO_ERR_ARG, dict(a=X)), (B.ECHO_ERR_ARG, dict(a=Y)), (B.ECHO_ERR_ARG, dict(a=OUT)), (B.ECHO_ERR_ARG, dict(a=GATE)),
    (B.ECHO_ERR_ARG, dict(a=WPRE + 1020)), (B.ECHO_ERR_ARG, dict(out=WPOST)),
    (B.ECHO_ERR_ARG, dict(y=None)), (B.ECHO_ERR_ARG, dict(y=None, out=None, a=None, w_pre=None)),
    (B.ECHO_ERR_ARG, dict(y=None, out=None, residual_scale=0.5)), (B.ECHO_ERR_ARG, dict(y=None, out=None, post_norm=1)),
    (B.ECHO_ERR_ARG, dict(y=None, out=None, gate=GATE)),
])
def test_block_norm_refusals(want, kw):
    assert norm(**kw) == want


def test_block_norm_of_nothing_is_a_no_op():
    assert norm(rows=0) == B.ECHO_OK and norm(cols=0, ldx=0) == B.ECHO_OK
    assert B.load_library().echo_block_norm(None, X, 8, None, 8, None, 8, A, 8, None) == B.ECHO_ERR_ARG


def backward(out=OUT, ldo=256, y=Y, ldy=256, dout=DOUT, lddo=256, da=DA, ldda=256, dx=DX, lddx=256, dy=DY, lddy=256, dgate=DGATE,
             ld_dgate=256, dw_post=DWPOST, dw_pre=DWPRE, ws=WS, ws_bytes=None, **kw):
    b = block(y is not None, **kw)
    if ws_bytes is None:
        ws_bytes = B.echo_block_norm_workspace(64, 256, 1)
    return B.load_library().echo_block_norm_backward(ctypes.byref(b), out, ldo, y, ldy, dout, lddo, da, ldda, dx, lddx, dy, lddy,
                                                     dgate, ld_dgate, dw_post, dw_pre, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", BAD_BLOCKS + [
    (B.ECHO_ERR_SHAPE, dict(ldo=1)), (B.ECHO_ERR_SHAPE, dict(ldy=1)), (B.ECHO_ERR_SHAPE, dict(lddo=1)),
    (B.ECHO_ERR_SHAPE, dict(ldda=1)), (B.ECHO_ERR_SHAPE, dict(lddx=1)), (B.ECHO_ERR_SHAPE, dict(lddy=1)),
    (B.ECHO_ERR_SHAPE, dict(gate_rows=2, ld_dgate=1)),
    (B.ECHO_ERR_WORKSPACE, dict(ws=None)), (B.ECHO_ERR_WORKSPACE, dict(ws_bytes=1024)), (B.ECHO_ERR_ARG, dict(ws=WS + 8)),
    (B.ECHO_ERR_ARG, dict(out=None)), (B.ECHO_ERR_ARG, dict(dout=None, da=None, w_pre=None, dw_pre=None)),
    (B.ECHO_ERR_ARG, dict(dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None)),
    (B.ECHO_ERR_ARG, dict(y=None)), (B.ECHO_ERR_ARG, dict(gate=None)), (B.ECHO_ERR_ARG, dict(w_post=None)),
    (B.ECHO_ERR_ARG, dict(w_pre=None)), (B.ECHO_ERR_ARG, dict(da=None)),
    (B.ECHO_ERR_ARG, dict(dx=DOUT + 2)), (B.ECHO_ERR_ARG, dict(dx=DOUT, lddx=512)), (B.ECHO_ERR_ARG, dict(dx=OUT)),
    (B.ECHO_ERR_ARG, dict(dy=Y)), (B.ECHO_ERR_ARG, dict(dy=DX)), (B.ECHO_ERR_ARG, dict(dx=DA)), (B.ECHO_ERR_ARG, dict(dgate=GATE)),
    (B.ECHO_ERR_ARG, dict(dw_post=WPOST + 4)), (B.ECHO_ERR_ARG, dict(dw_pre=DWPOST)), (B.ECHO_ERR_ARG, dict(ws=DX)),
    (B.ECHO_ERR_ARG, dict(ws=WPRE - 64)), (B.ECHO_ERR_ARG, dict(dgate=DGATE + 1)),
])
def test_block_norm_backward_refusals(want, kw):
    assert backward(**kw) == want


def test_block_norm_backward_of_no_columns_is_a_no_op():
    assert backward(cols=0) == B.ECHO_OK
    assert backward(rows=0, dgate=None, dw_post=None, dw_pre=None) == B.ECHO_OK


def test_block_norm_workspace():
    size = B.echo_block_norm_workspace
    assert size(1, 8) == 3 * 8 * 4 and size(0, 8) == 0 and size(8, 0) == 0 and size(-1, 8) == 0
    assert size(8, (1 << 22) + 1) == 0 and size(9, 8, 2) == 0 and size(9, 8, -1) == 0
    assert size(1 << 20, 64, 1 << 20) > 0


def tensors(*spec):
    """(address, numel, dtype) triples as the C ABI takes them."""
    p, n, t = zip(*spec) if spec else ((), (), ())
    return (ctypes.c_void_p * len(p))(*p), (ctypes.c_int64 * len(n))(*n), (ctypes.c_int32 * len(t))(*t)


F32, BF16 = B.ECHO_F32, B.ECHO_BF16
NORM = 20 * G


def clip(spec=((X, 100, F32), (Y, 100, BF16)), out=None, count=None, max_norm=1.0, norm=NORM, ws=WS, ws_bytes=1 << 20):
    p, n, t = tensors(*spec)
    o = p if out is None else (ctypes.c_void_p * len(out))(*out)
    return B.load_library().echo_clip_grads(p, o, n, t, len(spec) if count is None else count, max_norm, norm, ws, ws_bytes, None)


def grad_norm(spec=((X, 100, F32), (Y, 100, BF16)), count=None, norm=NORM, ws=WS, ws_bytes=1 << 20):
    p, n, t = tensors(*spec)
    return B.load_library().echo_grad_norm(p, n, t, len(spec) if count is None else count, norm, ws, ws_bytes, None)


BAD_TENSORS = [
    (B.ECHO_ERR_SHAPE, dict(count=-1)), (B.ECHO_ERR_SHAPE, dict(count=(1 << 24) + 1)),
    (B.ECHO_ERR_DTYPE, dict(spec=((X, 100, 3),))), (B.ECHO_ERR_SHAPE, dict(spec=((X, -1, F32),))),
    (B.ECHO_ERR_SHAPE, dict(spec=((X, (1 << 40) + 1, F32),))), (B.ECHO_ERR_SHAPE, dict(spec=((X, 1 << 40, F32),) * 33)),
    (B.ECHO_ERR_ARG, dict(spec=((None, 1, F32),))), (B.ECHO_ERR_ARG, dict(spec=((X + 2, 1, F32),))),
    (B.ECHO_ERR_ARG, dict(spec=((X + 1, 1, BF16),))), (B.ECHO_ERR_ARG, dict(norm=None)), (B.ECHO_ERR_ARG, dict(norm=NORM + 2)),
    (B.ECHO_ERR_ARG, dict(norm=X + 396)), (B.ECHO_ERR_WORKSPACE, dict(ws=None)), (B.ECHO_ERR_WORKSPACE, dict(ws_bytes=100)),
    (B.ECHO_ERR_ARG, dict(ws=WS + 4)), (B.ECHO_ERR_ARG, dict(ws=X + 8)), (B.ECHO_ERR_ARG, dict(ws=NORM - 64)),
]


@pytest.mark.parametrize("want,kw", BAD_TENSORS)
def test_grad_norm_refusals(want, kw):
    assert grad_norm(**kw) == want


@pytest.mark.parametrize("want,kw", BAD_TENSORS + [
    (B.ECHO_ERR_ARG, dict(max_norm=-1.0)), (B.ECHO_ERR_ARG, dict(max_norm=float("nan"))), (B.ECHO_ERR_ARG, dict(max_norm=float("inf"))),
    (B.ECHO_ERR_ARG, dict(out=(X, None))), (B.ECHO_ERR_ARG, dict(out=(X, OUT + 1))),
    (B.ECHO_ERR_ARG, dict(out=(X + 4, Y))), (B.ECHO_ERR_ARG, dict(out=(OUT, OUT + 200))), (B.ECHO_ERR_ARG, dict(out=(Y, OUT))),
    (B.ECHO_ERR_ARG, dict(out=(OUT, X))), (B.ECHO_ERR_ARG, dict(spec=((X, 100, F32), (X, 100, F32)))),  # the same tensor twice
    (B.ECHO_ERR_ARG, dict(spec=((X, 100, F32), (X + 8, 4, F32)))),  # one inside another
])
def test_clip_refusals(want, kw):
    assert clip(**kw) == want


def test_clip_workspace():
    size = B.echo_clip_workspace
    assert size(0) == 0 and size(-1) == 0 and size((1 << 24) + 1) == 0
    assert size(1) == size(280) > 0 and size(281) == 2 * size(1)


TOK = 21 * G


def ptrs(*p):
    return (ctypes.c_void_p * len(p))(*p)


def embed(tables=None, tokens=TOK, out=None, P=1, rows=100, cols=64, ldt=64, n=10, ldo=64, tt=F32, ot=BF16, tb=8, first=0, scale=1.0):
    return B.load_library().echo_embed(ptrs(X) if tables is None else tables, tokens, ptrs(OUT) if out is None else out, P, rows, cols,
                                       ldt, n, ldo, tt, ot, tb, first, scale, None)


BAD_EMBED = [
    (B.ECHO_ERR_DTYPE, dict(tt=3)), (B.ECHO_ERR_DTYPE, dict(ot=-1)), (B.ECHO_ERR_DTYPE, dict(tt=B.ECHO_F16)),
    (B.ECHO_ERR_DTYPE, dict(tb=2)), (B.ECHO_ERR_SHAPE, dict(P=0)), (B.ECHO_ERR_SHAPE, dict(P=17)), (B.ECHO_ERR_SHAPE, dict(rows=-1)),
    (B.ECHO_ERR_SHAPE, dict(rows=(1 << 31) - 1)), (B.ECHO_ERR_SHAPE, dict(P=2, rows=1 << 30)), (B.ECHO_ERR_SHAPE, dict(cols=-1)),
    (B.ECHO_ERR_SHAPE, dict(cols=(1 << 22) + 1)), (B.ECHO_ERR_SHAPE, dict(n=-1)), (B.ECHO_ERR_SHAPE, dict(n=(1 << 27) + 1)),
    (B.ECHO_ERR_SHAPE, dict(ldt=63)), (B.ECHO_ERR_ARG, dict(first=-1)),
    (B.ECHO_ERR_ARG, dict(first=(1 << 62) + 1)), (B.ECHO_ERR_ARG, dict(scale=float("nan"))), (B.ECHO_ERR_ARG, dict(scale=1e39)),
    (B.ECHO_ERR_ARG, dict(tokens=None)), (B.ECHO_ERR_ARG, dict(tokens=TOK + 4)), (B.ECHO_ERR_ARG, dict(tokens=TOK + 2, tb=4)),
]


@pytest.mark.parametrize("want,kw", BAD_EMBED + [
    (B.ECHO_ERR_SHAPE, dict(ldo=63)),
    (B.ECHO_ERR_ARG, dict(tables=ptrs(None))), (B.ECHO_ERR_ARG, dict(tables=ptrs(X + 2))), (B.ECHO_ERR_ARG, dict(out=ptrs(None))),
    (B.ECHO_ERR_ARG, dict(out=ptrs(OUT + 1))), (B.ECHO_ERR_ARG, dict(out=ptrs(X + 128))), (B.ECHO_ERR_ARG, dict(out=ptrs(TOK + 64))),
    (B.ECHO_ERR_ARG, dict(P=2, tables=ptrs(X, X), out=ptrs(OUT, OUT + 64))),
])
def test_embed_refusals(want, kw):
    assert embed(**kw) == want


def embed_backward(dout=DOUT, tokens=TOK, dtables=None, P=1, rows=100, cols=64, ldt=64, n=10, ldo=64, ot=BF16, tt=F32, tb=8, first=0,
                   scale=1.0, ws=WS, ws_bytes=1 << 20):
    return B.load_library().echo_embed_backward(dout, tokens, ptrs(OUT) if dtables is None else dtables, P, rows, cols, ldt, n, ldo,
                                                ot, tt, tb, first, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", BAD_EMBED + [
    (B.ECHO_ERR_SHAPE, dict(ldo=63)), (B.ECHO_ERR_ARG, dict(dout=None)), (B.ECHO_ERR_ARG, dict(dout=DOUT + 1)),
    (B.ECHO_ERR_ARG, dict(dtables=ptrs(None))), (B.ECHO_ERR_ARG, dict(dtables=ptrs(OUT + 2))),
    (B.ECHO_ERR_ARG, dict(dtables=ptrs(DOUT + 64))), (B.ECHO_ERR_ARG, dict(dtables=ptrs(TOK - 64))),
    (B.ECHO_ERR_ARG, dict(dtables=ptrs(WS + 256))), (B.ECHO_ERR_ARG, dict(P=2, dtables=ptrs(OUT, OUT + 128))),
    (B.ECHO_ERR_WORKSPACE, dict(ws=None)), (B.ECHO_ERR_WORKSPACE, dict(ws_bytes=64)), (B.ECHO_ERR_ARG, dict(ws=WS + 128)),
    (B.ECHO_ERR_ARG, dict(ws=TOK)), (B.ECHO_ERR_ARG, dict(ws=DOUT)),
])
def test_embed_backward_refusals(want, kw):
    assert embed_backward(**kw) == want


def test_embed_of_nothing_is_a_no_op():
    assert embed(n=0) == B.ECHO_OK and embed(cols=0) == B.ECHO_OK
    assert embed_backward(rows=0) == B.ECHO_OK and embed_backward(cols=0) == B.ECHO_OK
    size = B.echo_embed_workspace
    assert size(0, 8) == 0 and size(8, 0) == 0 and size((1 << 27) + 1, 8) == 0 and size(8, (1 << 22) + 1) == 0 and size(1, 1) > 0


def test_binding_refuses_what_is_not_on_a_gpu_or_not_alike():
    import torch
    x, w, n = torch.zeros(4, 8), torch.ones(8), torch.zeros(1)
    tok = torch.zeros(4, dtype=torch.long)
    cases = [
        lambda: B.echo_block_norm(x, a=x.clone()), lambda: B.echo_block_norm(None, a=x),
        lambda: B.echo_block_norm_backward(x, da=x, dx=x.clone()), lambda: B.echo_grad_norm([x], n),
        lambda: B.echo_clip_grads([x], 1.0, n), lambda: B.echo_clip_grads(x, 1.0, None), lambda: B.echo_grad_norm(3, n),
        lambda: B.echo_embed([x], tok, [x.clone()]), lambda: B.echo_embed([], tok, []),
        lambda: B.echo_embed_backward(x, tok, [x.clone()]),
    ]
    for f in cases:
        with pytest.raises(B.EchoError):
            f()


def test_references_agree_with_differentiating_the_definition():
    import torch
    rng = np.random.default_rng(1)
    T, C, alpha, offset, eps = 6, 17, 0.6, 0.25, 1e-5
    v = {n: rng.standard_normal(s) for n, s in dict(x=(T, C), y=(T, C), gate=(3, C), w_post=(C,), w_pre=(C,), dout=(T, C),
                                                    da=(T, C)).items()}
    leaf = {n: torch.from_numpy(a).requires_grad_() for n, a in v.items()}
    norm_ = lambda t, w: t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + eps) * (w + offset)
    out = alpha * leaf["x"] + leaf["gate"].repeat_interleave(2, 0) * norm_(leaf["y"], leaf["w_post"])
    a = norm_(out, leaf["w_pre"])
    want_out, _ = block_norm_ref(v["x"], v["y"], v["gate"], v["w_post"], True, alpha, offset, eps)
    s = out.detach().numpy()
    assert np.allclose(want_out, s, rtol=1e-12) and np.allclose(norm_ref(s, v["w_pre"], offset, eps)[0], a.detach().numpy(), rtol=1e-12)
    ((out * leaf["dout"]).sum() + (a * leaf["da"]).sum()).backward()
    got = block_norm_backward_ref(s, v["y"], v["dout"], v["da"], v["gate"], v["w_post"], v["w_pre"], True, alpha, offset, eps)
    for name, of in dict(dx="x", dy="y", dgate="gate", dw_post="w_post", dw_pre="w_pre").items():
        assert np.allclose(got[name][0], leaf[of].grad.numpy(), rtol=1e-10, atol=1e-12), name
