"""Echo inside tensor-parallel layers: autograd operators over one emulated TP group.

A tensor-parallel block needs two collectives (rit.work blog post
"echo-4-bit-gpu-communication", «Почему обычное 4-битное суммирование портит
модель»: the layer's matrices are split over the GPUs, each computes a part of
the result and an all-reduce sums the parts; in training it repeats on the
backward pass):

* ``g`` after a row-parallel product: forward sums the P partial outputs (an
  Echo all-reduce on the forward compensator state); backward hands the
  replicated gradient to every rank unchanged.
* ``f`` before a column-parallel product: forward gives every rank the same
  input; backward sums the P partial input gradients (an Echo all-reduce on
  the backward compensator state).

Forward and backward keep separate compensator state (same page, «Как Echo
возвращает ошибку в следующие вызовы»); one state per residual stream, shared
by all the block's calls of one pass and reset at the start of each step.
The P ranks are P tensors on one GPU; every reduction runs in libecho's
kernels through the C ABI.  A ``mode`` of "exact" replaces both collectives by
a plain sum (the bf16 wire values added in fp32), for comparison.

The row-parallel product and ``g`` can also run as one step in bfloat16
(``product="bf16_fused"``): libecho's MFMA product writes each rank's stage-1
payload straight from its accumulators, then the owner and decode stages
finish the all-reduce; ``"bf16"`` runs the same product written out followed
by a whole Echo call, which gives bit-identical results.  The same holds for
``f`` in the backward pass: the input-gradient products of the column-parallel
layer run on libecho's kernel, on the backward state.

With ``product="fp8"`` every product of the stack, forward, input gradients and
weight gradients, runs in 8-bit floating point with a scale per 128 elements
(e4m3 for activations and weights, e5m2 for gradients); the ranks' partials are
bfloat16 and reduced by Echo as before, and weight gradients come in fp32.
``dropout`` puts a dropout on each reduced output before it joins the residual
stream, with a mask that both passes draw from a counter-based generator.

Around the blocks, a stack can have learned norms before and after each block
with a gate and a scaled residual (``block_norms``; the end of a block and the
start of the next are one kernel), an embedding whose vocabulary is split over
the ranks and whose partials go through the same all-reduce (``vocab``), and
train_step can clip the gradients of all its shards by their common norm.
"""
from __future__ import annotations

import math
from typing import List, Optional

from . import binding as B


class EchoGroup:
    """P emulated ranks sharing one Echo state (forward and backward directions)
    for messages of ``numel`` elements in bfloat16 on the wire.  ``variant``
    passes the configuration switches ``sender_feedback``, ``state_bf16``,
    ``own_exact`` and ``group`` through to the state (the output stays fp32)."""

    VARIANT_KEYS = ("sender_feedback", "state_bf16", "own_exact", "group")

    def __init__(self, P: int, numel: int, mode: str = "echo", device=None, record: bool = False,
                 **variant):
        import torch

        if mode not in ("echo", "echo_off", "exact"):
            raise ValueError(f"mode {mode!r}")
        unknown = set(variant) - set(self.VARIANT_KEYS)
        if unknown:
            raise ValueError(f"unknown variant switches {sorted(unknown)}")
        self.P, self.numel, self.mode, self.variant = P, numel, mode, dict(variant)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.state = None
        if mode != "exact":
            cfg = B.EchoConfig.make(P, numel, "bf16", compensate=(mode == "echo"), **variant)
            self.state = B.echo_init_state(cfg, device=self.device)
        # when recording, every reduction appends (direction, [partials], out)
        self.record = record
        self.log: List[tuple] = []

    def reset(self):
        """Start of a step: fresh compensator for both directions."""
        if self.state is not None:
            B.echo_reset(self.state, 3)
        self.log.clear()

    def product_allreduce(self, A, W, fused: bool, direction: int = B.ECHO_FWD):
        """All-reduce of bf16(A_r @ W_r^T) (A_r [T, K], W_r [H, K] bf16) on the
        state of `direction`: fused, stage 1 runs in the product's epilogue;
        otherwise the product is written out and reduced by a whole call."""
        import torch

        if self.mode == "exact":
            raise ValueError("the bf16 product path needs an Echo state")
        if fused and (self.variant.get("own_exact") or self.variant.get("group", 32) != 32):
            raise ValueError("the fused product takes group 32 without the owners' own shares")
        T, H = A[0].shape[0], W[0].shape[0]
        out = torch.empty(self.numel, dtype=torch.float32, device=self.device)
        if fused:
            B.echo_gemm_stage1(A, W, self.state, direction)
            B.echo_owner(self.state, direction)
            B.echo_decode(out, self.state)
        else:
            parts = [torch.empty(T, H, dtype=torch.bfloat16, device=self.device) for _ in range(self.P)]
            B.echo_gemm_bf16(A, W, parts)
            B.echo_reduce([p.view(-1) for p in parts], out, self.state, direction)
        if self.record:
            self.log.append((direction, ("product", [a.detach().clone() for a in A],
                                         [w.detach().clone() for w in W]), out.detach().clone()))
        return out

    def allreduce(self, partials, direction: int):
        """Sum of the P bf16 partials ([..] contiguous, numel each) as fp32."""
        import torch

        parts = [p.contiguous() for p in partials]
        if self.mode == "exact":
            out = torch.zeros(self.numel, dtype=torch.float32, device=self.device)
            for p in parts:
                out += p.reshape(-1).float()
        else:
            out = torch.empty(self.numel, dtype=torch.float32, device=self.device)
            B.echo_reduce([p.reshape(-1) for p in parts], out, self.state, direction)
        if self.record:
            self.log.append((direction, [p.detach().clone() for p in parts], out.detach().clone()))
        return out


def _fns():
    import torch

    class RowParallelEcho(torch.autograd.Function):
        """g(h_r @ W2_r) with the products in bfloat16 on libecho's matrix-core
        kernel: forward gives sum_r bf16(bf16(h_r) @ bf16(W2_r)) through Echo
        (fused: stage 1 in the product's epilogue); backward is the fp32
        gradient of sum_r h_r @ W2_r (the rounding passed straight through)."""

        @staticmethod
        def forward(ctx, group: "EchoGroup", shape, fused: bool, *hw):
            P = group.P
            hs, ws = hw[:P], hw[P:]
            A = [h.to(torch.bfloat16).contiguous() for h in hs]   # [T, F/P]
            W = [w.t().to(torch.bfloat16).contiguous() for w in ws]  # [H, F/P]: output features by K
            out = group.product_allreduce(A, W, fused)
            ctx.save_for_backward(*hs, *ws)
            ctx.P = P
            return out.view(shape)

        @staticmethod
        def backward(ctx, grad):
            P = ctx.P
            saved = ctx.saved_tensors
            hs, ws = saved[:P], saved[P:]
            g = grad.contiguous()
            dh = [g @ w.t().contiguous() for w in ws]
            dw = [h.t().contiguous() @ g for h in hs]
            return (None, None, None) + tuple(dh) + tuple(dw)

    class ReduceForward(torch.autograd.Function):
        """g: forward all-reduce of the P partial outputs; backward identity per rank."""

        @staticmethod
        def forward(ctx, group: EchoGroup, shape, *partials):
            ctx.dtypes = [p.dtype for p in partials]
            return group.allreduce([p.to(torch.bfloat16) for p in partials], B.ECHO_FWD).view(shape)

        @staticmethod
        def backward(ctx, grad):
            g = grad.contiguous()
            return (None, None) + tuple(g.reshape(-1).to(dt) for dt in ctx.dtypes)

    class ReduceBackward(torch.autograd.Function):
        """f: forward replicates the input to every rank; backward all-reduces the
        P input gradients."""

        @staticmethod
        def forward(ctx, group: EchoGroup, x):
            ctx.group, ctx.shape, ctx.dtype = group, x.shape, x.dtype
            return tuple(x.clone() for _ in range(group.P))

        @staticmethod
        def backward(ctx, *grads):
            parts = [g.to(torch.bfloat16).contiguous() for g in grads]
            out = ctx.group.allreduce(parts, B.ECHO_BWD)
            return None, out.view(ctx.shape).to(ctx.dtype)

    class ColumnParallelEcho(torch.autograd.Function):
        """f(a) @ W1_r with the input-gradient products in bfloat16 on libecho's
        matrix-core kernel: forward gives every rank's pre-activation a @ W1_r
        (fp32, no reduction); backward gives dL/da through Echo on the backward
        state as sum_r bf16(bf16(dpre_r) @ bf16(W1_r)^T) (fused: stage 1 in the
        product's epilogue), and the fp32 weight gradients a^T dpre_r."""

        @staticmethod
        def forward(ctx, group: "EchoGroup", fused: bool, a, *w1s):
            ctx.save_for_backward(a, *w1s)
            ctx.group, ctx.fused = group, fused
            return tuple(a @ w for w in w1s)

        @staticmethod
        def backward(ctx, *gpres):
            a, *w1s = ctx.saved_tensors
            A = [g.to(torch.bfloat16).contiguous() for g in gpres]   # [T, F/P]
            W = [w.to(torch.bfloat16).contiguous() for w in w1s]     # [H, F/P]: output features by K
            da = ctx.group.product_allreduce(A, W, ctx.fused, B.ECHO_BWD).view(a.shape)
            dw = [a.t().contiguous() @ g for g in gpres]
            return (None, None, da) + tuple(dw)

    once = torch.autograd.function.once_differentiable

    def quantize(mats, fmt, straight=True, transposed=True):
        """Row blocks of fp32 or bf16 matrices [T, K], as they are and transposed (None: not
        wanted)."""
        R, C = mats[0].shape
        dev = mats[0].device
        rows = [B.EchoFp8.empty(R, C, fmt, device=dev) for _ in mats] if straight else None
        cols = [B.EchoFp8.empty(C, R, fmt, device=dev) for _ in mats] if transposed else None
        B.echo_quantize_fp8(mats, rows, cols)
        return rows, cols

    def kept(acts8t, w8, for_inputs, for_weights):
        """The operands of the backward products: transposed activations for the weights'
        gradients, weights for the inputs' (empty where not wanted)."""
        if for_inputs and w8[0] is None:
            raise ValueError("the weights were laid out for a pass without gradients")
        return (acts8t if for_weights else []), (w8[0] if for_inputs else [])

    def flat(*lists):
        """The tensors of lists of 8-bit matrices, for save_for_backward."""
        return [t for mats in lists for m in mats for t in m]

    def matrices(tensors):
        """8-bit matrices from saved tensors.  A hook may have moved them: codes that lost
        their rows' padding on the way get it back."""
        mats = []
        for codes, scales in zip(tensors[::2], tensors[1::2]):
            if codes.shape[0] > 1 and codes.stride(0) % 16:
                padded = codes.new_empty(codes.shape[0], (codes.shape[1] + 15) // 16 * 16)[:, :codes.shape[1]]
                codes = padded.copy_(codes)
            mats.append((codes, scales))
        return mats

    def products(A, W, dtype):
        out = [torch.empty(A[0][0].shape[0], W[0][0].shape[0], dtype=dtype, device=A[0][0].device) for _ in A]
        B.echo_gemm_fp8(A, W, out)
        return out

    class RowParallelFp8(torch.autograd.Function):
        """g(h_r @ W2_r) in 8-bit products: forward sums bf16(q(h_r) q(W2_r)) over the
        ranks through Echo; backward gives dh_r = q(g) q(W2_r)^T (bfloat16) and
        dW2_r = q(h_r^T) q(g^T)^T (fp32).  q is the rounding to 8 bits, with blocks
        along the dimension that is summed over; it passes gradients straight
        through.  ``w8``: the weights both ways (TPMLPStack.quantize_weights).  Only what
        the gradients asked for need is laid out and kept; ``grads`` false: none."""

        @staticmethod
        def forward(ctx, group: "EchoGroup", shape, w8, grads: bool, *hw):
            P = group.P
            hs, ws = hw[:P], hw[P:]
            for_h, for_w = (grads and any(ctx.needs_input_grad[i:i + P]) for i in (4, 4 + P))
            h8, h8t = quantize([h.detach().contiguous() for h in hs], "e4m3", True, for_w)
            h8t, w8b = kept(h8t, w8, for_h, for_w)
            ctx.save_for_backward(*flat(h8t, w8b))
            ctx.P, ctx.n_acts, ctx.h_dtype, ctx.w_dtype = P, 2 * len(h8t), hs[0].dtype, ws[0].dtype
            parts = products(h8, w8[1], torch.bfloat16)
            return group.allreduce([p.view(-1) for p in parts], B.ECHO_FWD).view(shape)

        @staticmethod
        @once
        def backward(ctx, grad):
            P = ctx.P
            saved = ctx.saved_tensors
            for_h, for_w = (any(ctx.needs_input_grad[i:i + P]) for i in (4, 4 + P))
            g8, g8t = quantize([grad.contiguous()], "e5m2", for_h, for_w)
            dh = dw = (None,) * P
            if for_h:
                dh = tuple(d.to(ctx.h_dtype) for d in products(g8 * P, matrices(saved[ctx.n_acts:]), torch.bfloat16))
            if for_w:
                dw = tuple(d.to(ctx.w_dtype) for d in products(matrices(saved[:ctx.n_acts]), g8t * P, torch.float32))
            return (None, None, None, None) + dh + dw

    class ColumnParallelFp8(torch.autograd.Function):
        """f(a) @ W1_r in 8-bit products: forward gives every rank's pre-activation
        q(a) q(W1_r) (bfloat16); backward gives dL/da through Echo on the backward
        state as the sum of bf16(q(dpre_r) q(W1_r)^T), and dW1_r = q(a^T) q(dpre_r^T)^T
        (fp32)."""

        @staticmethod
        def forward(ctx, group: "EchoGroup", w8, grads: bool, a, *w1s):
            for_a, for_w = grads and ctx.needs_input_grad[3], grads and any(ctx.needs_input_grad[4:])
            a8, a8t = quantize([a.detach().contiguous()], "e4m3", True, for_w)
            a8t, w8b = kept(a8t, w8, for_a, for_w)
            ctx.save_for_backward(*flat(a8t, w8b))
            ctx.n_acts = 2 * len(a8t)
            ctx.group, ctx.shape, ctx.a_dtype, ctx.w_dtype = group, a.shape, a.dtype, w1s[0].dtype
            return tuple(products(a8 * group.P, w8[1], torch.bfloat16))

        @staticmethod
        @once
        def backward(ctx, *gpres):
            P = ctx.group.P
            saved = ctx.saved_tensors
            for_a, for_w = ctx.needs_input_grad[3], any(ctx.needs_input_grad[4:])
            g8, g8t = quantize([g.contiguous() for g in gpres], "e5m2", for_a, for_w)
            da, dw = None, (None,) * P
            if for_a:
                parts = products(g8, matrices(saved[ctx.n_acts:]), torch.bfloat16)
                da = ctx.group.allreduce([p.view(-1) for p in parts], B.ECHO_BWD).view(ctx.shape).to(ctx.a_dtype)
            if for_w:
                dw = tuple(d.to(ctx.w_dtype) for d in products(matrices(saved[:ctx.n_acts]) * P, g8t, torch.float32))
            return (None, None, None, da) + dw

    class DropoutAdd(torch.autograd.Function):
        """residual + dropout(x); backward draws the same mask again.  ``rng`` must still
        hold the forward pass's values in the backward pass (autograd refuses a changed
        one)."""

        @staticmethod
        def forward(ctx, x, residual, p: float, rng, offset: int, first: int):
            ctx.save_for_backward(rng)
            ctx.args, ctx.x_dtype = (p, offset, first), x.dtype
            out = torch.empty_like(x if residual is None else residual, memory_format=torch.contiguous_format)
            return B.echo_dropout_add(x.contiguous(), out, p, rng, residual=None if residual is None else
                                      residual.contiguous(), offset=offset, first=first)

        @staticmethod
        @once
        def backward(ctx, grad):
            (rng,) = ctx.saved_tensors
            p, offset, first = ctx.args
            grad = grad.contiguous()
            dx = None
            if ctx.needs_input_grad[0]:
                dx = torch.empty_like(grad, dtype=ctx.x_dtype)
                B.echo_dropout_add(grad, dx, p, rng, offset=offset, first=first)
            return dx, grad if ctx.needs_input_grad[1] else None, None, None, None, None

    def gradient(ctx, i, like):
        """An empty gradient of input i, None where it is not wanted."""
        return torch.empty_like(like, memory_format=torch.contiguous_format) if ctx.needs_input_grad[i] else None

    class BlockNorm(torch.autograd.Function):
        """The end of a block and the start of the next (see echo_block_norm): (out, a), out
        alone without ``a_dtype``, a alone without ``y``.  The stored out is all that is kept
        beside the inputs."""

        @staticmethod
        def forward(ctx, x, y, gate, w_post, w_pre, options, a_dtype):
            x, y = x.contiguous(), None if y is None else y.contiguous()
            out = None if y is None else torch.empty_like(x)
            a = None if a_dtype is None else torch.empty_like(x, dtype=a_dtype)
            B.echo_block_norm(x, out, a, y=y, gate=gate, w_post=w_post, w_pre=w_pre, **options)
            ctx.save_for_backward(x if out is None else out, y, gate, w_post, w_pre)
            ctx.options = options
            ctx.set_materialize_grads(False)
            return a if out is None else out if a is None else (out, a)

        @staticmethod
        @once
        def backward(ctx, *grads):
            out, y, gate, w_post, w_pre = ctx.saved_tensors
            grads = [None if g is None else g.contiguous() for g in grads]
            dout, da = grads if len(grads) == 2 else (None, grads[0]) if y is None else (grads[0], None)
            if dout is None and da is None:
                return (None,) * 7
            dx = gradient(ctx, 0, out)
            dy, dgate, dw_post, dw_pre = (None if t is None else gradient(ctx, i, t)
                                          for i, t in ((1, y), (2, gate), (3, w_post), (4, w_pre)))
            if da is None:  # the next block's input was not used
                dw_pre = None if dw_pre is None else dw_pre.zero_()
                if not any(ctx.needs_input_grad[:4]):
                    return None, None, None, None, dw_pre, None, None
            B.echo_block_norm_backward(out, dout=dout, da=da, dx=dx, y=y, dy=dy, gate=gate, dgate=dgate, w_post=w_post,
                                       dw_post=dw_post, w_pre=None if da is None else w_pre,
                                       dw_pre=None if da is None else dw_pre, **ctx.options)
            return dx, dy, dgate, dw_post, dw_pre, None, None

    class VocabEmbed(torch.autograd.Function):
        """The all-reduce, on the forward state, of every rank's bfloat16 partial embedding
        (see echo_embed); the rounding passes gradients straight through."""

        @staticmethod
        def forward(ctx, group: "EchoGroup", tokens, scale: float, *tables):
            tokens = tokens.contiguous()
            shape = (tokens.numel(), tables[0].shape[1])
            parts = [torch.empty(shape, dtype=torch.bfloat16, device=t.device) for t in tables]
            B.echo_embed(tables, tokens, parts, scale=scale)
            ctx.save_for_backward(tokens)
            ctx.scale, ctx.like = scale, [(t.shape, t.dtype) for t in tables]
            return group.allreduce([p.view(-1) for p in parts], B.ECHO_FWD).view(tokens.shape + shape[1:])

        @staticmethod
        @once
        def backward(ctx, grad):
            (tokens,) = ctx.saved_tensors
            d = [torch.empty(shape, dtype=dtype, device=grad.device) for shape, dtype in ctx.like]
            B.echo_embed_backward(grad.contiguous().view(tokens.numel(), grad.shape[-1]), tokens, d, scale=ctx.scale)
            return (None, None, None) + tuple(d)

    return (ReduceForward, ReduceBackward, RowParallelEcho, ColumnParallelEcho, RowParallelFp8, ColumnParallelFp8, DropoutAdd,
            BlockNorm, VocabEmbed)


_FNS = None


def _grad_enabled() -> bool:
    import torch
    return torch.is_grad_enabled()  # always false inside a Function's forward


def row_parallel_echo(group: "EchoGroup", hs, ws, shape, fused: bool):
    """g(sum_r h_r @ W2_r) with bf16 products on libecho's kernel (see RowParallelEcho)."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[2].apply(group, shape, fused, *hs, *ws)


def column_parallel_echo(group: "EchoGroup", a, ws, fused: bool):
    """[a @ W1_r] with the input gradient through bf16 products on libecho's
    kernel and Echo's backward state (see ColumnParallelEcho)."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[3].apply(group, fused, a, *ws)


def row_parallel_fp8(group: "EchoGroup", hs, ws, shape, w8):
    """g(sum_r h_r @ W2_r) in 8-bit products (see RowParallelFp8)."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[4].apply(group, shape, w8, _grad_enabled(), *hs, *ws)


def column_parallel_fp8(group: "EchoGroup", a, ws, w8):
    """[a @ W1_r] in 8-bit products, the input gradient through Echo's backward state
    (see ColumnParallelFp8)."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[5].apply(group, w8, _grad_enabled(), a, *ws)


def dropout_add(x, residual, p: float, rng, offset: int = 0, first: int = 0):
    """residual + dropout(x), differentiable in both (``residual`` None: dropout(x));
    the mask is drawn from ``rng`` (int64 device tensor: key, step), ``offset`` and
    ``first`` in both passes (see echo_dropout_add)."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[6].apply(x, residual, p, rng, offset, first)


def block_norm(x, y=None, gate=None, w_post=None, w_pre=None, *, post_norm: bool = False, residual_scale: float = 1.0,
               weight_offset: float = 0.0, eps: float = 1e-6, a: bool = True, a_dtype=None):
    """(out, a): out = residual_scale * x + gate * n, n = rmsnorm(y) * (weight_offset + w_post)
    or y, and a = rmsnorm(out) * (weight_offset + w_pre) of ``a_dtype`` (x's by default),
    differentiable in x, y, gate and the weights (see echo_block_norm).  Without ``y`` out is
    x; ``a`` false: a is None."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    if y is None and not a:
        raise ValueError("neither a block's output nor a norm")
    options = dict(post_norm=post_norm, residual_scale=residual_scale, weight_offset=weight_offset, eps=eps)
    got = _FNS[7].apply(x, y, gate, w_post, w_pre, options, (a_dtype or x.dtype) if a else None)
    return (x, got) if y is None else got if a else (got, None)


def vocab_embed(group: "EchoGroup", tables, tokens, scale: float = 1.0):
    """The embedding [.., H] of ``tokens`` from P tables [rows, H] that hold consecutive
    stretches of the vocabulary: their partials through Echo's forward state (fp32),
    differentiable in the tables, which are float32 or bfloat16 (the partials are bfloat16,
    and float16 does not go with it).  Tokens outside the vocabulary give zeros."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[8].apply(group, tokens, scale, *tables)


def clip_grads(grads, max_norm: float):
    """Scales ``grads`` in place so that the norm of all of them together is at most
    ``max_norm``; returns the norm before (one float32 element, see echo_clip_grads)."""
    import torch

    grads = [g.detach() for g in grads]
    if not grads:
        raise ValueError("no gradients")
    return B.echo_clip_grads(grads, max_norm, torch.empty(1, dtype=torch.float32, device=grads[0].device))


def quantize_weights_fp8(ws, backward: bool = True):
    """P weights [K_in, K_out] in e4m3 with a scale per 128 x 128 block: (as they are,
    transposed), the operands of the input-gradient and of the forward products; the
    first None without ``backward``."""
    R, C = ws[0].shape
    dev = ws[0].device
    rows = [B.EchoFp8.empty(R, C, block_rows=B.ECHO_FP8_BLOCK, device=dev) for _ in ws] if backward else None
    cols = [B.EchoFp8.empty(C, R, block_rows=B.ECHO_FP8_BLOCK, device=dev) for _ in ws]
    B.echo_quantize_fp8([w.detach() for w in ws], rows, cols)
    return rows, cols


def reduce_forward(group: EchoGroup, partials, shape):
    """g(partials): all-reduce on the forward state; gradient passes through."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[0].apply(group, shape, *partials)


def replicate(group: EchoGroup, x):
    """f(x): P copies of x; their gradients are all-reduced on the backward state."""
    global _FNS
    if _FNS is None:
        _FNS = _fns()
    return _FNS[1].apply(group, x)


class TPMLPStack:
    """L pre-norm MLP blocks, each split over P ranks: W1 column-parallel
    ([H, F] in P slices of F/P columns), W2 row-parallel ([F, H] in P slices of
    F/P rows); x <- x + g(sum_r gelu(f(a)_r @ W1_r) @ W2_r), a = rmsnorm(x).
    Weights are fp32 and seeded.  product "f32": the products are taken in fp32
    and each rank's partial output is rounded to bf16 (the wire dtype);
    "bf16" / "bf16_fused": the products whose outputs are reduced run in
    bfloat16 on libecho's kernel, the row-parallel W2 product in the forward
    pass and the column-parallel W1 input-gradient product in the backward
    pass (written out, or with stage 1 in their epilogues; T a multiple of 64,
    H of 128, F/P of 64); "fp8": every product of both passes in 8-bit floating
    point (any sizes).  ``dropout``: probability with which an element of a reduced
    output is dropped before the residual add while ``training`` is set; the masks
    come from ``rng`` (key ``seed``, step), layer l's from step + l, and train_step
    moves the step on by the number of layers.

    ``block_norms``: x <- residual_scale * x + gate * rmsnorm(y) * w_post, a = rmsnorm(x) *
    w_pre, with a gate and two weights [H] per layer that start at 1; a dropout then
    applies to y.  ``vocab``: an embedding of that many rows (rounded up to a multiple of
    P) in P stretches, times sqrt(H); forward then takes tokens too."""

    def __init__(self, layers: int, hidden: int, ffn: int, P: int, seed: int = 0, device=None,
                 product: str = "f32", dropout: float = 0.0, block_norms: bool = False, residual_scale: float = 1.0,
                 vocab: int = 0):
        import torch

        if ffn % P:
            raise ValueError("ffn must be divisible by P")
        if product not in ("f32", "bf16", "bf16_fused", "fp8"):
            raise ValueError(f"product {product!r}")
        if not 0.0 <= dropout <= 1.0 - 2.0 ** -16:  # what echo_dropout_add takes
            raise ValueError(f"dropout {dropout!r}")
        if not math.isfinite(residual_scale) or (residual_scale != 1.0 and not block_norms):
            raise ValueError(f"residual_scale {residual_scale!r} (block_norms {block_norms!r})")
        if vocab < 0:
            raise ValueError(f"vocab {vocab!r}")
        self.L, self.H, self.F, self.P, self.product = layers, hidden, ffn, P, product
        self.block_norms, self.residual_scale = block_norms, residual_scale
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.dropout, self.training = dropout, True
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=dev) if dropout > 0 else None
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.w1, self.w2 = [], []
        for _ in range(layers):
            w1 = torch.randn(hidden, ffn, generator=g, device=dev) / hidden ** 0.5
            w2 = torch.randn(ffn, hidden, generator=g, device=dev) / ffn ** 0.5 * 0.5
            self.w1.append([w1[:, r * ffn // P:(r + 1) * ffn // P].contiguous().requires_grad_()
                            for r in range(P)])
            self.w2.append([w2[r * ffn // P:(r + 1) * ffn // P, :].contiguous().requires_grad_()
                            for r in range(P)])
        ones = lambda: [torch.ones(hidden, device=dev).requires_grad_() for _ in range(layers)] if block_norms else []
        self.w_pre, self.w_post, self.gate = ones(), ones(), ones()
        self.tables = [(torch.randn(-(-vocab // P), hidden, generator=g, device=dev) / hidden ** 0.5).requires_grad_()
                       for _ in range(P)] if vocab else []

    def parameters(self):
        return [w for layer in self.w1 + self.w2 for w in layer] + self.w_pre + self.w_post + self.gate + self.tables

    def quantize_weights(self):
        """The weights of every layer in 8 bits, for ``forward(..., weights8=...)`` as long
        as they do not change; without it a forward pass quantizes them itself."""
        return [(quantize_weights_fp8(w1), quantize_weights_fp8(w2)) for w1, w2 in zip(self.w1, self.w2)]

    def _block(self, l: int, a, shape, group: EchoGroup, weights8):
        """The reduced output of layer l's block for its normalised input."""
        import torch

        gelu = torch.nn.functional.gelu
        if self.product == "fp8":
            w8 = weights8[l] if weights8 is not None else [quantize_weights_fp8(w, torch.is_grad_enabled())
                                                           for w in (self.w1[l], self.w2[l])]
            pres = column_parallel_fp8(group, a, self.w1[l], w8[0])
            # gelu in fp32 of the bfloat16 pre-activations
            return row_parallel_fp8(group, [gelu(p.float()) for p in pres], self.w2[l], shape, w8[1])
        if self.product == "f32":
            xs = replicate(group, a)
            hs = [gelu(xs[r] @ self.w1[l][r]) for r in range(self.P)]
            partials = [(hs[r] @ self.w2[l][r]).to(torch.bfloat16) for r in range(self.P)]
            return reduce_forward(group, [p.reshape(-1) for p in partials], shape)
        pres = column_parallel_echo(group, a, self.w1[l], self.product == "bf16_fused")
        return row_parallel_echo(group, [gelu(p) for p in pres], self.w2[l], shape, self.product == "bf16_fused")

    def forward(self, x, group: EchoGroup, weights8=None):
        """``x``: the residual stream [T, H], or tokens [T] where there is a vocabulary."""
        import torch

        if weights8 is not None and self.product != "fp8":
            raise ValueError("weights8 goes with product 'fp8'")
        if not x.is_floating_point():
            if not self.tables:
                raise ValueError("tokens need a vocabulary")
            x = vocab_embed(group, self.tables, x, self.H ** 0.5)
        drop = self.dropout > 0 and self.training
        if self.block_norms:
            a = block_norm(x, w_pre=self.w_pre[0])[1] if self.L else None
            for l in range(self.L):
                y = self._block(l, a, x.shape, group, weights8)
                if drop:
                    y = dropout_add(y, None, self.dropout, self.rng, offset=l)
                more = l + 1 < self.L
                x, a = block_norm(x, y, self.gate[l], self.w_post[l], self.w_pre[l + 1] if more else None, post_norm=True,
                                  residual_scale=self.residual_scale, a=more)
            return x
        for l in range(self.L):
            a = x * torch.rsqrt(x.pow(2).mean(dim=-1, keepdim=True) + 1e-6)
            y = self._block(l, a, x.shape, group, weights8)
            x = dropout_add(y, x, self.dropout, self.rng, offset=l) if drop else x + y
        return x


def train_step(model: TPMLPStack, group: EchoGroup, x0, target, weights8=None, max_norm=None):
    """One forward + backward; returns (loss, dL/dx0, [dL/dW...]).  ``x0``: the residual
    stream (the gradients of a vocabulary's tables are zeros), or tokens (dL/dx0 is None).
    ``weights8``: the weights in 8 bits (quantize_weights), for several steps before they
    change.  ``max_norm``: the gradients of the parameters are clipped to that norm together,
    and the norm before is returned too, as a fourth value."""
    import torch

    group.reset()
    x = x0.detach().clone()
    if x.is_floating_point():
        x.requires_grad_()
    for p in model.parameters():
        p.grad = None
    y = model.forward(x, group, weights8=weights8)
    loss = torch.nn.functional.mse_loss(y, target)
    loss.backward()
    if model.rng is not None and model.training:
        model.rng[1] += model.L  # the next step draws other masks
    # a parameter without a part in the pass: the tables beside a residual stream
    grads = [torch.zeros_like(p) if p.grad is None else p.grad.detach() for p in model.parameters()]
    result = loss.detach(), None if x.grad is None else x.grad.detach(), grads
    return result if max_norm is None else result + (clip_grads(grads, max_norm),)
