"""A tensor-parallel training step with an embedding, block norms and clipping: each autograd
function against its formula in 64 bits, whole steps through Echo against the oracle, and the
operators run together as the stack runs them."""
import numpy as np
import pytest

from oracle import echo_oracle as eo
from step_helpers import U, assert_close, block_norm_backward_ref, block_norm_ref, embed_backward_ref, norm_ref, np64

pytestmark = pytest.mark.gpu

T, H, F, P, LAYERS, VOCAB, EPS = 96, 160, 256, 2, 3, 101, 1e-6


@pytest.fixture(scope="module")
def tp(cuda):
    from error_compensated_bit_echo_amd import tp
    return tp


def tensors(seed, *shapes):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda") for s in shapes]


def block(dtype, gates=2):
    import torch
    x, y, dout, da = [t.to(dtype) for t in tensors(1, *[(T, H)] * 4)]
    gate, w_post, w_pre = tensors(2, (gates, H), (H,), (H,))
    leaves = [t.requires_grad_() for t in (x, y, gate, w_post, w_pre)]
    return leaves, dout, da


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("used", ["both", "out", "a"])
def test_block_norm_follows_its_formula(cuda, tp, dtype, used):
    import torch
    dt = getattr(torch, dtype)
    (x, y, gate, w_post, w_pre), dout, da = block(dt)
    out, a = tp.block_norm(x, y, gate, w_post, w_pre, post_norm=True, residual_scale=0.5, weight_offset=0.25, a_dtype=torch.bfloat16)
    assert out.dtype == dt and a.dtype == torch.bfloat16
    want, off = block_norm_ref(np64(x), np64(y), np64(gate), np64(w_post), True, 0.5, 0.25, EPS)
    assert_close(out, want, off, dt, "out")
    assert_close(a, *norm_ref(np64(out), np64(w_pre), 0.25, EPS), torch.bfloat16, "a")
    loss = 0.0
    if used != "a":
        loss = loss + (out * dout).sum()
    if used != "out":
        loss = loss + (a * da.bfloat16()).sum()
    loss.backward()
    ref = block_norm_backward_ref(np64(out), np64(y), np64(dout) if used != "a" else None,
                                  np64(da.bfloat16()) if used != "out" else None, np64(gate), np64(w_post),
                                  np64(w_pre) if used != "out" else None, True, 0.5, 0.25, EPS)
    for name, t in dict(dx=x, dy=y, dgate=gate, dw_post=w_post, dw_pre=w_pre).items():
        if name == "dw_pre" and used == "out":
            assert t.grad is None or not t.grad.any()
        else:
            assert_close(t.grad, *ref[name], t.dtype, name)


def test_block_norm_of_a_stream_alone_and_of_a_last_block(cuda, tp):
    import torch
    (x, y, gate, w_post, w_pre), dout, da = block(torch.float32, 1)
    same, a = tp.block_norm(x, w_pre=w_pre)
    assert same is x
    (a * da).sum().backward()
    ref = block_norm_backward_ref(np64(x), None, None, np64(da), None, None, np64(w_pre), False, 1.0, 0.0, EPS)
    assert_close(x.grad, *ref["dx"], torch.float32)
    assert_close(w_pre.grad, *ref["dw_pre"], torch.float32)
    x.grad = None
    out, none = tp.block_norm(x, y, gate, w_post, post_norm=True, residual_scale=2.0, a=False)
    assert none is None
    out.backward(dout.expand_as(out))
    ref = block_norm_backward_ref(np64(out), np64(y), np64(dout), None, np64(gate), np64(w_post), None, True, 2.0, 0.0, EPS)
    for name, t in dict(dx=x, dy=y, dgate=gate, dw_post=w_post).items():
        assert_close(t.grad, *ref[name], torch.float32, name)


def test_only_wanted_gradients_are_given(cuda, tp):
    import torch
    (x, y, gate, w_post, w_pre), dout, da = block(torch.float32, 1)
    for t in (x, gate, w_pre):
        t.requires_grad_(False)
    out, a = tp.block_norm(x, y, gate, w_post, w_pre, post_norm=True)
    ((out * dout).sum() + (a * da).sum()).backward()
    assert x.grad is None and gate.grad is None and w_pre.grad is None
    ref = block_norm_backward_ref(np64(out), np64(y), np64(dout), np64(da), np64(gate), np64(w_post), np64(w_pre), True, 1.0, 0.0, EPS)
    assert_close(y.grad, *ref["dy"], y.dtype)
    assert_close(w_post.grad, *ref["dw_post"], y.dtype)


def test_a_weight_whose_output_is_not_used(cuda, tp):
    """The weight before the next block alone wants a gradient, and that block's input is dropped."""
    import torch
    leaves, dout, _ = block(torch.float32, 1)
    for t in leaves[:4]:
        t.requires_grad_(False)
    out, _ = tp.block_norm(*leaves, post_norm=True)
    (out * dout).sum().backward()
    assert leaves[4].grad.shape == (H,) and not leaves[4].grad.any()


def test_block_norm_gradient_against_differences(cuda, tp):
    """Along a direction, with a step of 2^-6: see the operator's own test for what a quotient may be off."""
    import torch
    leaves, dout, da = block(torch.float32)

    def loss(ls):
        out, a = tp.block_norm(*ls, post_norm=True, residual_scale=0.5)
        return (out.double() * dout.double()).sum() + (a.double() * da.double()).sum()

    loss(leaves).backward()
    h = 2.0 ** -6
    for i, t in enumerate(leaves):
        d, = tensors(30 + i, t.shape)
        with torch.no_grad():
            at = [[u.double() + s * h * d.double() if j == i else u for j, u in enumerate(leaves)] for s in (1, -1)]
            q = (loss([u.float() for u in at[0]]) - loss([u.float() for u in at[1]])).item() / (2 * h)
        exact = (t.grad.double() * d.double()).sum().item()
        size = (t.grad.double().abs() * d.double().abs()).sum().item()
        # third order: h^2 / 6 of sums of this size times a few; roundings: 2 T H outputs of up to 8, each off by
        # 30 U with a random sign, over 2 h
        assert abs(q - exact) <= 2e-3 * size + 8 * 30 * U * (2 * T * H) ** 0.5 / (2 * h) * 4, i


def test_dropout_without_a_residual(cuda, tp):
    import torch
    x, g = tensors(4, (T, H), (T, H))
    x.requires_grad_()
    rng = torch.tensor([7, 3], device="cuda")
    y = tp.dropout_add(x, None, 0.25, rng)
    z = tp.dropout_add(x.detach(), torch.zeros_like(x), 0.25, rng)
    assert torch.equal(y, z) and 0 < int((y == 0).sum()) < T * H
    y.backward(g)
    assert torch.equal(x.grad, tp.dropout_add(g, torch.zeros_like(g), 0.25, rng))


@pytest.mark.parametrize("mode", ["echo", "exact"])
@pytest.mark.parametrize("dtype", ["int64", "int32"])
def test_vocab_embed_follows_its_formula(cuda, tp, mode, dtype):
    import torch
    V = 40
    tables = [t.requires_grad_() for t in tensors(5, *[(V, H)] * P)]
    tokens = torch.randint(-2, V * P + 2, (8, 12), device="cuda").to(getattr(torch, dtype))
    group = tp.EchoGroup(P, 96 * H, mode=mode, device=cuda, record=True)
    x = tp.vocab_embed(group, tables, tokens, 3.0)
    assert x.shape == (8, 12, H) and x.dtype == torch.float32
    (d, parts, out), = group.log
    ids, whole = tokens.long().view(-1), torch.zeros(96, H, device="cuda")
    for r, p in enumerate(parts):
        here = (ids >= r * V) & (ids < (r + 1) * V)
        want = torch.zeros(96, H, device="cuda")
        want[here] = 3.0 * tables[r].detach()[ids[here] - r * V]
        assert torch.equal(p.view(96, H), want.bfloat16())
        whole += want.bfloat16().float()
    if mode == "exact":
        assert torch.equal(x.view(96, H), whole)
    else:
        host = np.stack([p.reshape(-1).float().cpu().numpy() for p in parts])
        o = eo.echo_call(host, eo.OracleState(96 * H), d)
        assert np.array_equal(x.detach().reshape(-1).cpu().numpy().view(np.uint32), o["out"].view(np.uint32))
    g, = tensors(6, (8, 12, H))
    x.backward(g)
    want, off = embed_backward_ref(np64(g).reshape(96, H), ids.cpu().numpy(), P * V, 0, 3.0)
    for r, t in enumerate(tables):
        assert_close(t.grad, want[r * V:(r + 1) * V], off[r * V:(r + 1) * V], torch.float32)


def test_clip_grads(cuda, tp):
    import torch
    grads = tensors(7, (5, 9), (1000,), ())
    before = [g.clone() for g in grads]
    norm = tp.clip_grads(grads, 2.0)
    total = np.sqrt(sum((np64(g) ** 2).sum() for g in before))
    assert abs(norm.item() - total) <= total * (U + 1e-12)
    for g, b in zip(grads, before):
        want = np64(b) * (2.0 / (total + 1e-6))
        assert_close(g, want, np.abs(want) * 3 * U, torch.float32)


def stack(cuda, tp, product="f32", **kw):
    import torch
    model = tp.TPMLPStack(LAYERS, H, F, P, seed=11, device=cuda, product=product, block_norms=True, residual_scale=0.75,
                          vocab=VOCAB, **kw)
    g = torch.Generator(device=cuda)
    g.manual_seed(12)
    with torch.no_grad():
        for w in model.w_pre + model.w_post + model.gate:
            w += 0.2 * torch.randn(H, generator=g, device=cuda)
    tokens = torch.randint(0, VOCAB, (T,), generator=g, device=cuda)
    return model, tokens, torch.randn(T, H, generator=g, device=cuda)


@pytest.mark.parametrize("product", ["f32", "fp8"])
@pytest.mark.parametrize("variant", [{}, {"sender_feedback": True, "state_bf16": True}])
def test_step_reductions_match_the_oracle(cuda, tp, product, variant):
    """Every reduction of a whole step is an Echo all-reduce of the recorded partials on its
    direction's state: the embedding's, then the layers', then the gradients'."""
    model, tokens, target = stack(cuda, tp, product, dropout=0.1)
    group = tp.EchoGroup(P, T * H, device=cuda, record=True, **variant)
    loss, dx, grads, norm = tp.train_step(model, group, tokens, target, max_norm=0.01)
    assert dx is None and len(grads) == len(model.parameters())
    assert [d for d, _, _ in group.log] == [0] * (LAYERS + 1) + [1] * LAYERS
    st = eo.OracleState(T * H)
    for k, (d, parts, out) in enumerate(group.log):
        host = np.stack([p.reshape(-1).float().cpu().numpy() for p in parts])
        o = eo.echo_call(host, st, d, **variant)
        assert np.array_equal(out.cpu().numpy().view(np.uint32), o["out"].view(np.uint32)), f"call {k} dir {d}"
    assert all(bool(g.isfinite().all()) and bool((g != 0).any()) for g in grads + [loss, norm])


def test_clipped_step_is_the_step_scaled(cuda, tp):
    import torch
    model, tokens, target = stack(cuda, tp)
    group = tp.EchoGroup(P, T * H, device=cuda)
    loss, _, grads = tp.train_step(model, group, tokens, target)
    before = [g.clone() for g in grads]
    loss2, _, clipped, norm = tp.train_step(model, group, tokens, target, max_norm=0.01)
    total = np.sqrt(sum((np64(g) ** 2).sum() for g in before))
    assert torch.equal(loss, loss2) and total > 0.02
    assert abs(norm.item() - total) <= total * (U + 1e-10)
    for c, b in zip(clipped, before):
        want = np64(b) * (0.01 / (total + 1e-6))
        assert_close(c, want, np.abs(want) * 3 * U, torch.float32)
    _, _, same, _ = tp.train_step(model, group, tokens, target, max_norm=1e9)
    assert all(torch.equal(a, b) for a, b in zip(same, before))


def test_forward_is_its_parts(cuda, tp):
    """The stack's forward pass is its functions put together by hand."""
    import torch
    model, tokens, target = stack(cuda, tp, dropout=0.2)
    group = tp.EchoGroup(P, T * H, device=cuda)
    loss, _, _ = tp.train_step(model, group, tokens, target)
    model.rng[1] -= LAYERS
    group.reset()
    x = tp.vocab_embed(group, model.tables, tokens, H ** 0.5)
    for l in range(LAYERS):
        # the norms apart: the fused one starts from the same stream
        _, a = tp.block_norm(x, w_pre=model.w_pre[l])
        y = model._block(l, a, x.shape, group, None)
        y = tp.dropout_add(y, None, model.dropout, model.rng, offset=l)
        x, _ = tp.block_norm(x, y, model.gate[l], model.w_post[l], post_norm=True, residual_scale=0.75, a=False)
    assert torch.equal(torch.nn.functional.mse_loss(x, target), loss)


def test_steps_repeat(cuda, tp):
    import torch
    model, tokens, target = stack(cuda, tp, "fp8", dropout=0.1)
    group = tp.EchoGroup(P, T * H, device=cuda)
    runs = []
    for _ in range(3):
        model.rng[1] = 0
        loss, _, grads, norm = tp.train_step(model, group, tokens, target, max_norm=1.0)
        runs.append([loss, norm] + [g.clone() for g in grads])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_captured_forward_pass(cuda, tp):
    """Tokens to the last stream in one graph, replayed on new tokens with eager passes between."""
    import torch
    model, tokens, _ = stack(cuda, tp, "fp8", dropout=0.1)
    w8 = model.quantize_weights()
    graphed, eager = (tp.EchoGroup(P, T * H, device=cuda) for _ in range(2))
    tokens = tokens.clone()

    def run(group):
        group.reset()
        return model.forward(tokens, group, weights8=w8)

    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(graphed)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(graphed)
        for i in range(4):
            tokens.copy_(torch.randint(0, VOCAB, (T,), device=cuda))
            model.rng[1] += LAYERS
            graph.replay()
            want = run(eager)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
