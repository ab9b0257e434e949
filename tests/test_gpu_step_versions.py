"""What the training step's operators write counts as written for autograd: a graph that saved a
tensor refuses its backward pass after a call has changed the tensor."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E(cuda):
    import error_compensated_bit_echo_amd as E
    return E


def calls(E):
    """name -> (call, what it writes, what it only reads)"""
    import torch
    new = lambda *shape: torch.ones(shape, device="cuda")
    T, C, V = 12, 40, 9
    x, y, out, a, dout, da, dx, dy = (new(T, C) for _ in range(8))
    gate, dgate, w_post, dw_post, w_pre, dw_pre = (new(C) for _ in range(6))
    tables, parts = [new(V, C) for _ in range(2)], [new(T, C) for _ in range(2)]
    tokens = torch.zeros(T, dtype=torch.long, device="cuda")
    grads, apart, norm = [new(7), new(3, 5)], [new(7), new(3, 5)], new(1)
    params = dict(y=y, gate=gate, w_post=w_post, w_pre=w_pre, post_norm=True)
    read = [y, gate, w_post, w_pre]
    return {
        "block norm": (lambda: E.echo_block_norm(x, out, a, **params), [out, a], [x] + read),
        "block norm in place": (lambda: E.echo_block_norm(x, x, a, **params), [x, a], read),
        "norm alone": (lambda: E.echo_block_norm(x, a=a), [a], [x]),
        "block norm backward": (lambda: E.echo_block_norm_backward(out, dout=dout, da=da, dx=dx, dy=dy, dgate=dgate, dw_post=dw_post,
                                                                   dw_pre=dw_pre, **params),
                                [dx, dy, dgate, dw_post, dw_pre], [out, dout, da] + read),
        "block norm backward in place": (lambda: E.echo_block_norm_backward(out, dout=dout, dx=dout), [dout], [out]),
        "grad norm": (lambda: E.echo_grad_norm(grads, norm), [norm], grads),
        "clip": (lambda: E.echo_clip_grads(grads, 1.0, norm, out=(t for t in apart)), apart + [norm], grads),
        "clip in place": (lambda: E.echo_clip_grads((g for g in grads), 1.0, norm), grads + [norm], []),
        "embed": (lambda: E.echo_embed(tables, tokens, parts), parts, tables + [tokens]),
        "embed backward": (lambda: E.echo_embed_backward(x, tokens, tables), tables, [x, tokens]),
    }


@pytest.mark.parametrize("name", ["block norm", "block norm in place", "norm alone", "block norm backward",
                                  "block norm backward in place", "grad norm", "clip", "clip in place", "embed", "embed backward"])
def test_written_tensors_change_their_version(E, name):
    import torch
    call, written, read = calls(E)[name]
    before = [t._version for t in written + read]
    call()
    after = [t._version for t in written + read]
    assert all(b > a for a, b in zip(before[:len(written)], after)) and before[len(written):] == after[len(written):]
    with torch.inference_mode():  # tensors without a version
        call, written, _ = calls(E)[name]
        call()
    call()
    assert all(t.is_inference() for t in written)


def test_clipping_what_a_graph_saved_is_noticed(cuda):
    """The clipped tensors are the caller's own, reached through detached ones."""
    import torch
    from error_compensated_bit_echo_amd import tp
    g = torch.randn(100, device="cuda", requires_grad=True)
    square = (g * g).sum()
    tp.clip_grads([g], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        square.backward()
    again = (g * g).sum()  # of the clipped values
    again.backward()
    assert torch.equal(g.grad, 2 * g.detach())


def test_a_stream_written_in_place_is_noticed(E):
    import torch
    x = torch.randn(8, 64, device="cuda")
    w = torch.randn(64, device="cuda", requires_grad=True)
    product = (x * w).sum()
    E.echo_block_norm(x, x, y=torch.ones_like(x), post_norm=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.backward()
