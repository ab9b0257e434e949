"""Training steps of the tensor-parallel stack at the edges of what they take, on the CPU (exact
reduction, products in fp32)."""
import pytest

from error_compensated_bit_echo_amd import tp

T, H, F, P = 6, 32, 64, 2


def stream():
    import torch
    g = torch.Generator().manual_seed(3)
    return torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)


@pytest.mark.parametrize("layers", [1, 2])
def test_step_on_a_residual_stream_of_a_stack_with_a_vocabulary(layers):
    """The tables take no part: the step is that of the stack without them, their gradients zeros."""
    import torch
    x0, target = stream()
    plain = tp.TPMLPStack(layers, H, F, P, seed=5, device="cpu")
    vocab = tp.TPMLPStack(layers, H, F, P, seed=5, device="cpu", vocab=11)
    loss, dx, grads = tp.train_step(plain, tp.EchoGroup(P, T * H, mode="exact", device="cpu"), x0, target)
    loss2, dx2, grads2 = tp.train_step(vocab, tp.EchoGroup(P, T * H, mode="exact", device="cpu"), x0, target)
    assert torch.equal(loss, loss2) and torch.equal(dx, dx2)
    assert len(grads2) == len(vocab.parameters()) == len(grads) + P
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
    for g, table in zip(grads2[-P:], vocab.tables):
        assert g.shape == table.shape and g.dtype == table.dtype and not g.requires_grad and not g.any()


@pytest.mark.parametrize("shape", [(0,), (3, 0)])
def test_embedding_of_no_tokens(monkeypatch, shape):
    """Both directions around the kernels, which stand-ins replace here."""
    import torch
    asked = []

    def backward(dout, tokens, dtables, scale=1.0):
        asked.append((tuple(dout.shape), tuple(tokens.shape)))
        for d in dtables:
            d.zero_()

    monkeypatch.setattr(tp.B, "echo_embed", lambda tables, tokens, out, scale=1.0: out)
    monkeypatch.setattr(tp.B, "echo_embed_backward", backward)
    tables = [torch.randn(4, H, requires_grad=True) for _ in range(P)]
    x = tp.vocab_embed(tp.EchoGroup(P, 0, mode="exact", device="cpu"), tables, torch.zeros(shape, dtype=torch.long), 2.0)
    assert x.shape == shape + (H,)
    x.sum().backward()
    assert asked == [((0, H), shape)]
    assert all(t.grad.shape == t.shape and not t.grad.any() for t in tables)
