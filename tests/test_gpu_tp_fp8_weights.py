"""Training steps of the tensor-parallel stack on weights laid out in 8 bits once."""
import pytest

pytestmark = pytest.mark.gpu

T, H, F, P, LAYERS = 70, 160, 2 * 96, 2, 3


def test_steps_on_weights_laid_out_once(cuda, monkeypatch):
    """Several steps over the same weights, as a caller that accumulates gradients runs them: the
    weights are not quantized again, and every step's results are those of a step that does."""
    import torch
    from error_compensated_bit_echo_amd import tp
    model = tp.TPMLPStack(LAYERS, H, F, P, seed=11, device=cuda, product="fp8", dropout=0.1)
    group = tp.EchoGroup(P, T * H, device=cuda)
    data = [(torch.randn(T, H, device=cuda), torch.randn(T, H, device=cuda)) for _ in range(3)]
    want = [tp.train_step(model, group, x, t) for x, t in data]
    model.rng[1] = 0
    w8 = model.quantize_weights()
    shapes = []
    plain = tp.B.echo_quantize_fp8

    def record(X, rows=None, cols=None, stream=None):
        shapes.append(tuple(X[0].shape))
        return plain(X, rows, cols, stream)

    monkeypatch.setattr(tp.B, "echo_quantize_fp8", record)
    got = [tp.train_step(model, group, x, t, weights8=w8) for x, t in data]
    assert shapes and {s[0] for s in shapes} == {T}
    for (l0, x0, w0), (l1, x1, w1) in zip(want, got):
        assert torch.equal(l0, l1) and torch.equal(x0, x1)
        assert all(torch.equal(a, b) for a, b in zip(w0, w1))


def test_step_refuses_such_weights_for_other_products(cuda):
    import torch
    from error_compensated_bit_echo_amd import tp
    model = tp.TPMLPStack(1, 64, 64, 2, device=cuda)
    x = torch.randn(4, 64, device=cuda)
    with pytest.raises(ValueError):
        tp.train_step(model, tp.EchoGroup(2, 256, device=cuda), x, x, weights8=[])
