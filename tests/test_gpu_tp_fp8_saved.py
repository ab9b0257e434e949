"""What the 8-bit products of the tensor-parallel stack keep for the backward pass: saved through
autograd, and no more than the gradients asked for need."""
import pytest

pytestmark = pytest.mark.gpu

# T is no multiple of 16, so codes along the tokens lie on padded rows
T, H, F, P = 70, 160, 2 * 96, 2


@pytest.fixture(scope="module")
def tp(cuda):
    from error_compensated_bit_echo_amd import tp
    return tp


def tensors(cuda, seed, *shapes):
    import torch
    g = torch.Generator(device=cuda)
    g.manual_seed(seed)
    return [torch.randn(*s, generator=g, device=cuda) for s in shapes]


def row(tp, cuda, w_grad=True, h_grad=True):
    """(group, output, its gradient, inputs) of a row-parallel product."""
    hs = [h.requires_grad_(h_grad) for h in tensors(cuda, 1, *[(T, F // P)] * P)]
    ws = [w.requires_grad_(w_grad) for w in tensors(cuda, 2, *[(F // P, H)] * P)]
    group = tp.EchoGroup(P, T * H, mode="exact", device=cuda, record=True)
    y = tp.row_parallel_fp8(group, hs, ws, (T, H), tp.quantize_weights_fp8(ws))
    return group, [y], tensors(cuda, 3, (T, H)), hs + ws


def column(tp, cuda, w_grad=True, a_grad=True):
    """The same of a column-parallel one."""
    a = [tensors(cuda, 1, (T, H))[0].requires_grad_(a_grad)]
    ws = [w.requires_grad_(w_grad) for w in tensors(cuda, 2, *[(H, F // P)] * P)]
    group = tp.EchoGroup(P, T * H, mode="exact", device=cuda, record=True)
    pres = tp.column_parallel_fp8(group, a[0], ws, tp.quantize_weights_fp8(ws))
    return group, list(pres), [g.bfloat16() for g in tensors(cuda, 3, *[(T, F // P)] * P)], a + ws


def backward(outs, grads, inputs):
    import torch
    torch.autograd.backward(outs, grads)
    return [t.grad for t in inputs]


@pytest.mark.parametrize("layer", [row, column])
def test_second_backward_pass_is_refused_before_any_reduction(cuda, tp, layer):
    group, outs, grads, inputs = layer(tp, cuda)
    backward(outs, grads, inputs)
    calls = len(group.log)
    with pytest.raises(RuntimeError, match="second time"):
        backward(outs, grads, inputs)
    assert len(group.log) == calls


@pytest.mark.parametrize("layer", [row, column])
def test_hooks_see_the_saved_operands_and_may_move_them(cuda, tp, layer):
    import torch
    _, outs, grads, inputs = layer(tp, cuda)
    want = backward(outs, grads, inputs)
    seen = []

    def pack(t):
        seen.append(t)
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        layer(tp, cuda)
    assert torch.float8_e4m3fn in [t.dtype for t in seen] and torch.float8_e8m0fnu in [t.dtype for t in seen]
    # activations transposed, and weights as they are, of every rank
    shapes = [tuple(t.shape) for t in seen if t.dtype == torch.float8_e4m3fn]
    k, n = (F // P, H) if layer is row else (H, F // P)
    assert shapes.count((k, T)) == (P if layer is row else 1) and shapes.count((k, n)) == P
    # moved away and back they come in another layout: rows without padding
    with torch.autograd.graph.save_on_cpu():
        _, outs, grads, inputs = layer(tp, cuda)
        got = backward(outs, grads, inputs)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.fixture
def quantized(tp, monkeypatch):
    """Records (rows of X, rows wanted, columns wanted) of every call of the quantizer."""
    calls = []
    plain = tp.B.echo_quantize_fp8

    def record(X, rows=None, cols=None, stream=None):
        calls.append((tuple(X[0].shape), rows is not None, cols is not None))
        return plain(X, rows, cols, stream)

    monkeypatch.setattr(tp.B, "echo_quantize_fp8", record)
    return calls


@pytest.mark.parametrize("layer", [row, column])
def test_a_pass_without_gradients_lays_nothing_out_for_them(cuda, tp, quantized, layer):
    import torch
    _, want, _, _ = layer(tp, cuda)
    quantized.clear()
    with torch.no_grad():
        _, got, _, _ = layer(tp, cuda)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    acts = (T, F // P) if layer is row else (T, H)
    assert [c for c in quantized if c[0] == acts] == [(acts, True, False)]


@pytest.mark.parametrize("layer", [row, column])
def test_only_the_gradients_asked_for_are_laid_out_for(cuda, tp, quantized, layer):
    import torch
    _, outs, grads, inputs = layer(tp, cuda)
    want = backward(outs, grads, inputs)
    n_w = P
    acts, back = ((T, F // P), (T, H)) if layer is row else ((T, H), (T, F // P))
    for w_grad, x_grad in ((True, False), (False, True)):
        quantized.clear()
        group, outs, grads, inputs = layer(tp, cuda, w_grad, x_grad)
        assert [c for c in quantized if c[0] == acts] == [(acts, True, w_grad)]
        quantized.clear()
        reductions = len(group.log)
        got = backward(outs, grads, inputs)
        assert quantized == [(back, x_grad, w_grad)]
        assert len(group.log) - reductions == (1 if layer is column and x_grad else 0)
        for i, (a, b) in enumerate(zip(got, want)):
            asked = w_grad if i >= len(inputs) - n_w else x_grad
            assert (a is None) if not asked else torch.equal(a, b)


def test_stack_without_gradients_lays_out_one_orientation(cuda, tp, quantized):
    """Weights too, where the pass quantizes them itself."""
    import torch
    model = tp.TPMLPStack(2, H, F, P, seed=11, device=cuda, product="fp8")
    x = tensors(cuda, 12, (T, H))[0]
    group = tp.EchoGroup(P, T * H, mode="exact", device=cuda)
    want = model.forward(x, group).detach()
    assert any(rows and cols for _, rows, cols in quantized)
    quantized.clear()
    with torch.no_grad():
        got = model.forward(x, group)
    assert torch.equal(got, want) and len(quantized) == 8
    assert not any(rows and cols for _, rows, cols in quantized)
    # weights laid out for such a pass alone do not serve a backward pass
    w8 = tp.quantize_weights_fp8(model.w1[0], backward=False)
    with pytest.raises(ValueError):
        tp.column_parallel_fp8(group, x.clone().requires_grad_(), model.w1[0], w8)
    with torch.no_grad():
        tp.column_parallel_fp8(group, x, model.w1[0], w8)
