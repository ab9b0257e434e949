"""The training step's operators at the edges of what they take: shapes that say nothing, and the
sizes at which another kernel takes over."""
import pytest

from test_gpu_step import BlockCase, E, dt  # noqa: F401 (E is a fixture)

pytestmark = pytest.mark.gpu


def test_a_gate_without_rows_is_no_missing_gate(E):
    import torch
    new = lambda *shape: torch.full(shape, 2.0, device="cuda")
    x, y, out, none, gate = new(4, 16), new(4, 16), new(4, 16), new(0, 16), new(1, 16)
    with pytest.raises(E.EchoError):
        E.echo_block_norm(x, out, y=y, gate=none)
    with pytest.raises(E.EchoError):
        E.echo_block_norm_backward(x, dout=x, dy=out, y=y, gate=none)
    with pytest.raises(E.EchoError):  # a gradient that would not be written
        E.echo_block_norm_backward(x, dout=x, dy=out, dgate=none, y=y, gate=gate)
    with pytest.raises(E.EchoError):
        E.echo_block_norm_backward(x, dout=x, dy=out, dgate=none, y=y)
    assert (out == 2).all()


def test_a_gate_per_token_of_no_tokens(E):
    import torch
    new = lambda *shape: torch.full(shape, 2.0, device="cuda")
    x, w, dw, dgate = new(0, 16), new(16), new(16), new(0, 16)
    params = dict(y=new(0, 16), gate=new(0, 16), w_post=w, w_pre=w, post_norm=True)
    E.echo_block_norm(x, new(0, 16), new(0, 16), **params)
    E.echo_block_norm_backward(x, dout=x.clone(), da=x.clone(), dx=x.clone(), dgate=dgate, dw_pre=dw, **params)
    assert not dw.any()


def test_no_tokens_through_autograd(cuda):
    import torch
    from error_compensated_bit_echo_amd import tp
    for gates in (0, 1):  # one per token, one for all
        leaves = [torch.ones(s, device="cuda", requires_grad=True) for s in ((0, 16), (0, 16), (gates, 16), (16,), (16,))]
        out, a = tp.block_norm(*leaves, post_norm=True)
        (out.sum() + a.sum()).backward()
        assert all(t.grad.shape == t.shape and not t.grad.any() for t in leaves)
