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


@pytest.mark.parametrize("C,T,gates", [(5, 600, 300), (5, 1025, 1025), (4100, 1100, 550), (8192, 600, 300), (8192, 515, 515),
                                       (9000, 600, 300), (9000, 515, 515), (9000, 600, 200), (17000, 339, 339), (17000, 226, 113)])
def test_block_norm_many_gates_of_any_width(E, C, T, gates):
    """A workgroup of the gradients with several whole gates (the last with fewer), and with a part of
    one, for rows in the registers, rows by columns, and rows of fewer than 8 columns."""
    for types in (("f32", "f32", "f32"), ("bf16", "bf16", "bf16")):
        c = BlockCase(T, C, types, "f32", gates=gates, seed=gates)
        c.check_forward(E)
        c.check_backward(E)


@pytest.mark.parametrize("T,C", [(8200, 4100), (4100, 9001)])
def test_block_norm_a_gate_per_token_of_more_than_the_cache_holds(E, T, C):
    """Gradients of a row and of its own gate are what a call on fewer rows gives."""
    import torch
    c = BlockCase(T, C, ("bf16", "bf16", "bf16"), "f32", gates=T, pad=3)
    got = c.gradients(E)
    for lo in range(0, T, 700):
        r = slice(lo, lo + 700)
        dx, dy, dgate = torch.empty_like(c.x[r]), torch.empty_like(c.y[r]), torch.empty_like(c.gate[r])
        E.echo_block_norm_backward(c.x[r], dout=c.dout[r], da=c.da[r], dx=dx, dy=dy, dgate=dgate,
                                   **dict(c.params, y=c.y[r], gate=c.gate[r]))
        assert torch.equal(dx, got["dx"].t[r]) and torch.equal(dy, got["dy"].t[r]) and torch.equal(dgate, got["dgate"][r])
    assert got["dx"].check() and got["dy"].check()


@pytest.mark.parametrize("types", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "f16", "f16")], ids="-".join)
@pytest.mark.parametrize("T,C", [(2049, 1025), (2304, 1032), (3000, 1600), (2100, 4100), (2049, 8191), (2049, 8192)])
def test_block_norm_two_runs_to_a_thread(E, types, T, C):
    """More rows than get a workgroup of one run to a thread: the formula's values, and to the bit
    those of calls on few rows."""
    import torch
    c = BlockCase(T, C, types, "f32", pad=5, at=1)
    c.check_forward(E)
    out, a = c.forward(E)
    alone = torch.empty_like(a.t)
    E.echo_block_norm(c.x, a=alone, w_pre=c.w_pre, weight_offset=c.offset)
    for lo in range(0, T, 1100):
        r = slice(lo, lo + 1100)
        o, b = torch.empty_like(c.x[r]), torch.empty_like(a.t[r])
        E.echo_block_norm(c.x[r], o, b, **dict(c.params, y=c.y[r]))
        assert torch.equal(o, out.t[r]) and torch.equal(b, a.t[r])
        E.echo_block_norm(c.x[r], a=b, w_pre=c.w_pre, weight_offset=c.offset)
        assert torch.equal(b, alone[r])


@pytest.mark.parametrize("T", [1025, 3000])
def test_block_norm_many_wide_rows(E, T):
    c = BlockCase(T, 9000, ("bf16", "f32", "bf16"), "bf16", seed=T)
    c.check_forward(E)
    c.check_backward(E)


@pytest.mark.parametrize("C", [5, 300, 9000, 17000])
def test_block_norm_parameters_of_the_other_16_bit_type(E, C):
    for types, param in ((("bf16", "bf16", "bf16"), "f16"), (("f16", "f32", "f16"), "bf16")):
        c = BlockCase(9, C, types, param, gates=3, pad=1, at=1)
        c.check_forward(E)
        c.check_backward(E)
