"""The tensor-parallel stack's options around the blocks, on the CPU."""
import pytest

from error_compensated_bit_echo_amd import tp


@pytest.mark.parametrize("kw", [dict(residual_scale=0.5), dict(block_norms=True, residual_scale=float("nan")),
                                dict(block_norms=True, residual_scale=float("inf")), dict(vocab=-1)])
def test_stack_refuses_options_that_do_not_go_together(kw):
    with pytest.raises(ValueError):
        tp.TPMLPStack(1, 32, 64, 2, device="cpu", **kw)


def test_stack_parameters_in_order():
    import torch
    plain = tp.TPMLPStack(2, 32, 64, 2, device="cpu", seed=5)
    more = tp.TPMLPStack(2, 32, 64, 2, device="cpu", seed=5, block_norms=True, residual_scale=0.5, vocab=11)
    assert len(plain.parameters()) == 8
    # the products' weights first, the same as without; then norms and gates, then the tables
    assert all(torch.equal(a, b) for a, b in zip(plain.parameters(), more.parameters()))
    assert [tuple(p.shape) for p in more.parameters()[8:]] == [(32,)] * 6 + [(6, 32)] * 2
    assert all(p.requires_grad for p in more.parameters())


def test_what_needs_more_is_refused():
    import torch
    model = tp.TPMLPStack(1, 32, 64, 2, device="cpu")
    with pytest.raises(ValueError):  # tokens without a vocabulary
        model.forward(torch.zeros(4, dtype=torch.long), None)
    with pytest.raises(ValueError):
        tp.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        tp.block_norm(torch.zeros(2, 8), a=False)
