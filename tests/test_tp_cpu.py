"""The tensor-parallel stack's construction, on the CPU."""
import pytest

from error_compensated_bit_echo_amd import tp


@pytest.mark.parametrize("p", [-0.1, 1.0 - 2.0 ** -17, 1.0, float("nan")])
def test_stack_refuses_a_dropout_that_the_operator_refuses(p):
    with pytest.raises(ValueError):
        tp.TPMLPStack(1, 32, 64, 2, device="cpu", dropout=p)


@pytest.mark.parametrize("p", [0.0, 0.5, 1.0 - 2.0 ** -16])
def test_stack_takes_every_dropout_that_the_operator_takes(p):
    model = tp.TPMLPStack(1, 32, 64, 2, device="cpu", dropout=p)
    assert (model.rng is None) == (p == 0.0)
