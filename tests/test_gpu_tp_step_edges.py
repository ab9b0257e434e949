"""The tensor-parallel stack's options around its blocks at the edges of what they take, on the GPU."""
import pytest

pytestmark = pytest.mark.gpu

T, H, F, P, LAYERS, VOCAB = 96, 160, 256, 2, 2, 101


@pytest.fixture(scope="module")
def tp(cuda):
    from error_compensated_bit_echo_amd import tp
    return tp


def normal(seed, *shapes):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda") for s in shapes]


@pytest.mark.parametrize("product", ["f32", "fp8"])
@pytest.mark.parametrize("max_norm", [None, 0.01])
def test_step_on_a_residual_stream_of_a_stack_with_a_vocabulary(cuda, tp, product, max_norm):
    """The tables take no part: the step is that of the stack without them, their gradients zeros."""
    import torch
    x0, target = normal(1, (T, H), (T, H))
    group = tp.EchoGroup(P, T * H, device=cuda)
    kw = dict(seed=5, device=cuda, product=product, block_norms=True)
    plain, vocab = tp.TPMLPStack(LAYERS, H, F, P, **kw), tp.TPMLPStack(LAYERS, H, F, P, vocab=VOCAB, **kw)
    want = tp.train_step(plain, group, x0, target, max_norm=max_norm)
    got = tp.train_step(vocab, group, x0, target, max_norm=max_norm)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert len(got[2]) == len(vocab.parameters()) == len(want[2]) + P
    assert all(torch.equal(a, b) for a, b in zip(want[2], got[2]))
    for g, table in zip(got[2][-P:], vocab.tables):
        assert g.shape == table.shape and not g.any()
    if max_norm is not None:  # zeros add nothing to the norm
        assert torch.equal(want[3], got[3])


@pytest.mark.parametrize("shape", [(0,), (3, 0)])
def test_embedding_of_no_tokens(cuda, tp, shape):
    import torch
    tables = [t.requires_grad_() for t in normal(2, *[(7, H)] * P)]
    group = tp.EchoGroup(P, 0, mode="exact", device=cuda)
    x = tp.vocab_embed(group, tables, torch.zeros(shape, dtype=torch.long, device=cuda), 2.0)
    assert x.shape == shape + (H,)
    x.sum().backward()
    assert all(t.grad.shape == t.shape and not t.grad.any() for t in tables)


def test_embedding_types(cuda, tp):
    """float32 and bfloat16 tables go with the bfloat16 partials, float16 ones do not."""
    import torch
    tokens = torch.arange(T, device=cuda) % 14
    group = tp.EchoGroup(P, T * H, mode="exact", device=cuda)
    for dtype in (torch.float32, torch.bfloat16):
        tables = [t.to(dtype).requires_grad_() for t in normal(3, *[(7, H)] * P)]
        x = tp.vocab_embed(group, tables, tokens)
        assert torch.equal(x, torch.cat(tables)[tokens].bfloat16().float())
        x.backward(torch.ones_like(x))
        # every token comes up 6 or 7 times
        assert torch.equal(torch.cat([t.grad for t in tables]),
                           torch.bincount(tokens, minlength=14)[:, None].expand(14, H).to(dtype))
    with pytest.raises(tp.B.EchoError):
        tp.vocab_embed(group, [t.half() for t in normal(3, *[(7, H)] * P)], tokens)
