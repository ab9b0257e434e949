"""The operators of a training step around the blocks on the GPU, against their formulas in 64 bits:
sizes, types, layouts and special values where they can go wrong, their order of sums, streams,
captured calls and what lies beside their outputs."""
import itertools

import numpy as np
import pytest

from step_helpers import (Guarded, assert_close, block_norm_backward_ref, block_norm_ref, embed_backward_ref, half_step, matrix,
                          norm_ref, np64, U)

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def E(cuda):
    import error_compensated_bit_echo_amd as E
    return E


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


ALL_TYPES = [c for c in itertools.product(("f32", "bf16", "f16"), repeat=3) if not {"bf16", "f16"} <= set(c)]


class BlockCase:
    def __init__(self, T, C, types=("bf16",) * 3, param="f32", y=True, post=True, gates=1, w_pre=True, w_post=True, alpha=0.75,
                 offset=0.5, pad=0, at=0, seed=0):
        g = gen(seed)
        self.T, self.C, self.pad, self.at = T, C, pad, at
        self.X, self.Y, self.A, self.W = dt(types[0]), dt(types[1]), dt(types[2]), dt(param)
        mat = lambda t, size=1.0: matrix(g, (T, C), t, pad, at, size)
        vec = lambda n: matrix(g, (n, C), self.W, 0, at, 0.3) + 0.75
        self.x, self.y = mat(self.X), mat(self.Y, 0.7) if y else None
        self.dout, self.da = mat(self.X, 0.1), mat(self.A, 0.1)
        self.gate = vec(gates) if y and gates else None
        self.w_post = vec(1)[0] if y and post and w_post else None
        self.w_pre = vec(1)[0] if w_pre else None
        self.post = bool(y and post)
        self.alpha, self.offset = alpha if y else 1.0, offset
        self.params = dict(y=self.y, gate=self.gate, w_post=self.w_post, w_pre=self.w_pre, post_norm=self.post,
                           residual_scale=self.alpha, weight_offset=offset, eps=EPS)

    def guarded(self, dtype):
        return Guarded((self.T, self.C), dtype, self.pad, self.at)

    def forward(self, E):
        out, a = self.guarded(self.X) if self.y is not None else None, self.guarded(self.A)
        E.echo_block_norm(self.x, None if out is None else out.t, a.t, **self.params)
        return out, a

    def check_forward(self, E):
        out, a = self.forward(E)
        stream = self.x
        if out is not None:
            want, off = block_norm_ref(np64(self.x), np64(self.y), np64(self.gate), np64(self.w_post), self.post, self.alpha,
                                       self.offset, EPS)
            assert_close(out.t, want, off, self.X, "out")
            stream = out.t.clone()
        want, off = norm_ref(np64(stream), np64(self.w_pre), self.offset, EPS)  # from the stream as stored
        assert_close(a.t, want, off, self.A, "a")
        assert a.check() and (out is None or out.check())

    def gradients(self, E, dout=True, da=True, workspace=None):
        import torch
        like = lambda t: None if t is None else torch.full_like(t, 7.25)
        got = dict(dx=self.guarded(self.X), dy=None if self.y is None else self.guarded(self.Y), dgate=like(self.gate),
                   dw_post=like(self.w_post), dw_pre=like(self.w_pre) if da else None)
        params = dict(self.params, w_pre=self.w_pre if da else None)
        E.echo_block_norm_backward(self.x, dout=self.dout if dout else None, da=self.da if da else None, dx=got["dx"].t,
                                   dy=None if got["dy"] is None else got["dy"].t, dgate=got["dgate"], dw_post=got["dw_post"],
                                   dw_pre=got["dw_pre"], workspace=workspace, **params)
        return got

    def check_backward(self, E, dout=True, da=True):
        got = self.gradients(E, dout, da)
        want = block_norm_backward_ref(np64(self.x), np64(self.y), np64(self.dout) if dout else None,
                                       np64(self.da) if da else None, np64(self.gate), np64(self.w_post),
                                       np64(self.w_pre) if da else None, self.post, self.alpha, self.offset, EPS)
        types = dict(dx=self.X, dy=self.Y, dgate=self.W, dw_post=self.W, dw_pre=self.W)
        for name, t in got.items():
            if t is not None:
                assert_close(t.t if isinstance(t, Guarded) else t, *want[name], types[name], name)
        assert got["dx"].check() and (got["dy"] is None or got["dy"].check())


@pytest.mark.parametrize("types", ALL_TYPES, ids="-".join)
@pytest.mark.parametrize("C", [200, 8200, 16500])
def test_block_norm_every_type(E, types, C):
    half = next((t for t in types if t != "f32"), "bf16")
    for param in ("f32", half):
        c = BlockCase(5, C, types, param, pad=3, at=1)
        c.check_forward(E)
        c.check_backward(E)


@pytest.mark.parametrize("C", [1, 7, 8, 9, 64, 511, 512, 513, 1000, 4096, 8191, 8192, 8193, 16383, 16384, 16385, 50001])
@pytest.mark.parametrize("T", [1, 3])
def test_block_norm_every_width(E, T, C):
    c = BlockCase(T, C, ("f32", "bf16", "bf16"), seed=C)
    c.check_forward(E)
    c.check_backward(E)


@pytest.mark.parametrize("T", [1, 2, 511, 512, 513, 1025, 3000])
@pytest.mark.parametrize("C", [40, 9000])
def test_block_norm_every_height(E, T, C):
    if C == 9000 and T > 600:
        pytest.skip("covered by the narrow rows")
    c = BlockCase(T, C, ("bf16", "f32", "bf16"), "bf16", seed=T)
    c.check_forward(E)
    c.check_backward(E)


@pytest.mark.parametrize("kw", [
    dict(y=False), dict(y=False, w_pre=False), dict(post=False), dict(post=False, gates=0), dict(gates=0), dict(w_post=False),
    dict(w_pre=False), dict(w_pre=False, w_post=False, gates=0), dict(gates=2), dict(gates=12), dict(gates=36),
    dict(gates=1, pad=1), dict(pad=8, at=3), dict(alpha=0.0, offset=0.0), dict(alpha=-2.5, offset=1.0)], ids=str)
@pytest.mark.parametrize("C", [136, 8192, 17000])
def test_block_norm_every_part(E, kw, C):
    c = BlockCase(36, C, ("bf16", "bf16", "f32"), **kw)
    c.check_forward(E)
    for dout, da in ((True, True), (True, False), (False, True)):
        c.check_backward(E, dout, da)


@pytest.mark.parametrize("T,gates", [(1200, 600), (1025, 1025), (2048, 512), (1533, 511), (513, 3)])
def test_block_norm_many_gates(E, T, gates):
    c = BlockCase(T, 72, ("f32", "f32", "f32"), gates=gates)
    c.check_forward(E)
    c.check_backward(E)


def test_block_norm_parts_wanted(E):
    import torch
    c = BlockCase(20, 300, ("f32", "f32", "f32"))
    want = c.gradients(E)
    out, a = c.forward(E)
    only = torch.empty_like(c.x)
    E.echo_block_norm(c.x, only, None, **dict(c.params, w_pre=None))  # the end of the last block
    assert torch.equal(only, out.t)
    for name in ("dx", "dy", "dgate", "dw_post", "dw_pre"):
        t = want[name].t if isinstance(want[name], Guarded) else want[name]
        got = torch.full_like(t, -1)
        E.echo_block_norm_backward(c.x, dout=c.dout, da=c.da, **{name: got}, **c.params)
        assert torch.equal(got, t), name


@pytest.mark.parametrize("T,C,types", [(8200, 4100, ("bf16",) * 3), (5000, 7001, ("f32", "f16", "f16")), (4100, 9001, ("bf16",) * 3)])
def test_block_norm_of_more_than_the_cache_holds(E, T, C, types):
    """Calls that move more than 256 MB, whose 16-bit results go past the caches, give row by row
    what small calls give; their column sums are the small calls' added up."""
    import torch
    c = BlockCase(T, C, types, "f32", pad=3)
    out, a = c.forward(E)
    got = c.gradients(E)
    sums = {n: torch.zeros(1, C, dtype=torch.float64, device="cuda") for n in ("dgate", "dw_post", "dw_pre")}
    for lo in range(0, T, 1000):
        r = slice(lo, lo + 1000)
        o, b = torch.empty_like(c.x[r]), torch.empty_like(a.t[r])
        E.echo_block_norm(c.x[r], o, b, **dict(c.params, y=c.y[r]))
        assert torch.equal(o, out.t[r]) and torch.equal(b, a.t[r])
        dx, dy = torch.empty_like(o), torch.empty_like(c.y[r])
        part = {n: torch.empty_like(got[n]) for n in sums}
        E.echo_block_norm_backward(c.x[r], dout=c.dout[r], da=c.da[r], dx=dx, dy=dy, **part, **dict(c.params, y=c.y[r]))
        assert torch.equal(dx, got["dx"].t[r]) and torch.equal(dy, got["dy"].t[r])
        for n, p in part.items():
            sums[n] += p.double()
    for n, want in sums.items():
        # both add T terms of random signs in fp32: a root of T of terms of at most 2 or so, and T roundings of them
        off = T * U * T ** 0.5 * 2
        assert float((got[n].double() - want).abs().max()) <= off, n
    assert out.check() and a.check() and got["dx"].check() and got["dy"].check()


def test_block_norm_in_place(E):
    import torch
    for C in (500, 20000):
        c = BlockCase(7, C, ("bf16", "f32", "bf16"))
        out, a = c.forward(E)
        x, a2 = c.x.clone(), torch.empty_like(a.t)
        E.echo_block_norm(x, x, a2, **c.params)
        assert torch.equal(x, out.t) and torch.equal(a2, a.t)
        want = c.gradients(E)
        dout, dy = c.dout.clone(), torch.empty_like(c.y)
        E.echo_block_norm_backward(c.x, dout=dout, da=c.da, dx=dout, dy=dy, **c.params)
        assert torch.equal(dout, want["dx"].t) and torch.equal(dy, want["dy"].t)


def test_block_norm_of_the_stored_stream_is_the_same(E):
    """The fused norm and a norm of the stream that it stored agree to the bit."""
    import torch
    for C in (333, 4096, 8200, 30000):
        c = BlockCase(4, C, ("bf16", "bf16", "bf16"))
        out, a = c.forward(E)
        alone = torch.empty_like(a.t)
        E.echo_block_norm(out.t, a=alone, w_pre=c.w_pre, weight_offset=c.offset, eps=EPS)
        assert torch.equal(alone, a.t)


def test_block_norm_of_nothing(E):
    import torch
    for shape in ((0, 64), (5, 0)):
        x = torch.empty(shape, device="cuda")
        w, gate = torch.ones(shape[1], device="cuda"), torch.ones(1, shape[1], device="cuda")
        params = dict(y=x.clone(), gate=gate, w_post=w, w_pre=w, post_norm=True)
        E.echo_block_norm(x, x.clone(), x.clone(), **params)
        dw, dw2, dg = torch.full_like(w, 3), torch.full_like(w, 3), torch.full_like(gate, 3)
        E.echo_block_norm_backward(x, dout=x.clone(), da=x.clone(), dx=x.clone(), dw_pre=dw, dw_post=dw2, dgate=dg, **params)
        assert not dw.any() and not dw2.any() and not dg.any()  # sums over no rows


@pytest.mark.parametrize("C", [300, 9000, 20000])
def test_block_norm_special_values(E, C):
    import torch
    for types in (("f32",) * 3, ("bf16",) * 3):
        X = dt(types[0])
        y = torch.ones(5, C, device="cuda").to(X)
        x = torch.zeros(5, C, device="cuda").to(X)
        y[0] = 0                 # nothing to normalise: zeros, not NaN
        y[1, C // 2] = float("nan")
        y[2, C // 2] = float("inf")
        y[3] = 1e-20             # squares below eps
        x[4, 1] = float("nan")   # of the stream only
        out, a = torch.empty_like(x), torch.empty_like(x)
        E.echo_block_norm(x, out, a, y=y, post_norm=True, eps=EPS)
        assert not out[0].any() and not a[0].any()
        assert out[1].isnan().all() and a[1].isnan().all()
        assert out[2, C // 2].isnan() and out[2].isnan().sum() == 1 and a[2].isnan().all()
        want = 1e-20 / np.sqrt(EPS)
        # two roundings to the type (the value and what it is made of) and those of the norm in fp32
        assert (np.abs(np64(out[3]) - want) <= want * (torch.finfo(X).eps + 40 * U)).all()
        assert out[4].isnan().sum() == 1 and a[4].isnan().all()


@pytest.mark.parametrize("C", [5, 300, 9000, 20000])
def test_block_norm_gradient_beside_an_infinite_output(E, C):
    """Without a post-norm y's gradient does not depend on y."""
    import torch
    for types in (("f32",) * 3, ("bf16",) * 3):
        c = BlockCase(3, C, types, post=False, w_pre=False)
        c.y[1, C // 2], c.y[2, 0] = float("inf"), float("-inf")
        dy = torch.empty_like(c.y)
        E.echo_block_norm_backward(c.x, dout=c.dout, dy=dy, **c.params)
        want = np64(c.dout) * np64(c.gate)
        assert_close(dy, want, np.abs(want) * U, c.Y, "dy")  # one product in fp32


def test_block_norm_gradient_against_differences(E):
    """d loss along a direction, in fp32 with steps of 2^-7: the difference quotient is off by the
    third derivative (h^2 / 6, below 1e-4 of these sums) and by the forward pass's roundings / h."""
    import torch
    c = BlockCase(6, 96, ("f32", "f32", "f32"), gates=2)
    g = gen(5)
    names = ("x", "y", "gate", "w_post", "w_pre")
    base = {n: getattr(c, n) for n in names}
    dirs = {n: torch.randn(v.shape, generator=g, device="cuda") for n, v in base.items()}
    out, a = torch.empty_like(c.x), torch.empty_like(c.x)

    def loss(name, h):
        v = {n: (t.double() + (h * dirs[n].double() if n == name else 0)).float() for n, t in base.items()}
        E.echo_block_norm(v["x"], out, a, **dict(c.params, y=v["y"], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"]))
        return (out.double() * c.dout.double()).sum().item() + (a.double() * c.da.double()).sum().item()

    E.echo_block_norm(c.x, out, a, **c.params)
    grads = {n: torch.empty_like(v) for n, v in base.items()}
    E.echo_block_norm_backward(out.clone(), dout=c.dout, da=c.da, dx=grads["x"], dy=grads["y"], dgate=grads["gate"],
                               dw_post=grads["w_post"], dw_pre=grads["w_pre"], **c.params)
    h = 2.0 ** -7
    for n in names:
        quotient = (loss(n, h) - loss(n, -h)) / (2 * h)
        exact = (grads[n].double() * dirs[n].double()).sum().item()
        size = (grads[n].double().abs() * dirs[n].double().abs()).sum().item()
        # 576 outputs of size up to 4, gradients of 0.1, each off by 30 U: 576 * 4 * 0.1 * 30 U * 2 / (2 h) = 0.05
        # at the worst; their signs are random: a root of 576 of that
        assert abs(quotient - exact) <= 1e-3 * size + 0.05 / 24 * 4, n


# ---- gradient norm and clipping ----------------------------------------------------------------


def clip_factor(grads, max_norm):
    total = np.sqrt(sum(float((np64(g) ** 2).sum()) for g in grads))
    return total, min(1.0, max_norm / (total + 1e-6))


def check_clip(E, grads, max_norm, in_place=False, **kw):
    import torch
    norm, alone = (torch.full((1,), -1.0, device="cuda") for _ in range(2))
    total, f = clip_factor(grads, max_norm)
    wide = [np64(g) for g in grads]
    E.echo_grad_norm(grads, alone, **kw)
    if in_place:
        out = grads
        E.echo_clip_grads(grads, max_norm, norm, **kw)
    else:
        out = [torch.full_like(g, 7.25) for g in grads]
        E.echo_clip_grads(grads, max_norm, norm, out=out, **kw)
    assert torch.equal(norm, alone)
    assert abs(norm.item() - total) <= total * (U + 1e-10)  # sums in 64 bits: 2^-53 for each of up to 2^20 terms
    for g, o in zip(wide, out):
        # the factor's rounding and the product's, in fp32
        assert_close(o, g * f, np.abs(g * f) * (2 * U + 1e-9) * (f < 1), o.dtype)


@pytest.mark.parametrize("sizes", [[], [0], [1], [0, 3, 0], [7, 8, 9], [255, 16383, 16384, 16385], [100003], [40000, 1, 32768]],
                         ids=str)
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip_sizes(E, sizes, max_norm):
    import torch
    g = gen(1)
    for t in ("f32", "bf16", "f16"):
        check_clip(E, [torch.randn(n, generator=g, device="cuda").to(dt(t)) for n in sizes], max_norm)


def test_clip_many_tensors_of_mixed_types_at_any_element(E):
    """More tensors than a launch takes, lying next to each other in one buffer."""
    import torch
    g, rng = gen(2), np.random.default_rng(3)
    for count in (175, 176, 177, 280, 281, 700):
        bufs = {t: torch.randn(1 << 19, generator=g, device="cuda").to(dt(t)) for t in ("f32", "bf16", "f16")}
        at, grads = dict.fromkeys(bufs, 0), []
        for _ in range(count):
            t, n = ("f32", "bf16", "f16")[rng.integers(3)], int(rng.integers(0, 900))
            grads.append(bufs[t][at[t]:at[t] + n])
            at[t] += n
        rest = {t: b[at[t]:].clone() for t, b in bufs.items()}
        check_clip(E, grads, 3.0)
        check_clip(E, grads, 3.0, in_place=True)
        for t, b in bufs.items():
            assert torch.equal(b[at[t]:], rest[t])


def test_clip_more_sums_than_a_launch_leaves(E):
    import torch
    g = gen(7)
    grads = [torch.randn(1 << 16, generator=g, device="cuda") for _ in range(301)]
    check_clip(E, grads, 3.0)
    check_clip(E, grads, 5.0, in_place=True)


def test_clip_is_the_same_every_time_and_in_place(E):
    import torch
    g = gen(4)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (1 << 22, 5, 777777)]
    outs, norms = [], []
    for _ in range(3):
        out, norm = [torch.empty_like(x) for x in grads], torch.empty(1, device="cuda")
        E.echo_clip_grads(grads, 1.0, norm, out=out)
        outs.append(out)
        norms.append(norm)
    mine = [x.clone() for x in grads]
    norm = torch.empty(1, device="cuda")
    E.echo_clip_grads(mine, 1.0, norm)
    outs.append(mine)
    norms.append(norm)
    for out, norm in zip(outs[1:], norms[1:]):
        assert torch.equal(norm, norms[0]) and all(torch.equal(a, b) for a, b in zip(out, outs[0]))


def test_clip_over_the_whole_range_of_the_types(E):
    """Squares of elements of 1e30 and of 1e-30 leave the range of 32 bits."""
    import torch
    for v in (1e30, 1e-30):
        check_clip(E, [torch.full((1000,), v, device="cuda")], v)
        check_clip(E, [torch.full((1000,), v, device="cuda").bfloat16()], v)


def test_clip_special_values(E):
    import torch
    inf, nan = float("inf"), float("nan")
    for bad in (inf, nan):
        g = torch.ones(5000, device="cuda")
        g[4321] = bad
        norm, out = torch.empty(1, device="cuda"), [torch.empty_like(g)]
        E.echo_clip_grads([g], 1.0, norm, out=out)
        if bad == inf:
            assert norm.item() == inf and out[0].isnan().sum() == 1 and not out[0].nan_to_num(0).any()
        else:
            assert norm.isnan().all() and out[0].isnan().all()
    z, norm = torch.zeros(100, device="cuda"), torch.empty(1, device="cuda")
    E.echo_clip_grads([z], 1.0, norm)
    assert norm.item() == 0 and not z.any()
    g = torch.ones(100, device="cuda")
    E.echo_clip_grads([g], 0.0, norm)
    assert norm.item() == 10 and not g.any()


# ---- embedding ---------------------------------------------------------------------------------


def embed_case(P, V, T, C, table, seed=0, pad=0, at=0, first=0, spread=None, wide=True):
    import torch
    g = gen(seed)
    tables = [matrix(g, (V, C), dt(table), pad, at) for _ in range(P)]
    lo, hi = spread if spread else (first - V // 2 - 1, first + P * V + V // 2 + 1)
    tokens = torch.randint(lo, hi, (T,), generator=g, device="cuda")
    return tables, tokens if wide else tokens.int()


def check_embed(E, P, V, T, C, table, out, scale=1.0, first=0, pad=0, at=0, **kw):
    import torch
    tables, tokens = embed_case(P, V, T, C, table, pad=pad, at=at, first=first, **kw)
    got = [Guarded((T, C), dt(out), pad, at) for _ in range(P)]
    E.echo_embed(tables, tokens, [o.t for o in got], scale=scale, first=first)
    ids = tokens.long() - first
    for r, o in enumerate(got):
        here = (ids >= r * V) & (ids < (r + 1) * V)
        want = torch.zeros(T, C, device="cuda")
        want[here] = tables[r][ids[here] - r * V].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")
        assert torch.equal(o.t, want.to(dt(out))), r
        assert o.check()


@pytest.mark.parametrize("table,out", [(t, o) for t in ("f32", "bf16", "f16") for o in ("f32", "bf16", "f16") if {t, o} != {"bf16", "f16"}])
def test_embed_every_type(E, table, out):
    check_embed(E, 2, 37, 50, 100, table, out, scale=10.0, pad=3, at=1)


@pytest.mark.parametrize("C", [1, 7, 8, 9, 63, 64, 65, 1000, 2048, 2056, 5000])
@pytest.mark.parametrize("T", [1, 3, 300])
def test_embed_every_size(E, T, C):
    check_embed(E, 1, 20, T, C, "bf16", "bf16")
    check_embed(E, 3, 20, T, C, "f32", "bf16", scale=0.3, first=11, wide=False)


def test_embed_sixteen_ranks_and_far_tokens(E):
    import torch
    check_embed(E, 16, 5, 200, 64, "bf16", "f32", scale=3.0)
    check_embed(E, 2, 5, 200, 64, "bf16", "f32", first=1 << 62)
    table, out = torch.ones(4, 8, device="cuda"), torch.full((4, 8), 5.0, device="cuda")
    tokens = torch.tensor([-2 ** 63, 2 ** 63 - 1, -1, 3], device="cuda")
    E.echo_embed([table], tokens, [out])
    assert not out[:3].any() and (out[3] == 1).all()
    out.fill_(5.0)
    E.echo_embed([table], tokens, [out], first=1 << 62)
    assert not out.any()


def test_embed_of_nothing(E):
    import torch
    table = torch.ones(4, 8, device="cuda")
    none = torch.empty(0, dtype=torch.long, device="cuda")
    E.echo_embed([table], none, [torch.empty(0, 8, device="cuda")])
    out = torch.ones(3, 8, device="cuda")
    E.echo_embed([torch.empty(0, 8, device="cuda")], torch.zeros(3, dtype=torch.long, device="cuda"), [out])
    assert not out.any()
    d = torch.ones(4, 8, device="cuda")
    E.echo_embed_backward(torch.empty(0, 8, device="cuda"), none, [d])
    assert not d.any()


def check_embed_backward(E, P, V, T, C, out, table, tokens=None, scale=1.0, first=0, pad=0, at=0, seed=0, wide=True):
    import torch
    dout = matrix(gen(seed + 1), (T, C), dt(out), pad, at)
    if tokens is None:
        tokens = embed_case(1, max(P * V, 1), T, 1, "f32", seed, first=first)[1]
    got = [Guarded((V, C), dt(table), pad, at) for _ in range(P)]
    ids = tokens if wide else tokens.int()
    E.echo_embed_backward(dout, ids, [d.t for d in got], scale=scale, first=first)
    want, off = embed_backward_ref(np64(dout), tokens.cpu().numpy(), P * V, first, float(np.float32(scale)))
    for r, d in enumerate(got):
        assert_close(d.t, want[r * V:(r + 1) * V], off[r * V:(r + 1) * V], dt(table), f"rank {r}")
    again = [torch.empty_like(d.t) for d in got]
    E.echo_embed_backward(dout, ids, again, scale=scale, first=first)
    assert all(torch.equal(a, d.t) for a, d in zip(again, got))  # no order that changes
    assert all(d.check() for d in got)


@pytest.mark.parametrize("out,table", [(o, t) for t in ("f32", "bf16", "f16") for o in ("f32", "bf16", "f16") if {t, o} != {"bf16", "f16"}])
def test_embed_backward_every_type(E, out, table):
    check_embed_backward(E, 2, 37, 500, 100, out, table, scale=10.0, pad=3, at=1)


@pytest.mark.parametrize("C", [1, 8, 9, 65, 2048, 2060])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 1000])
def test_embed_backward_every_size(E, T, C):
    check_embed_backward(E, 1, 20, T, C, "bf16", "f32")
    check_embed_backward(E, 3, 50, T, C, "f32", "bf16", scale=0.3, first=11, wide=False)


@pytest.mark.parametrize("T", [3, 5000, 20000])
@pytest.mark.parametrize("V,C", [(1000, 77), (257, 1024), (70001, 5), (1, 300001), (2100, 2048)])
def test_embed_backward_clears_what_no_token_has(E, V, C, T):
    """Tables without gaps, their ends inside a page and at any element; and with gaps."""
    for at in (0, 1):
        check_embed_backward(E, 3, V, min(T, 40000000 // C), C, "bf16", "bf16", at=at)
    check_embed_backward(E, 2, V, min(T, 40000000 // C), C, "f32", "f32", at=3, pad=0 if C > 2000 else 9)


@pytest.mark.parametrize("T", [1023, 1024, 1025, 16383, 16384, 16385, 20480, 20481, 70000])
@pytest.mark.parametrize("n", [200, 255, 256, 65535, 65536, 70001])
def test_embed_backward_sorts_any_number_of_tokens(E, T, n):
    check_embed_backward(E, 1, n, T, 8, "f32", "f32", seed=T + n)


@pytest.mark.parametrize("T", [64, 5000, 40000])
def test_embed_backward_of_runs(E, T):
    """One token only, none that a rank holds, each once, two that take turns, all but one the same."""
    import torch
    n = 300
    t = torch.arange(T, device="cuda")
    for tokens in (torch.full_like(t, 7), torch.full_like(t, n), torch.full_like(t, -1), t % n, t % 2, (t == T // 2).long(),
                   torch.where(t < T // 2, n - 1, 0), torch.where(t % 3 == 0, n + 5, 3)):
        check_embed_backward(E, 3, n // 3, T, 24, "f32", "f32", tokens=tokens)


def test_embed_backward_of_a_large_vocabulary(E):
    """Row numbers of four digits, tables beyond 4 GiB."""
    import torch
    V, C, T = (1 << 24) + 77, 136, 3000
    tokens = torch.randint(0, V, (T,), generator=gen(3), device="cuda")
    tokens[:3] = torch.tensor([0, V - 1, V - 1], device="cuda")
    dout = torch.randn(T, C, generator=gen(4), device="cuda").bfloat16()
    d = torch.full((V, C), 3.0, dtype=torch.bfloat16, device="cuda")
    E.echo_embed_backward(dout, tokens, [d])
    ids, inverse = tokens.unique(return_inverse=True)
    want, off = embed_backward_ref(np64(dout), inverse.cpu().numpy(), len(ids), 0, 1.0)
    assert_close(d[ids], want, off, torch.bfloat16)
    d[ids] = 0
    assert not d.view(torch.int16).any()
    out = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    d[ids] = torch.randn(len(ids), C, generator=gen(5), device="cuda").bfloat16()
    E.echo_embed([d], tokens, [out])
    assert torch.equal(out, d[tokens])


def test_more_threads_than_a_launch_numbers(E):
    """Launches number their threads along an axis in 32 bits: 2^26 rows of 64 threads, 2^24 of 256."""
    import torch
    R, C = (1 << 26) + 5, 8
    x = torch.randn(R, C, generator=gen(6), device="cuda").bfloat16()
    w = torch.rand(C, generator=gen(7), device="cuda")
    a, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.empty_like(w)
    E.echo_block_norm(x, a=a, w_pre=w)
    E.echo_block_norm_backward(x, da=x, dx=dx, w_pre=w, dw_pre=dw)
    some = torch.randint(0, R, (2000,), generator=gen(8), device="cuda")
    some[:4] = torch.tensor([0, R - 1, R - 5, R - 6], device="cuda")
    assert_close(a[some], *norm_ref(np64(x[some]), np64(w), 0.0, 1e-6), torch.bfloat16)
    ref = block_norm_backward_ref(np64(x[some]), None, None, np64(x[some]), None, None, np64(w), False, 1.0, 0.0, 1e-6)
    assert_close(dx[some], *ref["dx"], torch.bfloat16)
    del a, dx
    # sums of 2^26 terms, of about 0.5 each, in 4096 workgroups of 16384 rows: 16384 additions in a row and 70 more
    total = sum((t.double() ** 2 / (t.double() ** 2).mean(1, keepdim=True).add(1e-6).sqrt()).sum(0) for t in x.split(1 << 22))
    assert (np.abs(np64(dw) - total.cpu().numpy()) <= (16384 + 100) * U * total.abs().cpu().numpy()).all()
    del x
    T, C = (1 << 24) + 3, 2048
    table = torch.randn(100, C, generator=gen(9), device="cuda").bfloat16()
    tokens = torch.randint(0, 100, (T,), generator=gen(10), device="cuda")
    out = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    E.echo_embed([table], tokens, [out])
    for lo in range(0, T, 1 << 20):
        assert torch.equal(out[lo:lo + (1 << 20)], table[tokens[lo:lo + (1 << 20)]])


# ---- streams, graphs ---------------------------------------------------------------------------


def test_calls_on_another_stream(E):
    import torch
    c = BlockCase(300, 1000, ("bf16", "f32", "bf16"), seed=9)
    want = c.gradients(E)
    s = torch.cuda.Stream()
    ws = torch.empty(E.echo_block_norm_workspace(c.T, c.C, 1), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(c.x), torch.empty_like(c.w_pre)
    s.wait_stream(torch.cuda.current_stream())
    E.echo_block_norm_backward(c.x, dout=c.dout, da=c.da, dx=dx, dw_pre=dw, workspace=ws, stream=s, **c.params)
    with pytest.raises(E.EchoError):  # torch's allocator would hand a workspace of this stream to the next call on it
        E.echo_block_norm_backward(c.x, dout=c.dout, da=c.da, dx=dx, dw_pre=dw, stream=s, **c.params)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(dx, want["dx"].t) and torch.equal(dw, want["dw_pre"])
    with torch.cuda.stream(s):  # torch's current stream
        E.echo_block_norm_backward(c.x, dout=c.dout, da=c.da, dx=dx.zero_(), dw_pre=dw.zero_(), **c.params)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(dx, want["dx"].t) and torch.equal(dw, want["dw_pre"])


def test_calls_on_two_streams_at_once(E):
    """Each with its own workspace: what they give alone."""
    import torch
    T, V, C = 20000, 700, 512
    g = gen(13)
    tokens = [torch.randint(0, V, (T,), generator=g, device="cuda") for _ in range(2)]
    d = [torch.randn(T, C, generator=g, device="cuda") for _ in range(2)]
    x = torch.randn(T, C, generator=g, device="cuda")
    w = torch.rand(C, generator=g, device="cuda")
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    sizes = E.echo_block_norm_workspace(T, C), E.echo_embed_workspace(T, C), E.echo_clip_workspace(2)

    def buffers():
        return dict(dx=torch.empty(T, C, device="cuda"), dw=torch.empty(C, device="cuda"), dt=torch.empty(V, C, device="cuda"),
                    norm=torch.empty(1, device="cuda"), ws=[u8(n) for n in sizes])

    def run(i, b, stream):
        E.echo_block_norm_backward(x, da=d[i], dx=b["dx"], w_pre=w, dw_pre=b["dw"], workspace=b["ws"][0], stream=stream)
        E.echo_embed_backward(b["dx"], tokens[i], [b["dt"]], workspace=b["ws"][1], stream=stream)
        E.echo_clip_grads([b["dt"], b["dw"]], 0.5, b["norm"], workspace=b["ws"][2], stream=stream)

    want, got, streams = [buffers() for _ in range(2)], [buffers() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        run(i, want[i], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            run(i, got[i], streams[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in ("dx", "dw", "dt", "norm"))


@pytest.mark.parametrize("T", [200, 20000])
def test_captured_step(E, T):
    """Embedding, block norm, their gradients and the clipping in one graph, replayed on new inputs."""
    import torch
    V, C, P = 90, 72, 2
    g = gen(11)
    tables = [torch.randn(V, C, generator=g, device="cuda") for _ in range(P)]
    tokens = torch.zeros(T, dtype=torch.long, device="cuda")
    w = torch.rand(C, generator=g, device="cuda")
    d = torch.randn(T, C, generator=g, device="cuda")

    def step():
        parts = [torch.empty(T, C, device="cuda") for _ in range(P)]
        E.echo_embed(tables, tokens, parts, scale=2.0)
        a, dx, dw = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda"), torch.empty_like(w)
        x = parts[0] + parts[1]
        E.echo_block_norm(x, a=a, w_pre=w)
        E.echo_block_norm_backward(x, da=a * d, dx=dx, w_pre=w, dw_pre=dw)
        dt_ = [torch.empty_like(t) for t in tables]
        E.echo_embed_backward(dx, tokens, dt_, scale=2.0)
        norm = torch.empty(1, device="cuda")
        E.echo_clip_grads(dt_ + [dw], 0.25, norm)
        return [norm, dw] + dt_

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(4):
        tokens.copy_(torch.randint(-3, P * V + 3, (T,), generator=gen(seed), device="cuda"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
