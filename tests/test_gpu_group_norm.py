"""Group norm with an activation on the GPU against its 64-bit definition.

Tolerances (2-norm, relative): fp32 outputs are sums over a group and a few
operations per value, 2e-5 leaves a factor of ten over the roundings; bf16 outputs
are rounded once, by at most 2^-8 each, 2^-8 / sqrt(3) = 2.3e-3 in the 2-norm when
uniform: 2.5e-3.  Of fewer than 64 values that average says nothing and the largest
rounding, 2^-8 = 3.9e-3 for every value, bounds the norm."""
import pytest
import torch

import gdr_reference as R
import momentum_delta_rule_mdn_b200 as mdn

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 2.5e-3}


def tol(t):
    return 2.0 ** -8 if t.dtype == BF16 and t.numel() < 64 else TOL[t.dtype]


F32, BF16 = torch.float32, torch.bfloat16


def make(N, L, C, dtype, gate, affine, seed, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = (r(N, L, C) + shift).to(dtype)
    return (x, 1 + 0.3 * r(C) if affine else None, 0.2 * r(C) if affine else None,
            r(N, L, C).to(dtype) if gate else None, r(N, L, C).to(dtype))


def cu(t):
    return None if t is None else t.cuda()


SHAPES = [  # N, L, C, G
    (1, 1, 1, 1), (1, 1, 7, 1), (5, 1, 24, 3), (3, 1, 2048, 16), (70, 1, 640, 5), (9, 1, 1024, 1),
    (4, 1, 96, 96), (2, 1, 4096, 4), (33, 1, 2040, 8), (2, 1, 250, 1), (1000, 1, 128, 2),
    (2, 3, 24, 3), (1, 64, 100, 5), (3, 333, 64, 2), (2, 1000, 640, 20), (1, 17, 7, 7), (5, 40, 520, 1),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act,gate,affine", [("silu", True, True), ("silu", False, True),
                                             ("none", False, False), ("none", True, True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradients(shape, act, gate, affine, dtype):
    N, L, C, G = shape
    x, w, b, z, dy = make(N, L, C, dtype, gate, affine, seed=N + C)
    ry, rm, rr, rg = R.group_norm(x, G, w, b, z, act, 1e-3, dy)
    y, mean, rstd = mdn.group_norm_fwd(x.cuda(), G, cu(w), cu(b), cu(z), 1e-3, act)
    assert R.rel(y, ry) <= tol(y) or float(ry.norm()) < 1e-6
    # a mean's error is relative to the values, not to the mean
    assert float((mean.cpu() - rm).abs().max()) <= 2e-6 * float(x.double().abs().max() + 1)
    assert R.rel(rstd, rr) <= 2e-5
    g = mdn.group_norm_bwd(x.cuda(), G, mean, rstd, dy.cuda(), cu(w), cu(b), cu(z), act)
    assert set(g) == set(rg)
    for n in rg:
        if n == "dx" and L * C // G <= 2:
            # dx is a difference of equal terms there: absolute against those
            assert float((g[n].cpu() - rg[n]).abs().max()) <= 2e-2 * float(rr.max())
        else:
            assert R.rel(g[n], rg[n]) <= tol(g[n]), n


@pytest.mark.parametrize("L", [1, 130])
def test_large_mean(L):
    """A mean a hundred times the spread: the variance is taken about the mean, so that
    only the input's own rounding (2^-24 of the mean, 100 / 2^24 of the spread) is left."""
    x, w, b, z, dy = make(6, L, 512, F32, False, True, 3, shift=100.0)
    ry, rm, rr, rg = R.group_norm(x, 4, w, b, None, "silu", 1e-5, dy)
    y, mean, rstd = mdn.group_norm_fwd(x.cuda(), 4, cu(w), cu(b))
    assert R.rel(mean, rm) <= 1e-6 and R.rel(rstd, rr) <= 2e-5 and R.rel(y, ry) <= 5e-5


def test_constant_group_and_not_finite():
    """No spread: xhat = 0.  A NaN or infinity stays in its group."""
    x = torch.full((3, 1, 64), 2.5, device="cuda")
    y, mean, rstd = mdn.group_norm_fwd(x, 4, act="none")
    assert (y == 0).all() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))
    for L in (1, 50):
        x = torch.randn(3, L, 64, device="cuda")
        x[1, L // 2, 20] = float("nan")
        x[2, 0, 3] = float("inf")
        y, mean, rstd = mdn.group_norm_fwd(x, 4)
        bad = ~torch.isfinite(y.reshape(3, L, 4, 16)).all(3).all(1)
        expect = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
        expect[1, 1] = expect[2, 0] = True
        assert torch.equal(bad, expect)


def test_unaligned_tensors_take_the_scalar_path():
    x, w, b, z, dy = make(40, 1, 256, BF16, True, True, 9)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)]).cuda()[1:].view(t.shape)
    a = mdn.group_norm_fwd(x.cuda(), 2, cu(w), cu(b), cu(z))
    c = mdn.group_norm_fwd(off(x), 2, off(w), off(b), off(z))
    ry = R.group_norm(x, 2, w, b, z, "silu", 1e-5)[0]
    assert R.rel(a[0], ry) <= TOL[BF16] and R.rel(c[0], ry) <= TOL[BF16]
    g = mdn.group_norm_bwd(off(x), 2, c[1], c[2], off(dy), off(w), off(b), off(z))
    rg = R.group_norm(x, 2, w, b, z, "silu", 1e-5, dy)[3]
    for n in rg:
        assert R.rel(g[n], rg[n]) <= TOL[g[n].dtype], n


@pytest.mark.parametrize("L", [1, 77])
def test_repeatable_captured_and_empty(L):
    x, w, b, z, dy = (cu(t) for t in make(300, L, 256, BF16, True, True, 4))

    def call(**kw):
        y, mean, rstd = mdn.group_norm_fwd(x, 4, w, b, z, **kw)
        return [y, mean, rstd, *mdn.group_norm_bwd(x, 4, mean, rstd, dy, w, b, z, **kw).values()]
    first = call()
    assert all(torch.equal(p, q) for p, q in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    x.copy_(torch.randn_like(x.float()))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, call()))
    e = x[:0].contiguous()
    y, mean, rstd = mdn.group_norm_fwd(e, 4, w, b)
    g = mdn.group_norm_bwd(e, 4, mean, rstd, e, w, b)
    assert y.shape == e.shape and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_more_rows_than_a_grid_dimension():
    """More than 65535 tokens (the tokens form has no such limit)."""
    x = torch.randn(70001, 1, 64, device="cuda")
    y, mean, rstd = mdn.group_norm_fwd(x, 2, act="none")
    r = x.double().reshape(70001, 2, 32)
    ref = ((r - r.mean(2, keepdim=True)) / (r.var(2, unbiased=False, keepdim=True) + 1e-5).sqrt())
    assert R.rel(y.reshape(70001, 2, 32), ref.cpu()) <= 2e-5
