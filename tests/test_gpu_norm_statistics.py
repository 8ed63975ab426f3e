"""Statistics of group norm over long rows in which a few values lie far from the rest, against
the definition in 64 bits.

Tolerances.  A block of rows is summed in 64 bits and its mean and sum of squared distances
are rounded to fp32 once (2^-24 each); at most 592 blocks join in 19 additions a lane and 5
across lanes.  Their sum of squares is then off by at most 26 roundings, 1.6e-6, rstd by half
of that and rsqrtf's 2 ulp: 2e-6.  The mean is off by as many roundings of a block's mean, which
is at most about the group's standard deviation here: 4e-6 of that.  y adds the roundings of
the normed value and the few 1e-7 of the sigmoid: 1e-5 in the 2-norm; in bf16 also the store's
half step, at most 2^-8 of each value and so of the norm (the far values' few roundings make up
the norm, so that no average holds: 569.5 is stored as 568, 2.6e-3 off)."""
import pytest
import torch

import momentum_delta_rule_mdn_b200 as mdn

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def stats(x, G):
    N, L, C = x.shape
    h = x.double().reshape(N, L, G, C // G)
    mean = h.mean((1, 3))
    var = (h - mean[:, None, :, None]).square().mean((1, 3))
    return mean, var.sqrt(), 1 / (var + 1e-5).sqrt()


def check(x, G):
    y, mean, rstd = mdn.group_norm_fwd(x, G, act="silu")
    rm, std, rr = stats(x, G)
    assert float((rstd.double() / rr - 1).abs().max()) <= 2e-6
    assert float(((mean.double() - rm).abs() / std).max()) <= 4e-6
    N, L, C = x.shape
    n = ((x.double().reshape(N, L, G, -1) - rm[:, None, :, None]) * rr[:, None, :, None]).reshape(x.shape)
    ry = n * torch.sigmoid(n)
    tol = 1e-5 if x.dtype is F32 else 1e-5 + 2.0 ** -8
    assert float((y.double() - ry).norm() / ry.norm()) <= tol


SHAPES = [  # N, L, C, G: one to many row blocks a sequence, one row of a wide group
    (600, 700, 64, 2), (200, 900, 256, 4), (3, 5000, 128, 4), (1, 60000, 24, 3), (5, 1, 4096, 2),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [30.0, -100.0, 1000.0, 1e4])
@pytest.mark.parametrize("shape", SHAPES)
def test_first_value_far_from_the_rest(shape, far, dtype):
    """A first token with huge activations."""
    N, L, C, G = shape
    g = torch.Generator(device="cuda").manual_seed(N + C)
    x = torch.randn(N, L, C, generator=g, device="cuda")
    x[:, 0, ::C // G] = far
    check(x.to(dtype), G)


@pytest.mark.parametrize("shape", SHAPES)
def test_far_values_anywhere(shape):
    """Far values of both signs at seeded places, on a mean of some spreads."""
    N, L, C, G = shape
    g = torch.Generator(device="cuda").manual_seed(L)
    x = torch.randn(N, L, C, generator=g, device="cuda") + 5
    at = torch.randint(0, x.numel(), (max(4, x.numel() // 20000),), generator=g, device="cuda")
    x.view(-1)[at] = 2000 * torch.randn(at.numel(), generator=g, device="cuda")
    check(x, G)


@pytest.mark.parametrize("eps", [1e-5, 0.25, 0.0])
@pytest.mark.parametrize("given", [False, True])
def test_no_rows(given, eps):
    """Groups of no rows: mean 0 and rstd 1 / sqrt(eps), whatever the memory held."""
    x = torch.empty(3, 0, 64, device="cuda")
    held = torch.full((3, 4), 7.0, device="cuda"), torch.full((3, 4), 7.0, device="cuda")
    out = (torch.empty_like(x), *held) if given else None
    del held
    y, mean, rstd = mdn.group_norm_fwd(x, 4, eps=eps, out=out)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4)
    assert (mean == 0).all()
    want = torch.tensor(eps, dtype=torch.float64).rsqrt().float().expand(3, 4)
    assert torch.allclose(rstd.cpu(), want, rtol=2.0 ** -22, atol=0)   # eps and the result in fp32
    w = torch.ones(64, device="cuda")
    g = mdn.group_norm_bwd(x, 4, mean, rstd, x, w, w)
    assert g["dx"].shape == x.shape and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
