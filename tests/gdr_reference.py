"""The gated delta rule and group norm in 64 bits on the CPU, token by token and
by their definitions, and seeded inputs for their tests."""
import torch

F64 = torch.float64


def rep(x, H):
    return x.to(F64).repeat_interleave(H // x.shape[-2], dim=-2)


def fwd(q, k, v, alpha_log, beta, scale, S0=None):
    """[B,T,...] inputs -> o, vtilde, S_T."""
    B, T, H, d = v.shape
    q, k, v = rep(q, H), rep(k, H), v.to(F64)
    a, b = alpha_log.to(F64).exp(), beta.to(F64)
    S = torch.zeros(B, H, d, d, dtype=F64) if S0 is None else S0.to(F64).clone()
    o, vt = torch.empty_like(v), torch.empty_like(v)
    for t in range(T):
        S = a[:, t, :, None, None] * S
        vt[:, t] = v[:, t] - (S.transpose(-1, -2) @ k[:, t, :, :, None])[..., 0]
        S = S + b[:, t, :, None, None] * k[:, t, :, :, None] * vt[:, t, :, None, :]
        o[:, t] = scale * (S.transpose(-1, -2) @ q[:, t, :, :, None])[..., 0]
    return o, vt, S


def bwd(q, k, alpha_log, beta, scale, vt, do, S0=None, dS_T=None):
    """The adjoint from the given vtilde (the states are rebuilt from it)."""
    B, T, H, d = vt.shape
    Hk = q.shape[2]
    q, k, vt, do = rep(q, H), rep(k, H), vt.to(F64), do.to(F64)
    a, b = alpha_log.to(F64).exp(), beta.to(F64)
    S = [torch.zeros(B, H, d, d, dtype=F64) if S0 is None else S0.to(F64)]
    for t in range(T):
        S.append(a[:, t, :, None, None] * S[-1]
                 + b[:, t, :, None, None] * k[:, t, :, :, None] * vt[:, t, :, None, :])
    G = torch.zeros(B, H, d, d, dtype=F64) if dS_T is None else dS_T.to(F64)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(vt)
    da, db = torch.empty_like(a), torch.empty_like(b)
    mv = lambda M, x: (M @ x[..., None])[..., 0]
    for t in reversed(range(T)):
        at, bt = a[:, t, :, None], b[:, t, :, None]
        G = G + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * mv(S[t + 1], do[:, t])
        dv[:, t] = bt * mv(G.transpose(-1, -2), k[:, t])
        Gv = mv(G, vt[:, t])
        dk[:, t] = bt * Gv - at * mv(S[t], dv[:, t])
        db[:, t] = (k[:, t] * Gv).sum(-1)
        G = G - k[:, t, :, :, None] * dv[:, t, :, None, :]
        da[:, t] = a[:, t] * (G * S[t]).sum((-1, -2))
        G = at[..., None] * G
    fold = lambda x: x.unflatten(2, (Hk, H // Hk)).sum(3)
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dalpha_log=da, dbeta=db, dS0=G)


def inputs(B, T, H, Hk, d, dtype, seed, state=True, decay=-3.0):
    """Seeded inputs as stored (CPU): k normed, gates in their usual range."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = dict(q=r(B, T, Hk, d).to(dtype),
             k=torch.nn.functional.normalize(r(B, T, Hk, d), dim=-1).to(dtype),
             v=r(B, T, H, d).to(dtype),
             alpha_log=-torch.nn.functional.softplus(r(B, T, H) + decay),
             beta=torch.sigmoid(r(B, T, H)), do=r(B, T, H, d).to(dtype),
             S0=0.1 * r(B, H, d, d) if state else None,
             dS_T=0.1 * r(B, H, d, d) if state else None)
    return x


def group_norm(x, G, weight, bias, gate, act, eps, dy=None):
    """y, mean, rstd and (with dy) the gradients by autograd, in 64 bits."""
    leaf = lambda t: None if t is None else t.to(F64).requires_grad_(True)
    x, weight, bias, gate = leaf(x), leaf(weight), leaf(bias), leaf(gate)
    N, L, C = x.shape
    h = x.reshape(N, L, G, C // G)
    mean = h.mean((1, 3), keepdim=True)
    rstd = 1 / ((h - mean).square().mean((1, 3), keepdim=True) + eps).sqrt()
    n = ((h - mean) * rstd).reshape(N, L, C)
    if weight is not None:
        n = n * weight + bias
    f = (lambda z: z * torch.sigmoid(z)) if act == "silu" else (lambda z: z)
    y = f(n) if gate is None else n * f(gate)
    grads = {}
    if dy is not None:
        (y * dy.to(F64)).sum().backward()
        grads = {n_: t.grad for n_, t in (("dx", x), ("dgate", gate), ("dweight", weight),
                                          ("dbias", bias)) if t is not None}
    return y.detach(), mean.detach().reshape(N, G), rstd.detach().reshape(N, G), grads


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    n = ref.norm()
    return float((got - ref).norm() / n) if n > 0 else float(got.norm())
