"""dalpha_log of the gated delta rule token by token: strong decays and resets among slow tokens,
each against its own size.

With S the state before token t and G' the adjoint it is paired with, dalpha_log_t =
alpha_t <G', S>, an inner product of d x d matrices, of size alpha_t |G'| |S| / d where they are
not related.  Tolerances, of that size: fp32, some ten sums of d products, each off by some
sqrt(d) roundings of 2^-24 / sqrt(3): 1.3e-6 in the mean square, three times that at the worst
of some hundred tokens, and a factor of two: 1e-5.  Tensor cores: seven factors on the way
are two bf16 terms, 2^-17 / sqrt(3) each in the mean square, 1.2e-5, three times that: 4e-5.
Where alpha is 0 in fp32 every term is, and the result."""
import pytest
import torch

import gdr_reference as R
import momentum_delta_rule_mdn_b200 as mdn
from momentum_delta_rule_mdn_b200 import _lib as E

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def sizes(q, k, alpha_log, beta, scale, vt, do, S0, dS_T):
    """(dalpha_log, alpha |G'| |S| / d) by the recurrences in 64 bits; [T,...] inputs."""
    T, H, d = vt.shape
    q, k, vt, do = R.rep(q, H), R.rep(k, H), vt.to(R.F64), do.to(R.F64)
    a, b = alpha_log.to(R.F64).exp(), beta.to(R.F64)
    S = [S0.to(R.F64)]
    for t in range(T):
        S.append(a[t, :, None, None] * S[-1] + b[t, :, None, None] * k[t, :, :, None] * vt[t, :, None, :])
    G, da, size = dS_T.to(R.F64), torch.empty_like(a), torch.empty_like(a)
    for t in reversed(range(T)):
        G = G + scale * q[t, :, :, None] * do[t, :, None, :]
        dv = b[t, :, None] * (G.transpose(-1, -2) @ k[t, :, :, None])[..., 0]
        G = G - k[t, :, :, None] * dv[:, None, :]
        da[t] = a[t] * (G * S[t]).sum((-1, -2))
        size[t] = a[t] * G.flatten(1).norm(dim=1) * S[t].flatten(1).norm(dim=1) / d
        G = a[t, :, None, None] * G
    return da, size


@pytest.mark.parametrize("off", [(0, 200), (0, 33, 33, 170, 200)])
@pytest.mark.parametrize("dtype,d,flags", [(F32, 64, 0), (F32, 128, 0), (BF16, 64, 0), (BF16, 128, 0),
                                           (BF16, 128, E.MDN_FORCE_SIMT)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (24, 24)])
def test_single_tokens_of_strong_decay(H, Hk, dtype, d, flags, off):
    """alpha of e^-8 to e^-14, and 0, at a chunk's ends and inside its blocks of 16."""
    T, N = off[-1], len(off) - 1
    x = R.inputs(1, T, H, Hk, d, dtype, seed=17, state=False)
    g = torch.Generator().manual_seed(18)
    S0, dST = (0.1 * torch.randn(N, H, d, d, generator=g) for _ in range(2))
    for t, a in ((5, -8.0), (16, -10.0), (31, -12.0), (32, -8.0), (47, -9.0), (63, -8.0), (64, -14.0),
                 (65, -8.0), (100, -200.0), (117, -11.0), (130, float("-inf")), (191, -8.0), (199, -12.0)):
        x["alpha_log"][:, t] = a
    one = {n: t[0] for n, t in x.items() if t is not None}
    q, k, v, al, be, do = (one[n].cuda() for n in ("q", "k", "v", "alpha_log", "beta", "do"))
    if N == 1:
        vt = mdn.gdr_chunk_fwd(q[None], k[None], v[None], al[None], be[None], None, S0.cuda(), flags=flags)[1][0]
        got = mdn.gdr_chunk_bwd(q[None], k[None], al[None], be[None], None, vt[None], do[None], S0.cuda(),
                                dST.cuda(), flags=flags)["dalpha_log"][0]
    else:
        cu = torch.tensor(off, dtype=torch.int32, device="cuda")
        vt = mdn.gdr_chunk_fwd_varlen(q, k, v, al, be, cu, None, S0.cuda(), flags=flags)[1]
        got = mdn.gdr_chunk_bwd_varlen(q, k, al, be, cu, None, vt, do, S0.cuda(), dST.cuda(),
                                       flags=flags)["dalpha_log"]
    got, vt = got.cpu().to(R.F64), vt.cpu()
    tol = 4e-5 if (dtype, d, flags) == (BF16, 128, 0) else 1e-5
    for s in range(N):
        sl = slice(off[s], off[s + 1])
        ref, size = sizes(*(one[n][sl] for n in ("q", "k", "alpha_log", "beta")), d ** -0.5, vt[sl],
                          one["do"][sl], S0[s], dST[s])
        err = ((got[sl] - ref).abs() / size.clamp_min(1e-37)).amax(1)   # 1e-37: alpha is 0 in fp32
        bad = {off[s] + t: float(e) for t, e in enumerate(err) if not e <= tol}
        assert not bad, bad
