"""The gated delta rule's and group norm's entry points without a GPU: workspace
sizes, and refusals before any device work."""
import pytest
import torch

import gdr_reference as R
import momentum_delta_rule_mdn_b200 as mdn
from momentum_delta_rule_mdn_b200 import _lib as E
from momentum_delta_rule_mdn_b200 import build_lib

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return E.load()


def test_reference_gradient_against_differences():
    """The reference adjoint is the derivative of the reference forward pass."""
    x = R.inputs(1, 5, 2, 1, 3, torch.float64, 3)
    x = {n: t.to(R.F64) for n, t in x.items()}
    sc = 0.6

    def loss(**kw):
        y = {**x, **kw}
        o, _, S = R.fwd(y["q"], y["k"], y["v"], y["alpha_log"], y["beta"], sc, y["S0"])
        return (o * x["do"]).sum() + (S * x["dS_T"]).sum()
    _, vt, _ = R.fwd(x["q"], x["k"], x["v"], x["alpha_log"], x["beta"], sc, x["S0"])
    g = R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], sc, vt, x["do"], x["S0"], x["dS_T"])
    h = 1e-6
    for name in ("q", "k", "v", "alpha_log", "beta", "S0"):
        flat = x[name].reshape(-1)
        num = torch.empty_like(flat)
        for i in range(flat.numel()):
            e = torch.zeros_like(flat)
            e[i] = h
            e = e.reshape(x[name].shape)
            num[i] = (loss(**{name: x[name] + e}) - loss(**{name: x[name] - e})) / (2 * h)
        # central differences: h^2 of curvature and eps / h of rounding, both below 1e-8
        assert R.rel(g["d" + name], num.reshape(x[name].shape)) < 1e-7, name


def test_workspace_sizes(lib):
    f, b = lib.mdn_gdr_chunk_fwd_workspace_size, lib.mdn_gdr_chunk_bwd_workspace_size
    fv, bv = lib.mdn_gdr_chunk_fwd_varlen_workspace_size, lib.mdn_gdr_chunk_bwd_varlen_workspace_size
    for w in (f, b, fv, bv):
        assert w(2, 300, 2, 4, 128, 128, 64, E.MDN_BF16, 0) > 0
        assert w(2, 0, 2, 4, 64, 64, 64, E.MDN_F32, 0) > 0
        assert w(2, 300, 3, 4, 128, 128, 64, E.MDN_BF16, 0) == 0   # 4 heads on 3 key heads
        assert w(2, 300, 2, 4, 96, 96, 64, E.MDN_BF16, 0) == 0
        assert w(2, 300, 2, 4, 128, 64, 64, E.MDN_BF16, 0) == 0
        assert w(2, 300, 2, 4, 128, 128, 32, E.MDN_BF16, 0) == 0
        assert w(2, 300, 2, 4, 128, 128, 64, 9, 0) == 0
        assert w(-1, 300, 2, 4, 128, 128, 64, E.MDN_BF16, 0) == 0
        # beyond 2^31 chunk-heads (a packed call's T is the tokens of all its sequences)
        assert w(1 << 15, (1 << 31) - 1, 64, 64, 128, 128, 64, E.MDN_BF16, 0) == 0
    assert b(2, 300, 4, 4, 128, 128, 64, E.MDN_BF16, 0) > f(2, 300, 4, 4, 128, 128, 64, E.MDN_BF16, 0)
    g = lib.mdn_group_norm_workspace_size
    assert g(8, 1, 2048, 16, E.MDN_BF16, 0) == 0
    assert g(8, 1, 2048, 16, E.MDN_BF16, 1) > 0
    assert g(2, 100, 2048, 16, E.MDN_F32, 0) > 0
    assert g(2, 100, 100, 16, E.MDN_F32, 0) == 0


def _fwd(lib, varlen=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=E.MDN_F32, al=FAKE, be=FAKE, sc=0.1, S0=None, B=1, T=100,
             Hk=1, H=2, dk=64, dv=64, C=64, o=FAKE, vt=FAKE, ST=FAKE, ws=FAKE, wsb=1 << 30, flags=0,
             cu=FAKE)
    a.update(kw)
    if varlen:
        return lib.mdn_gdr_chunk_fwd_varlen(
            a["q"], a["k"], a["v"], a["dt"], a["al"], a["be"], a["sc"], a["cu"], a["B"], a["T"],
            a["S0"], a["Hk"], a["H"], a["dk"], a["dv"], a["C"], a["o"], a["vt"], a["ST"], a["ws"],
            a["wsb"], a["flags"], None)
    return lib.mdn_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["dt"], a["al"], a["be"], a["sc"], a["S0"],
                                 a["B"], a["T"], a["Hk"], a["H"], a["dk"], a["dv"], a["C"], a["o"],
                                 a["vt"], a["ST"], a["ws"], a["wsb"], a["flags"], None)


BAD = [dict(q=None), dict(k=FAKE + 4), dict(v=None), dict(o=None), dict(vt=FAKE + 8), dict(al=None),
       dict(be=FAKE + 2), dict(S0=FAKE + 4), dict(ST=None), dict(ws=None), dict(ws=FAKE + 16),
       dict(wsb=0), dict(flags=4), dict(Hk=0), dict(Hk=4, H=6), dict(B=-1), dict(T=-1), dict(C=0),
       dict(sc=float("nan")), dict(sc=float("inf"))]


@pytest.mark.parametrize("varlen", [False, True])
def test_fwd_refusals(lib, varlen):
    for kw in BAD:
        assert _fwd(lib, varlen, **kw) == E.MDN_ERR_INVALID_ARG, kw
    for kw in (dict(dk=96, dv=96), dict(dv=128), dict(C=32), dict(dt=5),
               dict(B=1 << 15, T=(1 << 31) - 1, Hk=64, H=64)):
        assert _fwd(lib, varlen, **kw) == E.MDN_ERR_UNSUPPORTED, kw
    assert _fwd(lib, varlen, B=0, q=None, cu=None) == E.MDN_OK
    assert _fwd(lib, varlen, H=0, Hk=0, q=None) == E.MDN_OK
    zero = E.MDN_ZERO_BEHIND
    assert _fwd(lib, varlen, flags=zero, q=None) == E.MDN_ERR_INVALID_ARG
    assert _fwd(lib, varlen, flags=zero, H=0, Hk=0, q=None) == (E.MDN_OK if varlen else E.MDN_ERR_INVALID_ARG)
    if varlen:
        assert _fwd(lib, True, flags=zero, B=0, o=None) == E.MDN_ERR_INVALID_ARG
        assert _fwd(lib, True, flags=zero, B=0, T=0, o=None) == E.MDN_OK
        assert _fwd(lib, True, cu=None) == E.MDN_ERR_INVALID_ARG
        assert _fwd(lib, True, cu=FAKE + 2) == E.MDN_ERR_INVALID_ARG


def test_bwd_refusals(lib):
    def bw(vt=FAKE, do=FAKE, dST=None, dq=FAKE, da=FAKE, dS0=FAKE, wsb=1 << 30, flags=0, Hk=1, S0=None,
           sc=0.1, B=1):
        return lib.mdn_gdr_chunk_bwd(FAKE, FAKE, E.MDN_F32, FAKE, FAKE, sc, S0, vt, do, dST, B, 100,
                                     Hk, 2, 64, 64, 64, dq, FAKE, FAKE, da, FAKE, dS0, FAKE, wsb,
                                     flags, None)
    for kw in (dict(vt=None), dict(do=FAKE + 4), dict(dST=FAKE + 8), dict(dq=None), dict(da=None),
               dict(da=FAKE + 1), dict(dS0=None), dict(wsb=100), dict(flags=8), dict(Hk=3),
               dict(S0=FAKE + 2), dict(sc=float("inf"))):
        assert bw(**kw) == E.MDN_ERR_INVALID_ARG, kw
    assert bw(B=0, vt=None) == E.MDN_OK


def test_step_refusals(lib):
    def st(q=FAKE, S=FAKE, So=FAKE, B=2, Hk=1, H=2, d=64, dt=E.MDN_BF16, flags=0, vt=None, sc=1.0,
           be=FAKE):
        return lib.mdn_gdr_step(q, FAKE, FAKE, dt, FAKE, be, sc, S, So, B, Hk, H, d, d, FAKE, vt,
                                flags, None)
    for kw in (dict(q=None), dict(q=FAKE + 1), dict(S=None), dict(So=FAKE + 8), dict(Hk=0),
               dict(Hk=2, H=3), dict(flags=1), dict(vt=FAKE + 1), dict(sc=float("nan")),
               dict(be=FAKE + 2), dict(B=-1)):
        assert st(**kw) == E.MDN_ERR_INVALID_ARG, kw
    assert st(d=32) == E.MDN_ERR_UNSUPPORTED
    assert st(dt=3) == E.MDN_ERR_UNSUPPORTED
    assert st(B=0, q=None) == E.MDN_OK


def test_group_norm_refusals(lib):
    def fw(x=FAKE, y=FAKE, gate=None, w=FAKE, b=FAKE, N=4, L=1, C=64, G=4, eps=1e-5, act=1, mean=FAKE,
           dt=E.MDN_BF16, ws=FAKE, wsb=1 << 30):
        return lib.mdn_group_norm_fwd(x, gate, dt, w, b, N, L, C, G, eps, act, y, mean, FAKE, ws, wsb,
                                      None)
    for kw in (dict(x=None), dict(y=FAKE + 1), dict(gate=FAKE + 1), dict(w=None), dict(b=None),
               dict(w=FAKE + 2), dict(N=-1), dict(L=-1), dict(C=0), dict(G=0), dict(G=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(act=2), dict(mean=None),
               dict(L=5, ws=None), dict(L=5, wsb=3), dict(L=5, ws=FAKE + 4)):
        assert fw(**kw) == E.MDN_ERR_INVALID_ARG, kw
    assert fw(dt=4) == E.MDN_ERR_UNSUPPORTED
    assert fw(N=1 << 17, L=2) == E.MDN_ERR_UNSUPPORTED
    assert fw(C=1 << 22, G=1) == E.MDN_ERR_UNSUPPORTED
    assert fw(C=1 << 20, G=1 << 20, N=1, L=2) == E.MDN_ERR_UNSUPPORTED
    assert fw(C=1, G=1, N=1, L=(1 << 31) - 4) == E.MDN_ERR_UNSUPPORTED
    assert fw(N=0, x=None) == E.MDN_OK and fw(L=0, x=None) == E.MDN_OK

    def bw(dy=FAKE, dx=FAKE, gate=None, dg=None, w=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30,
           rstd=FAKE):
        return lib.mdn_group_norm_bwd(FAKE, gate, E.MDN_BF16, w, w, FAKE, rstd, dy, 4, 1, 64, 4, 1, dx,
                                      dg, dw, db, ws, wsb, None)
    for kw in (dict(dy=None), dict(dx=None), dict(gate=FAKE), dict(dg=FAKE), dict(w=None),
               dict(dw=None), dict(db=None), dict(db=FAKE + 2), dict(ws=None), dict(wsb=1),
               dict(rstd=None)):
        assert bw(**kw) == E.MDN_ERR_INVALID_ARG, kw


def test_python_refusals(lib):
    """Shapes, types and devices are checked before the library is called."""
    x = R.inputs(1, 4, 2, 2, 64, torch.float32, 1)
    with pytest.raises(ValueError, match="CUDA"):
        mdn.gdr_chunk_fwd(x["q"], x["k"], x["v"], x["alpha_log"], x["beta"])
    with pytest.raises(ValueError, match="multiple"):
        mdn.gdr_chunk_fwd(torch.zeros(1, 4, 3, 64), x["k"], x["v"], x["alpha_log"], x["beta"])
    with pytest.raises(ValueError, match="v: expected"):
        mdn.gdr_chunk_fwd(x["q"], x["k"], x["v"].double(), x["alpha_log"], x["beta"])
    with pytest.raises(ValueError, match="k: expected"):
        mdn.gdr_chunk_fwd(x["q"], x["k"].transpose(1, 2), x["v"], x["alpha_log"], x["beta"])
    with pytest.raises(ValueError, match="finite"):
        mdn.gdr_chunk_fwd(x["q"], x["k"], x["v"], x["alpha_log"], x["beta"], float("nan"))
    with pytest.raises(ValueError, match="cu_seqlens"):
        mdn.gdr_chunk_fwd_varlen(x["q"][0], x["k"][0], x["v"][0], x["alpha_log"][0], x["beta"][0],
                                 torch.tensor([0, 4]))
    with pytest.raises(TypeError):
        mdn.gdr_chunk_fwd(x["q"].half(), x["k"], x["v"], x["alpha_log"], x["beta"])
    with pytest.raises(ValueError, match="vtilde"):
        mdn.gdr_chunk_bwd(x["q"], x["k"], x["alpha_log"], x["beta"], None, x["v"][:, :2], x["v"])
    with pytest.raises(ValueError, match="S: expected"):
        mdn.gdr_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["alpha_log"][:, 0], x["beta"][:, 0],
                     None, torch.zeros(1, 2, 64, 32))
    with pytest.raises(ValueError, match="groups"):
        mdn.group_norm_fwd(torch.zeros(2, 1, 10), 3)
    with pytest.raises(ValueError, match="both or neither"):
        mdn.group_norm_fwd(torch.zeros(2, 1, 10), 2, torch.ones(10))
    with pytest.raises(ValueError, match="act"):
        mdn.group_norm_fwd(torch.zeros(2, 1, 10), 2, act="gelu")
    with pytest.raises(ValueError, match="dimensions"):
        mdn.group_norm_fwd(torch.zeros(2, 10), 2)
    with pytest.raises(ValueError, match="CUDA"):
        mdn.group_norm_fwd(torch.zeros(2, 1, 10), 2)
