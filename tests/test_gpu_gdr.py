"""The gated delta rule on the GPU against its 64-bit token-by-token reference.

Tolerances (2-norm, relative).  fp32 outputs: sums of at most d = 128 terms a
token and a contracting state, so a few tens of roundings of 2^-24 in a row at
random signs: 2e-5 leaves a factor of ten.  bf16 outputs: one store rounding of at
most 2^-8 relative, and at most three bf16-rounded factors in front of it (the
state, the chunk matrix, vtilde); independent and uniform, their 2-norm is at most
sqrt(4) 2^-8 / sqrt(3) = 4.5e-3."""
import pytest
import torch

import gdr_reference as R
import momentum_delta_rule_mdn_b200 as mdn
from momentum_delta_rule_mdn_b200 import _lib as E

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 4.5e-3}
F32, BF16 = torch.float32, torch.bfloat16


def cuda(x, *names):
    return [None if x[n] is None else x[n].cuda() for n in names]


def check(got, ref, names=None):
    bad = {}
    for n in names or ref:
        e = R.rel(got[n], ref[n])
        if not e <= TOL[got[n].dtype]:
            bad[n] = e
    assert not bad, bad


SHAPES = [  # B, T, H, Hk, d
    (1, 1, 1, 1, 64), (2, 1, 4, 2, 128), (1, 2, 2, 2, 128), (1, 63, 2, 1, 64), (2, 64, 3, 3, 128),
    (1, 65, 4, 1, 128), (1, 127, 2, 2, 128), (2, 129, 2, 1, 64), (3, 200, 6, 2, 128),
    (1, 517, 2, 2, 128), (1, 1000, 1, 1, 64), (40, 70, 16, 4, 128),
]


@pytest.mark.parametrize("flags", [0, E.MDN_FORCE_SIMT])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradients(shape, dtype, flags):
    B, T, H, Hk, d = shape
    x = R.inputs(B, T, H, Hk, d, dtype, seed=T * 7 + H, state=T % 2 == 1)
    sc = d ** -0.5
    q, k, v, al, be, S0, do, dST = cuda(x, "q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=flags)
    ref = dict(zip(("o", "vt", "S"), R.fwd(x["q"], x["k"], x["v"], x["alpha_log"], x["beta"], sc,
                                           x["S0"])))
    check(dict(o=o, vt=vt, S=S), ref)
    g = mdn.gdr_chunk_bwd(q, k, al, be, None, vt, do, S0, dST, flags=flags)
    ref = R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], sc, vt.cpu(), x["do"], x["S0"], x["dS_T"])
    assert g["dq"].dtype == dtype and g["dalpha_log"].dtype == F32
    check(g, ref)


@pytest.mark.parametrize("B,T,H,Hk", [(4, 2048, 8, 8), (1, 3000, 2, 1), (5, 777, 16, 4), (1, 4100, 37, 37)])
def test_many_chunks_both_paths(B, T, H, Hk):
    """Sequences of many chunks with few and many chains: the tensor-core kernels against the
    fp32 CUDA-core ones (2e-5 covers both sides' fp32 error, 4.5e-3 the bf16 roundings of the
    one and 2^-8 / sqrt(3) of the other's stores: 6.8e-3), and no wait that ran out."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, v, do = r(B, T, Hk, 128).to(BF16), r(B, T, H, 128).to(BF16), r(B, T, H, 128).to(BF16)
    k = torch.nn.functional.normalize(r(B, T, Hk, 128), dim=-1).to(BF16)
    al, be = -torch.nn.functional.softplus(r(B, T, H) - 3), torch.sigmoid(r(B, T, H))
    S0, dST = 0.1 * r(B, H, 128, 128), 0.1 * r(B, H, 128, 128)
    chk = E.MDN_CHECK_FINITE
    a = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=chk)
    b = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=chk | E.MDN_FORCE_SIMT)
    ga = mdn.gdr_chunk_bwd(q, k, al, be, None, b[1], do, S0, dST, flags=chk)
    gb = mdn.gdr_chunk_bwd(q, k, al, be, None, b[1], do, S0, dST, flags=chk | E.MDN_FORCE_SIMT)
    both = dict(zip(("o", "vt", "S"), zip(a, b))) | {n: (ga[n], gb[n]) for n in ga}
    bad = {}
    for n, (x, y) in both.items():
        e = float((x.double() - y.double()).norm() / y.double().norm())
        if not e <= (6.8e-3 if x.dtype == BF16 else 2e-5):
            bad[n] = e
    assert not bad, bad


@pytest.mark.parametrize("decay", [-12.0, 3.0])
def test_extreme_decay(decay):
    """alpha close to 1 (nothing forgotten over the whole sequence), and alpha ~ e^-3
    and less (a chunk's products of decays underflow)."""
    x = R.inputs(1, 300, 2, 2, 128, BF16, seed=5, decay=decay)
    x["alpha_log"][0, 100:110] = -200.0   # and a hard reset
    q, k, v, al, be, S0, do, dST = cuda(x, "q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, 0.3, S0)
    check(dict(o=o, vt=vt, S=S), dict(zip(("o", "vt", "S"), R.fwd(
        x["q"], x["k"], x["v"], x["alpha_log"], x["beta"], 0.3, x["S0"]))))
    g = mdn.gdr_chunk_bwd(q, k, al, be, 0.3, vt, do, S0, dST)
    check(g, R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], 0.3, vt.cpu(), x["do"], x["S0"],
                   x["dS_T"]))


def test_zero_and_one_gates():
    """beta = 0 writes nothing; alpha = 1, beta = 1 with a repeated unit key overwrites."""
    x = R.inputs(1, 130, 2, 2, 128, F32, seed=6)
    x["beta"][:, 40:80] = 0.0
    x["beta"][:, 80:] = 1.0
    x["alpha_log"][:, 80:] = 0.0
    x["k"][:, 100:] = x["k"][:, 100:101]
    for dtype in (F32, BF16):
        y = {n: t.to(dtype) if n in ("q", "k", "v", "do") else t for n, t in x.items()}
        q, k, v, al, be, S0, do, dST = cuda(y, "q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
        o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, 1.0, S0)
        check(dict(o=o, vt=vt, S=S), dict(zip(("o", "vt", "S"), R.fwd(
            y["q"], y["k"], y["v"], y["alpha_log"], y["beta"], 1.0, y["S0"]))))
        g = mdn.gdr_chunk_bwd(q, k, al, be, 1.0, vt, do, S0, dST)
        check(g, R.bwd(y["q"], y["k"], y["alpha_log"], y["beta"], 1.0, vt.cpu(), y["do"], y["S0"],
                       y["dS_T"]))


LENGTHS = [(5,), (64, 1, 0, 130), (1, 1, 1), (0, 0, 77, 0), (300, 65, 63, 2, 0, 128), (0,)]


@pytest.mark.parametrize("dtype,d,Hk", [(F32, 64, 2), (BF16, 128, 4), (BF16, 128, 1), (BF16, 64, 4)])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_packed(lengths, dtype, d, Hk):
    """Each sequence as if it were alone; rows behind the last one untouched, and not
    read into any result (they hold NaN)."""
    H, extra, N = 4, 5, len(lengths)
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    x = R.inputs(1, off[-1] + extra, H, Hk, d, dtype, seed=11 + N, state=False)
    x = {n: t[0] if t is not None else None for n, t in x.items()}
    g = torch.Generator().manual_seed(9)
    S0, dST = (0.1 * torch.randn(N, H, d, d, generator=g) for _ in range(2))
    for n in ("q", "k", "v", "do", "alpha_log", "beta"):
        x[n][off[-1]:] = float("nan")
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    q, k, v, al, be, do = cuda(x, "q", "k", "v", "alpha_log", "beta", "do")
    mark = lambda t: torch.full_like(t, 7.0)
    out = (mark(v), mark(v), torch.empty(N, H, d, d, device="cuda"))
    o, vt, S = mdn.gdr_chunk_fwd_varlen(q, k, v, al, be, cu, None, S0.cuda(), out=out)
    assert (o[off[-1]:] == 7).all() and (vt[off[-1]:] == 7).all()
    vt[off[-1]:] = float("nan")
    gr = mdn.gdr_chunk_bwd_varlen(q, k, al, be, cu, None, vt, do, S0.cuda(), dST.cuda())
    for n in ("dq", "dk", "dv", "dalpha_log", "dbeta"):
        assert (gr[n][off[-1]:] == 0).all(), n
    for s in range(N):
        sl = slice(off[s], off[s + 1])
        one = lambda t: t[None, sl].cpu()
        r = R.fwd(one(x["q"]), one(x["k"]), one(x["v"]), one(x["alpha_log"]), one(x["beta"]),
                  d ** -0.5, S0[s:s + 1])
        check(dict(o=o[None, sl], vt=vt[None, sl], S=S[s:s + 1]), dict(zip(("o", "vt", "S"), r)))
        r = R.bwd(one(x["q"]), one(x["k"]), one(x["alpha_log"]), one(x["beta"]), d ** -0.5, one(vt),
                  one(x["do"]), S0[s:s + 1], dST[s:s + 1])
        check({n: gr[n][s:s + 1] if n == "dS0" else gr[n][None, sl] for n in r}, r)


@pytest.mark.parametrize("off", [(0, 70, 60, 90), (1, 20, 30, 90), (0, 20, 30, 200), (0, -5, 30, 90)])
def test_packed_bad_offsets(off):
    """Broken offsets make every sequence empty and are reported."""
    x = R.inputs(1, 100, 2, 2, 128, BF16, seed=2)
    q, k, v, al, be = (t[0].cuda() for t in (x["q"], x["k"], x["v"], x["alpha_log"], x["beta"]))
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    S0 = torch.randn(3, 2, 128, 128, device="cuda")
    ws = torch.empty(mdn.gdr_chunk_workspace_size(3, 100, 2, 2, 128, packed=True), dtype=torch.uint8,
                     device="cuda")
    o, vt, S = mdn.gdr_chunk_fwd_varlen(q, k, v, al, be, cu, None, S0, workspace=ws)
    assert (o == 0).all() and (vt == 0).all() and torch.equal(S, S0)
    assert mdn.chunk_fwd_status(ws) == E.MDN_ERR_INVALID_ARG
    with pytest.raises(mdn.MDNError):
        mdn.gdr_chunk_fwd_varlen(q, k, v, al, be, cu, None, S0, flags=E.MDN_CHECK_FINITE)
    g = mdn.gdr_chunk_bwd_varlen(q, k, al, be, cu, None, v, v, S0, S0)
    assert (g["dq"] == 0).all() and (g["dv"] == 0).all() and torch.equal(g["dS0"], S0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,d", [(1, 1, 1, 64), (1, 16, 4, 128), (3, 6, 2, 64), (5, 8, 8, 128),
                                      (19, 8, 1, 128), (40, 16, 16, 128), (75, 8, 2, 64)])
def test_step(B, H, Hk, d, dtype):
    """Tokens one by one, in place and into another buffer, against the recurrence."""
    T = 3
    x = R.inputs(B, T, H, Hk, d, dtype, seed=B)
    o_ref, vt_ref, S_ref = R.fwd(x["q"], x["k"], x["v"], x["alpha_log"], x["beta"], d ** -0.5, x["S0"])
    S = x["S0"].cuda()
    for t in range(T):
        args = [x[n][:, t].cuda().contiguous() for n in ("q", "k", "v", "alpha_log", "beta")]
        before = S.clone()
        S2 = torch.empty_like(S)
        o2, none = mdn.gdr_step(*args, None, S, S_out=S2, want_vtilde=False)
        assert none is None and torch.equal(S, before)
        o, vt = mdn.gdr_step(*args, None, S)
        assert torch.equal(S, S2) and torch.equal(o, o2)
        check(dict(o=o, vt=vt), dict(o=o_ref[:, t], vt=vt_ref[:, t]))
    check(dict(S=S), dict(S=S_ref))


def test_prefill_then_decode_and_layer_gradients():
    """The operators as a layer uses them: a prompt through the chunk pass, tokens after it
    one by one, the output norm over both; then the gradients of the prompt's part through
    norm and rule against the same chain in 64 bits."""
    B, T, H, Hk, d, extra = 2, 150, 4, 2, 128, 3
    x = R.inputs(B, T + extra, H, Hk, d, BF16, seed=21)
    names = ("q", "k", "v", "alpha_log", "beta")
    head = [x[n][:, :T].contiguous().cuda() for n in names]
    o, vt, S = mdn.gdr_chunk_fwd(*head, None, x["S0"].cuda())
    state = S.clone()
    steps = []
    for t in range(T, T + extra):
        o1, _ = mdn.gdr_step(*[x[n][:, t].contiguous().cuda() for n in names], None, state)
        steps.append(o1)
    ro, _, rS = R.fwd(*[x[n] for n in names], d ** -0.5, x["S0"])
    check(dict(o=torch.cat([o, torch.stack(steps, 1)], 1), S=state), dict(o=ro, S=rS))
    g = torch.Generator().manual_seed(4)
    w, b = 1 + 0.1 * torch.randn(H * d, generator=g), 0.1 * torch.randn(H * d, generator=g)
    gate = torch.randn(B * T, 1, H * d, generator=g).to(BF16)
    dy = torch.randn(B * T, 1, H * d, generator=g).to(BF16)
    flat = o.view(B * T, 1, H * d)
    y, mean, rstd = mdn.group_norm_fwd(flat, H, w.cuda(), b.cuda(), gate.cuda())
    n = mdn.group_norm_bwd(flat, H, mean, rstd, dy.cuda(), w.cuda(), b.cuda(), gate.cuda())
    grads = mdn.gdr_chunk_bwd(head[0], head[1], head[3], head[4], None, vt,
                              n["dx"].view(B, T, H, d), x["S0"].cuda())
    ry, _, _, rn = R.group_norm(flat.cpu(), H, w, b, gate, "silu", 1e-5, dy)
    check(dict(y=y, **n), dict(y=ry, **rn))
    cut = lambda t: t[:, :T]
    ref = R.bwd(cut(x["q"]), cut(x["k"]), cut(x["alpha_log"]), cut(x["beta"]), d ** -0.5, vt.cpu(),
                n["dx"].view(B, T, H, d).cpu(), x["S0"])
    check(grads, ref)


def test_gradients_against_differences():
    """Central differences of the 64-bit loss against the fp32 gradients: the differences are
    good to 1e-8, the gradients and the saved vtilde to some 1e-6."""
    x = R.inputs(1, 70, 1, 1, 64, F32, seed=8)
    q, k, v, al, be, S0, do, dST = cuda(x, "q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    _, vt, _ = mdn.gdr_chunk_fwd(q, k, v, al, be, 0.4, S0)
    g = mdn.gdr_chunk_bwd(q, k, al, be, 0.4, vt, do, S0, dST)
    x = {n: t.double() for n, t in x.items()}

    def loss(y):
        o, _, S = R.fwd(y["q"], y["k"], y["v"], y["alpha_log"], y["beta"], 0.4, y["S0"])
        return float((o * y["do"]).sum() + (S * y["dS_T"]).sum())
    gen = torch.Generator().manual_seed(1)
    for n in ("q", "k", "v", "alpha_log", "beta", "S0"):
        e = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        num = (loss({**x, n: x[n] + h * e}) - loss({**x, n: x[n] - h * e})) / (2 * h)
        got = float((g["d" + n].double().cpu() * e).sum())
        size = float(g["d" + n].double().norm() * e.norm()) / e.numel() ** 0.5
        assert abs(got - num) <= 2e-5 * max(size, abs(num)), (n, got, num)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeatable_captured_and_on_another_stream(dtype):
    """Equal calls give equal bits; so do a captured and replayed call with new inputs in the
    same buffers, and a call on a side stream."""
    B, T, H, Hk, d = 2, 190, 6, 2, 128
    x, x2 = (R.inputs(B, T, H, Hk, d, dtype, seed=s) for s in (31, 32))
    names = ("q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    buf = dict(zip(names, cuda(x, *names)))

    def call(**kw):
        o, vt, S = mdn.gdr_chunk_fwd(*[buf[n] for n in names[:5]], None, buf["S0"], **kw)
        g = mdn.gdr_chunk_bwd(buf["q"], buf["k"], buf["alpha_log"], buf["beta"], None, vt, buf["do"],
                              buf["S0"], buf["dS_T"], **kw)
        return [o, vt, S, *g.values()]
    first = call()
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for n, t in zip(names, cuda(x2, *names)):
        buf[n].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, call()))


def test_state_may_alias_and_empty_sequence():
    x = R.inputs(2, 100, 2, 2, 128, BF16, seed=3)
    q, k, v, al, be, S0 = cuda(x, "q", "k", "v", "alpha_log", "beta", "S0")
    o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0)
    A = S0.clone()
    o2, none, S2 = mdn.gdr_chunk_fwd(q, k, v, al, be, None, A, out=(torch.empty_like(v), None, A))
    assert none is None and S2 is A and torch.equal(A, S) and torch.equal(o, o2)
    cut = [t[:, :0].contiguous() for t in (q, k, v, al, be)]
    o, vt, S = mdn.gdr_chunk_fwd(*cut, None, S0)
    assert torch.equal(S, S0) and o.shape[1] == 0
    g = mdn.gdr_chunk_bwd(cut[0], cut[1], cut[3], cut[4], None, vt, vt, S0, S)
    assert torch.equal(g["dS0"], S)
    none = [t[:0].contiguous() for t in (q, k, v, al, be)]
    assert mdn.gdr_chunk_fwd(*none)[2].shape[0] == 0


def test_check_finite_reports():
    x = R.inputs(1, 80, 2, 2, 128, BF16, seed=3)
    q, k, v, al, be, S0 = cuda(x, "q", "k", "v", "alpha_log", "beta", "S0")
    mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=E.MDN_CHECK_FINITE)
    v[0, 70, 1, 5] = float("inf")
    with pytest.raises(mdn.MDNError) as e:
        mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=E.MDN_CHECK_FINITE)
    assert e.value.status == E.MDN_ERR_NONFINITE
    # the infinity stays in its head and behind its token
    o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0)
    assert torch.isfinite(o[0, :, 0]).all() and torch.isfinite(S[0, 0]).all()
    assert not torch.isfinite(vt[0, 70, 1, 5])
