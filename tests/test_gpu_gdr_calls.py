"""How calls of the gated delta rule and of the norms meet: back to back, on two streams at
once, in captured graphs that share a workspace, and packed calls of many sequences."""
import pytest
import torch

import gdr_reference as R
import momentum_delta_rule_mdn_b200 as mdn
from momentum_delta_rule_mdn_b200 import _lib as E

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(lead, H, Hk, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*lead, *s, generator=g, device="cuda")
    k = torch.nn.functional.normalize(r(Hk, d), dim=-1)
    return dict(q=r(Hk, d).to(dtype), k=k.to(dtype), v=r(H, d).to(dtype),
                al=-torch.nn.functional.softplus(r(H) - 3), be=torch.sigmoid(r(H)), do=r(H, d).to(dtype))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def layer(x, ws=None, stream=None, cu=None):
    """Forward, norm and the gradients of both, as a layer uses them."""
    kw = dict(workspace=ws, stream=stream)
    if cu is None:
        o, vt, S = mdn.gdr_chunk_fwd(x["q"], x["k"], x["v"], x["al"], x["be"], **kw)
    else:
        o, vt, S = mdn.gdr_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["al"], x["be"], cu, **kw)
    rows, H = o.numel() // (o.shape[-1] * o.shape[-2]), o.shape[-2]
    on = o.view(rows, 1, -1)
    y, m, r = mdn.group_norm_fwd(on, H, gate=x["do"].view_as(on), stream=stream)
    g = mdn.group_norm_bwd(on, H, m, r, y, gate=x["do"].view_as(on), stream=stream)
    args = (x["q"], x["k"], x["al"], x["be"])
    if cu is None:
        b = mdn.gdr_chunk_bwd(*args, None, vt, g["dx"].view_as(o), **kw)
    else:
        b = mdn.gdr_chunk_bwd_varlen(*args, cu, None, vt, g["dx"].view_as(o), **kw)
    return [o, vt, S, y, m, r, g["dx"], g["dgate"], *b.values()]


def scratch(B, T, Hk, H, d, dtype, packed=False):
    n = max(mdn.gdr_chunk_workspace_size(B, T, Hk, H, d, dtype=dtype, packed=packed, backward=b)
            for b in (False, True))
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("B,T,H,Hk,d,dtype", [(4, 2048, 8, 8, 128, BF16), (1, 3000, 16, 4, 128, BF16),
                                              (2, 700, 3, 3, 64, BF16), (2, 300, 4, 2, 64, F32)])
def test_back_to_back_on_one_workspace(B, T, H, Hk, d, dtype):
    """Each call clears and reuses what the call before it left running last."""
    x, ws = inputs((B, T), H, Hk, d, dtype, 1), scratch(B, T, Hk, H, d, dtype)
    first = layer(x, ws)
    torch.cuda.synchronize()
    runs = [layer(x, ws) for _ in range(8)]
    assert all(same(first, r) for r in runs)


@pytest.mark.parametrize("B,T,H,Hk,dtype", [(4, 1024, 8, 8, BF16), (1, 4000, 16, 4, BF16), (2, 200, 4, 2, F32)])
def test_two_streams_at_once(B, T, H, Hk, dtype):
    xs = [inputs((B, T), H, Hk, 128, dtype, s) for s in (2, 3)]
    want = [layer(x) for x in xs]
    wss = [scratch(B, T, Hk, H, 128, dtype) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(layer(xs[i], wss[i], streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(same(want[i], g) for g in got[i])


def test_graphs_that_share_a_workspace():
    """Two captured layers on one workspace, replayed in turn with other inputs and offsets in
    the same buffers."""
    H, Hk, d, T = 4, 2, 128, 700
    xa, xb = inputs((T,), H, Hk, d, BF16, 4), inputs((2, 350), H, Hk, d, BF16, 5)
    cu = torch.tensor([0, 200, 201, 201, 640], dtype=torch.int32, device="cuda")
    n = max(scratch(4, T, Hk, H, d, BF16, True).numel(), scratch(2, 350, Hk, H, d, BF16).numel())
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    layer(xa, ws, cu=cu), layer(xb, ws)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a = layer(xa, ws, cu=cu)
    with torch.cuda.graph(gb):
        b = layer(xb, ws)
    for x, seed in ((xa, 6), (xb, 7)):
        for n, t in inputs(x["al"].shape[:-1], H, Hk, d, BF16, seed).items():
            x[n].copy_(t)
    cu.copy_(torch.tensor([0, 0, 333, 340, 699], dtype=torch.int32))
    for t in a:  # rows behind the last sequence are left as they were
        t.zero_()
    for g in (ga, gb, gb, ga, gb):
        g.replay()
    torch.cuda.synchronize()
    wa, wb = layer(xa, cu=cu), layer(xb)
    keep = [t[:699] if t.shape[0] == T else t for t in wa]
    assert same([t[:699] if t.shape[0] == T else t for t in a], keep) and same(b, wb)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_many_short_sequences(dtype, d):
    """300 sequences of 0 to 130 tokens, some sequences against the 64-bit reference; the state
    of each is its own."""
    gen = torch.Generator().manual_seed(8)
    n = torch.randint(0, 131, (300,), generator=gen)
    n[::7] = 0
    off = [0] + torch.cumsum(n, 0).tolist()
    H, Hk, T = 4, 2, off[-1]
    x = inputs((T,), H, Hk, d, dtype, 9)
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    o, vt, S = mdn.gdr_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["al"], x["be"], cu)
    g = mdn.gdr_chunk_bwd_varlen(x["q"], x["k"], x["al"], x["be"], cu, None, vt, x["do"])
    assert (S[n == 0] == 0).all()
    tol = {F32: 2e-5, BF16: 4.5e-3}
    for s in (1, 2, 5, 100, 298, 299):
        sl = slice(off[s], off[s + 1])
        c = {k: t[None, sl].cpu() for k, t in x.items()}
        ref = dict(zip(("o", "vt", "S"), R.fwd(c["q"], c["k"], c["v"], c["al"], c["be"], d ** -0.5)))
        got = dict(o=o[None, sl], vt=vt[None, sl], S=S[s:s + 1])
        ref |= R.bwd(c["q"], c["k"], c["al"], c["be"], d ** -0.5, got["vt"].cpu(), c["do"])
        got |= {k: t[s:s + 1] if k == "dS0" else t[None, sl] for k, t in g.items()}
        for k, r in ref.items():
            assert R.rel(got[k], r) <= tol[got[k].dtype], (s, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [(0,), (0, 0), (0, 3, 10), (0, 3, 11)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 3)])
def test_new_outputs_are_zero_behind_the_last_sequence(H, Hk, off, dtype):
    """Freshly allocated outputs, on memory that held something else; with no sequence at all
    every row is behind."""
    x = inputs((11,), H, Hk, 64, dtype, 15)
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    full = [torch.full((11, H, 64), 7.0, device="cuda", dtype=dtype) for _ in range(8)]
    full += [torch.full((11, H), 7.0, device="cuda") for _ in range(4)]
    del full
    o, vt, S = mdn.gdr_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["al"], x["be"], cu)
    g = mdn.gdr_chunk_bwd_varlen(x["q"], x["k"], x["al"], x["be"], cu, None, vt, x["do"])
    assert S.shape == g["dS0"].shape == (len(off) - 1, H, 64, 64)
    for t in (o, vt, *(g[n] for n in ("dq", "dk", "dv", "dalpha_log", "dbeta"))):
        assert (t[off[-1]:] == 0).all()
        assert torch.isfinite(t).all() and (off[-1] == 0 or t[1:off[-1]].ne(0).any())


@pytest.mark.parametrize("T", [1, 3, 4, 5, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("d,H,Hk", [(128, 6, 2), (64, 5, 5)])
def test_few_tokens(d, H, Hk, packed, T):
    """Lengths at which bf16 calls change between the CUDA cores and the tensor cores."""
    x = R.inputs(1, T, H, Hk, d, BF16, seed=T + 20)
    n = ("q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    q, k, v, al, be, S0, do, dST = (x[i].cuda() if x[i] is not None else None for i in n)
    if packed:
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        o, vt, S = mdn.gdr_chunk_fwd_varlen(q[0], k[0], v[0], al[0], be[0], cu, None, S0)
        g = mdn.gdr_chunk_bwd_varlen(q[0], k[0], al[0], be[0], cu, None, vt, do[0], S0, dST)
        got = dict(o=o[None], vt=vt[None], S=S) | {i: t if i == "dS0" else t[None] for i, t in g.items()}
    else:
        o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0)
        got = dict(o=o, vt=vt, S=S) | mdn.gdr_chunk_bwd(q, k, al, be, None, vt, do, S0, dST)
    ref = dict(zip(("o", "vt", "S"), R.fwd(*[x[i] for i in n[:5]], d ** -0.5, x["S0"])))
    ref |= R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], d ** -0.5, got["vt"].cpu(), x["do"], x["S0"],
                 x["dS_T"])
    tol = {F32: 2e-5, BF16: 4.5e-3}
    for i, r in ref.items():
        assert R.rel(got[i], r) <= tol[got[i].dtype], i


@pytest.mark.parametrize("flags", [0, E.MDN_FORCE_SIMT])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_minus_infinity_resets(dtype, d, flags):
    """alpha = 0: at the first token, at a chunk's first and last, and inside."""
    x = R.inputs(1, 200, 2, 1, d, dtype, seed=10)
    for t in (0, 63, 64, 90, 199):
        x["alpha_log"][:, t] = float("-inf")
    n = ("q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T")
    q, k, v, al, be, S0, do, dST = (x[i].cuda() for i in n)
    o, vt, S = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=flags)
    ref = dict(zip(("o", "vt", "S"), R.fwd(*[x[i] for i in n[:5]], d ** -0.5, x["S0"])))
    got = dict(o=o, vt=vt, S=S)
    got |= mdn.gdr_chunk_bwd(q, k, al, be, None, vt, do, S0, dST, flags=flags)
    ref |= R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], d ** -0.5, vt.cpu(), x["do"], x["S0"], x["dS_T"])
    tol = {F32: 2e-5, BF16: 4.5e-3}
    for i, r in ref.items():
        if float(r.norm()) == 0:
            assert (got[i] == 0).all(), i
        else:
            assert R.rel(got[i], r) <= tol[got[i].dtype], i


@pytest.mark.parametrize("dtype,d,flags", [(F32, 64, 0), (F32, 128, 0), (BF16, 64, 0), (BF16, 128, 0),
                                           (BF16, 128, E.MDN_FORCE_SIMT)])
@pytest.mark.parametrize("decay", [3.0, 8.0])
def test_strong_decay_keeps_the_gates_gradients(decay, dtype, d, flags):
    """alpha of e^-3 and e^-8: what a token's decay acts on is a small rest beside what the token
    writes itself."""
    x = R.inputs(1, 200, 2, 2, d, dtype, seed=5, decay=decay)
    q, k, v, al, be, S0, do, dST = (x[i].cuda() if x[i] is not None else None
                                    for i in ("q", "k", "v", "alpha_log", "beta", "S0", "do", "dS_T"))
    vt = mdn.gdr_chunk_fwd(q, k, v, al, be, None, S0, flags=flags)[1]
    g = mdn.gdr_chunk_bwd(q, k, al, be, None, vt, do, S0, dST, flags=flags)
    r = R.bwd(x["q"], x["k"], x["alpha_log"], x["beta"], d ** -0.5, vt.cpu(), x["do"], x["S0"], x["dS_T"])
    for i in ("dalpha_log", "dbeta", "dS0"):
        assert R.rel(g[i], r[i]) <= 2e-5, i


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_a_sequence_that_is_not_finite_stays_alone(dtype, d):
    """Packed neighbours, in the same 64-token tile of the buffer, are not reached."""
    off, H = [0, 30, 100, 170], 2
    x = inputs((170,), H, H, d, dtype, 11)
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    clean = layer(x, cu=cu)
    for n in ("q", "k", "v", "do"):
        x[n][40] = float("nan")
    x["al"][41], x["be"][42] = float("nan"), float("inf")
    got = layer(x, cu=cu)
    for i, (a, b) in enumerate(zip(got, clean)):
        if a.shape[0] == 170:
            assert torch.equal(a[:30], b[:30]) and torch.equal(a[100:], b[100:]), i
        elif a.shape[0] == 3:
            assert torch.equal(a[[0, 2]], b[[0, 2]]), i


def test_step_and_norm_captured_with_a_kept_state():
    """Decode with the state kept (S_out) and in place, in one graph."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = inputs((3,), 4, 2, 128, BF16, 13)
    S = 0.1 * torch.randn(3, 4, 128, 128, generator=g, device="cuda")
    S0, out = S.clone(), torch.empty_like(S)
    w = lambda: mdn.gdr_step(x["q"], x["k"], x["v"], x["al"], x["be"], None, S, S_out=out)
    w()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, vt = w()
        y, m, r = mdn.group_norm_fwd(o.view(3, 1, -1), 4)
    for n, t in inputs((3,), 4, 2, 128, BF16, 14).items():
        x[n].copy_(t)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, S0)
    o2, vt2 = mdn.gdr_step(x["q"], x["k"], x["v"], x["al"], x["be"], None, S0)
    assert same((o, vt, out), (o2, vt2, S0))
    assert same((y, m, r), mdn.group_norm_fwd(o2.view(3, 1, -1), 4))
