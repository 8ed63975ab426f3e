"""What is measured of the gated delta rule and of the output norm beside it.

Two kinds of operators, each as a user's program calls it:

- the gated delta rule over whole sequences (``chunk``, ``varlen`` and their
  gradients ``chunk_bwd``, ``varlen_bwd``) and for one decode token (``step``);
- group norm with an activation, channels last (``norm``, ``norm_bwd``), which
  takes the mixer's output head by head (rows = tokens, groups = heads, the
  activation on a gate) or a whole sequence of rows per group.

Per head, with S of d x d entries, alpha = exp(alpha_log):

    vt_t = v_t - alpha_t S_{t-1}^T k_t,  S_t = alpha_t S_{t-1} + beta_t k_t vt_t^T,
    o_t  = scale S_t^T q_t.

The gradients are those of <do, o> + <dS_T, S_T>, from the vt that the forward
pass saved (stored in the type of v): S is rebuilt from that vt.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_C = 64


# ----------------------------------------------------------------- the cases
def _seq(op, name, B, T, H, Hk, d, dtype, state, decay):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "Hk": Hk, "d": d, "dtype": dtype,
            "state": state, "decay": decay}


def _packed(op, name, lengths, H, Hk, d, dtype, state, decay):
    return {"name": name, "op": op, "lengths": " ".join(str(n) for n in lengths), "H": H,
            "Hk": Hk, "d": d, "dtype": dtype, "state": state, "decay": decay}


def _norm(op, name, N, L, C, G, dtype, act, gate, affine):
    return {"name": name, "op": op, "N": N, "L": L, "C": C, "G": G, "dtype": dtype, "act": act,
            "gate": gate, "affine": affine}


def listed():
    return [
        # one decode token of one sequence: nothing but latency
        _seq("step", "step_one", 1, 1, 16, 16, 128, "bf16", True, -3.0),
        # one decode token of a full batch: the states stream through once
        _seq("step", "step_batch", 256, 1, 16, 16, 128, "bf16", True, -3.0),
        # the smallest layer: a few chunks of one fp32 head
        _seq("chunk", "chunk_tiny", 1, 256, 1, 1, 64, "f32", False, -3.0),
        # prefill or training forward of a 400M layer's shape
        _seq("chunk", "chunk_400m", 4, 2048, 8, 8, 128, "bf16", False, -3.0),
        # the same of a 1.3B layer's shape, continuing from entering states
        _seq("chunk", "chunk_1p3b", 8, 4096, 16, 16, 128, "bf16", True, -3.0),
        # one long context with slow decay, four value heads to a key head
        _seq("chunk", "chunk_long_shared", 1, 16384, 16, 4, 128, "bf16", False, -6.0),
        # packed prompts of very different lengths
        _packed("varlen", "varlen_mix", (3000, 1500, 64, 2500, 1, 700, 300, 127, 24576), 16, 16,
                128, "bf16", True, -4.0),
        # training: the gradients at the 400M layer's shape
        _seq("chunk_bwd", "bwd_400m", 4, 2048, 8, 8, 128, "bf16", False, -3.0),
        # training on packed fp32 sequences with shared key heads, one of them empty
        _packed("varlen_bwd", "bwd_packed_shared", (517, 64, 1, 0, 1203, 259), 8, 2, 64, "f32",
                True, -3.0),
        # the output norm of 16 heads over a batch of tokens, gated
        _norm("norm", "norm_tokens", 32768, 1, 2048, 16, "bf16", "silu", True, True),
        # its gradients at the 400M layer's shape
        _norm("norm_bwd", "norm_bwd_tokens", 8192, 1, 1024, 8, "bf16", "silu", True, True),
        # groups over whole sequences of rows, the activation on the normed value
        _norm("norm_bwd", "norm_bwd_rows", 3, 1111, 640, 20, "f32", "silu", False, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "chunk", "chunk", "varlen", "chunk_bwd", "varlen_bwd", "norm",
                     "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        G = rng.choice([1, 2, 5, 8, 16, 32])
        C = G * rng.choice([8, 24, 40, 64, 80, 128, 256])
        rows = _log(rng, 1, min(32768, (1 << 24) // C))
        L = rng.choice([1, 1, _log(rng, 1, rows)])
        return _norm(op, "", max(1, rows // L), L, C, G, dtype, rng.choice(["silu", "none"]),
                     rng.random() < 0.5, rng.random() < 0.75)
    H = rng.choice([1, 2, 3, 4, 6, 8, 16])
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
    d = rng.choice([64, 128, 128])
    state, decay = rng.random() < 0.5, rng.choice([-1.0, -3.0, -6.0])
    if op == "step":
        return _seq(op, "", _log(rng, 1, 256), 1, H, Hk, d, dtype, True, decay)
    most = (1 << 16) if op.endswith("bwd") else (1 << 18)   # tokens x heads
    if op.startswith("chunk"):
        T = _log(rng, 1, min(8192, most // H))
        return _seq(op, "", rng.randint(1, max(1, min(8, most // (H * T)))), T, H, Hk, d, dtype,
                    state or T < 2, decay)   # one token from no state has no decay to learn
    lengths = [_log(rng, 1, 4096) if rng.random() < 0.9 else 0 for _ in range(rng.randint(1, 12))]
    while sum(lengths) * H > most or not any(lengths):
        lengths = [max(1, n // 2) for n in lengths]
    return _packed(op, "", lengths, H, Hk, d, dtype, state or max(lengths) < 2, decay)


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) + 1) % (1 << 40))
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    dt, op = _DT[case["dtype"]], case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        N, L, C, G = (case[k] for k in ("N", "L", "C", "G"))
        s["x"] = (rand(N, L, C) * 0.7 + 0.3 * rand(1, 1, C)).to(dt)
        s["gate"] = rand(N, L, C).to(dt) if case["gate"] else None
        s["weight"] = 1.0 + 0.2 * rand(C) if case["affine"] else None
        s["bias"] = 0.2 * rand(C) if case["affine"] else None
        if op == "norm_bwd":
            s["dy"] = rand(N, L, C).to(dt)
            _, s["mean"], s["rstd"] = _norm_plain(s["x"], G, s["weight"], s["bias"], s["gate"],
                                                  case["act"])
        return s
    H, Hk, d = case["H"], case["Hk"], case["d"]
    packed = "lengths" in case
    if packed:
        lens = [int(n) for n in case["lengths"].split()]
        lead, nseq = (sum(lens),), len(lens)
        off = torch.tensor([0] + lens).cumsum(0)
        s["cu"] = off.to(device="cuda", dtype=torch.int32)
        s["offsets"] = [int(n) for n in off]
    else:
        lead, nseq = ((case["B"],) if op == "step" else (case["B"], case["T"])), case["B"]
    s["q"] = rand(*lead, Hk, d).to(dt)
    s["k"] = torch.nn.functional.normalize(rand(*lead, Hk, d), dim=-1).to(dt)
    s["v"] = rand(*lead, H, d).to(dt)
    s["alpha_log"] = -torch.nn.functional.softplus(rand(*lead, H) + case["decay"])
    s["beta"] = torch.sigmoid(rand(*lead, H))
    s["scale"] = d ** -0.5
    s["S0"] = 0.1 * rand(nseq, H, d, d) if case["state"] else None
    if op == "step":
        s["S"] = torch.empty_like(s["S0"])
    if op.endswith("bwd"):
        s["vt"] = _gdr_plain(s)[1]
        s["do"] = rand(*lead, H, d).to(dt)
        s["dS_T"] = 0.1 * rand(nseq, H, d, d) if case["state"] else None
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import momentum_delta_rule_mdn_b200 as mdn
    op = s["case"]["op"]
    if op == "norm":
        return dict(zip(("y", "mean", "rstd"), mdn.group_norm_fwd(
            s["x"], s["case"]["G"], s["weight"], s["bias"], s["gate"], act=s["case"]["act"])))
    if op == "norm_bwd":
        return mdn.group_norm_bwd(s["x"], s["case"]["G"], s["mean"], s["rstd"], s["dy"],
                                  s["weight"], s["bias"], s["gate"], act=s["case"]["act"])
    a = (s["q"], s["k"], s["v"], s["alpha_log"], s["beta"])
    if op == "step":
        # the state before the token is kept, as a program does that may have to drop the token
        o, vt = mdn.gdr_step(*a, s["scale"], s["S0"], S_out=s["S"])
        return {"o": o, "vt": vt, "S": s["S"]}
    if op == "chunk":
        return dict(zip(("o", "vt", "S"), mdn.gdr_chunk_fwd(*a, s["scale"], s["S0"])))
    if op == "varlen":
        return dict(zip(("o", "vt", "S"),
                        mdn.gdr_chunk_fwd_varlen(*a, s["cu"], s["scale"], s["S0"])))
    a, b = a[:2] + a[3:], (s["scale"], s["vt"].contiguous(), s["do"], s["S0"], s["dS_T"])
    if op == "chunk_bwd":
        return mdn.gdr_chunk_bwd(*a, *b)
    return mdn.gdr_chunk_bwd_varlen(*a, s["cu"], *b)


def _run_plain(s):
    op, c = s["case"]["op"], s["case"]
    if op == "norm":
        return dict(zip(("y", "mean", "rstd"), _norm_plain(s["x"], c["G"], s["weight"], s["bias"],
                                                           s["gate"], c["act"])))
    if op == "norm_bwd":
        return _norm_bwd_plain(s, c)
    if op == "step":
        return _step_plain(s)
    if op in ("chunk", "varlen"):
        return dict(zip(("o", "vt", "S"), _gdr_plain(s)))
    return _gdr_bwd_plain(s)


# ----------------------------------------------------------------- plain forms, 32 bits
def _shared(x, H):
    """The key heads repeated for the value heads that share them."""
    return x.float().repeat_interleave(H // x.shape[-2], dim=-2)


def _step_plain(s):
    H = s["case"]["H"]
    q, k, v = _shared(s["q"], H), _shared(s["k"], H), s["v"].float()
    al = s["alpha_log"].exp()[..., None, None]
    S = s["S0"] * al
    vt = v - (S * k[..., None]).sum(-2)
    S = S + s["beta"][..., None, None] * k[..., None] * vt[..., None, :]
    o = s["scale"] * (S * q[..., None]).sum(-2)
    return {"o": o.to(s["v"].dtype), "vt": vt.to(s["v"].dtype), "S": S}


def _chunks(s, names, b0, b1):
    """The named inputs of batch row or packed sequence b0:b1 as [rows, H, chunks, 64, ...],
    zeros behind the last token (a token with k = 0 and alpha_log = 0 changes nothing)."""
    H, out = s["case"]["H"], []
    for n in names:
        x = s[n]
        x = _shared(x, H) if n in ("q", "k") else x.float()
        x = x[None, b0:b1] if "offsets" in s else x
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, -x.shape[1] % _C))
        x = x.reshape(x.shape[0], -1, _C, *x.shape[2:])
        out.append(x.permute(0, 3, 1, 2, *range(4, x.dim())))
    return out


def _tokens(x, T):
    """[rows, H, chunks, 64, ...] -> [rows, T, H, ...]"""
    x = x.permute(0, 2, 3, 1, *range(4, x.dim()))
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :T]


def _rows(s):
    """(row range of the tokens, row range of the states) of each independent piece."""
    if "offsets" in s:
        f = s["offsets"]
        return [(f[i], f[i + 1], i, i + 1) for i in range(len(f) - 1)]
    return [(0, s["q"].shape[1], 0, s["q"].shape[0])]


def _local(k, alpha_log, beta):
    """la, the decay L, L (k_r . k_i) below the diagonal and T = (I + that Diag(beta))^-1."""
    la = alpha_log.cumsum(-1)
    lower = torch.ones(_C, _C, device=k.device, dtype=torch.bool).tril()
    L = (la[..., :, None] - la[..., None, :]).masked_fill(~lower, -math.inf).exp()
    A = (k @ k.transpose(-1, -2) * L).tril(-1)
    T = torch.eye(_C, device=k.device).expand(A.shape).clone()
    Ab = A * beta[..., None, :]
    for r in range(1, _C):                       # forward substitution
        T[..., r, :r] = -(Ab[..., r, None, :r] @ T[..., :r, :r])[..., 0, :]
    return la, L, A, T


def _gdr_plain(s):
    H, d, dt = s["case"]["H"], s["case"]["d"], s["v"].dtype
    os_, vts, Ss = [], [], []
    for t0, t1, r0, r1 in _rows(s):
        S = s["S0"][r0:r1] if s["S0"] is not None else torch.zeros(r1 - r0, H, d, d, device="cuda")
        if t1 > t0:
            q, k, v, al, be = _chunks(s, ("q", "k", "v", "alpha_log", "beta"), t0, t1)
            la, L, A, T = _local(k, al, be)
            D = la.exp()[..., None]
            P = q @ k.transpose(-1, -2) * L * be[..., None, :]
            wr = (k * (be * (la[..., -1:] - la).exp())[..., None]).transpose(-1, -2)
            vt, o = torch.empty_like(v), torch.empty_like(v)
            for n in range(v.shape[2]):
                x = T[:, :, n] @ (v[:, :, n] - D[:, :, n] * (k[:, :, n] @ S))
                o[:, :, n] = D[:, :, n] * (q[:, :, n] @ S) + P[:, :, n] @ x
                S = D[:, :, n, -1:] * S + wr[:, :, n] @ x
                vt[:, :, n] = x
            os_.append(_tokens(s["scale"] * o, t1 - t0).to(dt))
            vts.append(_tokens(vt, t1 - t0).to(dt))
        Ss.append(S)
    if "offsets" in s:
        return torch.cat(os_, 1)[0], torch.cat(vts, 1)[0], torch.cat(Ss)
    return os_[0], vts[0], Ss[0]


def _gdr_bwd_plain(s):
    c, sc, dt = s["case"], s["scale"], s["v"].dtype
    H, Hk, d = c["H"], c["Hk"], c["d"]
    parts, dS0 = {n: [] for n in ("dq", "dk", "dv", "dalpha_log", "dbeta")}, []
    for t0, t1, r0, r1 in _rows(s):
        zero = torch.zeros(r1 - r0, H, d, d, device="cuda")
        S = s["S0"][r0:r1] if s["S0"] is not None else zero
        G = s["dS_T"][r0:r1] if s["dS_T"] is not None else zero
        if t1 > t0:
            q, k, al, be, vt, do = _chunks(s, ("q", "k", "alpha_log", "beta", "vt", "do"), t0, t1)
            la, L, A, T = _local(k, al, be)
            D, w = la.exp()[..., None], (la[..., -1:] - la).exp()[..., None]
            b, NT = be[..., None], k.shape[2]
            Sn, Gn = [], [None] * NT                      # entering S, adjoint of the leaving S
            for n in range(NT):
                Sn.append(S)
                S = D[:, :, n, -1:] * S + (k * w * b)[:, :, n].transpose(-1, -2) @ vt[:, :, n]
            end = Sn[1:] + [S]
            P = sc * (q @ k.transpose(-1, -2)) * L
            Pdo = P.transpose(-1, -2) @ do
            Ab = A * be[..., None, :]
            dv = torch.empty_like(vt)
            for n in reversed(range(NT)):
                Gn[n] = G
                direct = b[:, :, n] * (Pdo[:, :, n] + w[:, :, n] * (k[:, :, n] @ G))
                dv[:, :, n] = T[:, :, n].transpose(-1, -2) @ direct
                G = D[:, :, n, -1:] * G + (sc * q * D)[:, :, n].transpose(-1, -2) @ do[:, :, n] \
                    - (k * D)[:, :, n].transpose(-1, -2) @ dv[:, :, n]
            Sn, Gn, end = torch.stack(Sn, 2), torch.stack(Gn, 2), torch.stack(end, 2)
            M1 = sc * (do @ vt.transpose(-1, -2)) * L
            M2 = (dv @ vt.transpose(-1, -2)) * L.tril(-1)
            dqq = sc * D * (do @ Sn.transpose(-1, -2)) + (M1 * be[..., None, :]) @ k
            kS = D * (dv @ Sn.transpose(-1, -2))          # = D S dv, row by row
            Gv = w * (vt @ Gn.transpose(-1, -2))
            dkk = b * (M1.transpose(-1, -2) @ q + Gv - M2.transpose(-1, -2) @ k) - kS \
                - (M2 * be[..., None, :]) @ k
            kk = k @ k.transpose(-1, -2)
            dbe = (M1 * (q @ k.transpose(-1, -2))).sum(-2) + (k * Gv).sum(-1) - (M2 * kk).sum(-2)
            x = (k * kS).sum(-1) + (M2 * kk * be[..., None, :]).sum(-1)
            cc = (q * dqq).sum(-1) - be * dbe - x
            dal = cc.flip(-1).cumsum(-1).flip(-1) + (Gn * end).sum((-1, -2))[..., None]
            fold = lambda y: _tokens(y, t1 - t0).unflatten(2, (Hk, H // Hk)).sum(3)
            for n, y in (("dq", fold(dqq).to(dt)), ("dk", fold(dkk).to(dt)),
                         ("dv", _tokens(dv, t1 - t0).to(dt)),
                         ("dalpha_log", _tokens(dal, t1 - t0)), ("dbeta", _tokens(dbe, t1 - t0))):
                parts[n].append(y)
        dS0.append(G)
    out = {n: torch.cat(x, 1)[0] if "offsets" in s else x[0] for n, x in parts.items()}
    return {**out, "dS0": torch.cat(dS0)}


def _act(x, act):
    return x * torch.sigmoid(x) if act == "silu" else x


def _act_d(x, act):
    if act != "silu":
        return torch.ones_like(x)
    y = torch.sigmoid(x)
    return y * (1 + x * (1 - y))


def _norm_plain(x, G, weight, bias, gate, act, eps=1e-5):
    N, L, C = x.shape
    h = x.float().reshape(N, L, G, C // G)
    mean = h.mean((1, 3))
    rstd = ((h - mean[:, None, :, None]).square().mean((1, 3)) + eps).rsqrt()
    n = ((h - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, L, C)
    n = n * weight + bias if weight is not None else n
    y = _act(n, act) if gate is None else n * _act(gate.float(), act)
    return y.to(x.dtype), mean, rstd


def _norm_bwd_plain(s, c):
    N, L, C, G = c["N"], c["L"], c["C"], c["G"]
    wide = lambda z: z[:, None, :, None].expand(N, L, G, C // G).reshape(N, L, C)
    xh = (s["x"].float() - wide(s["mean"])) * wide(s["rstd"])
    n = xh * s["weight"] + s["bias"] if c["affine"] else xh
    dy, out = s["dy"].float(), {}
    if c["gate"]:
        z = s["gate"].float()
        dn = dy * _act(z, c["act"])
        out["dgate"] = (dy * n * _act_d(z, c["act"])).to(s["x"].dtype)
    else:
        dn = dy * _act_d(n, c["act"])
    dh = dn * s["weight"] if c["affine"] else dn
    avg = lambda z: wide(z.reshape(N, L, G, C // G).mean((1, 3)))
    out["dx"] = (wide(s["rstd"]) * (dh - avg(dh) - xh * avg(dh * xh))).to(s["x"].dtype)
    if c["affine"]:
        out["dweight"], out["dbias"] = (dn * xh).sum((0, 1)), dn.sum((0, 1))
    return out


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        n, st = case["N"] * case["L"] * case["C"], 8 * case["N"] * case["G"]
        wb = (8 * case["C"]) if case["affine"] else 0
        if op == "norm":
            return {"bytes": n * e * (3 if case["gate"] else 2) + st + wb, "flops": 10 * n}
        return {"bytes": n * e * (5 if case["gate"] else 3) + st + 2 * wb, "flops": 24 * n}
    H, Hk, d = case["H"], case["Hk"], case["d"]
    if "lengths" in case:
        lens = [int(n) for n in case["lengths"].split()]
        tok, nseq = sum(lens), len(lens)
    else:
        tok, nseq = case["B"] * (1 if op == "step" else case["T"]), case["B"]
    st = 4 * nseq * H * d * d
    if op.endswith("bwd"):
        # q, k, dq, dk; v's cotangent, vt, do; gates and their gradients; S0, dS_T, dS0
        return {"bytes": tok * (4 * Hk * d * e + 3 * H * d * e + 16 * H) + st * (3 if case["state"] else 1),
                "flops": 14 * d * d * tok * H}
    return {"bytes": tok * (2 * Hk * d * e + 3 * H * d * e + 8 * H) + st * (2 if case["state"] else 1),
            "flops": 6 * d * d * tok * H}


# ----------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    s = {n: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x
         for n, x in s.items()}
    if op in ("norm", "norm_bwd"):
        return _exact_norm(s, case)
    if "offsets" not in s:
        lead = 1 if op == "step" else None
        s = {n: (x[:, None] if lead and n in ("q", "k", "v", "alpha_log", "beta") else x)
             for n, x in s.items()}
        out = _exact_gdr(s, case)
        return {n: x[:, 0] if lead and n in ("o", "vt") else x for n, x in out.items()}
    f, got = s["offsets"], []
    for i in range(len(f) - 1):
        p = {}
        for n, x in s.items():
            if n in ("q", "k", "v", "alpha_log", "beta", "vt", "do"):
                p[n] = x[None, f[i]:f[i + 1]]
            elif n in ("S0", "dS_T"):
                p[n] = x[i:i + 1] if x is not None else None
            else:
                p[n] = x
        got.append(_exact_gdr(p, case))
    return {n: torch.cat([g[n] for g in got]) if n in ("S", "dS0")
            else torch.cat([g[n] for g in got], 1)[0] for n in got[0]}


def _exact_gdr(s, case):
    """Token by token, as the recurrence and its adjoint are written."""
    q, k, v = s["q"], s["k"], s["v"]
    (B, T, H, d), Hk, sc = v.shape, q.shape[2], s["scale"]
    rep = H // Hk
    alpha, beta = s["alpha_log"].exp(), s["beta"]
    head = lambda x, t: x[:, t].repeat_interleave(rep, 1)
    S = s["S0"] if s["S0"] is not None else v.new_zeros(B, H, d, d)
    if "vt" not in s:
        o, vt = torch.empty_like(v), torch.empty_like(v)
        for t in range(T):
            kt = head(k, t)
            S = alpha[:, t, :, None, None] * S
            vt[:, t] = v[:, t] - torch.einsum("bhij,bhi->bhj", S, kt)
            S = S + torch.einsum("bhi,bhj->bhij", beta[:, t, :, None] * kt, vt[:, t])
            o[:, t] = sc * torch.einsum("bhij,bhi->bhj", S, head(q, t))
        return {"o": o, "vt": vt, "S": S}
    vt, do = s["vt"], s["do"]
    seg = max(1, int(math.isqrt(max(T, 1))))
    kept = {}                                      # S entering every seg-th token

    def forward(S, t):
        return alpha[:, t, :, None, None] * S + torch.einsum(
            "bhi,bhj->bhij", beta[:, t, :, None] * head(k, t), vt[:, t])
    for t in range(T):
        if t % seg == 0:
            kept[t] = S
        S = forward(S, t)
    G = s["dS_T"] if s["dS_T"] is not None else v.new_zeros(B, H, d, d)
    dq, dk, dv = v.new_empty(B, T, H, d), v.new_empty(B, T, H, d), torch.empty_like(v)
    da, db = torch.empty_like(beta), torch.empty_like(beta)
    for t0 in sorted(kept, reverse=True):
        run_ = [kept[t0]]
        for t in range(t0, min(t0 + seg, T)):
            run_.append(forward(run_[-1], t))
        for t in reversed(range(t0, min(t0 + seg, T))):
            before, after = run_[t - t0], run_[t - t0 + 1]
            kt, qt, a, b = head(k, t), head(q, t), alpha[:, t], beta[:, t]
            dq[:, t] = sc * torch.einsum("bhij,bhj->bhi", after, do[:, t])
            G = G + sc * torch.einsum("bhi,bhj->bhij", qt, do[:, t])     # adjoint of S_t
            db[:, t] = torch.einsum("bhij,bhi,bhj->bh", G, kt, vt[:, t])
            dv[:, t] = b[..., None] * torch.einsum("bhij,bhi->bhj", G, kt)
            Sdv = torch.einsum("bhij,bhj->bhi", before, dv[:, t])
            dk[:, t] = b[..., None] * torch.einsum("bhij,bhj->bhi", G, vt[:, t]) \
                - a[..., None] * Sdv
            G1 = G - torch.einsum("bhi,bhj->bhij", kt, dv[:, t])
            da[:, t] = a * (G1 * before).sum((-1, -2))
            G = a[..., None, None] * G1
    fold = lambda x: x.unflatten(2, (Hk, rep)).sum(3)
    return {"dq": fold(dq), "dk": fold(dk), "dv": dv, "dalpha_log": da, "dbeta": db, "dS0": G}


def _exact_norm(s, case):
    N, L, C, G = (case[n] for n in ("N", "L", "C", "G"))
    split = lambda z: z.reshape(N, L, G, C // G).transpose(1, 2).reshape(N, G, -1)
    join = lambda z: z.reshape(N, G, L, C // G).transpose(1, 2).reshape(N, L, C)
    x = split(s["x"])
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=2, unbiased=False)
        rstd = 1 / torch.sqrt(var + 1e-5)
    else:
        mean, rstd = s["mean"], s["rstd"]
    hat = (x - mean[..., None]) * rstd[..., None]
    n = join(hat)
    if case["affine"]:
        n = n * s["weight"] + s["bias"]
    sig = lambda z: 1 / (1 + torch.exp(-z))
    f = (lambda z: z * sig(z)) if case["act"] == "silu" else (lambda z: z)
    df = (lambda z: sig(z) + z * sig(z) * (1 - sig(z))) if case["act"] == "silu" else torch.ones_like
    if case["op"] == "norm":
        return {"y": f(n) if s["gate"] is None else n * f(s["gate"]), "mean": mean, "rstd": rstd}
    out = {}
    if case["gate"]:
        dn = s["dy"] * f(s["gate"])
        out["dgate"] = s["dy"] * n * df(s["gate"])
    else:
        dn = s["dy"] * df(n)
    dh = split(dn * s["weight"] if case["affine"] else dn)
    m = dh.shape[2]
    out["dx"] = join(rstd[..., None] * (dh - dh.sum(2, keepdim=True) / m
                                        - hat * (dh * hat).sum(2, keepdim=True) / m))
    if case["affine"]:
        out["dweight"] = (dn * join(hat)).sum((0, 1))
        out["dbias"] = dn.sum((0, 1))
    return out
