"""The block around the fast-weight read, as cases to be timed: the gated delta rule (forward, single step, backward)
and the root-mean-square norm with the residual's addition and an output in 8 bits (forward, backward).

Gated delta rule, per head with a state S [dk, dv]: S_t = a_t S_{t-1} + k_t (beta_t (v_t - a_t S_{t-1}^T k_t))^T with
a_t = e^{g_t}, out_t = scale S_t^T q_t. q and k may have fewer heads than v: each is then shared by a group of them.
Norm, per token: h = x + residual, y = weight h / sqrt(mean h^2 + eps), y in x's type or as e4m3 values with one scale a
token (the largest |y| of the token is 448 of them).

``run`` with ``own`` false computes each in elementary torch operations (the delta rule in chunks of 64 tokens, the
chunks' maps composed by doubling); with ``own`` true it calls the library. Layout "bhtd" is dense, "bthd" the
projection's: q, k and v are column blocks of one [B,T,...] product, beta and g [B,T,H]."""

import math

import torch

own = False

EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # one decoding step of 256 sequences, 12 heads of 64: the state is read and written once
        dict(name="gdr_step_b256_bf16", op="gdr_fwd", batch=256, heads=12, heads_qk=12, seqlen=1, dk=64, dv=64,
             dtype="bf16", layout="bthd", ragged=False),
        # the 130M model's training batch
        dict(name="gdr_fwd_b8t1024_bf16", op="gdr_fwd", batch=8, heads=12, heads_qk=12, seqlen=1024, dk=64, dv=64,
             dtype="bf16", layout="bhtd", ragged=False),
        # a padded batch of prompts, wide heads, two value heads to each key head
        dict(name="gdr_fwd_b4t4096d128_ragged", op="gdr_fwd", batch=4, heads=16, heads_qk=8, seqlen=4096, dk=128,
             dv=128, dtype="bf16", layout="bthd", ragged=True),
        # fp32, odd sizes
        dict(name="gdr_fwd_b3h5t2047_f32", op="gdr_fwd", batch=3, heads=5, heads_qk=5, seqlen=2047, dk=48, dv=80,
             dtype="f32", layout="bthd", ragged=False),
        # one very long document: few heads, the states' chain is the limit
        dict(name="gdr_fwd_b1t65536_bf16", op="gdr_fwd", batch=1, heads=12, heads_qk=12, seqlen=65536, dk=64, dv=64,
             dtype="bf16", layout="bhtd", ragged=False),
        # backward of the training batch
        dict(name="gdr_bwd_b8t1024_bf16", op="gdr_bwd", batch=8, heads=12, heads_qk=12, seqlen=1024, dk=64, dv=64,
             dtype="bf16", layout="bhtd", ragged=False),
        # backward in fp32, padded, shared keys
        dict(name="gdr_bwd_b2h6t4095_f32", op="gdr_bwd", batch=2, heads=6, heads_qk=3, seqlen=4095, dk=64, dv=64,
             dtype="f32", layout="bthd", ragged=True),
        # the norm before a block in a decoding step: latency
        dict(name="rms_fwd_b256t1_bf16", op="rms_fwd", batch=256, seqlen=1, d=768, dtype="bf16", residual=True,
             eight=False, ragged=False),
        # the training batch at length 2048
        dict(name="rms_fwd_b8t2048_bf16", op="rms_fwd", batch=8, seqlen=2048, d=768, dtype="bf16", residual=True,
             eight=False, ragged=False),
        # 16384 tokens of a wide model into an 8-bit product
        dict(name="rms_fwd_b4t4096d4096_e4m3", op="rms_fwd", batch=4, seqlen=4096, d=4096, dtype="bf16", residual=True,
             eight=True, ragged=False),
        # backward of the training batch
        dict(name="rms_bwd_b8t1024_bf16", op="rms_bwd", batch=8, seqlen=1024, d=768, dtype="bf16", residual=True,
             ragged=False),
        # backward, fp32, odd width, padded
        dict(name="rms_bwd_b3t5001d1000_f32", op="rms_bwd", batch=3, seqlen=5001, d=1000, dtype="f32", residual=True,
             ragged=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_bwd", "gdr_fwd", "gdr_bwd", "rms_fwd", "rms_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ragged = rng.random() < 0.4
    if op.startswith("rms"):
        d = _log_uniform(rng, 64, 8192) if rng.random() < 0.5 else rng.choice([512, 768, 1024, 1536, 2048, 4096])
        rows = _log_uniform(rng, 1, max(2, min(32768, (48 if op == "rms_fwd" else 24) * 2 ** 20 // d)))
        batch = rng.randint(1, min(rows, 16))
        c = dict(op=op, batch=batch, seqlen=max(1, rows // batch), d=d, dtype=dtype, residual=rng.random() < 0.7,
                 ragged=ragged)
        if op == "rms_fwd":
            c["eight"] = rng.random() < 0.4
        return c
    dk, dv = (rng.choice([16, 32, 64, 64, 64, 128, 40, 100, 33]) for _ in range(2))
    heads_qk, group = rng.randint(1, 12), rng.choice([1, 1, 1, 2, 3])
    heads = heads_qk * group
    # tokens x heads: at most half of what the largest listed case has, and less where heads are wide or in fp32
    most = (384 if op == "gdr_fwd" else 96) * 1024 // (2 if dtype == "f32" else 1) // (2 if max(dk, dv) > 64 else 1)
    seqlen = 1 if rng.random() < 0.1 else _log_uniform(rng, 2, min(32768 if op == "gdr_fwd" else 8192, most // heads))
    batch = _log_uniform(rng, 1, max(1, min(128, most // (heads * seqlen))))
    return dict(op=op, batch=batch, heads=heads, heads_qk=heads_qk, seqlen=seqlen, dk=dk, dv=dv, dtype=dtype,
                layout=rng.choice(["bhtd", "bthd"]), ragged=ragged)


def _lengths(case):
    """A padded batch's lengths: the first sequence full, the others spread down to an eighth, a batch of more than
    four with an empty one."""
    B, T = case["batch"], case["seqlen"]
    n = [T - (7 * T * b) // (8 * B) for b in range(B)]
    if B > 4:
        n[B // 2] = 0
    return n


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = case["batch"], case["seqlen"]
    live = sum(_lengths(case)) if case["ragged"] else B * T  # tokens read; outputs are written whole
    if case["op"].startswith("rms"):
        d, r = case["d"], case["residual"]
        if case["op"] == "rms_fwd":
            y = 1 if case["eight"] else e
            return {"bytes": live * d * e * (2 if r else 1) + B * T * (d * (y + (e if r else 0)) + (4 if case["eight"] else 0))
                    + 4 * d, "flops": 5 * live * d}
        return {"bytes": live * d * e * (3 if r else 2) + B * T * d * e + 8 * d, "flops": 10 * live * d}
    H, Hk, dk, dv = (case[k] for k in ("heads", "heads_qk", "dk", "dv"))
    inputs = live * (e * (2 * Hk * dk + H * dv) + 8 * H)
    state = 4 * B * H * dk * dv
    if case["op"] == "gdr_fwd":
        # the recurrence's own products: S^T k, the update, S^T q
        return {"bytes": inputs + B * T * H * dv * e + 2 * state, "flops": 7 * live * H * dk * dv}
    # forward states again, then five products a token and the state's adjoint
    return {"bytes": inputs + live * H * dv * e + B * T * (e * (2 * Hk * dk + H * dv) + 8 * H) + 3 * state,
            "flops": 21 * live * H * dk * dv}


# ---- inputs


def _view(buf):
    return buf.transpose(1, 2)  # [B,T,H,d] -> a [B,H,T,d] view


def _place(case, *tensors):
    """Tensors [B,Hi,T,di] in the case's type and layout: dense, or column blocks of one [B,T,...] buffer."""
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["layout"] == "bhtd":
        return [t.to(dt).contiguous() for t in tensors]
    B, T = case["batch"], case["seqlen"]
    buf = torch.empty(B, T, sum(t.shape[1] * t.shape[3] for t in tensors), dtype=dt, device="cuda")
    views, at = [], 0
    for t in tensors:
        n = t.shape[1] * t.shape[3]
        views.append(_view(buf[:, :, at:at + n].view(B, T, t.shape[1], t.shape[3])).copy_(t))
        at += n
    return views


def _place_gate(case, t):
    """[B,H,T] fp32, dense or a view of [B,T,H]."""
    return t.contiguous() if case["layout"] == "bhtd" else t.transpose(1, 2).contiguous().transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, T = case["batch"], case["seqlen"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"].startswith("rms"):
        d = case["d"]
        s["weight"] = 1 + 0.2 * normal(d)
        # a residual stream: tokens of unlike sizes, channels of unlike sizes
        stream = normal(B, T, d) * torch.exp(0.5 * normal(B, T, 1)) * torch.exp(0.5 * normal(d))
        if case["op"] == "rms_fwd":
            s["x"] = normal(B, T, d).to(dt)
            s["residual"] = stream.to(dt) if case["residual"] else None
            s["y_buf"] = torch.empty(B, T, d, dtype=torch.float8_e4m3fn if case["eight"] else dt, device="cuda")
            s["h_buf"] = torch.empty(B, T, d, dtype=dt, device="cuda") if case["residual"] else None
            s["scale_buf"] = torch.empty(B, T, device="cuda") if case["eight"] else None
        else:
            s["h"], s["dy"] = stream.to(dt), normal(B, T, d).to(dt)
            s["dh"] = normal(B, T, d).to(dt) if case["residual"] else None
            s["dx_buf"], s["dw_buf"] = torch.empty(B, T, d, dtype=dt, device="cuda"), torch.empty(d, device="cuda")
        return s
    H, Hk, dk, dv = (case[k] for k in ("heads", "heads_qk", "dk", "dv"))

    def unit(t):
        return t / t.norm(dim=-1, keepdim=True)

    s["q"], s["k"], s["v"] = _place(case, unit(normal(B, Hk, T, dk)), unit(normal(B, Hk, T, dk)), normal(B, H, T, dv))
    # log decays around -0.05 and gains between 0 and 1: memories of a few to a few hundred tokens
    s["beta"] = _place_gate(case, torch.sigmoid(normal(B, H, T)))
    s["g"] = _place_gate(case, -torch.exp(normal(B, H, T) - 3))
    s["S0"] = normal(B, H, dk, dv) / dk ** 0.5
    s["state_buf"] = torch.empty(B, H, dk, dv, device="cuda")
    if case["op"] == "gdr_fwd":
        s["out_buf"] = torch.empty(B, T, H, dv, dtype=dt, device="cuda").transpose(1, 2)
    else:
        s["dout"] = _view(normal(B, T, H, dv).to(dt))
        s["dS_final"] = normal(B, H, dk, dv) / dk ** 0.5
        s["dq_buf"], s["dk_buf"], s["dv_buf"] = _place(case, *(torch.zeros_like(s[n]) for n in ("q", "k", "v")))
        s["dbeta_buf"], s["dg_buf"] = (_place_gate(case, torch.zeros(B, H, T, device="cuda")) for _ in range(2))
    return s


# ---- plain forms, 32 bits


def _valid(s, B, T):
    """[B,T] truth values of the tokens inside their sequence."""
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"]
    return torch.arange(T, device="cuda") < n[:, None]


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular [.., C, C], C a power of two: the inverses of the diagonal blocks,
    doubled in size until there is one."""
    C = A.shape[-1]
    inv, n = torch.ones(*A.shape[:-2], C, 1, 1, device=A.device, dtype=A.dtype), 1
    while n < C:
        m = C // (2 * n)
        blocks = A.reshape(*A.shape[:-2], m, 2, n, m, 2, n)
        low = torch.diagonal(blocks[..., :, 1, :, :, 0, :], dim1=-4, dim2=-2).movedim(-1, -3)
        first, second = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        corner = -(second @ (low @ first))
        inv = torch.cat([torch.cat([first, torch.zeros_like(first)], -1), torch.cat([corner, second], -1)], -2)
        n *= 2
    return inv[..., 0, :, :]


def _states(M, N):
    """X_n = M_n X_{n-1} + N_n along dim 2 from X = 0, by doubling: each pass composes neighbouring spans' maps."""
    n, L = 1, M.shape[2]
    while n < L:
        N = torch.cat([N[:, :, :n], N[:, :, n:] + M[:, :, n:] @ N[:, :, :-n]], 2)
        if 2 * n < L:
            M = torch.cat([M[:, :, :n], M[:, :, n:] @ M[:, :, :-n]], 2)
        n *= 2
    return N


def _chunked(s):
    """The call's tensors in chunks [B,H,n,C,d], zero behind each sequence's end, and the chunks' maps."""
    c = s["case"]
    B, H, T, dk = c["batch"], c["heads"], c["seqlen"], c["dk"]
    C = min(CHUNK, 1 << (T - 1).bit_length())
    n = -(-T // C)
    ok = _valid(s, B, T)[:, None, :, None]

    def cut(t):
        t = torch.where(ok, t.float(), 0.0)
        if t.shape[1] != H:
            t = t.repeat_interleave(H // t.shape[1], 1)
        return torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).view(B, H, n, C, t.shape[-1])

    f = {"C": C, "n": n, "ok": ok, "scale": dk ** -0.5}
    f["q"], f["k"], f["v"] = cut(s["q"]), cut(s["k"]), cut(s["v"])
    f["beta"], g = cut(s["beta"][..., None]), cut(s["g"][..., None])
    G = g.double().cumsum(-2)  # differences of far sums: 64 bits
    lower = torch.ones(C, C, device="cuda").tril()
    f["D"] = torch.where(lower > 0, G - G.transpose(-1, -2), 0.0).float().exp() * lower
    f["eG"], f["w"], f["eC"] = G.float().exp(), (G[..., -1:, :] - G).float().exp(), G[..., -1:, :].float().exp()
    f["strict"] = lower - torch.eye(C, device="cuda")
    f["N"] = f["D"] * f["strict"] * (f["k"] @ f["k"].transpose(-1, -2))
    f["P"] = f["D"] * (f["q"] @ f["k"].transpose(-1, -2)) * f["scale"]
    f["inv"] = _inverse(f["N"] * f["beta"].transpose(-1, -2))
    # E = inv (v - e^G k S): what the state does not predict; U = beta E enters it
    f["kw"] = f["k"] * f["w"] * f["beta"]
    f["M"] = f["eC"] * torch.eye(dk, device="cuda") - f["kw"].transpose(-1, -2) @ (f["inv"] @ (f["eG"] * f["k"]))
    add = f["kw"].transpose(-1, -2) @ (f["inv"] @ f["v"])
    add[:, :, 0] += f["M"][:, :, 0] @ s["S0"]
    ends = _states(f["M"], add)
    f["S"] = torch.cat([s["S0"][:, :, None], ends[:, :, :-1]], 2)
    f["last"] = ends[:, :, -1].contiguous()
    f["E"] = f["inv"] @ (f["v"] - f["eG"] * (f["k"] @ f["S"]))
    f["U"] = f["beta"] * f["E"]
    return f


def _joined(f, t, T, like=None):
    """[B,H,n,C,d] -> [B,H,T,d], zero behind the sequences' ends; summed over the heads that share `like`'s."""
    t = t.reshape(*t.shape[:2], -1, t.shape[-1])[:, :, :T]
    if like is not None and like.shape[1] != t.shape[1]:
        t = t.view(t.shape[0], like.shape[1], -1, *t.shape[2:]).sum(2)
    return torch.where(f["ok"], t, 0.0)


def _gdr_fwd(s):
    f, T = _chunked(s), s["case"]["seqlen"]
    out = f["scale"] * f["eG"] * (f["q"] @ f["S"]) + f["P"] @ f["U"]
    return {"out": _joined(f, out, T).to(s["q"].dtype), "S_final": f["last"]}


def _gdr_bwd(s):
    f, T = _chunked(s), s["case"]["seqlen"]
    dt = s["q"].dtype
    tr = lambda t: t.transpose(-1, -2)  # noqa: E731
    dout = torch.where(f["ok"], s["dout"].float(), 0.0)
    dout = torch.nn.functional.pad(dout, (0, 0, 0, f["n"] * f["C"] - T)).view(f["v"].shape)
    read = f["scale"] * f["eG"] * f["q"]
    local = tr(f["inv"]) @ (f["beta"] * (tr(f["P"]) @ dout))
    add = tr(read) @ dout - tr(f["eG"] * f["k"]) @ local
    add[:, :, -1] += tr(f["M"][:, :, -1]) @ s["dS_final"]
    starts = _states(tr(f["M"]).flip(2), add.flip(2)).flip(2)  # adjoint of the state before each chunk
    dS = torch.cat([starts[:, :, 1:], s["dS_final"][:, :, None]], 2)  # and behind it
    dU = tr(f["P"]) @ dout + f["w"] * (f["k"] @ dS)
    dV = tr(f["inv"]) @ (f["beta"] * dU)
    dP = f["scale"] * f["D"] * (dout @ tr(f["U"]))
    dN = -f["D"] * f["strict"] * (dV @ tr(f["U"]))
    dq = f["scale"] * f["eG"] * (dout @ tr(f["S"])) + dP @ f["k"]
    dk = tr(dP) @ f["q"] + (dN + tr(dN)) @ f["k"] - f["eG"] * (dV @ tr(f["S"])) + f["w"] * (f["U"] @ tr(dS))
    dbeta = (f["E"] * (dU - tr(f["N"]) @ dV)).sum(-1, keepdim=True)
    # g scales what each later token reads and writes of the state: <dq, q> - <dv, v>, and the state behind the chunk
    after = torch.cat([f["S"][:, :, 1:], f["last"][:, :, None]], 2)
    own_part = (dq.double() * f["q"]).sum(-1) - (dV.double() * f["v"]).sum(-1)
    dg = own_part.flip(-1).cumsum(-1).flip(-1) + (dS.double() * after).sum((-1, -2))[..., None]
    return {"dq": _joined(f, dq, T, s["q"]).to(dt), "dk": _joined(f, dk, T, s["k"]).to(dt),
            "dv": _joined(f, dV, T).to(dt), "dbeta": _joined(f, dbeta, T)[..., 0],
            "dg": _joined(f, dg[..., None].float(), T)[..., 0], "dS0": starts[:, :, 0].contiguous()}


def _rms_fwd(s):
    c = s["case"]
    dt = s["x"].dtype
    ok = _valid(s, c["batch"], c["seqlen"])[..., None]
    h = s["x"].float() if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt).float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    y, h = torch.where(ok, y, 0.0), torch.where(ok, h, 0.0)
    out = {} if s["residual"] is None else {"h": h.to(dt)}
    if not c["eight"]:
        return {"y": y.to(dt), **out}
    scale = y.abs().amax(-1) / 448
    q = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0)
    return {"y": q.clamp(-448, 448).to(torch.float8_e4m3fn), "scales": scale, **out}


def _rms_bwd(s):
    c = s["case"]
    ok = _valid(s, c["batch"], c["seqlen"])[..., None]
    h, dy = torch.where(ok, s["h"].float(), 0.0), torch.where(ok, s["dy"].float(), 0.0)
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    p = dy * s["weight"]
    dx = rstd * (p - h * (rstd * rstd * (p * h).mean(-1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + torch.where(ok, s["dh"].float(), 0.0)
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * h * rstd).sum((0, 1))}


# ---- the passes


def run(state):
    s, c = state, state["case"]
    if own:
        from weight_linear_attention_gb300 import falcon as F

        if c["op"] == "gdr_fwd":
            out, S = F.gdr_forward(s["q"], s["k"], s["v"], s["beta"], s["g"], s["S0"], lengths=s["lengths"],
                                   out=s["out_buf"], S_final=s["state_buf"])
            return {"out": out, "S_final": S}
        if c["op"] == "gdr_bwd":
            return F.gdr_backward(s["q"], s["k"], s["v"], s["beta"], s["g"], s["dout"], s["S0"], s["dS_final"],
                                  lengths=s["lengths"], dq=s["dq_buf"], dk=s["dk_buf"], dv=s["dv_buf"],
                                  dbeta=s["dbeta_buf"], dg=s["dg_buf"], dS0=s["state_buf"])
        if c["op"] == "rms_fwd":
            y, h, scales = F.rmsnorm_forward(s["x"], s["weight"], s["residual"], eps=EPS, lengths=s["lengths"],
                                             y=s["y_buf"], h=s["h_buf"], scales=s["scale_buf"])
            return {k: v for k, v in (("y", y), ("h", h if c["residual"] else None), ("scales", scales))
                    if v is not None}
        return F.rmsnorm_backward(s["h"], s["dy"], s["weight"], s["dh"], eps=EPS, lengths=s["lengths"],
                                  dx=s["dx_buf"], dweight=s["dw_buf"])
    return {"gdr_fwd": _gdr_fwd, "gdr_bwd": _gdr_bwd, "rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd}[c["op"]](s)


# ---- 64 bits, token by token from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rms"):
        return _exact_rms(s, case)
    B, T, H, Hk, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "heads_qk", "dk", "dv"))
    forward = case["op"] == "gdr_fwd"
    if not forward and B * H * T * dk * dv * 8 > 40 << 30:  # every state is kept
        return None
    n = torch.tensor(_lengths(case) if case["ragged"] else [T] * B, device="cuda")
    share = torch.arange(H, device="cuda") // (H // Hk)
    by_token = lambda t: t.double().movedim(2, 0).contiguous()  # noqa: E731
    q, k = by_token(s["q"][:, share]), by_token(s["k"][:, share])
    v, beta, a = by_token(s["v"]), by_token(s["beta"])[..., None, None], by_token(s["g"]).exp()[..., None, None]
    live = (torch.arange(T, device="cuda")[:, None] < n)[..., None, None, None]
    scale = 1 / math.sqrt(dk)
    S = s["S0"].double()
    out = torch.zeros(T, B, H, dv, dtype=torch.double, device="cuda")
    states = []
    for t in range(T):
        if not forward:
            states.append(S)
        kept = a[t] * S
        err = v[t][..., None, :] - (k[t][..., :, None] * kept).sum(-2, keepdim=True)
        new = kept + k[t][..., :, None] * (beta[t] * err)
        S = torch.where(live[t], new, S)
        out[t] = torch.where(live[t, ..., 0], scale * (q[t][..., :, None] * new).sum(-2), 0.0)
    if forward:
        return {"out": out.movedim(0, 2).contiguous(), "S_final": S}
    do = by_token(s["dout"])
    dS = s["dS_final"].double()
    got = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v),
           "dbeta": torch.zeros(T, B, H, dtype=torch.double, device="cuda"),
           "dg": torch.zeros(T, B, H, dtype=torch.double, device="cuda")}
    for t in reversed(range(T)):
        kt, qt, dot = k[t][..., :, None], q[t][..., :, None], do[t][..., None, :]
        kept = a[t] * states[t]
        err = v[t][..., None, :] - (kt * kept).sum(-2, keepdim=True)
        new = kept + kt * (beta[t] * err)
        total = dS + scale * qt * dot                       # adjoint of the state behind the token
        pulled = (kt * total).sum(-2, keepdim=True)         # and of beta err
        derr = beta[t] * pulled
        ok = live[t]
        put = lambda name, x, m: got[name].__setitem__(t, torch.where(m, x, 0.0))  # noqa: E731
        put("dq", scale * (new * dot).sum(-1), ok[..., 0])
        put("dk", (total * (beta[t] * err)).sum(-1) - (kept * derr).sum(-1), ok[..., 0])
        put("dv", derr[..., 0, :], ok[..., 0])
        put("dbeta", (pulled * err).sum((-1, -2)), ok[..., 0, 0])
        dkept = total - kt * derr
        put("dg", (dkept * kept).sum((-1, -2)), ok[..., 0, 0])
        dS = torch.where(ok, a[t] * dkept, dS)
        states.pop()
    got = {name: t.movedim(0, 2).contiguous() for name, t in got.items()}
    for name in ("dq", "dk"):
        got[name] = got[name].view(B, Hk, H // Hk, T, dk).sum(2)
    got["dS0"] = dS
    return got


def _exact_rms(s, case):
    B, T, d = case["batch"], case["seqlen"], case["d"]
    live = (torch.arange(T, device="cuda") < torch.tensor(_lengths(case) if case["ragged"] else [T] * B,
                                                          device="cuda")[:, None])[..., None]
    w = s["weight"].double()
    if case["op"] == "rms_bwd":
        h, dy = s["h"].double() * live, s["dy"].double() * live
        r = (h.square().sum(-1, keepdim=True) / d + EPS) ** -0.5
        dx = r * w * dy - h * r ** 3 / d * (w * dy * h).sum(-1, keepdim=True)
        if s["dh"] is not None:
            dx = dx + s["dh"].double() * live
        return {"dx": dx, "dweight": (dy * h * r).sum(0).sum(0)}
    h = s["x"].double()
    got = {}
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()  # the sum as it is stored is what is normalised
        got["h"] = h * live
    y = h * (h.square().sum(-1, keepdim=True) / d + EPS) ** -0.5 * w * live
    if not case["eight"]:
        return {"y": y, **got}
    scales = y.abs().amax(-1) / 448
    codes = torch.where(scales[..., None] > 0, y / scales[..., None], 0.0)
    # e4m3: four significant bits, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(codes.abs().clamp(min=2.0 ** -6))) - 3)
    return {"y": torch.round(codes / step) * step, "scales": scales, **got}
