"""Cases that measure the per-head scan and the block norms.

Operators: the scan with one decay per head (forward over packed sequences,
backward, one decode token) and the norms around a mixer block (residual add +
scale + norm before it, gate + norm after it). `run` computes them with plain
torch operations, or, where `own` is set, through the package's entry points.
"""

import math
import random

import torch

own = False

Q = 128  # chunk of the plain form


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    scan = dict(op="scan", dtype="bf16", P=64, N=128, G=1, h0=False, bwd=False)
    return [
        # three short prompts (one of them empty), fp32: latency of a whole call
        dict(scan, name="scan_tiny_f32", dtype="f32", tok=17, S=3, empty=1, H=24, h0=True),
        # a dense training batch of one 1536-channel layer
        dict(scan, name="scan_layer_8x2048", tok=16384, S=8, ragged=False, H=24),
        # packed prefill of 43 sequences, 5120 channels
        dict(scan, name="scan_packed_65536x5120", tok=65536, S=43, H=80),
        # one 8192-token call of a long prompt, 8192 channels, state carried in and out
        dict(scan, name="scan_long_8192x8192", tok=8192, S=1, H=128, G=8, h0=True),
        # the training step's backward on the 1536-channel layer, ragged batch
        dict(scan, name="scan_bwd_layer", tok=16384, S=8, H=24, bwd=True),
        # backward of packed training sequences, 5120 channels
        dict(scan, name="scan_bwd_packed_32768x5120", tok=32768, S=21, H=80, bwd=True, h0=True),
        # one chat's next token
        dict(op="step", name="step_1x1536", dtype="bf16", rows=1, slots=1, H=24, P=64, N=128, G=1),
        # a serving batch of 256 sequences, slots in no order
        dict(op="step", name="step_256x8192", dtype="bf16", rows=256, slots=260, H=128, P=64, N=128, G=8),
        # norm and gate after the block: one decode batch, grouped
        dict(op="gated", name="gated_256x8192", dtype="bf16", tok=256, D=8192, group=1024, before=False, train=False),
        # the same in training, forward and backward
        dict(op="gated", name="gated_train_16384x5120", dtype="bf16", tok=16384, D=5120, group=5120, before=False, train=True),
        # residual add and norm before the block: one decode batch
        dict(op="residual", name="residual_256x4096", dtype="bf16", tok=256, D=4096, res="f32", scaled=False, train=False),
        # the same in training with a learned residual scale, forward and backward
        dict(op="residual", name="residual_train_16384x2560", dtype="bf16", tok=16384, D=2560, res="f32", scaled=True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "step", "gated", "residual"])
    dtype = "bf16" if rng.random() < 0.8 else "f32"
    if op in ("scan", "scan_bwd"):
        G = rng.choice([1, 1, 2, 4, 8])
        H = G * rng.choice([1, 2, 5, 7, 8, 10, 16])
        P = rng.choice([64, 64, 64, 32, 128, 40])
        N = rng.choice([128, 128, 64, 16, 96, 37])
        most = 16384 * 24 * 64 * 128 // (H * P * N)
        if dtype == "f32":
            most //= 8
        tok = _log(rng, 1, max(64, min(32768, most)))
        S = rng.choice([1, 1, 2, 5, _log(rng, 1, 64)])
        S = min(S, tok)
        return dict(op="scan", dtype=dtype, tok=tok, S=S, empty=rng.choice([0, 0, 1]), H=H, P=P, N=N, G=G,
                    h0=rng.random() < 0.5, bwd=op == "scan_bwd")
    if op == "step":
        G = rng.choice([1, 1, 2, 8])
        H = G * rng.choice([1, 5, 8, 16])
        rows = _log(rng, 1, 256)
        return dict(op="step", dtype=dtype, rows=rows, slots=rows + rng.choice([0, 3]), H=H, P=rng.choice([64, 64, 32, 128, 40]),
                    N=rng.choice([128, 128, 64, 16, 96, 37]), G=G)
    tok = _log(rng, 1, 16384)
    if op == "gated":
        group = rng.choice([64, 192, 640, 1024, 1536, 2560, 5120, 4097])
        D = group * rng.choice([1, 1, 2, 4]) if group <= 1024 else group
        return dict(op="gated", dtype=dtype, tok=tok, D=D, group=group, before=rng.random() < 0.5, train=rng.random() < 0.6)
    return dict(op="residual", dtype=dtype, tok=tok, D=rng.choice([768, 1536, 2560, 4096, 5120, 1031]), res=rng.choice(["f32", "same"]),
                scaled=rng.random() < 0.5, train=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
class State:
    pass


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Lengths of the packed sequences: fixed by the case, since `work` counts with them."""
    tok, S = case["tok"], case["S"]
    if not case.get("ragged", True):
        return [tok // S] * S
    r = random.Random(tok * 1000003 + S)
    empty = min(case.get("empty", 0), S - 1)
    live = S - empty
    cuts = sorted(r.sample(range(1, tok), live - 1)) if live > 1 else []
    lens = [b - a for a, b in zip([0] + cuts, cuts + [tok])]
    for _ in range(empty):
        lens.insert(r.randrange(len(lens) + 1), 0)
    return lens


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _head_params(g, H):
    """A in [-16, -1], time steps log-uniform in [1e-3, 1e-1], as such layers are initialised."""
    A = -(1.0 + 15.0 * torch.rand(H, generator=g, device="cuda"))
    dt0 = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    bias = dt0 + torch.log(-torch.expm1(-dt0))
    D = 1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")
    return A, bias, D


def prepare(case, seed):
    g, st = _gen(seed), State()
    st.case, dt = case, _dt(case)
    st.ws = None
    if case["op"] in ("scan", "step"):
        H, P, N, G = case["H"], case["P"], case["N"], case["G"]
        rows = case["tok"] if case["op"] == "scan" else case["rows"]
        # u, B and C are slices of one projection's rows, as the conv leaves them
        xbc = _normal(g, (rows, H * P + 2 * G * N), dt)
        st.u = xbc[:, : H * P].view(rows, H, P)
        st.B = xbc[:, H * P : H * P + G * N].view(rows, G, N)
        st.C = xbc[:, H * P + G * N :].view(rows, G, N)
        st.delta = _normal(g, (rows, H), dt, 0.5)
        st.A, st.bias, st.D = _head_params(g, H)
        st.y = torch.empty((rows, H, P), dtype=dt, device="cuda")
    if case["op"] == "scan":
        st.lens = _lengths(case)
        S = len(st.lens)
        cu = [0]
        for n in st.lens:
            cu.append(cu[-1] + n)
        st.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st.h0 = _normal(g, (S, H, P, N), torch.float32, 0.3) if case["h0"] else None
        st.hf = torch.empty((S, H, P, N), device="cuda")
        # chunks of the plain form: token index (or -1) of each place, and each chunk's sequence
        idx, seq = [], []
        for s, n in enumerate(st.lens):
            k = -(-n // Q)
            i = torch.arange(k * Q).view(k, Q)
            idx.append(torch.where(i < n, i + cu[s], -1))
            seq += [s] * k
        st.idx = torch.cat(idx).cuda()
        st.seq = torch.tensor(seq, device="cuda")
        if case["bwd"]:
            st.dy = _normal(g, (rows, H, P), dt)
            st.dhf = _normal(g, (S, H, P, N), torch.float32, 0.1)
            f32 = dict(device="cuda", dtype=torch.float32)
            st.grads = {"du": torch.empty((rows, H, P), dtype=dt, device="cuda"), "ddelta": torch.empty((rows, H), dtype=dt, device="cuda"),
                        "dB": torch.empty((rows, G, N), dtype=dt, device="cuda"), "dC": torch.empty((rows, G, N), dtype=dt, device="cuda"),
                        "dA": torch.empty(H, **f32), "dDskip": torch.empty(H, **f32), "ddt_bias": torch.empty(H, **f32)}
            if case["h0"]:
                st.grads["dh0"] = torch.empty((S, H, P, N), **f32)
    elif case["op"] == "step":
        st.state = _normal(g, (case["slots"], H, P, N), torch.float32, 0.3)
        st.slots = torch.randperm(case["slots"], generator=g, device="cuda")[: case["rows"]].to(torch.int32)
    else:
        tok, D = case["tok"], case["D"]
        st.x = _normal(g, (tok, D), dt)
        st.w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
        st.y = torch.empty((tok, D), dtype=dt, device="cuda")
        st.dy = _normal(g, (tok, D), dt)
        if case["op"] == "gated":
            st.z = _normal(g, (tok, D), dt)
            st.grads = {"dx": torch.empty_like(st.x), "dz": torch.empty_like(st.x), "dweight": torch.empty(D, device="cuda")}
        else:
            rdt = torch.float32 if case["res"] == "f32" else dt
            st.res = _normal(g, (tok, D), rdt)
            st.res_out = torch.empty_like(st.res)
            st.scale = (0.1 + 0.02 * torch.randn(D, generator=g, device="cuda")) if case["scaled"] else None
            st.dres = _normal(g, (tok, D), rdt)
            st.grads = {"dx": torch.empty_like(st.x), "dresidual": torch.empty_like(st.res), "dweight": torch.empty(D, device="cuda")}
            if case["scaled"]:
                st.grads["dx_scale"] = torch.empty(D, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _chunked(u, delta, A, B, C, D, bias, h0, idx, seq, S):
    """y (fp32, packed) and the final states; fp32, with the decays' sums in 64 bits."""
    nc = idx.shape[0]
    H, P, N, G = u.shape[1], u.shape[2], B.shape[2], B.shape[1]
    mask = idx >= 0
    at = idx.clamp(min=0)
    keep = mask[..., None]
    d = torch.where(keep, _softplus(delta[at].double() + bias.double()), 0.0)  # (nc, Q, H)
    c = torch.cumsum(d * A.double(), 1)
    uc = torch.where(keep[..., None], u[at], 0.0).permute(0, 2, 1, 3)  # (nc, H, Q, P)
    Bc = torch.where(keep[..., None], B[at], 0.0).permute(0, 2, 1, 3)  # (nc, G, Q, N)
    Cc = torch.where(keep[..., None], C[at], 0.0).permute(0, 2, 1, 3)
    ch, dh = c.transpose(1, 2), d.float().transpose(1, 2)  # (nc, H, Q)
    causal = torch.ones(Q, Q, dtype=torch.bool, device=u.device).tril()
    gap = (ch[..., :, None] - ch[..., None, :]).float()
    M = torch.exp(torch.where(causal, gap, float("-inf"))) * dh[..., None, :]
    M = (M.view(nc, G, H // G, Q, Q) * (Cc @ Bc.transpose(-1, -2))[:, :, None]).view(nc, H, Q, Q)
    y = M @ uc
    total = ch[..., -1]  # (nc, H)
    w = (torch.exp((total[..., None] - ch).float()) * dh)[..., None] * uc
    add = (w.transpose(-1, -2).reshape(nc, G, H // G * P, Q) @ Bc).view(nc, H, P, N)
    # states: every chunk start and sequence end as a sum over the chunks before it in its sequence
    before = torch.cumsum(total, 0) - total  # (nc, H), over all chunks
    chunk = torch.arange(nc, device=u.device)
    ends = torch.cumsum(torch.bincount(seq, minlength=S), 0)  # one past the last chunk of each sequence
    firsts = ends - torch.bincount(seq, minlength=S)
    upto = torch.cat([before, total.sum(0, keepdim=True)])  # (nc + 1, H)
    row_at, row_seq = torch.cat([chunk, ends]), torch.cat([seq, torch.arange(S, device=u.device)])
    from_chunk = (chunk[None, :] < row_at[:, None]) & (seq[None, :] == row_seq[:, None])
    e = upto[row_at][:, None, :] - (before + total)[None]
    W = torch.exp(torch.where(from_chunk[..., None], e, float("-inf")).float()).permute(2, 0, 1)  # (H, rows, nc)
    states = W @ add.permute(1, 0, 2, 3).reshape(H, nc, P * N)
    if h0 is not None:
        e0 = torch.exp((upto[row_at] - upto[firsts][row_seq]).float())  # (rows, H)
        states = states + e0.t()[..., None] * h0.permute(1, 0, 2, 3).reshape(H, S, P * N)[:, row_seq]
    states = states.view(H, nc + S, P, N).transpose(0, 1)
    S0 = states[:nc].reshape(nc, G, H // G * P, N)
    inter = (S0 @ Cc.transpose(-1, -2)).view(nc, H, P, Q).transpose(-1, -2)
    y = y + torch.exp(ch.float())[..., None] * inter + D[:, None, None] * uc
    y = y.permute(0, 2, 1, 3)[mask]
    return y, states[nc:]


def _scan(st):
    case, S = st.case, len(st.lens)
    if not case["bwd"]:
        y, hf = _chunked(st.u.float(), st.delta.float(), st.A, st.B.float(), st.C.float(), st.D, st.bias, st.h0, st.idx, st.seq, S)
        return {"y": y.to(st.u.dtype), "h_final": hf.contiguous()}
    leaves = {"du": st.u.float(), "ddelta": st.delta.float(), "dA": st.A, "dB": st.B.float(), "dC": st.C.float(), "dDskip": st.D,
              "ddt_bias": st.bias}
    if st.h0 is not None:
        leaves["dh0"] = st.h0
    leaves = {k: v.detach().requires_grad_() for k, v in leaves.items()}
    v = leaves
    y, hf = _chunked(v["du"], v["ddelta"], v["dA"], v["dB"], v["dC"], v["dDskip"], v["ddt_bias"], v.get("dh0"), st.idx, st.seq, S)
    got = torch.autograd.grad([y, hf], list(leaves.values()), [st.dy.float(), st.dhf])
    return {k: x.to(st.grads[k].dtype) for k, x in zip(leaves, got)}


def _step(st):
    rep = st.case["H"] // st.case["G"]
    at = st.slots.long()
    d = _softplus(st.delta.float() + st.bias)
    B = st.B.float().repeat_interleave(rep, 1)
    C = st.C.float().repeat_interleave(rep, 1)
    u = st.u.float()
    h = st.state[at] * torch.exp(d * st.A)[..., None, None] + (d[..., None] * u)[..., None] * B[:, :, None, :]
    st.state[at] = h
    y = (h * C[:, :, None, :]).sum(-1) + st.D[:, None] * u
    return {"y": y.to(st.u.dtype), "state": st.state}


EPS = 1e-5


def _gated(st):
    case = st.case
    n, gs = case["D"] // case["group"], case["group"]
    x, z, w = st.x.float(), st.z.float(), st.w
    sg = 1 / (1 + torch.exp(-z))
    gate = z * sg
    v = x if case["before"] else x * gate
    vg = v.view(-1, n, gs)
    rstd = torch.rsqrt((vg * vg).mean(-1, keepdim=True) + EPS)
    vh = (vg * rstd).view_as(x)
    y = vh * w * gate if case["before"] else vh * w
    out = {"y": y.to(st.x.dtype)}
    if not case["train"]:
        return out
    dy = st.dy.float()
    dn = dy * gate if case["before"] else dy
    out["dweight"] = (dn * vh).double().sum(0).float()
    dh = (dn * w).view(-1, n, gs)
    dv = (rstd * (dh - vh.view_as(dh) * (dh * vh.view_as(dh)).mean(-1, keepdim=True))).view_as(x)
    dgate = dy * vh * w if case["before"] else dv * x
    out["dx"] = (dv if case["before"] else dv * gate).to(st.x.dtype)
    out["dz"] = (dgate * sg * (1 + z * (1 - sg))).to(st.x.dtype)
    return out


ALPHA = 0.7


def _residual(st):
    case = st.case
    x = st.x.float()
    s = ALPHA * st.scale if case["scaled"] else ALPHA
    r = (st.res.float() + s * x).to(st.res.dtype)
    rf = r.float()
    rstd = torch.rsqrt((rf * rf).mean(-1, keepdim=True) + EPS)
    rh = rf * rstd
    out = {"y": (rh * st.w).to(st.x.dtype), "residual_out": r}
    if not case["train"]:
        return out
    dy = st.dy.float()
    dh = dy * st.w
    dr = rstd * (dh - rh * (dh * rh).mean(-1, keepdim=True)) + st.dres.float()
    out["dresidual"] = dr.to(st.res.dtype)
    out["dx"] = (s * dr).to(st.x.dtype)
    out["dweight"] = (dy * rh).double().sum(0).float()
    if case["scaled"]:
        out["dx_scale"] = ALPHA * (dr * x).double().sum(0).float()
    return out


# ---------------------------------------------------------------------------
# the package's entry points
# ---------------------------------------------------------------------------
def _workspace(st, nbytes):
    if st.ws is None:
        st.ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device="cuda")
    return st.ws


def _run_own(st):
    import selective_state_space_causal_b200 as ssm

    case = st.case
    if case["op"] == "scan":
        H, P, N, G, S = case["H"], case["P"], case["N"], case["G"], len(st.lens)
        sizes = (case["tok"], H, P, G, N, S, st.u.dtype)
        if not case["bwd"]:
            if st.ws is None:
                _workspace(st, ssm.ssm_head_scan_workspace_size(*sizes))
            ssm.ssm_head_scan_fwd(st.u, st.delta, st.A, st.B, st.C, st.y, Dskip=st.D, dt_bias=st.bias, h0=st.h0, h_final=st.hf,
                                  cu_seqlens=st.cu, workspace=st.ws)
            return {"y": st.y, "h_final": st.hf}
        if st.ws is None:
            _workspace(st, ssm.ssm_head_scan_bwd_workspace_size(*sizes))
        ssm.ssm_head_scan_bwd(st.u, st.delta, st.A, st.B, st.C, st.dy, st.grads, Dskip=st.D, dt_bias=st.bias, h0=st.h0,
                              dh_final=st.dhf, cu_seqlens=st.cu, workspace=st.ws)
        return dict(st.grads)
    if case["op"] == "step":
        ssm.ssm_head_state_update(st.state, st.u, st.delta, st.B, st.C, st.y, st.A, Dskip=st.D, dt_bias=st.bias,
                                  state_indices=st.slots)
        return {"y": st.y, "state": st.state}
    if st.ws is None and case["train"]:
        _workspace(st, ssm.ssm_norm_bwd_workspace_size(case["tok"], case["D"]))
    if case["op"] == "gated":
        ssm.ssm_gated_norm_fwd(st.x, st.y, weight=st.w, z=st.z, group_size=case["group"], eps=EPS, norm_before_gate=case["before"])
        if not case["train"]:
            return {"y": st.y}
        ssm.ssm_gated_norm_bwd(st.x, st.dy, st.grads, weight=st.w, z=st.z, group_size=case["group"], eps=EPS,
                               norm_before_gate=case["before"], workspace=st.ws)
        return {"y": st.y, **st.grads}
    ssm.ssm_residual_norm_fwd(st.x, st.y, residual=st.res, residual_out=st.res_out, weight=st.w, x_scale=st.scale, alpha=ALPHA, eps=EPS)
    if not case["train"]:
        return {"y": st.y, "residual_out": st.res_out}
    ssm.ssm_residual_norm_bwd(st.res_out, st.dy, st.grads, x=st.x, weight=st.w, x_scale=st.scale, alpha=ALPHA, eps=EPS,
                              dresidual_out=st.dres, workspace=st.ws)
    return {"y": st.y, "residual_out": st.res_out, **st.grads}


def run(state):
    if own:
        return _run_own(state)
    return {"scan": _scan, "step": _step, "gated": _gated, "residual": _residual}[state.case["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "scan":
        tok, S, H, P, N, G = case["tok"], case["S"], case["H"], case["P"], case["N"], case["G"]
        state = 4 * S * H * P * N
        row = H * P + 2 * G * N + H
        if not case["bwd"]:
            return {"bytes": es * tok * (row + H * P) + state * (2 if case["h0"] else 1), "flops": 4 * tok * H * P * N}
        return {"bytes": es * tok * (2 * row + H * P) + state * (3 if case["h0"] else 1), "flops": 12 * tok * H * P * N}
    if case["op"] == "step":
        rows, H, P, N, G = case["rows"], case["H"], case["P"], case["N"], case["G"]
        return {"bytes": rows * (8 * H * P * N + es * (2 * H * P + 2 * G * N + H)), "flops": 6 * rows * H * P * N}
    n = case["tok"] * case["D"]
    if case["op"] == "gated":
        return {"bytes": es * n * (3 + (5 if case["train"] else 0)), "flops": n * (10 + (25 if case["train"] else 0))}
    rs = 4 if case["res"] == "f32" else es
    fwd = 2 * es + 2 * rs
    bwd = 2 * es + 3 * rs + (es if case["scaled"] else 0)
    return {"bytes": n * (fwd + (bwd if case["train"] else 0)), "flops": n * (6 + (14 if case["train"] else 0))}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _token_rows(st, t):
    """Sequences (longest first) that have a token t, and that token's row."""
    n = sum(1 for s in st.order if st.lens[s] > t)
    return n, st.starts[:n] + t


def _exact_scan(st):
    """Token by token: h = exp(d A) h + d u B^T, y = h C + D u; the backward by
    the chain rule through that recurrence, its states recomputed from marks."""
    case = st.case
    H, P, N, G, S = case["H"], case["P"], case["N"], case["G"], len(st.lens)
    longest = max(st.lens)
    padded = longest * S * H * P * N
    if longest > 9000 or padded * (5 if case["bwd"] else 1) > 2.5e12:
        return None
    st.order = sorted(range(S), key=lambda s: -st.lens[s])
    order = torch.tensor(st.order, device="cuda")
    st.starts = st.cu[:-1].long()[order]
    f = torch.float64
    raw = st.delta.to(f) + st.bias.to(f)
    d = torch.logaddexp(raw, torch.zeros_like(raw))
    a = torch.exp(d * st.A.to(f))
    D = st.D.to(f)[:, None]
    start = st.h0.to(f)[order] if st.h0 is not None else torch.zeros((S, H, P, N), dtype=f, device="cuda")

    def heads(x, rows):
        return x[rows].to(f).repeat_interleave(H // G, 1)

    def advance(h, t):
        n, rows = _token_rows(st, t)
        h[:n].mul_(a[rows][..., None, None])
        h[:n].add_((d[rows][..., None] * st.u[rows].to(f))[..., None] * heads(st.B, rows)[:, :, None, :])
        return n, rows

    h = start.clone()
    if not case["bwd"]:
        y = torch.empty(st.u.shape, dtype=f, device="cuda")
        for t in range(longest):
            n, rows = advance(h, t)
            y[rows] = (h[:n] @ heads(st.C, rows)[..., None])[..., 0] + D * st.u[rows].to(f)
        back = torch.empty_like(h)
        back[order] = h
        return {"y": y, "h_final": back}
    span = max(1, int(math.isqrt(longest)))
    marks = []
    for t in range(longest):
        if t % span == 0:
            marks.append(h.clone())
        advance(h, t)
    dh = st.dhf.to(f)[order].clone()
    du, dB, dC = (torch.zeros(x.shape, dtype=f, device="cuda") for x in (st.u, st.B, st.C))
    dd = torch.zeros(st.delta.shape, dtype=f, device="cuda")
    dA = torch.zeros(H, dtype=f, device="cuda")
    dy_all = st.dy
    for k in reversed(range(len(marks))):
        first, last = k * span, min((k + 1) * span, longest)
        h, prior = marks[k].clone(), []
        for t in range(first, last):
            prior.append(h[: _token_rows(st, t)[0]].clone())
            advance(h, t)
        for t in reversed(range(first, last)):
            n, rows = _token_rows(st, t)
            hp, ar = prior.pop(), a[rows][..., None, None]
            Bt, Ct = heads(st.B, rows), heads(st.C, rows)
            ut, dy, dt = st.u[rows].to(f), dy_all[rows].to(f), d[rows]
            now = ar * hp + (dt[..., None] * ut)[..., None] * Bt[:, :, None, :]
            dC[rows] = (now.transpose(-1, -2) @ dy[..., None])[..., 0].view(n, G, H // G, N).sum(2)
            gh = dh[:n]
            gh += dy[..., None] * Ct[:, :, None, :]
            gB = (gh @ Bt[..., None])[..., 0]  # (n, H, P)
            du[rows] = dt[..., None] * gB + D * dy
            dB[rows] = (dt[..., None] * (gh.transpose(-1, -2) @ ut[..., None])[..., 0]).view(n, G, H // G, N).sum(2)
            dlog = (gh * ar * hp).sum((-1, -2))
            dd[rows] = (gB * ut).sum(-1) + dlog * st.A.to(f)
            dA += (dlog * dt).sum(0)
            gh *= ar
        marks[k] = None
    ddelta = dd * torch.sigmoid(raw)
    out = {"du": du, "ddelta": ddelta, "dA": dA, "dB": dB, "dC": dC, "dDskip": (st.dy.to(f) * st.u.to(f)).sum((0, 2)),
           "ddt_bias": ddelta.sum(0)}
    if st.h0 is not None:
        out["dh0"] = torch.empty_like(dh)
        out["dh0"][order] = dh
    return out


def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "scan":
        return _exact_scan(st)
    if case["op"] == "step":
        H, G = case["H"], case["G"]
        at = st.slots.long()
        raw = st.delta.to(f) + st.bias.to(f)
        d = torch.logaddexp(raw, torch.zeros_like(raw))
        new = st.state.to(f)
        y = torch.empty(st.u.shape, dtype=f, device="cuda")
        for b in range(0, at.numel(), 16):
            s = at[b : b + 16]
            B, C = (x[b : b + 16].to(f).repeat_interleave(H // G, 1) for x in (st.B, st.C))
            u, db = st.u[b : b + 16].to(f), d[b : b + 16]
            h = torch.exp(db * st.A.to(f))[..., None, None] * new[s] + torch.einsum("bh,bhp,bhn->bhpn", db, u, B)
            new[s] = h
            y[b : b + 16] = torch.einsum("bhpn,bhn->bhp", h, C) + st.D.to(f)[:, None] * u
        return {"y": y, "state": new}
    x, w = st.x.to(f).requires_grad_(), st.w.to(f).requires_grad_()
    tok, D = x.shape
    if case["op"] == "gated":
        z = st.z.to(f).requires_grad_()
        act = z * torch.sigmoid(z)

        def norm(v):
            v = v.reshape(tok, -1, case["group"])
            return (v / torch.sqrt(v.pow(2).mean(2, keepdim=True) + EPS)).reshape(tok, D)

        y = norm(x) * w * act if case["before"] else norm(x * act) * w
        out = {"y": y.detach()}
        if case["train"]:
            out["dx"], out["dz"], out["dweight"] = torch.autograd.grad(y, [x, z, w], st.dy.to(f))
        return out
    # the norm is of the residual stream as it is stored
    gamma = (st.scale if case["scaled"] else torch.ones(D, device="cuda")).to(f)
    s = ALPHA * gamma
    r = st.res.to(f) + s * x.detach()
    kept = r.to(st.res.dtype).to(f) if case["res"] == "same" and case["dtype"] == "bf16" else r
    leaf = kept.clone().requires_grad_()
    y = leaf / torch.sqrt(leaf.pow(2).mean(1, keepdim=True) + EPS) * w
    # a residual stream stored in bf16 rounds to a neighbour where 32 and 64 bits disagree: no value for it then
    exact_r = None if case["res"] == "same" and case["dtype"] == "bf16" else r
    out = {"y": y.detach(), "residual_out": exact_r}
    if case["train"]:
        dr, dw = torch.autograd.grad(y, [leaf, w], st.dy.to(f))
        dr = dr + st.dres.to(f)
        out |= {"dresidual": dr, "dx": s * dr, "dweight": dw}
        if case["scaled"]:
            out["dx_scale"] = ALPHA * (dr * x.detach()).sum(0)
    return out
