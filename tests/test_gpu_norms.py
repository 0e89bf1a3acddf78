"""The norms around a block on the GPU, forward and backward, against 64 bits.

Bounds as in head_oracle.py; nothing is rounded before the store, so bf16 results are
held to 1e-4 of the rms plus half a bf16 step."""

import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def ws_of(tok, D):
    return torch.empty(ssm.ssm_norm_bwd_workspace_size(tok, D), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("mode", ["plain", "gate_then_norm", "norm_then_gate"])
@pytest.mark.parametrize("tok,D,group,pad", [
    (1, 64, 64, 0), (3, 1536, 1536, 0), (33, 8, 8, 8), (9, 4096, 1024, 64), (5, 8192, 8192, 0),
    (4, 16384, 16384, 0), (2, 20000, 20000, 0), (7, 37, 37, 0), (6, 96, 3, 0), (1300, 64, 32, 0),
    (10, 1032, 1032, 3), (2500, 520, 520, 0), (0, 64, 64, 0), (6, 5120, 2560, 0),
])
def test_gated(tok, D, group, pad, mode, dt):
    g = torch.Generator().manual_seed(tok + D)
    wide = torch.randn(tok, 2 * D + pad, generator=g).to(dt)
    w = 1.0 + 0.3 * torch.randn(D, generator=g)
    dy = torch.randn(tok, D, generator=g).to(dt)
    gw = wide.cuda()
    x, z = gw[:, :D], gw[:, D:2 * D]
    before = mode == "norm_then_gate"
    if mode == "plain":
        z = None
    y = torch.empty((tok, D), dtype=dt, device="cuda")
    kw = dict(weight=w.cuda(), z=z, group_size=group, eps=EPS, norm_before_gate=before)
    ssm.ssm_gated_norm_fwd(x, y, **kw)
    gr = {"dx": torch.empty_like(y), "dz": torch.empty_like(y) if z is not None else None,
          "dweight": torch.full((D,), 5.0, device="cuda")}
    ssm.ssm_gated_norm_bwd(x, dy.cuda(), gr, workspace=ws_of(tok, D), **kw)
    rx = wide[:, :D].double().requires_grad_()
    rz = wide[:, D:2 * D].double().requires_grad_() if z is not None else None
    rw = w.double().requires_grad_()
    ry = ho.gated(rx, rz, rw, group, EPS, before)
    leaves = [rx, rw] + ([rz] if rz is not None else [])
    rg = torch.autograd.grad(ry, leaves, dy.double())
    ho.close(y, ry, dt == BF, 1e-4, "y")
    ho.close(gr["dx"], rg[0], dt == BF, 1e-4, "dx")
    ho.close(gr["dweight"], rg[1], False, 1e-4, "dweight")
    if rz is not None:
        ho.close(gr["dz"], rg[2], dt == BF, 1e-4, "dz")
    # the same bits again, and without the optional parts
    y2, g2 = torch.empty_like(y), {"dx": torch.empty_like(y), "dweight": torch.empty_like(gr["dweight"])}
    ssm.ssm_gated_norm_fwd(x, y2, **kw)
    ssm.ssm_gated_norm_bwd(x, dy.cuda(), g2, workspace=ws_of(tok, D), **kw)
    assert torch.equal(y, y2) and torch.equal(g2["dx"], gr["dx"]) and torch.equal(g2["dweight"], gr["dweight"])
    ssm.ssm_gated_norm_bwd(x, dy.cuda(), {"dx": g2["dx"]}, **kw)
    assert torch.equal(g2["dx"], gr["dx"])


@pytest.mark.parametrize("dt,rdt", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16_f32", "bf16"])
@pytest.mark.parametrize("tok,D", [(1, 64), (5, 2560), (40, 4096), (3, 37), (2, 20000), (1300, 256),
                                   (0, 8), (600, 1031)])
@pytest.mark.parametrize("scaled", [False, True])
def test_residual(tok, D, scaled, dt, rdt):
    g = torch.Generator().manual_seed(tok + D + scaled)
    x, dy = (torch.randn(tok, D, generator=g).to(dt) for _ in range(2))
    res, dro = (torch.randn(tok, D, generator=g).to(rdt) for _ in range(2))
    w = 1.0 + 0.3 * torch.randn(D, generator=g)
    sc = 0.1 + 0.02 * torch.randn(D, generator=g) if scaled else None
    alpha = 0.625
    gx, gw, gsc = x.cuda(), w.cuda(), sc.cuda() if scaled else None
    y = torch.empty_like(gx)
    ro = torch.empty((tok, D), dtype=rdt, device="cuda")
    kw = dict(weight=gw, x_scale=gsc, alpha=alpha, eps=EPS)
    ssm.ssm_residual_norm_fwd(gx, y, residual=res.cuda(), residual_out=ro, **kw)
    s = alpha * sc.double() if scaled else torch.tensor(alpha, dtype=torch.float64)
    rr = res.double() + s * x.double()
    # fp32 arithmetic, then one rounding to the stream's type
    ho.close(ro, rr, rdt == BF, 1e-5, "residual_out")
    leaf = ro.double().cpu().requires_grad_()
    lw = w.double().requires_grad_()
    ry = ho.norm(leaf, D, EPS) * lw
    ho.close(y, ry, dt == BF, 1e-4, "y")
    gr = {"dx": torch.empty_like(gx), "dresidual": torch.empty_like(ro), "dweight": torch.empty_like(gw)}
    if scaled:
        gr["dx_scale"] = torch.empty_like(gsc)
    ssm.ssm_residual_norm_bwd(ro, dy.cuda(), gr, x=gx, dresidual_out=dro.cuda(), workspace=ws_of(tok, D), **kw)
    dr, dw = torch.autograd.grad(ry, [leaf, lw], dy.double())
    dr = dr + dro.double()
    ho.close(gr["dresidual"], dr, rdt == BF, 1e-4, "dresidual")
    ho.close(gr["dx"], s * dr, dt == BF, 1e-4, "dx")
    ho.close(gr["dweight"], dw, False, 1e-4, "dweight")
    if scaled:
        ho.close(gr["dx_scale"], alpha * (dr * x.double()).sum(0), False, 1e-4, "dx_scale")
    # in place: the stream, and its gradient
    r2, y2 = res.cuda(), torch.empty_like(y)
    ssm.ssm_residual_norm_fwd(gx, y2, residual=r2, residual_out=r2, **kw)
    assert torch.equal(r2, ro) and torch.equal(y2, y)
    d2 = dro.cuda()
    ssm.ssm_residual_norm_bwd(ro, dy.cuda(), {"dresidual": d2}, dresidual_out=d2, **kw)
    assert torch.equal(d2, gr["dresidual"])


def test_first_block_has_no_residual():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 640, generator=g).to(BF)
    y, ro = torch.empty((9, 640), dtype=BF, device="cuda"), torch.empty((9, 640), device="cuda")
    ssm.ssm_residual_norm_fwd(x.cuda(), y, residual_out=ro)
    assert torch.equal(ro.cpu(), x.float())
    ho.close(y, ho.norm(x.double(), 640, EPS), True, 1e-4, "y")


def test_zero_rows_and_extreme_gates():
    """A row of zeros norms to zeros; gates of +-100 and the norm's gradient stay finite."""
    x = torch.zeros(3, 512)
    x[1] = 2.0
    z = torch.zeros(3, 512)
    z[1, ::2], z[1, 1::2] = 100.0, -100.0
    for dt in (F32, BF):
        y = torch.empty((3, 512), dtype=dt, device="cuda")
        gr = {"dx": torch.empty_like(y), "dz": torch.empty_like(y)}
        ssm.ssm_gated_norm_fwd(x.to(dt).cuda(), y, z=z.to(dt).cuda())
        ssm.ssm_gated_norm_bwd(x.to(dt).cuda(), torch.ones_like(y), gr, z=z.to(dt).cuda())
        assert (y[[0, 2]] == 0).all()
        for t in (y, gr["dx"], gr["dz"]):
            assert torch.isfinite(t.float()).all()


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_a_block_end_to_end(dt):
    """Residual norm, scan with a decay per head and gated norm as one mixer, forward and
    backward. (The projections of a real block sit between them; here the normed stream
    itself is the scan's value.) Every stage is held to its own bound on the inputs that
    it really had, the rounded outputs of the stage before; in fp32 the whole chain is
    also compared with autograd through the 64-bit forms, where three stages each add at
    most what their own bound allows."""
    lens, H, P, G, N = [90, 45], 4, 32, 2, 64
    tok, D = sum(lens), H * P
    g = torch.Generator().manual_seed(3)
    x, z, dout = (torch.randn(tok, D, generator=g).to(dt) for _ in range(3))
    B, C = (torch.randn(tok, G, N, generator=g).to(dt) for _ in range(2))
    delta = (0.5 * torch.randn(tok, H, generator=g)).to(dt)
    res = torch.randn(tok, D, generator=g)
    w1, w2 = (1.0 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    A, bias, Dk = -(1 + 8 * torch.rand(H, generator=g)), -3 + torch.randn(H, generator=g), torch.randn(H, generator=g)
    cu = torch.tensor([0, 90, 135], dtype=torch.int32).cuda()
    G_ = lambda t: t.cuda()  # noqa: E731
    n1, r, yo, out = (torch.empty((tok, D), dtype=d, device="cuda") for d in (dt, F32, dt, dt))
    ssm.ssm_residual_norm_fwd(G_(x), n1, residual=G_(res), residual_out=r, weight=G_(w1))
    args = (n1.view(tok, H, P), G_(delta), G_(A), G_(B), G_(C))
    opt = dict(Dskip=G_(Dk), dt_bias=G_(bias), cu_seqlens=cu)
    nb = ssm.ssm_head_scan_workspace_size(tok, H, P, G, N, 2, dt)
    ssm.ssm_head_scan_fwd(*args, yo.view(tok, H, P), workspace=torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda"), **opt)
    ssm.ssm_gated_norm_fwd(yo, out, weight=G_(w2), z=G_(z), group_size=D // 2)
    dyo, dz, dn1 = (torch.empty((tok, D), dtype=dt, device="cuda") for _ in range(3))
    dw1, dw2 = (torch.empty(D, device="cuda") for _ in range(2))
    ssm.ssm_gated_norm_bwd(yo, G_(dout), {"dx": dyo, "dz": dz, "dweight": dw2}, weight=G_(w2), z=G_(z),
                           group_size=D // 2, workspace=ws_of(tok, D))
    gr = {"du": dn1.view(tok, H, P), "ddelta": torch.empty((tok, H), dtype=dt, device="cuda"),
          "dB": torch.empty((tok, G, N), dtype=dt, device="cuda"), "dC": torch.empty((tok, G, N), dtype=dt, device="cuda"),
          "dA": torch.empty(H, device="cuda"), "dDskip": torch.empty(H, device="cuda"), "ddt_bias": torch.empty(H, device="cuda")}
    nb = ssm.ssm_head_scan_bwd_workspace_size(tok, H, P, G, N, 2, dt)
    ssm.ssm_head_scan_bwd(*args, dyo.view(tok, H, P), gr, workspace=torch.empty(nb, dtype=torch.uint8, device="cuda"), **opt)
    dx, dres = torch.empty((tok, D), dtype=dt, device="cuda"), torch.empty((tok, D), device="cuda")
    ssm.ssm_residual_norm_bwd(r, dn1, {"dx": dx, "dresidual": dres, "dweight": dw1}, x=G_(x), weight=G_(w1),
                              workspace=ws_of(tok, D))
    b = dt == BF
    f = lambda t: t.detach().double().cpu()  # noqa: E731

    def stage(fn, leaves, grad, out_want, wants, sizes={}):
        leaves = [v.requires_grad_() for v in leaves]
        ref = fn(*leaves)
        ho.close(out_want[1], ref, b, 1e-4, out_want[0], sizes.get(out_want[0]))
        for (name, got), r in zip(wants, torch.autograd.grad(ref, leaves, grad)):
            if got is not None:
                ho.close(got, r, b and got.dtype == BF, 1e-4, name, sizes.get(name))

    stage(lambda v, w: ho.norm(v, D, EPS) * w, [f(r), w1.double()], f(dn1), ("n1", n1), [("dres", dres), ("dw1", dw1)])
    stage(lambda v, zz, w: ho.gated(v, zz, w, D // 2, EPS, False), [f(yo), z.double(), w2.double()], dout.double(),
          ("out", out), [("dyo", dyo), ("dz", dz), ("dw2", dw2)])
    scan_in = (f(n1).view(tok, H, P), f(delta), f(A), f(B), f(C), f(Dk), f(bias), True, None, lens)
    size = ho.sizes(*scan_in, f(dyo).view(tok, H, P), None) if b else {}
    ry, _ = ho.scan(*scan_in)
    ho.close(yo.view(tok, H, P), ry, b, 1e-4, "yo", size.get("y"))
    rs = ho.scan_bwd(*scan_in, f(dyo).view(tok, H, P), None)
    for k in ("du", "ddelta", "dB", "dC"):
        ho.close(gr[k], rs[k], b, 1e-4, k, size.get(k))
    for k, total in (("dA", "dA_size"), ("ddt_bias", "dbias_size")):
        assert ((f(gr[k]) - rs[k]).abs() <= (1e-5 if k == "dA" else 1e-4) * rs[total] + 1e-6).all(), k
    ho.close(gr["dDskip"], rs["dDskip"], False, 1e-4, "dDskip")
    if b:
        return
    L = {k: v.double().requires_grad_() for k, v in dict(x=x, z=z, B=B, C=C, delta=delta, res=res, w1=w1, w2=w2, A=A,
                                                         bias=bias, Dk=Dk).items()}
    rn = ho.norm(L["res"] + L["x"], D, EPS) * L["w1"]
    ry, _ = ho.scan(rn.view(tok, H, P), L["delta"], L["A"], L["B"], L["C"], L["Dk"], L["bias"], True, None, lens)
    rout = ho.gated(ry.reshape(tok, D), L["z"], L["w2"], D // 2, EPS, False)
    rg = dict(zip(L, torch.autograd.grad(rout, list(L.values()), dout.double())))
    ho.close(out, rout, False, 3e-4, "out")
    for name, got in dict(x=dx, z=dz, B=gr["dB"], C=gr["dC"], delta=gr["ddelta"], res=dres, w1=dw1, w2=dw2,
                          Dk=gr["dDskip"], bias=gr["ddt_bias"], A=gr["dA"]).items():
        ho.close(got, rg[name], False, 3e-4, name)


@pytest.mark.parametrize("dt,rdt", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16_f32", "bf16"])
@pytest.mark.parametrize("D", [5120, 8192, 9000])
def test_wide_rows(D, dt, rdt):
    """Rows of more than 4096 columns, gate and stream, more rows than blocks."""
    tok = 700
    g = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, z, dy, ro, dro = r(tok, D).to(dt), r(tok, D).to(dt), r(tok, D).to(dt), r(tok, D).to(rdt), r(tok, D).to(rdt)
    w = 1.0 + 0.3 * r(D)
    gw = w.cuda()
    gr = {"dx": torch.empty_like(x, device="cuda"), "dz": torch.empty_like(x, device="cuda"), "dweight": torch.empty_like(gw)}
    ssm.ssm_gated_norm_bwd(x.cuda(), dy.cuda(), gr, weight=gw, z=z.cuda(), workspace=ws_of(tok, D))
    lx, lz, lw = (t.double().requires_grad_() for t in (x, z, w))
    ref = torch.autograd.grad(ho.norm(lx * torch.nn.functional.silu(lz), D, EPS) * lw, [lx, lz, lw], dy.double())
    for k, v in zip(("dx", "dz", "dweight"), ref):
        ho.close(gr[k], v, dt == BF and k != "dweight", 1e-4, k)
    g2 = {"dresidual": torch.empty_like(ro, device="cuda"), "dweight": torch.empty_like(gw), "dx_scale": torch.empty_like(gw)}
    ssm.ssm_residual_norm_bwd(ro.cuda(), dy.cuda(), g2, x=x.cuda(), weight=gw, alpha=0.5, dresidual_out=dro.cuda(),
                              workspace=ws_of(tok, D))
    lr, lw = ro.double().requires_grad_(), w.double().requires_grad_()
    dr, dw = torch.autograd.grad(ho.norm(lr, D, EPS) * lw, [lr, lw], dy.double())
    dr = dr + dro.double()
    ho.close(g2["dresidual"], dr, rdt == BF, 1e-4, "dresidual")
    ho.close(g2["dweight"], dw, False, 1e-4, "dweight")
    ho.close(g2["dx_scale"], 0.5 * (dr * x.double()).sum(0), False, 1e-4, "dx_scale")


def test_captured_and_on_another_stream():
    """A block's norms, forward and backward, captured beside each other on a side stream
    with a workspace each: replays give the eager results for inputs changed in place."""
    tok, D = 300, 1536
    side = torch.cuda.Stream()
    runs = []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(i)
        x, z, dy = (torch.randn(tok, D, generator=g, device="cuda").to(BF) for _ in range(3))
        res, w = torch.randn(tok, D, generator=g, device="cuda"), torch.rand(D, generator=g, device="cuda")
        o = {k: torch.zeros_like(x) for k in ("y", "n", "dx", "dz")}
        o.update(ro=torch.zeros_like(res), dweight=torch.zeros_like(w), dw2=torch.zeros_like(w))
        ws = ws_of(tok, D)

        def block(x=x, z=z, dy=dy, res=res, w=w, o=o, ws=ws):
            ssm.ssm_residual_norm_fwd(x, o["n"], residual=res, residual_out=o["ro"], weight=w)
            ssm.ssm_gated_norm_fwd(o["n"], o["y"], weight=w, z=z)
            ssm.ssm_gated_norm_bwd(o["n"], dy, {"dx": o["dx"], "dz": o["dz"], "dweight": o["dweight"]}, weight=w,
                                   z=z, workspace=ws)
            ssm.ssm_residual_norm_bwd(o["ro"], o["dx"], {"dweight": o["dw2"]}, weight=w, workspace=ws)

        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            block()
        runs.append((graph, block, x, o))
    for graph, block, x, o in runs:
        x.mul_(0.5)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        runs[0][0].replay()
    runs[1][0].replay()
    torch.cuda.synchronize()
    for graph, block, x, o in runs:
        got = {k: v.clone() for k, v in o.items()}
        block()
        torch.cuda.synchronize()
        for k, v in got.items():
            assert torch.equal(v, o[k]), k
            assert v.abs().sum() > 0
