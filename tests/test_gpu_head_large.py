"""The scan with one decay per head at sizes that small tests cannot show: offsets past
2^31 elements, thousands of sequences, heads and groups independent of one another."""

import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def fwd(u, delta, A, B, C, D, bias, h0, cu, S):
    tok, H, P = u.shape
    y = torch.empty((tok, H, P), dtype=u.dtype, device="cuda")
    hf = torch.empty((S, H, P, B.shape[2]), device="cuda")
    n = ssm.ssm_head_scan_workspace_size(tok, H, P, B.shape[1], B.shape[2], S, u.dtype)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    ssm.ssm_head_scan_fwd(u, delta, A, B, C, y, Dskip=D, dt_bias=bias, h0=h0, h_final=hf, cu_seqlens=cu,
                          S=S, workspace=ws)
    return y, hf


def bwd(u, delta, A, B, C, D, bias, h0, cu, S, dy):
    tok, H, P = u.shape
    g = {"du": torch.empty_like(dy), "ddelta": torch.empty((tok, H), dtype=u.dtype, device="cuda"),
         "dB": torch.empty(B.shape, dtype=u.dtype, device="cuda"), "dC": torch.empty(B.shape, dtype=u.dtype, device="cuda"),
         "dA": torch.empty(H, device="cuda"), "dh0": torch.empty((S, H, P, B.shape[2]), device="cuda")}
    n = ssm.ssm_head_scan_bwd_workspace_size(tok, H, P, B.shape[1], B.shape[2], S, u.dtype)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ssm.ssm_head_scan_bwd(u, delta, A, B, C, dy, g, Dskip=D, dt_bias=bias, h0=h0, cu_seqlens=cu, S=S, workspace=ws)
    return g


def inputs(tok, H, P, G, N, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u = torch.empty((tok, H, P), dtype=dt, device="cuda")
    for i in range(0, tok, 1 << 15):
        u[i:i + (1 << 15)] = r(min(1 << 15, tok - i), H, P).to(dt)
    return (u, (0.5 * r(tok, H)).to(dt), -(1 + 8 * torch.rand(H, generator=g, device="cuda")), r(tok, G, N).to(dt),
            r(tok, G, N).to(dt), r(H), -3 + r(H))


def test_offsets_past_2_31_elements():
    """u and y of 2.2e9 elements: the last heads' results equal those of a call that has
    these heads alone (a head's arithmetic does not depend on the others)."""
    tok, H, P, G, N = 270336, 128, 64, 2, 64
    u, delta, A, B, C, D, bias = inputs(tok, H, P, G, N, BF, 1)
    cu = torch.tensor([0, 100000, 100000, 270336], dtype=torch.int32, device="cuda")
    y, hf = fwd(u, delta, A, B, C, D, bias, None, cu, 3)
    k = H - 2
    y2, hf2 = fwd(u[:, k:].contiguous(), delta[:, k:].contiguous(), A[k:].clone(), B[:, 1:].contiguous(),
                  C[:, 1:].contiguous(), D[k:].clone(), bias[k:].clone(), None, cu, 3)
    assert torch.equal(y[:, k:], y2) and torch.equal(hf[:, k:], hf2)
    assert ssm.ssm_device_status() == 0


def test_states_past_2_31_elements():
    """A decode cache of 2.3e9 entries: only the named slots change, and rightly."""
    slots, H, P, G, N = 2200, 128, 64, 1, 128
    st = torch.zeros((slots, H, P, N), device="cuda")
    x, dt, A, B, C, D, bias = inputs(3, H, P, G, N, BF, 2)
    idx = torch.tensor([2199, 0, 2100], dtype=torch.int32, device="cuda")
    st[idx.long()] = 0.5
    y = torch.empty_like(x)
    ssm.ssm_head_state_update(st, x, dt, B, C, y, A, Dskip=D, dt_bias=bias, state_indices=idx)
    f = lambda t: t.double().cpu()  # noqa: E731
    ry, rh = ho.scan(f(x), f(dt), f(A), f(B), f(C), f(D), f(bias), True, torch.full((3, H, P, N), 0.5, dtype=torch.float64),
                     [1, 1, 1])
    ho.close(y, ry, True, 1e-4, "y")
    ho.close(st[idx.long()], rh, False, 1e-4, "state")
    st[idx.long()] = 0.0
    assert not bool(st.any())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_thousands_of_short_sequences(dt):
    """3000 sequences of 0 to 4 tokens, forward and backward."""
    r = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 5, (3000,), generator=r).tolist()
    tok, H, P, G, N = sum(lens), 2, 16, 1, 8
    u, delta, A, B, C, D, bias = inputs(tok, H, P, G, N, dt, 3)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    h0 = torch.randn((3000, H, P, N), device="cuda") * 0.3
    dy = torch.randn(tok, H, P, device="cuda").to(dt)
    y, hf = fwd(u, delta, A, B, C, D, bias, h0, cu, 3000)
    g = bwd(u, delta, A, B, C, D, bias, h0, cu, 3000, dy)
    f = lambda t: t.double().cpu()  # noqa: E731
    a = (f(u), f(delta), f(A), f(B), f(C), f(D), f(bias), True, f(h0), lens)
    ry, rh = ho.scan(*a)
    rg = ho.scan_bwd(*a, f(dy), None)
    size = ho.sizes(*a, f(dy), None) if dt == BF else {}
    ho.close(y, ry, dt == BF, 1e-4, "y", size.get("y"))
    ho.close(hf, rh, False, 1e-4, "h_final")
    for k in ("du", "ddelta", "dB", "dC"):
        ho.close(g[k], rg[k], dt == BF, 1e-4, k, size.get(k))
    ho.close(g["dh0"], rg["dh0"], False, 1e-4, "dh0")


@pytest.mark.parametrize("S,tok", [(1, 5000), (2, 6000)])
def test_split_walks(S, tok):
    """Few walks of many chunks are cut into segments that run side by side and are joined:
    against the 64-bit recurrence in matrix form, chunk by chunk."""
    H, P, G, N = 2, 64, 1, 128
    u, delta, A, B, C, D, bias = inputs(tok, H, P, G, N, BF, 4)
    A = A * 0.02  # states that last for thousands of tokens
    h0 = torch.randn((S, H, P, N), device="cuda") * 0.3
    dy = torch.randn(tok, H, P, device="cuda").to(BF)
    cut = tok // 3 if S == 2 else tok
    lens = [cut, tok - cut][:S]
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    y, hf = fwd(u, delta, A, B, C, D, bias, h0, cu, S)
    g = bwd(u, delta, A, B, C, D, bias, h0, cu, S, dy)
    f = lambda t: t.double()  # noqa: E731
    d = ho.softplus(f(delta) + f(bias))
    uc, Bc, Cc, yc = f(u), f(B)[:, 0], f(C)[:, 0], f(dy)
    for s, (lo, hi) in enumerate(ho.bounds_of(lens)):
        h, marks = f(h0[s]), []
        for a in range(lo, hi, 128):
            b = min(a + 128, hi)
            c = torch.cumsum(d[a:b] * f(A), 0).t()
            L = torch.exp(c[:, :, None] - c[:, None, :]).tril() * d[a:b].t()[:, None, :]
            M = (Cc[a:b] @ Bc[a:b].t()) * L
            ua, e = uc[a:b].transpose(0, 1), torch.exp(c)[..., None]
            ry = M @ ua + e * (Cc[a:b] @ h.transpose(1, 2)) + f(D)[:, None, None] * ua
            size = M.abs() @ ua.abs() + e * (Cc[a:b].abs() @ h.abs().transpose(1, 2))
            ho.close(y[a:b], ry.transpose(0, 1).cpu(), True, 1e-4, "y", size.transpose(0, 1).cpu())
            marks.append((a, b, c, L, M, h))
            w = d[a:b].t() * torch.exp(c[:, -1:] - c)
            h = torch.exp(c[:, -1])[:, None, None] * h + (w[..., None] * ua).transpose(1, 2) @ Bc[a:b]
        ho.close(hf[s], h.cpu(), False, 1e-4, "h_final")
        gs = torch.zeros_like(h)
        for a, b, c, L, M, h in reversed(marks):
            ya, e = yc[a:b].transpose(0, 1), torch.exp(c)[..., None]
            w = d[a:b].t() * torch.exp(c[:, -1:] - c)
            rdu = M.transpose(1, 2) @ ya + w[..., None] * (Bc[a:b] @ gs.transpose(1, 2)) + f(D)[:, None, None] * ya
            size = M.abs().transpose(1, 2) @ ya.abs()
            ho.close(g["du"][a:b], rdu.transpose(0, 1).cpu(), True, 1e-4, "du", size.transpose(0, 1).cpu())
            gs = torch.exp(c[:, -1])[:, None, None] * gs + (e * ya).transpose(1, 2) @ Cc[a:b]
        ho.close(g["dh0"][s], gs.cpu(), False, 1e-4, "dh0")


def test_split_walks_with_the_state_in_place():
    """h_final may be h0: every segment of a cut walk starts from h0, the last one ends in it.
    Dense and packed, against the same call with its own h_final, bit for bit."""
    tok, H, P, G, N = 8200, 2, 96, 1, 40
    u, delta, A, B, C, D, bias = inputs(tok, H, P, G, N, BF, 9)
    A = A * 0.02
    for S, cu in ((1, None), (2, None), (3, torch.tensor([0, 7000, 7000, tok], dtype=torch.int32, device="cuda"))):
        h0 = torch.randn((S, H, P, N), device="cuda")
        y, hf = fwd(u, delta, A, B, C, D, bias, h0, cu, S)
        y2, h2 = torch.empty_like(y), h0.clone()
        n = ssm.ssm_head_scan_workspace_size(tok, H, P, G, N, S, BF)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        ssm.ssm_head_scan_fwd(u, delta, A, B, C, y2, Dskip=D, dt_bias=bias, h0=h2, h_final=h2, cu_seqlens=cu,
                              S=S, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(hf, h2)
        # and the 64-bit recurrence's end, a chunk at a time
        f = lambda t: t.double()  # noqa: E731
        d = ho.softplus(f(delta) + f(bias))
        lens = [tok // S] * S if cu is None else (cu[1:] - cu[:-1]).tolist()
        for s, (lo, hi) in enumerate(ho.bounds_of(lens)):
            h = f(h0[s])
            for a in range(lo, hi, 128):
                b = min(a + 128, hi)
                c = torch.cumsum(d[a:b] * f(A), 0).t()
                w = d[a:b].t() * torch.exp(c[:, -1:] - c)
                h = torch.exp(c[:, -1])[:, None, None] * h + (w[..., None] * f(u[a:b]).transpose(0, 1)).transpose(1, 2) @ f(B[a:b, 0])
            ho.close(hf[s], h.cpu(), False, 1e-4, "h_final")


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_tens_of_thousands_of_heads(dt):
    """As many heads as the checks allow, each with its own B and C, two tokens."""
    tok, H, P, N = 2, 65535, 40, 3
    u, delta, A, B, C, D, bias = inputs(tok, H, P, H, N, dt, 5)
    dy = torch.randn(tok, H, P, device="cuda").to(dt)
    y, hf = fwd(u, delta, A, B, C, D, bias, None, None, 1)
    g = bwd(u, delta, A, B, C, D, bias, None, None, 1, dy)
    f = lambda t: t.double().cpu()  # noqa: E731
    a = [f(t) for t in (u, delta, A, B, C, D, bias)] + [True, None, [tok]]
    ry, rh = ho.scan(*a)
    rg = ho.scan_bwd(*a, f(dy), None)
    size = ho.sizes(*a, f(dy), None) if dt == BF else {}
    ho.close(y, ry, dt == BF, 1e-4, "y", size.get("y"))
    ho.close(hf, rh, False, 1e-4, "h_final")
    for k in ("du", "ddelta", "dB", "dC"):
        ho.close(g[k], rg[k], dt == BF, 1e-4, k, size.get(k))
