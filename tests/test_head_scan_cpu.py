"""The scan with one decay per head and the block norms on the host: their refusals
(fake addresses, nothing reaches a device), the chunk slots, and the 64-bit forms that
the GPU tests use, against differences."""

import ctypes

import numpy as np
import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm

L = ssm.lib
A16 = 0x10000
M = 1 << 20


def _err():
    return ssm.ssm_last_error()


def fwd(**kw):
    a = dict(u=A16, us=128, d=A16 + M, ds=2, A=A16 + 2 * M, B=A16 + 3 * M, C=A16 + 4 * M, bs=64, D=None, b=None, sp=1,
             h0=None, cu=None, S=1, y=A16 + 5 * M, hf=None, tok=64, H=2, P=64, G=1, N=64, dt=1,
             ws=A16 - A16 % 256 + 16 * M, wsb=1 << 30)
    a.update(kw)
    return L.ssm_head_scan_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), -2), (dict(H=0), -1), (dict(G=2, H=3), -1), (dict(P=0), -1), (dict(P=257), -1), (dict(N=0), -1),
    (dict(N=129), -1), (dict(G=3), -1), (dict(S=0), -1), (dict(tok=63, S=2), -1), (dict(tok=-1), -1), (dict(u=None), -1),
    (dict(A=None), -1), (dict(y=None), -1), (dict(us=127), -1), (dict(ds=1), -1), (dict(bs=63), -1),
    (dict(u=A16 + 1), -3), (dict(A=A16 + 2), -3), (dict(h0=A16 + 9 * M + 2), -3), (dict(y=A16), -1), (dict(y=A16 + 3 * M + 2), -1),
    (dict(cu=A16 + 2), -3), (dict(H=40000, P=128, us=40000 * 128, ds=40000), -1),
    (dict(h0=A16 + 9 * M, hf=A16 + 9 * M + 64), -1), (dict(S=65536, tok=65536), -1),
])
def test_head_scan_rejects(kw, code):
    assert fwd(**kw) == code
    assert "ssm_head_scan_fwd" in _err()


def bwd(**kw):
    a = dict(u=A16, us=128, d=A16 + M, ds=2, A=A16 + 2 * M, B=A16 + 3 * M, C=A16 + 4 * M, bs=64, D=None, b=None, sp=1,
             h0=None, cu=None, S=1, dy=A16 + 5 * M, dhf=None, du=A16 + 6 * M, dd=A16 + 7 * M, dB=A16 + 8 * M,
             dC=A16 + 9 * M, dA=A16 + 10 * M, dD=None, db=None, dh0=None, tok=64, H=2, P=64, G=1, N=64, dt=1,
             ws=A16 - A16 % 256 + 64 * M, wsb=1 << 30)
    a.update(kw)
    return L.ssm_head_scan_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), -2), (dict(dA=None), -1), (dict(dy=None), -1), (dict(du=None), -1), (dict(dd=None), -1),
    (dict(dB=None), -1), (dict(dC=None), -1), (dict(ws=None), -5), (dict(wsb=100), -5), (dict(ws=A16 + 64 * M + 16), -3),
    (dict(du=A16), -1), (dict(du=A16 + 5 * M), -1), (dict(dB=A16 + 9 * M), -1), (dict(dA=A16 + 2 * M), -1),
    (dict(dh0=A16 + 64 * M), -1), (dict(N=200), -1), (dict(P=300), -1),
])
def test_head_scan_bwd_rejects(kw, code):
    assert bwd(**kw) == code
    assert "ssm_head_scan_bwd" in _err()


def step(**kw):
    a = dict(st=A16, x=A16 + 2 * M, xs=128, dt_=A16 + 3 * M, ds=2, B=A16 + 4 * M, C=A16 + 5 * M, bs=64, A=A16, D=None,
             b=None, sp=1, idx=None, slots=4, y=A16 + 6 * M, Bt=4, H=2, P=64, G=1, N=64, dt=1)
    a.update(kw)
    return L.ssm_head_state_update(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=4), -2), (dict(N=129), -1), (dict(slots=3), -1), (dict(Bt=70000, slots=70000), -1), (dict(x=None), -1),
    (dict(st=A16 + 2), -3), (dict(y=A16 + 2 * M), -1), (dict(xs=5), -1), (dict(slots=-1), -1), (dict(idx=A16 + 1), -3),
    (dict(H=65535, Bt=65535, xs=1 << 30, ds=1 << 30, slots=65535), -1),
])
def test_head_step_rejects(kw, code):
    assert step(**kw) == code
    assert "ssm_head_state_update" in _err()


def test_no_rows_is_no_work():
    assert step(Bt=0, st=None, x=None, dt_=None, B=None, C=None, A=None, y=None) == 0


class Scalars(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("alpha", ctypes.c_float)]


SC = Scalars(1e-5, 1.0)
BAD = Scalars(float("nan"), 1.0)


def norm(name, **kw):
    sc = ctypes.addressof(SC)
    rows = {
        "gated_fwd": dict(x=A16, xs=64, z=A16 + M, zs=64, w=None, sc=sc, before=0, y=A16 + 2 * M, tok=4, D=64, gs=64, dt=1),
        "gated_bwd": dict(x=A16, xs=64, z=A16 + M, zs=64, w=None, sc=sc, before=0, dy=A16 + 2 * M, dx=A16 + 3 * M,
                          dz=A16 + 4 * M, dw=A16 + 5 * M, tok=4, D=64, gs=64, dt=1, ws=A16 + 16 * M, wsb=1 << 30),
        "residual_fwd": dict(x=A16, r=A16 + M, s=None, w=None, sc=sc, y=A16 + 2 * M, ro=A16 + M, tok=4, D=64, dt=1, rdt=0),
        "residual_bwd": dict(r=A16, x=A16 + M, s=None, w=None, sc=sc, dy=A16 + 2 * M, dro=A16 + 3 * M, dx=A16 + 4 * M,
                             dr=A16 + 3 * M, dw=A16 + 5 * M, dsc=None, tok=4, D=64, dt=1, rdt=0, ws=A16 + 16 * M, wsb=1 << 30),
    }[name]
    rows.update(kw)
    kind, way = name.split("_")
    return getattr(L, f"ssm_{kind}_norm_{way}")(*rows.values(), None)


@pytest.mark.parametrize("name,kw,code", [
    ("gated_fwd", dict(dt=3), -2), ("gated_fwd", dict(gs=7), -1), ("gated_fwd", dict(gs=0), -1), ("gated_fwd", dict(x=None), -1),
    ("gated_fwd", dict(sc=None), -1), ("gated_fwd", dict(sc=ctypes.addressof(BAD)), -1), ("gated_fwd", dict(xs=10), -1),
    ("gated_fwd", dict(zs=10), -1), ("gated_fwd", dict(y=A16 + 100), -1), ("gated_fwd", dict(x=A16 + 1), -3),
    ("gated_fwd", dict(D=0), -1), ("gated_fwd", dict(tok=-1), -1), ("gated_fwd", dict(D=65536 * 2, xs=1 << 20, zs=1 << 20, gs=1), -1),
    ("gated_bwd", dict(ws=None), -5), ("gated_bwd", dict(wsb=64), -5), ("gated_bwd", dict(dx=A16 + 2 * M), -1),
    ("gated_bwd", dict(dz=A16 + 3 * M), -1), ("gated_bwd", dict(dy=None), -1), ("gated_bwd", dict(ws=A16 + 16 * M + 8), -3),
    ("residual_fwd", dict(rdt=1, dt=0), -2), ("residual_fwd", dict(y=None), -1), ("residual_fwd", dict(ro=A16 + M + 8), -1),
    ("residual_fwd", dict(r=A16 + M + 2), -3), ("residual_fwd", dict(y=A16 + M), -1),
    ("residual_bwd", dict(r=None), -1), ("residual_bwd", dict(x=None, dsc=A16 + 6 * M), -1), ("residual_bwd", dict(ws=None), -5),
    ("residual_bwd", dict(dr=A16 + 3 * M + 8), -1), ("residual_bwd", dict(dx=A16), -1),
])
def test_norms_reject(name, kw, code):
    assert norm(name, **kw) == code
    assert "norm" in _err()


def test_workspace_sizes_of_bad_arguments_are_zero():
    assert ssm.ssm_head_scan_bwd_workspace_size(64, 2, 64, 1, 129, 1, torch.bfloat16) == 0
    assert ssm.ssm_head_scan_bwd_workspace_size(64, 2, 64, 1, 64, 0, torch.bfloat16) == 0
    assert ssm.ssm_head_scan_bwd_workspace_size(64, 2, 64, 1, 64, 1, torch.float32) % 256 == 0
    assert ssm.ssm_norm_bwd_workspace_size(-1, 64) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Shapes, dtypes, inner strides: refused before a pointer is passed."""
    tok, H, P, G, N = 6, 2, 8, 1, 4
    z = torch.zeros
    good = dict(u=z(tok, H, P), delta=z(tok, H), A=z(H), B=z(tok, G, N), C=z(tok, G, N), y=z(tok, H, P))
    for kw in (dict(u=z(tok, H, P).bfloat16()), dict(delta=z(tok, H + 1)), dict(A=z(H + 1)), dict(C=z(tok, G, N + 1)),
               dict(y=z(tok, P, H).transpose(1, 2)), dict(u=z(tok, P, H).transpose(1, 2)), dict(B=z(tok - 1, G, N)),
               dict(C=z(tok, 2 * G * N)[:, :G * N].view(tok, G, N)), dict(A=z(H).double())):
        a = {**good, **kw}
        with pytest.raises(ssm.SsmError):
            ssm.ssm_head_scan_fwd(a["u"], a["delta"], a["A"], a["B"], a["C"], a["y"], stream=0)
    with pytest.raises(ssm.SsmError):  # memory of the host
        ssm.ssm_head_scan_fwd(*good.values(), stream=0)
    with pytest.raises(ssm.SsmError):
        ssm.ssm_gated_norm_fwd(z(4, 8), z(4, 8), stream=0)
    with pytest.raises(ssm.SsmError):
        ssm.ssm_residual_norm_fwd(z(4, 8), z(4, 8), residual=z(4, 8), stream=0)
    with pytest.raises(ssm.SsmError):
        ssm.ssm_head_state_update(z(tok, H, P, N), good["u"], good["delta"], good["B"], good["C"], good["y"], good["A"], stream=0)


@pytest.mark.parametrize("span", [32, 128, 512])
def test_chunk_slots_are_distinct_and_found_again(span):
    """Chunk k of sequence s has slot floor(start / span) + s + k: no two share one, all
    lie below tok / span + S, and the search from the slot finds the chunk."""
    rng = np.random.default_rng(span)
    for _ in range(100):
        S = int(rng.integers(1, 40))
        lens = rng.integers(0, 5 * span, size=S) * (rng.random(S) > 0.3)
        cu = np.concatenate([[0], np.cumsum(lens)])
        tok = int(cu[-1])
        used = {}
        for s in range(S):
            for k in range(-(-int(lens[s]) // span)):
                slot = int(cu[s]) // span + s + k
                assert slot not in used and slot < tok // span + S
                used[slot] = (s, k)
        for slot in range(tok // span + S):
            lo, hi = 0, S - 1
            while lo < hi:
                mid = (lo + hi + 1) >> 1
                if cu[mid] // span + mid <= slot:
                    lo = mid
                else:
                    hi = mid - 1
            k = slot - (cu[lo] // span + lo)
            found = (lo, int(k)) if k >= 0 and cu[lo] + k * span < cu[lo + 1] else None
            assert found == used.get(slot)


def test_sizes_bound_what_a_rounded_factor_does():
    """Rounding M, or the state a chunk starts from, by up to 2^-8 moves y by at most 2^-8
    of `sizes`: shown on the matrix form with random roundings."""
    g = torch.Generator().manual_seed(5)
    lens, H, P, G, N = [150], 2, 4, 1, 6
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    u, delta, B, C, h0 = r(150, H, P), r(150, H), r(150, G, N), r(150, G, N), r(1, H, P, N)
    A = -torch.rand(H, generator=g, dtype=torch.float64)
    y, _ = ho.scan(u, delta, A, B, C, None, None, True, h0, lens)
    size = ho.sizes(u, delta, A, B, C, None, None, True, h0, lens)["y"]
    d = ho.softplus(delta)
    got = torch.zeros_like(y)
    h = h0[0]
    for a, b in ((0, 128), (128, 150)):
        c = torch.cumsum(d[a:b] * A, 0).t()
        L = torch.exp(c[:, :, None] - c[:, None, :]).tril() * d[a:b].t()[:, None, :]
        Bh, Ch, uh = B[a:b, 0], C[a:b, 0], u[a:b].transpose(0, 1)
        M = (Ch @ Bh.t()) * L
        M = M * (1 + (2 * torch.rand(M.shape, generator=g, dtype=torch.float64) - 1) * 2.0 ** -8)
        hr = h * (1 + (2 * torch.rand(h.shape, generator=g, dtype=torch.float64) - 1) * 2.0 ** -8)
        got[a:b] = (M @ uh + torch.exp(c)[..., None] * (Ch @ hr.transpose(1, 2))).transpose(0, 1)
        w = d[a:b].t() * torch.exp(c[:, -1:] - c)
        h = torch.exp(c[:, -1])[:, None, None] * h + (w[..., None] * uh).transpose(1, 2) @ Bh
    off = (got - y).abs()
    assert (off <= 2.0 ** -8 * size + 1e-12).all() and off.max() > 2.0 ** -12


@pytest.mark.parametrize("sp", [True, False])
def test_written_out_gradients_match_autograd_and_differences(sp):
    g = torch.Generator().manual_seed(0)
    lens, H, P, G, N = [4, 0, 3], 4, 3, 2, 5
    tok = sum(lens)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    t = dict(u=r(tok, H, P), delta=r(tok, H), A=-torch.rand(H, generator=g, dtype=torch.float64) - 0.2, B=r(tok, G, N),
             C=r(tok, G, N), D=r(H), bias=r(H), h0=r(3, H, P, N))
    dy, dhf = r(tok, H, P), r(3, H, P, N)

    def loss(v):
        y, hf = ho.scan(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["bias"], sp, v["h0"], lens)
        return (dy * y).sum() + (dhf * hf).sum()

    got = ho.scan_bwd(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"], t["bias"], sp, t["h0"], lens, dy, dhf)
    names = dict(u="du", delta="ddelta", A="dA", B="dB", C="dC", D="dDskip", bias="ddt_bias", h0="dh0")
    leaf = {k: v.clone().requires_grad_() for k, v in t.items()}
    auto = torch.autograd.grad(loss(leaf), list(leaf.values()))
    for (k, v), a in zip(t.items(), auto):
        assert torch.allclose(got[names[k]], a, rtol=1e-10, atol=1e-10), k
        step = r(*v.shape)
        e = 1e-6
        diff = (loss({**t, k: v + e * step}) - loss({**t, k: v - e * step})) / (2 * e)
        want = (got[names[k]] * step).sum()
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), k


def _plan(tok, H, P, G, S, known):
    """How the bf16 kernels walk the sequences: ("whole", None), or ("cut" / "ask", tokens a segment)."""
    npan = H // G * -(-P // 64)
    walks = G * -(-npan // 2)
    longest = -(-(tok // S) // 128)
    chunks = longest * S if known else tok // 128 + S
    load = (chunks * walks + 147) // 148
    limit, span = load * 11 // 5 + 4, max(load, 4) * 128
    if known:
        return ("cut", span) if longest > limit else ("whole", None)
    return ("whole", None) if walks * S >= 296 or tok // 128 + 1 <= limit else ("ask", span)


def _up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("bwd", [False, True])
def test_workspaces_hold_dense_and_packed_walks(bwd):
    """The size is asked for without cu_seqlens, so it covers the tables, the segments' states,
    the marks and the rest of either kind of call, whichever needs more."""
    rng = np.random.default_rng(1)
    cases = [(270336, 2, 64, 1, 64, 3), (270336, 128, 64, 2, 64, 3), (16384, 24, 64, 1, 128, 8), (8192, 128, 64, 8, 128, 1),
             (5000, 2, 64, 1, 128, 1), (6000, 2, 64, 1, 128, 2), (0, 2, 64, 1, 64, 2), (1, 1, 1, 1, 1, 1)]
    for _ in range(300):
        G = int(rng.choice([1, 2, 8]))
        cases.append((int(np.exp(rng.uniform(0, 13))), G * int(rng.integers(1, 20)), int(rng.integers(1, 257)), G,
                      int(rng.integers(1, 129)), int(rng.integers(1, 60))))
    packed_larger = 0
    for tok, H, P, G, N, S in cases:
        size = (ssm.ssm_head_scan_bwd_workspace_size if bwd else ssm.ssm_head_scan_workspace_size)(
            tok, H, P, G, N, S, torch.bfloat16)
        slots, np_ = tok // 128 + S, -(-P // 64)
        panel = H * np_ * 64 * (128 if N > 64 else 64)
        need = []
        for known in (True, False):
            mode, span = _plan(tok, H, P, G, S, known)
            segs = 0 if mode == "whole" else tok // span + S
            marks = _up(slots * panel * 2 * (2 if bwd else 1))
            n = _up(slots * H * (7 * 128 + 192) * 4) + _up(segs * panel * 4) + _up(segs * H * 4) + marks
            n += _up(4 * S if S > 1 else 0) + 256
            if bwd:  # the gradients' marks, at least one range of dG tiles, the chunks' shares
                n += marks + _up(slots * G * 128 * 128 * 4) + _up(slots * H * 12)
            need.append(n)
        assert size >= max(need), (tok, H, P, G, N, S, size, need)
        packed_larger += need[1] > need[0]
    assert packed_larger  # the case that a size from the dense plan alone would miss
