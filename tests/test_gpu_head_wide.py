"""Backward of the per-head scan with heads of several 64-row panels, several of them in one
CTA, and every gradient across the joints of cut walks. References in 64 bits, on the GPU where
they are long; bounds as derived in head_oracle.py."""

import random

import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm
from test_gpu_head_scan import BF, F32, Case

pytestmark = pytest.mark.gpu


def heads_of_cta(tok, S, H, P, G):
    """Heads that one CTA of the bf16 backward takes: the fewest whole waves over 148 SMs, a
    CTA's start and end counted as two panels."""
    ctas, heads, start = (tok // 128 + S) * G, H // G, 2.0 / -(-P // 64)
    best, cost = heads, None
    for waves in range(1, 17):
        r = min(max(waves * 148 // ctas, 1), heads)
        per = -(-heads // r)
        c = (ctas * -(-heads // per) + 147) // 148 * (per + start)
        if cost is None or c < cost:
            best, cost = per, c
        if r == heads:
            break
    return best


def check(c, got):
    """Case.check_bwd with the 64-bit recurrence on the GPU."""
    with torch.device("cuda"):
        a = [t.cuda() if torch.is_tensor(t) else t for t in c.ref_args()]
        dy, dhf = c.dy.double().cuda(), c.dhf.double().cuda() if c.dhf is not None else None
        r = {k: v.cpu() for k, v in ho.scan_bwd(*a, dy, dhf).items()}
        size = {k: v.cpu() for k, v in ho.sizes(*a, dy, dhf).items()} if c.dt == BF else {}
    for k in ("du", "ddelta", "dB", "dC"):
        ho.close(got[k], r[k], c.dt == BF, 1e-4, k, size.get(k))
    for k in ("dh0", "dDskip"):
        ho.close(got[k], r[k], False, 1e-4, k)
    # <g, S> takes two factors in two bf16 planes each with bf16 activations: each is off by at
    # most half a step of half a step, 2^-16
    planes = 2.0 ** -15 if c.dt == BF else 0.0
    for k, size, tol in (("dA", r["dA_size"], 1e-5 + planes), ("ddt_bias", r["dbias_size"], 1e-4)):
        off = (got[k].double().cpu() - r[k]).abs()
        lim = tol * size + 1e-6
        assert (off <= lim).all(), f"{k}: off by {(off / lim).max():.3g} x the bound"


def many(S, seed, *longer):
    """S lengths: mostly none to three tokens, the given longer ones among them."""
    r = random.Random(seed)
    lens = [r.randrange(4) for _ in range(S - len(longer))] + list(longer)
    r.shuffle(lens)
    return lens


# lens, H, P, G, N, heads of a CTA
WIDE = [
    (many(60, 1, 130), 8, 128, 1, 128, 4),
    (many(301, 2, 128, 200), 6, 128, 1, 64, 3),
    (many(301, 3, 129), 14, 96, 2, 40, 7),     # an odd number of heads
    (many(60, 4, 260), 7, 192, 1, 16, 4),      # three panels a head, the last CTA has fewer heads
    (many(200, 5, 100), 5, 200, 1, 128, 3),
    (many(260, 6), 8, 66, 1, 19, 8),           # rows that no tile copy takes
    (many(200, 7, 131), 3, 256, 1, 64, 3),     # four panels a head
    (many(150, 8, 64), 12, 256, 2, 32, 3),
    (many(299, 9, 127), 6, 64, 1, 128, 6),     # one panel a head
    (many(299, 10, 140), 5, 32, 1, 128, 5),
    ([700, 0, 128, 1, 600, 619], 16, 128, 1, 64, 3),
]


@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "-".join(map(str, [sum(s[0]), *s[1:]])))
def test_backward_of_several_heads_in_a_cta(shape):
    lens, H, P, G, N, heads = shape
    assert heads_of_cta(sum(lens), len(lens), H, P, G) == heads
    c = Case(lens, H, P, G, N, BF, seed=20)
    got = c.bwd()
    torch.cuda.synchronize()
    assert ssm.ssm_device_status() == 0
    check(c, got)
    again = c.bwd()
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_forward_of_several_wide_heads_in_a_cta():
    c = Case(many(301, 11, 128, 200), 6, 192, 1, 64, BF, seed=21)
    c.check_fwd(*c.fwd())
    assert ssm.ssm_device_status() == 0


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("lens", [[5000], [2000, 4000], [2500, 2500]], ids=["one", "packed", "dense"])
def test_every_gradient_across_cut_walks(lens, P):
    """Few walks of many chunks are cut into segments: the gradients of the decays, of B and of
    C see the states and their gradients from other segments."""
    c = Case(lens, 2, P, 1, 128, BF, seed=22, decay=(0.02, 0.2))
    got = c.bwd(dense=lens[0] == lens[-1])
    torch.cuda.synchronize()
    assert ssm.ssm_device_status() == 0
    check(c, got)


def test_wide_training_step_in_a_graph():
    """Forward and backward of wide heads, captured and replayed on another stream."""
    c = Case(many(120, 12, 300), 6, 128, 1, 128, BF, seed=23)
    assert heads_of_cta(sum(c.lens), len(c.lens), 6, 128, 1) >= 2
    y, hf = c.fwd()
    want = c.bwd()
    d, A, D, b, dy, h0, dhf = (c.g(t) for t in (c.delta, c.A, c.D, c.bias, c.dy, c.h0, c.dhf))
    ws, wsb = c.ws(False), c.ws(True)
    y2, hf2, g = torch.empty_like(y), torch.empty_like(hf), {k: torch.empty_like(v) for k, v in want.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.ssm_head_scan_fwd(c.gu, d, A, c.gB, c.gC, y2, Dskip=D, dt_bias=b, h0=h0, h_final=hf2, cu_seqlens=c.cu,
                              workspace=ws)
        ssm.ssm_head_scan_bwd(c.gu, d, A, c.gB, c.gC, dy, g, Dskip=D, dt_bias=b, h0=h0, dh_final=dhf,
                              cu_seqlens=c.cu, workspace=wsb)
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(hf, hf2)
    assert all(torch.equal(want[k], g[k]) for k in want)


def test_wide_heads_in_fp32():
    check(c := Case(many(60, 13, 130), 4, 192, 2, 40, F32, seed=24), c.bwd())
