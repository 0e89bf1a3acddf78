"""The scan with one decay per head on the GPU: forward, backward, one decode token,
against the plain 64-bit forms of head_oracle.py, with the bounds derived there."""

import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Case:
    """Seeded inputs on the CPU in 64 bits (rounded to dt first) and on the GPU."""

    def __init__(self, lens, H, P, G, N, dt, seed=0, h0=True, D=True, bias=True, sp=True,
                 sliced=False, decay=(1.0, 16.0), pad=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.P, self.G, self.N, self.dt, self.sp = lens, H, P, G, N, dt, sp
        tok = sum(lens)
        S = len(lens)

        def rnd(*shape):
            return torch.randn(*shape, generator=g).to(dt)

        if sliced:  # one wide row per token, as a projection leaves it
            wide = rnd(tok, H * P + 2 * G * N + pad)
            gw = wide.cuda()

            def cut(w):
                return (w[:, :H * P].view(tok, H, P), w[:, H * P:H * P + G * N].view(tok, G, N),
                        w[:, H * P + G * N:H * P + 2 * G * N].view(tok, G, N))
            self.u, self.B, self.C = cut(wide)
            self.gu, self.gB, self.gC = cut(gw)
        else:
            self.u, self.B, self.C = rnd(tok, H, P), rnd(tok, G, N), rnd(tok, G, N)
            self.gu, self.gB, self.gC = self.u.cuda(), self.B.cuda(), self.C.cuda()
        self.delta = (0.5 * torch.randn(tok, H, generator=g)).to(dt)
        if not sp:
            self.delta = (self.delta.float().abs() * 0.2).to(dt)
        self.A = -(decay[0] + (decay[1] - decay[0]) * torch.rand(H, generator=g))
        self.bias = (-3.0 + torch.randn(H, generator=g)) if bias and sp else None
        self.D = torch.randn(H, generator=g) if D else None
        self.h0 = torch.randn(S, H, P, N, generator=g) * 0.3 if h0 else None
        self.dy = rnd(tok, H, P)
        self.dhf = torch.randn(S, H, P, N, generator=g) * 0.1 if h0 else None
        self.cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()

    def f(self, t):
        return t.double() if t is not None else None

    def g(self, t):
        return t.cuda() if t is not None else None

    def ref_args(self):
        f = self.f
        return (f(self.u), f(self.delta), f(self.A), f(self.B), f(self.C), f(self.D), f(self.bias),
                self.sp, f(self.h0), self.lens)

    def ws(self, bwd):
        size = ssm.ssm_head_scan_bwd_workspace_size if bwd else ssm.ssm_head_scan_workspace_size
        n = size(sum(self.lens), self.H, self.P, self.G, self.N, len(self.lens), self.dt)
        return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

    def fwd(self, dense=False, h_final=None, y_fill=None, stream=None, h0=None):
        S = len(self.lens)
        y = torch.empty(self.gu.shape, dtype=self.dt, device="cuda")
        if y_fill is not None:
            y.fill_(y_fill)
        hf = torch.full((S, self.H, self.P, self.N), 5.0, device="cuda") if h_final is None else h_final
        ssm.ssm_head_scan_fwd(self.gu, self.g(self.delta), self.g(self.A), self.gB, self.gC, y,
                              Dskip=self.g(self.D), dt_bias=self.g(self.bias), delta_softplus=self.sp,
                              h0=self.g(self.h0) if h0 is None else h0, h_final=hf,
                              cu_seqlens=None if dense else self.cu, S=S, workspace=self.ws(False))
        return y, hf

    def bwd(self, dense=False):
        S, tok = len(self.lens), sum(self.lens)
        new = lambda *s, dt=F32: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
        g = {"du": new(tok, self.H, self.P, dt=self.dt), "ddelta": new(tok, self.H, dt=self.dt),
             "dB": new(tok, self.G, self.N, dt=self.dt), "dC": new(tok, self.G, self.N, dt=self.dt),
             "dA": new(self.H), "dDskip": new(self.H), "ddt_bias": new(self.H),
             "dh0": new(S, self.H, self.P, self.N)}
        ssm.ssm_head_scan_bwd(self.gu, self.g(self.delta), self.g(self.A), self.gB, self.gC,
                              self.dy.cuda(), g, Dskip=self.g(self.D), dt_bias=self.g(self.bias),
                              delta_softplus=self.sp, h0=self.g(self.h0), dh_final=self.g(self.dhf),
                              cu_seqlens=None if dense else self.cu, S=S, workspace=self.ws(True))
        return g

    def size(self, bwd=False):
        """The sizes that bf16 roundings go by (None: nothing is rounded)."""
        if self.dt != BF:
            return {}
        return ho.sizes(*self.ref_args(), *((self.dy.double(), self.f(self.dhf)) if bwd else ()))

    def check_fwd(self, y, hf):
        ry, rh = ho.scan(*self.ref_args())
        ho.close(y, ry, self.dt == BF, 1e-4, "y", self.size().get("y"))
        ho.close(hf, rh, False, 1e-4, "h_final")

    def check_bwd(self, g):
        r = ho.scan_bwd(*self.ref_args(), self.dy.double(), self.f(self.dhf))
        size = self.size(bwd=True)
        for k in ("du", "ddelta", "dB", "dC"):
            ho.close(g[k], r[k], self.dt == BF, 1e-4, k, size.get(k))
        ho.close(g["dh0"], r["dh0"], False, 1e-4, "dh0")
        # sums over tokens: against the size of what is summed, which their rounding goes by
        for k, size in (("dA", r["dA_size"]), ("ddt_bias", r["dbias_size"])):
            off = (g[k].double().cpu() - r[k]).abs()
            lim = (1e-5 if k == "dA" else 1e-4) * size + 1e-6
            assert (off <= lim).all(), f"{k}: off by {(off / lim).max():.3g} x the bound"
        ho.close(g["dDskip"], r["dDskip"], False, 1e-4, "dDskip")


SHAPES = [
    # lens, H, P, G, N
    ([1], 1, 64, 1, 128),
    ([17], 3, 64, 1, 128),
    ([128], 2, 64, 1, 128),
    ([129], 2, 64, 2, 64),
    ([5, 0, 130, 1, 31], 4, 64, 2, 128),
    ([300], 6, 32, 3, 16),
    ([260, 40], 2, 128, 1, 128),
    ([77, 90], 3, 48, 1, 96),
    ([33, 64, 7], 2, 37, 1, 19),
    ([140], 2, 200, 2, 128),
    ([0, 0], 2, 64, 1, 128),
]


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, [sum(s[0]), *s[1:]])))
def test_forward(shape, dt):
    c = Case(*shape, dt)
    c.check_fwd(*c.fwd())
    assert ssm.ssm_device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, [sum(s[0]), *s[1:]])))
def test_backward(shape, dt):
    c = Case(*shape, dt, seed=1)
    c.check_bwd(c.bwd())
    assert ssm.ssm_device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(h0=False, D=False, bias=False), dict(sp=False), dict(sliced=True),
                                dict(sliced=True, pad=3), dict(decay=(200.0, 3000.0)),
                                dict(decay=(0.0, 1e-3))],
                         ids=["bare", "no_softplus", "sliced", "odd_stride", "resets", "no_decay"])
def test_options(kw, dt):
    c = Case([150, 9], 4, 64, 2, 64, dt, seed=2, **kw)
    c.check_fwd(*c.fwd())
    c.check_bwd(c.bwd())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_dense_rows_equal_packed_rows(dt):
    c = Case([131, 131, 131], 3, 64, 1, 128, dt, seed=3)
    for a, b in zip(c.fwd(), c.fwd(dense=True)):
        assert torch.equal(a, b)
    p, d = c.bwd(), c.bwd(dense=True)
    assert all(torch.equal(p[k], d[k]) for k in p)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_same_bits_twice_and_state_in_place(dt):
    c = Case([400, 3, 150], 8, 64, 2, 128, dt, seed=4)
    y, hf = c.fwd()
    h = c.g(c.h0).clone()
    y2, h2 = c.fwd(h_final=h, h0=h)
    assert torch.equal(y, y2) and torch.equal(hf, h2)
    a, b = c.bwd(), c.bwd()
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_sequences_do_not_touch_each_other(dt):
    """NaN and infinity in one sequence stay there, tokens behind the last sequence and
    rows of an empty one keep what they hold."""
    c = Case([70, 0, 140, 60], 2, 64, 1, 64, dt, seed=5)
    y, hf = c.fwd()
    g = c.bwd()
    c.gu[80] = float("nan")
    c.gB[90] = float("inf")
    c.dy[81] = float("nan")
    y2, hf2 = c.fwd()
    g2 = c.bwd()
    keep = [i for i in range(270) if not 70 <= i < 210]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(hf[[0, 1, 3]], hf2[[0, 1, 3]])
    for k in ("du", "ddelta", "dB", "dC"):
        assert torch.equal(g[k][keep], g2[k][keep]), k
    assert torch.equal(g["dh0"][[0, 1, 3]], g2["dh0"][[0, 1, 3]])
    # the last sequence ends early: its tail is nobody's
    c = Case([70, 60], 2, 64, 1, 64, dt, seed=6)
    cu = c.cu.clone()
    cu[2] = 100
    c.cu = cu
    y3, _ = c.fwd(y_fill=3.0)
    assert (y3[100:] == 3.0).all()
    c.lens = [70, 30]
    c.u, c.delta, c.B, c.C = c.u[:100], c.delta[:100], c.B[:100], c.C[:100]
    c.h0 = c.h0[:2]
    ry, _ = ho.scan(*c.ref_args())
    ho.close(y3[:100], ry, dt == BF, 1e-4, "y", c.size().get("y"))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_chunks_carry_the_state(dt):
    """A prompt in three calls, the state carried in place, equals one call."""
    c = Case([700], 4, 64, 1, 128, dt, seed=7)
    c.check_fwd(*c.fwd())
    h = c.g(c.h0).clone()
    ys = []
    for lo, hi in ((0, 256), (256, 301), (301, 700)):
        y = torch.empty((hi - lo, 4, 64), dtype=dt, device="cuda")
        n = ssm.ssm_head_scan_workspace_size(hi - lo, 4, 64, 1, 128, 1, dt)
        ssm.ssm_head_scan_fwd(c.gu[lo:hi], c.g(c.delta)[lo:hi], c.g(c.A), c.gB[lo:hi], c.gC[lo:hi], y,
                              Dskip=c.g(c.D), dt_bias=c.g(c.bias), h0=h, h_final=h,
                              workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
        ys.append(y)
    # chunks start with each call, so the calls' own roundings are the sizes of three sequences
    ry, rh = ho.scan(*c.ref_args())
    size = None
    if dt == BF:
        parts, start = [], c.f(c.h0)
        for lo, hi in ((0, 256), (256, 301), (301, 700)):
            a = list(c.ref_args())
            for i in (0, 1, 3, 4):
                a[i] = a[i][lo:hi]
            a[8], a[9] = start, [hi - lo]
            parts.append(ho.sizes(*a)["y"])
            start = ho.scan(*a)[1]
        size = torch.cat(parts)
    ho.close(torch.cat(ys), ry, dt == BF, 1e-4, "y", size)
    ho.close(h, rh, False, 1e-4, "h_final")


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 64, 1, 128), (5, 6, 64, 3, 128), (3, 4, 48, 1, 37),
                                   (7, 2, 128, 2, 16), (2, 2, 200, 1, 64), (4, 3, 1, 1, 1)])
def test_decode_token(shape, dt):
    Bt, H, P, G, N = shape
    c = Case([1] * Bt, H, P, G, N, dt, seed=8)
    ry, rh = ho.scan(*c.ref_args())
    st = torch.full((Bt + 2, H, P, N), 9.0, device="cuda")
    order = torch.randperm(Bt + 2, generator=torch.Generator().manual_seed(1))[:Bt]
    st[order.cuda()] = c.g(c.h0)
    y = torch.empty((Bt, H, P), dtype=dt, device="cuda")
    ssm.ssm_head_state_update(st, c.gu, c.g(c.delta), c.gB, c.gC, y, c.g(c.A), Dskip=c.g(c.D),
                              dt_bias=c.g(c.bias), state_indices=order.to(torch.int32).cuda())
    # no product is rounded here: fp32 throughout, bf16 only where y is stored
    ho.close(y, ry, dt == BF, 1e-4, "y")
    ho.close(st[order.cuda()], rh, False, 1e-4, "state")
    others = [i for i in range(Bt + 2) if i not in order.tolist()]
    assert (st[others] == 9.0).all()


def test_decode_skips_rows_without_a_slot():
    c = Case([1] * 4, 2, 64, 1, 128, BF, seed=9)
    st = c.g(c.h0).clone()
    y = torch.full((4, 2, 64), 3.0, dtype=BF, device="cuda")
    idx = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    ssm.ssm_head_state_update(st, c.gu, c.g(c.delta), c.gB, c.gC, y, c.g(c.A), state_indices=idx)
    assert (y[[1, 2]] == 3.0).all() and (y[[0, 3]] != 3.0).any()
    assert torch.equal(st[[1, 3]], c.g(c.h0)[[1, 3]])


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_prompt_then_tokens(dt):
    """What a server does: a prompt through the scan, then tokens one by one in a captured
    graph, equals the whole text through the scan."""
    T, n = 150, 6
    c = Case([T + n], 4, 64, 2, 64, dt, seed=10)
    ry, rh = ho.scan(*c.ref_args())
    d, A, D, b = c.g(c.delta), c.g(c.A), c.g(c.D), c.g(c.bias)
    h = c.g(c.h0).clone()
    y = torch.empty((T, 4, 64), dtype=dt, device="cuda")
    ws = c.ws(False)
    ssm.ssm_head_scan_fwd(c.gu[:T], d[:T], A, c.gB[:T], c.gC[:T], y, Dskip=D, dt_bias=b, h0=h,
                          h_final=h, workspace=ws)
    x1, d1, B1, C1 = (t[T:T + 1].clone() for t in (c.gu, d, c.gB, c.gC))
    y1 = torch.empty((1, 4, 64), dtype=dt, device="cuda")
    keep = h.clone()

    def step():
        ssm.ssm_head_state_update(h, x1, d1, B1, C1, y1, A, Dskip=D, dt_bias=b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    h.copy_(keep)
    ys = [y]
    for i in range(n):
        for dst, src in ((x1, c.gu), (d1, d), (B1, c.gB), (C1, c.gC)):
            dst.copy_(src[T + i:T + i + 1])
        graph.replay()
        ys.append(y1.clone())
    # the prompt's chunks are the whole text's, and a token by itself rounds nothing
    ho.close(torch.cat(ys), ry, dt == BF, 1e-4, "y", c.size().get("y"))
    ho.close(h, rh[0:1], False, 1e-4, "state")


def test_two_captured_graphs_and_another_stream():
    """Two captured training steps with workspaces of their own, replayed on two streams."""
    cases = [Case([260, 40], 4, 64, 2, 128, BF, seed=s) for s in (11, 12)]
    want = [(c.fwd(), c.bwd()) for c in cases]
    runs = []
    for c in cases:
        S, tok = 2, 300
        d, A, D, b, dy = c.g(c.delta), c.g(c.A), c.g(c.D), c.g(c.bias), c.dy.cuda()
        h0, dhf, ws, wsb = c.g(c.h0), c.g(c.dhf), c.ws(False), c.ws(True)
        y, hf = torch.empty_like(c.gu), torch.empty_like(h0)
        g = {k: torch.empty_like(v) for k, v in c.bwd().items()}

        def go(c=c, d=d, A=A, D=D, b=b, dy=dy, h0=h0, dhf=dhf, ws=ws, wsb=wsb, y=y, hf=hf, g=g):
            ssm.ssm_head_scan_fwd(c.gu, d, A, c.gB, c.gC, y, Dskip=D, dt_bias=b, h0=h0, h_final=hf,
                                  cu_seqlens=c.cu, workspace=ws)
            ssm.ssm_head_scan_bwd(c.gu, d, A, c.gB, c.gC, dy, g, Dskip=D, dt_bias=b, h0=h0,
                                  dh_final=dhf, cu_seqlens=c.cu, workspace=wsb)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        runs.append((graph, y, hf, g))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                r[0].replay()
    torch.cuda.synchronize()
    for (fw, bw), (_, y, hf, g) in zip(want, runs):
        assert torch.equal(fw[0], y) and torch.equal(fw[1], hf)
        assert all(torch.equal(bw[k], g[k]) for k in g)


def test_malformed_cu_seqlens_stays_in_bounds():
    """Offsets that decrease or leave [0, tok] give wrong values, never an access outside."""
    c = Case([100, 100], 2, 64, 1, 64, BF, seed=13)
    for bad in ([0, 500, 200], [0, 150, 50], [-7, 90, 1 << 30], [200, 100, 0]):
        c.cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c.fwd()
        c.bwd()
    torch.cuda.synchronize()
