"""Plain 64-bit forms of the scan with one decay per head and of the block norms,
on the CPU, token by token, and the bounds that the GPU results are held to.

Bounds. The kernels keep states, decays and sums in fp32. With fp32 activations every
product and sum is fp32 too: a sum of n terms of like size is off by about
sqrt(n) 2^-24 of its own size (n <= a few thousand here, so below 4e-6), a decay's
exponent by 2^-24 of its size (below 1e-5 at exponents of 100); 1e-4 of the tensor's
rms covers both.

With bf16 activations one factor of each product is rounded to bf16 once: inside a
chunk of 128 tokens the weights M = (C.B) decay d (for y and du) or dM decay d (for dB
and dC), across chunks the state that a chunk starts from (or its gradient). bf16 keeps
8 bits, so a rounded factor is off by at most 2^-8 of itself, and a sum of products
with it by at most 2^-8 of the sum of the products' sizes, which `sizes` computes
element by element. A value stored in bf16 is off by half a step on top, 2^-8 of it.
(A fixed fraction of the tensor's rms is no bound: heads with large steps d have
outputs, and so roundings, many times the rms.) Outputs kept in fp32 (states,
gradients of A, of the biases and of D) are products of the given inputs and unrounded
weights, and are held to 1e-4.
"""

import numpy as np
import torch

F64 = torch.float64


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def bounds_of(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def scan(u, delta, A, B, C, D, bias, sp, h0, lens):
    """y, final states; every tensor float64 on the CPU. Works under autograd."""
    tok, H, P = u.shape
    G, N = B.shape[1:]
    rep = H // G
    raw = delta + (bias if bias is not None else 0.0)
    d = softplus(raw) if sp else raw
    a = torch.exp(d * A)
    ys, finals = [], []
    for s, (lo, hi) in enumerate(bounds_of(lens)):
        h = h0[s] if h0 is not None else torch.zeros((H, P, N), dtype=F64)
        for t in range(lo, hi):
            Bt, Ct = B[t].repeat_interleave(rep, 0), C[t].repeat_interleave(rep, 0)
            h = a[t][:, None, None] * h + (d[t][:, None] * u[t])[:, :, None] * Bt[:, None, :]
            y = (h * Ct[:, None, :]).sum(-1)
            if D is not None:
                y = y + D[:, None] * u[t]
            ys.append(y)
        finals.append(h)
    y = torch.stack(ys) if ys else torch.zeros((0, H, P), dtype=F64)
    return y, torch.stack(finals)


def scan_bwd(u, delta, A, B, C, D, bias, sp, h0, lens, dy, dhf):
    """Every gradient by the chain rule through the recurrence, written out, and for
    dA the sum of its terms' sizes (what its rounding error goes by)."""
    tok, H, P = u.shape
    G, N = B.shape[1:]
    rep = H // G
    raw = delta + (bias if bias is not None else 0.0)
    d = softplus(raw) if sp else raw
    slope = torch.sigmoid(raw) if sp else torch.ones_like(raw)
    a = torch.exp(d * A)
    g = {"du": torch.zeros_like(u), "dB": torch.zeros_like(B), "dC": torch.zeros_like(C),
         "ddelta": torch.zeros_like(delta), "dA": torch.zeros(H, dtype=F64),
         "dh0": torch.zeros((len(lens), H, P, N), dtype=F64)}
    size = torch.zeros(H, dtype=F64)
    for s, (lo, hi) in enumerate(bounds_of(lens)):
        h = h0[s] if h0 is not None else torch.zeros((H, P, N), dtype=F64)
        states = [h]
        for t in range(lo, hi):
            Bt = B[t].repeat_interleave(rep, 0)
            h = a[t][:, None, None] * h + (d[t][:, None] * u[t])[:, :, None] * Bt[:, None, :]
            states.append(h)
        gh = dhf[s].clone() if dhf is not None else torch.zeros((H, P, N), dtype=F64)
        for t in reversed(range(lo, hi)):
            Bt, Ct = B[t].repeat_interleave(rep, 0), C[t].repeat_interleave(rep, 0)
            prev, now = states[t - lo], states[t - lo + 1]
            g["dC"][t] = (now * dy[t][:, :, None]).sum(1).view(G, rep, N).sum(1)
            gh = gh + dy[t][:, :, None] * Ct[:, None, :]
            gB = (gh * Bt[:, None, :]).sum(-1)
            g["du"][t] = d[t][:, None] * gB + (D[:, None] * dy[t] if D is not None else 0.0)
            g["dB"][t] = (gh * (d[t][:, None] * u[t])[:, :, None]).sum(1).view(G, rep, N).sum(1)
            dlog = (gh * a[t][:, None, None] * prev).sum((1, 2))
            g["ddelta"][t] = ((gB * u[t]).sum(-1) + A * dlog) * slope[t]
            g["dA"] += d[t] * dlog
            size += d[t].abs() * (gh * a[t][:, None, None] * prev).abs().sum((1, 2))
            gh = a[t][:, None, None] * gh
        g["dh0"][s] = gh
    g["dDskip"] = (dy * u).sum((0, 2))
    g["ddt_bias"] = g["ddelta"].sum(0)
    g["dA_size"] = size
    g["dbias_size"] = g["ddelta"].abs().sum(0)
    return g


CHUNK = 128


def sizes(u, delta, A, B, C, D, bias, sp, h0, lens, dy=None, dhf=None):
    """Per element, the sum of the sizes of the products with one rounded factor."""
    tok, H, P = u.shape
    G, N = B.shape[1:]
    rep = H // G
    raw = delta + (bias if bias is not None else 0.0)
    d = softplus(raw) if sp else raw
    out = {"y": torch.zeros_like(u), "du": torch.zeros_like(u), "dB": torch.zeros_like(B), "dC": torch.zeros_like(C)}
    for s, (lo, hi) in enumerate(bounds_of(lens)):
        cuts = [(a, min(a + CHUNK, hi)) for a in range(lo, hi, CHUNK)]
        per = []
        h = h0[s] if h0 is not None else torch.zeros((H, P, N), dtype=F64)
        for a, b in cuts:
            dc = d[a:b].t()                                   # (H, Q)
            c = torch.cumsum(dc * A[:, None], 1)
            Bh, Ch = (x[a:b].repeat_interleave(rep, 1).transpose(0, 1) for x in (B, C))  # (H, Q, N)
            uh = u[a:b].transpose(0, 1)
            L = torch.exp(c[:, :, None] - c[:, None, :]).tril() * dc[:, None, :]
            w = dc * torch.exp(c[:, -1:] - c)
            per.append((a, b, c, Bh, Ch, uh, L, w, h))
            h = torch.exp(c[:, -1])[:, None, None] * h + (w[..., None] * uh).transpose(1, 2) @ Bh
        for a, b, c, Bh, Ch, uh, L, w, h in per:
            M = (Ch @ Bh.transpose(1, 2)).abs() * L
            e = torch.exp(c)[..., None]
            out["y"][a:b] = (M @ uh.abs() + e * (Ch.abs() @ h.abs().transpose(1, 2))).transpose(0, 1)
        if dy is None:
            continue
        g = dhf[s] if dhf is not None else torch.zeros((H, P, N), dtype=F64)
        for a, b, c, Bh, Ch, uh, L, w, h in reversed(per):
            yh = dy[a:b].transpose(0, 1)
            e = torch.exp(c)[..., None]
            M = (Ch @ Bh.transpose(1, 2)).abs() * L
            out["du"][a:b] = (M.transpose(1, 2) @ yh.abs()).transpose(0, 1)
            X = (yh @ uh.transpose(1, 2)).abs() * L
            dC = X @ Bh.abs() + e * (yh.abs() @ h.abs())
            dB = X.transpose(1, 2) @ Ch.abs() + w[..., None] * (uh.abs() @ g.abs())
            for k, v in (("dC", dC), ("dB", dB)):
                out[k][a:b] = v.view(G, rep, b - a, N).sum(1).transpose(0, 1)
            g = torch.exp(c[:, -1])[:, None, None] * g + (e * yh).transpose(1, 2) @ Ch
    return out


def norm(v, group, eps):
    vg = v.reshape(v.shape[0], v.shape[1] // group, group)
    return (vg / torch.sqrt((vg * vg).mean(-1, keepdim=True) + eps)).reshape(v.shape)


def gated(x, z, w, group, eps, before):
    gate = z * torch.sigmoid(z) if z is not None else torch.ones_like(x)
    y = norm(x, group, eps) * gate if before else norm(x * gate, group, eps)
    return y * w if w is not None else y


def worst(gpu, ref, stored_bf16, tol, size=None):
    """Largest error over its bound: tol * rms(ref), plus half a bf16 step where stored so,
    plus 2^-8 of `size` where a factor was rounded."""
    g, r = gpu.detach().double().cpu().numpy(), ref.detach().double().numpy()
    assert g.shape == r.shape, (g.shape, r.shape)
    if r.size == 0:
        return 0.0
    if not np.isfinite(g).all():
        return float("inf")
    rms = float(np.sqrt(np.mean(r * r)))
    off = np.abs(g - r) - (2.0 ** -8 * np.abs(r) if stored_bf16 else 0.0)
    if size is not None:  # the half step is of the rounded value: 2^-8 (|r| + its error)
        off = off - 2.0 ** -8 * (1 + 2.0 ** -8) * size.numpy()
    return float(off.max()) / (tol * rms if rms else tol)


def close(gpu, ref, stored_bf16, tol, what, size=None):
    w = worst(gpu, ref, stored_bf16, tol, size)
    assert w <= 1.0, f"{what}: error is {w:.3g} x the bound"
