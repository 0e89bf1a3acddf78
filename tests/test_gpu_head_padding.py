"""Padded batches and masked tokens of the per-head scan: what stands behind the last sequence
is neither read into a result nor written, a token whose step is zero changes no state."""

import pytest
import torch

import head_oracle as ho
import selective_state_space_causal_b200 as ssm
from test_gpu_head_scan import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 64, 1, 128, 0), (4, 128, 2, 64, 0), (2, 64, 1, 64, 3), (2, 37, 1, 19, 0)],
                         ids=["64", "128", "odd_stride", "odd"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_padding_behind_the_last_sequence(shape, dt, bad):
    H, P, G, N, pad = shape
    live, rows = 200, 350  # 150 rows that belong to nobody, past the last chunk's end
    c = Case([70, 0, 60, rows - 130], H, P, G, N, dt, seed=30, sliced=pad > 0, pad=pad)
    c.cu = torch.tensor([0, 70, 70, 130, live], dtype=torch.int32, device="cuda")
    y, hf = c.fwd(y_fill=3.0)
    g = c.bwd()
    for t in (c.gu, c.gB, c.gC):
        t[live:] = bad
    c.delta[live:] = bad
    c.dy[live:] = bad
    y2, hf2 = c.fwd(y_fill=3.0)
    g2 = c.bwd()
    torch.cuda.synchronize()
    assert ssm.ssm_device_status() == 0
    assert torch.equal(y, y2) and torch.equal(hf, hf2) and torch.isfinite(y2[:live]).all()
    assert all(torch.equal(g[k], g2[k]) for k in g)
    assert (y2[live:] == 3.0).all()
    for k in ("du", "ddelta", "dB", "dC"):
        assert (g2[k][live:] == 7.0).all(), k


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("low", [float("-inf"), None], ids=["inf", "lowest"])
def test_masked_tokens_leave_the_state(dt, low):
    """A step of softplus(-inf) is zero: the token leaves the state as it is, reads it, and its
    delta gets no gradient. One sequence is masked throughout."""
    c = Case([140, 40, 33], 4, 64, 2, 128, dt, seed=31)
    value = torch.finfo(dt).min if low is None else low
    mask = torch.zeros(213, dtype=torch.bool)
    mask[::3] = True
    mask[140:180] = True
    c.delta[mask] = value
    y, hf = c.fwd()
    g = c.bwd()
    # in 64 bits the lowest fp32 value is no step either, and -inf has no defined gradient there
    c.delta = torch.where(mask[:, None], torch.tensor(-1e30 if dt == F32 else torch.finfo(BF).min), c.delta.float()).to(dt)
    c.check_fwd(y, hf)
    c.check_bwd(g)
    assert (g["ddelta"][mask.cuda()] == 0).all()
    assert torch.equal(hf[1], c.g(c.h0)[1])


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_longer_cu_seqlens_with_s_given(dt):
    """S may be less than the offsets allow: the first S sequences are taken."""
    c = Case([30, 100, 20], 2, 64, 1, 64, dt, seed=32)
    y, hf = c.fwd()
    c.cu = torch.cat([c.cu, torch.full((5,), 150, dtype=torch.int32, device="cuda")])
    y2, hf2 = c.fwd()
    assert torch.equal(y, y2) and torch.equal(hf, hf2)
    ho.close(y2, ho.scan(*c.ref_args())[0], dt == BF, 1e-4, "y", c.size().get("y"))
