"""What the Python binding refuses before a pointer reaches the library: tensors that the
library would read as something else, or past their end. Host memory throughout."""

import pytest
import torch

import selective_state_space_causal_b200 as ssm

z = torch.zeros


def cu(*offsets, dt=torch.int32):
    return torch.tensor(offsets, dtype=dt)


BAD_CU = [dict(cu_seqlens=cu(0, 2, 6, dt=torch.int64)), dict(cu_seqlens=cu(0, 2, 6).float()),
          dict(cu_seqlens=cu(0, 9, 2, 9, 6, 9)[::2]), dict(cu_seqlens=cu(0, 2, 6)[None]), dict(cu_seqlens=cu(0, 2, 6), S=3)]


def head_scan(way, **kw):
    tok, H, P, G, N = 6, 2, 8, 1, 4
    args = z(tok, H, P), z(tok, H), z(H), z(tok, G, N), z(tok, G, N), z(tok, H, P)
    if way == "fwd":
        return ssm.ssm_head_scan_fwd(*args, stream=0, **kw)
    grads = {"du": z(tok, H, P), "ddelta": z(tok, H), "dB": z(tok, G, N), "dC": z(tok, G, N), "dA": z(H)}
    return ssm.ssm_head_scan_bwd(*args, grads, stream=0, **kw)


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("kw", BAD_CU, ids=["int64", "float", "strided", "two_dims", "too_few"])
def test_head_scan_refuses_cu_seqlens(way, kw):
    with pytest.raises(ssm.SsmError, match="cu_seqlens"):
        head_scan(way, **kw)


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("kw", [dict(cu_seqlens=cu(0, 2, 6)), dict(cu_seqlens=cu(0, 2, 6, 6), S=2), dict(S=2)])
def test_head_scan_takes_good_sequences(way, kw):
    """The next thing in the way is that these tensors are in host memory."""
    with pytest.raises(ssm.SsmError, match="not on the current CUDA device"):
        head_scan(way, **kw)
