"""What the Python binding refuses before a pointer reaches the library: tensors that the
library would read as something else, or past their end. Host memory throughout."""

import pytest
import torch

import selective_state_space_causal_b200 as ssm

z = torch.zeros


def cu(*offsets, dt=torch.int32):
    return torch.tensor(offsets, dtype=dt)


BAD_CU = [dict(cu_seqlens=cu(0, 2, 6, dt=torch.int64)), dict(cu_seqlens=cu(0, 2, 6).float()),
          dict(cu_seqlens=cu(0, 9, 2, 9, 6, 9)[::2]), dict(cu_seqlens=cu(0, 2, 6), S=3)]


def head_scan(way, **kw):
    tok, H, P, G, N = 6, 2, 8, 1, 4
    args = z(tok, H, P), z(tok, H), z(H), z(tok, G, N), z(tok, G, N), z(tok, H, P)
    if way == "fwd":
        return ssm.ssm_head_scan_fwd(*args, stream=0, **kw)
    grads = {"du": z(tok, H, P), "ddelta": z(tok, H), "dB": z(tok, G, N), "dC": z(tok, G, N), "dA": z(H)}
    return ssm.ssm_head_scan_bwd(*args, grads, stream=0, **kw)


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("kw", BAD_CU, ids=["int64", "float", "strided", "too_few"])
def test_head_scan_refuses_cu_seqlens(way, kw):
    with pytest.raises(ssm.SsmError, match="cu_seqlens"):
        head_scan(way, **kw)


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("kw", [dict(cu_seqlens=cu(0, 2, 6)), dict(cu_seqlens=cu(0, 2, 6, 6), S=2), dict(cu_seqlens=cu(0, 2, 6)[None]), dict(S=2)])
def test_head_scan_takes_good_sequences(way, kw):
    """The next thing in the way is that these tensors are in host memory."""
    with pytest.raises(ssm.SsmError, match="not on the current CUDA device"):
        head_scan(way, **kw)


def channel_call(name, **kw):
    """The calls with a decay per channel; `tok` tokens of `D` channels."""
    tok, D, N, K = 6, 8, 16, 4
    r, bc, A, w = z(tok, D), z(tok, N), z(D, N), z(D, K)
    if name == "conv":
        return ssm.ssm_causal_conv1d(r, z(tok, D), w, stream=0, **kw)
    if name == "conv_scan":
        return ssm.ssm_conv_scan_fwd(r, w, r, A, bc, bc, z(tok, D), stream=0, **kw)
    if name == "bwd":
        grads = {"du": z(tok, D), "ddelta": z(tok, D), "dB": z(tok, N), "dC": z(tok, N), "dA": z(D, N)}
        return ssm.ssm_selective_scan_bwd(r, r, A, bc, bc, r, grads, stream=0, **kw)
    fn = {"fwd": ssm.ssm_selective_scan_fwd, "noalloc": ssm.ssm_selective_scan_fwd_noalloc,
          "ckpt": ssm.ssm_selective_scan_fwd_ckpt}[name]
    more = (z(64, dtype=torch.uint8),) if name == "ckpt" else ()
    return fn(r, r, A, bc, bc, z(tok, D), *more, stream=0, **kw)


@pytest.fixture
def no_launch(monkeypatch):
    """Nothing gets past the binding: a call that does returns the sequences it was given."""
    import ctypes

    from selective_state_space_causal_b200 import _lib

    class Stub:
        def __getattr__(self, name):
            at = [i for i, t in enumerate(dict((n, a) for n, _, a in _lib.SIGNATURES)[name]) if t is ctypes.c_int64]

            def fn(*args):
                Stub.got = [args[i] for i in at]
                return 0
            return fn

    monkeypatch.setattr(_lib, "lib", Stub())
    return Stub


CHANNEL = ["conv", "fwd", "ckpt", "noalloc", "bwd", "conv_scan"]


@pytest.mark.parametrize("name", CHANNEL)
@pytest.mark.parametrize("kw", BAD_CU, ids=["int64", "float", "strided", "too_few"])
def test_channel_calls_refuse_cu_seqlens(no_launch, name, kw):
    with pytest.raises(ssm.SsmError, match="cu_seqlens"):
        channel_call(name, **kw)


@pytest.mark.parametrize("name", CHANNEL)
@pytest.mark.parametrize("kw,S", [(dict(), 1), (dict(S=3), 3), (dict(cu_seqlens=cu(0, 2, 6)), 2), (dict(cu_seqlens=cu(0, 2, 6, 6), S=2), 2),
                                  (dict(cu_seqlens=cu(0, 2, 6)[None]), 2), (dict(cu_seqlens=1 << 20, S=5), 5)],
                         ids=["one", "dense", "packed", "longer", "two_dims", "address"])
def test_channel_calls_take_good_sequences(no_launch, name, kw, S):
    channel_call(name, **kw)
    assert S in no_launch.got


BYTES = z(64, dtype=torch.uint8)


@pytest.mark.parametrize("ws", [BYTES[:1].expand(1 << 30), BYTES[::2]], ids=["repeats", "skips"])
@pytest.mark.parametrize("name", ["fwd", "ckpt", "bwd", "head_fwd", "head_bwd", "gated", "residual"])
def test_workspaces_in_one_piece(no_launch, monkeypatch, name, ws):
    """A view's elements are not the bytes that lie behind its address."""
    from selective_state_space_causal_b200 import _lib

    monkeypatch.setattr(_lib, "_on_gpu", lambda *t: None)
    with pytest.raises(ssm.SsmError, match="contiguous"):
        if name.startswith("head"):
            head_scan(name[5:], workspace=ws)
        elif name == "gated":
            ssm.ssm_gated_norm_bwd(z(4, 8), z(4, 8), {"dx": z(4, 8), "dweight": z(8)}, workspace=ws, stream=0)
        elif name == "residual":
            ssm.ssm_residual_norm_bwd(z(4, 8), z(4, 8), {"dweight": z(8)}, workspace=ws, stream=0)
        else:
            channel_call(name, workspace=ws)
    if name == "ckpt":
        with pytest.raises(ssm.SsmError, match="contiguous"):
            a = z(6, 8), z(6, 8), z(8, 16), z(6, 16), z(6, 16), z(6, 8)
            ssm.ssm_selective_scan_fwd_ckpt(*a, ws, stream=0)


def test_addresses_of_an_int_subclass():
    class Address(int):
        pass

    from selective_state_space_causal_b200._lib import _ptr

    assert _ptr(Address(64)) == 64 and _ptr(64) == 64 and _ptr(None) is None
    assert _ptr(BYTES) == BYTES.data_ptr()
