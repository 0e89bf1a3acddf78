"""The per-head calls refuse outputs that lie over inputs, whichever input it is (fake
addresses, nothing reaches a device)."""

import pytest

from test_head_scan_cpu import A16, M, _err, bwd, fwd, step

F = A16 + 40 * M  # free room
STATE = 2 * 64 * 64 * 4  # bytes of a sequence's state


@pytest.mark.parametrize("at", [0, M, 2 * M, 3 * M, 4 * M], ids=["u", "delta", "A", "B", "C"])
def test_final_state_over_an_input(at):
    for h0 in (None, F):
        assert fwd(h0=h0, hf=A16 + at) == -1
        assert "overlap" in _err()


@pytest.mark.parametrize("name", ["y", "hf", "ws"])
@pytest.mark.parametrize("kw", [dict(D=F), dict(b=F), dict(cu=F)], ids=["Dskip", "dt_bias", "cu_seqlens"])
def test_forward_outputs_over_small_inputs(name, kw):
    assert fwd(**kw, **{name: F}) == -1
    assert "overlap" in _err()


def test_forward_outputs_over_each_other_and_h0():
    assert fwd(hf=A16 + 5 * M) == -1 and "overlap" in _err()                  # y
    assert fwd(hf=A16 - A16 % 256 + 16 * M) == -1 and "overlap" in _err()     # workspace
    assert fwd(h0=F, hf=F + STATE - 4) == -1 and "overlap" in _err()          # h0, but not the same
    assert fwd(h0=F, hf=F, y=F + 128) == -1 and "overlap" in _err()           # y over the state in place


@pytest.mark.parametrize("name", ["du", "dd", "dB", "dC", "dA", "dD", "db", "dh0", "ws"])
def test_backward_outputs_over_cu_seqlens(name):
    assert bwd(cu=F, **{name: F}) == -1
    assert "overlap" in _err()


@pytest.mark.parametrize("kw", [dict(A=F), dict(D=F), dict(b=F), dict(idx=F)], ids=["A", "Dskip", "dt_bias", "state_indices"])
def test_decode_output_over_small_inputs(kw):
    assert step(y=F, **kw) == -1
    assert "overlap" in _err()
