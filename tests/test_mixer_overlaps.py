"""Which tensors of a call of the operators around the token mixers may share memory; no GPU: a call that
passes the checks fails at its launch (or, with a GPU, is not made here)."""
import pytest
import torch

import linear_attention_attn_b200 as la

MB = 1 << 24          # spacing of the made-up addresses
INVALID = 1
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")


def _call(f, names, args, over):
    at = {n: (i + 1) * MB for i, n in enumerate(names)}
    at.update(over)
    status = getattr(la.raw_lib(), f)(*(at[n] for n in names), *args)
    return status, la.raw_lib().la_last_error().decode()


def _rotary(f, **over):
    return _call(f, ["q", "k", "oq", "ok", "freqs", "pos"], (0, 0, 0, 1.0, 1, 2, 2, 4, 8, 8, 2, None), over)


@pytest.mark.parametrize("f", ["la_rotary_fwd", "la_rotary_bwd"])
def test_rotary_in_place_of_a_tensor_that_is_also_the_other_input(f):
    assert _rotary(f, oq=MB)[0] != INVALID and _rotary(f, ok=2 * MB)[0] != INVALID
    assert _rotary(f, oq=MB, ok=2 * MB)[0] != INVALID
    assert _rotary(f, k=MB)[0] != INVALID                 # one tensor for both inputs: only read
    status, text = _rotary(f, k=MB, oq=MB)                # k's heads would be read after oq is written
    assert status == INVALID and "overlaps" in text
    assert _rotary(f, k=MB, ok=MB)[0] == INVALID


def test_convolution_state_in_place_of_a_buffer_that_is_also_x():
    names = ["x", "w", "bias", "si", "y", "so", "len"]

    def conv(**over):
        return _call("la_short_conv_fwd", names, (1, 1, 3, 8, 4, 2, None), over)        # T = W - 1: x and the state fit
    assert conv(so=4 * MB)[0] != INVALID
    assert conv(si=MB)[0] != INVALID
    status, text = conv(si=MB, so=MB)
    assert status == INVALID and "overlaps" in text


def test_scan_state_in_place_of_a_buffer_that_is_also_another_input():
    names = ["x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "si", "y", "so", "len"]

    def scan(**over):
        return _call("la_selective_scan_fwd", names, (1, 1, 8, 8, 1, 4, 0, None, 0, None), over)      # f32, T = C
    assert scan(so=9 * MB)[0] != INVALID
    for other in ("Bm", "Cm", "A"):
        status, text = scan(so=9 * MB, **{other: 9 * MB})
        assert status == INVALID and "overlaps" in text, other


def test_norm_in_place():
    def fwd(**over):
        return _call("la_group_norm_fwd", ["x", "ga", "be", "y", "m", "r"], (1e-5, 1, 1, 1, 8, 2, 0, None, 0, None), over)
    assert fwd(y=MB)[0] != INVALID
    status, text = fwd(y=MB, ga=MB)                       # one row of x is as long as gamma
    assert status == INVALID and "overlaps" in text

    def bwd(**over):
        return _call("la_group_norm_bwd", ["x", "dy", "m", "r", "ga", "be", "dx", "dga", "dbe"],
                     (1, 1, 4, 8, 2, 2, 40 * MB, MB, None), over)
    assert bwd(dx=2 * MB)[0] != INVALID
    assert bwd(dy=MB, dx=MB)[0] != INVALID                # dy is x
    assert bwd(dx=MB)[0] == INVALID                       # in place of x alone is not offered
    assert bwd(dx=2 * MB, ga=2 * MB)[0] == INVALID
