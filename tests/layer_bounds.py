"""Bounds for the layers around the mixer, derived from the number of fp32 roundings.

Every output is a sum of products; ``scale`` is the sum of the absolute values of its terms (the
oracle's ``absolute`` form). One fp32 rounding moves a term by at most U = 2^-24 of itself. A
fast function (2^x, quotient, reciprocal root) is within 2^-22 = 4 U, and an exponent of size E
adds 2 E U through the roundings of the step size and the product; the tests keep E <= 8.
So one step of a recurrence costs at most 4 + 16 + 4 = 24 U of the state, a term that
passed T steps 24 T U, and the ends (softplus, silu, its slope, the sums over N, the skip) are
covered by 96 U more; sums over n terms in any order add n U. A store in bf16 adds half a step,
at most 2^-8 of the value.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def assert_bound(got, ref, scale, roundings, what):
    """|got - ref| <= roundings U scale + the half step of got's type, elementwise."""
    g = np64(got)
    ref, scale = np.asarray(ref), np.asarray(scale)
    assert g.shape == ref.shape == scale.shape, (what, g.shape, ref.shape, scale.shape)
    if g.size == 0:
        return
    # fp32 ends at 3e38, and a scan with steps of the sign that grows passes it (1e183 after 70 tokens).
    # A term is a state, or its gradient, times inputs, which are above 1e-8 in size here: where the
    # terms stay below 1e30 those states stay below 1e38; elsewhere there is no fp32 value to compare.
    held = scale < 1e30
    g, ref, scale = g[held], ref[held], scale[held]
    if g.size == 0:
        return
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    arithmetic = roundings * U * scale
    limit = arithmetic + HALF_STEP[got.dtype] * (np.abs(ref) + arithmetic) + 1e-37
    over = np.abs(g - ref) / limit
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 1.0, f"{what}: {over[at]:.2f} of the bound at {at}: got {g[at]!r}, expected {ref[at]!r}"


def recurrence(T, sums=0):
    """Roundings of a value that passed T steps of the scan, and sums of `sums` terms."""
    return 24 * T + 96 + sums
