"""Edges of the layers around the mixer: steps that a mask drives to the type's lowest value."""
import numpy as np
import pytest
import torch

from gated_delta_rule_wy_b200 import gdr2_ssm_scan, gdr2_ssm_scan_backward, gdr2_ssm_step, gdr2_sync_status
from layer_bounds import U, np64
from oracle import layers as OL
from test_gpu_ssm import backward, check_gradients, check_scan, cuda, make

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
SMALLEST = 2.0 ** -126  # results below it are zero


def slope_of_the_step(v):
    """ddt of one token per channel with x = B = 1, A = C = 0 and dS_T = 1 on one state: softplus'(v)."""
    C = v.numel()
    one, zero = torch.ones((1, 1, C), device="cuda"), torch.zeros((1, 1, 8), device="cuda")
    dS = torch.zeros((1, C, 8), device="cuda")
    dS[..., 0] = 1.0
    g = gdr2_ssm_scan_backward(one, v.view(1, 1, C).cuda(), torch.zeros((C, 8), device="cuda"), zero + 1.0, zero,
                               torch.zeros_like(one), dS_T=dS)
    gdr2_sync_status()
    return np64(g["ddt"][0, 0])


def test_slope_of_the_step_over_every_finite_step():
    """softplus' = e / (1 + e) or 1 / (1 + e), e = e^-|v|: 2^x 4 U and the product that puts its argument's rounding
    back 1 U, which the denominator has again by half at most and adds 1 U; the quotient 2 U, the last product
    1 U: 11.5 U at any v, and nothing below the smallest normal value."""
    v = torch.cat([torch.linspace(-130, 130, 8001), torch.tensor([-1e4, -3.3e38, -torch.inf, 1e4, 3.3e38])])
    r = np64(v)
    with np.errstate(over="ignore"):
        want = 1 / (1 + np.exp(-r))
    got = slope_of_the_step(v)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= 12 * U * want + SMALLEST)


def test_gates_over_every_finite_argument():
    """silu(z) and its slope below z = -80: both end in zero, and never in NaN. The terms are at most |z| sigma(z), and
    where sigma is below the smallest normal value |z| sigma is below 90 times that."""
    z = torch.cat([torch.linspace(-130, -80, 2001), torch.tensor([-1e4, -3.3e38])])
    C = z.numel()
    one, zero = torch.ones((1, 1, C), device="cuda"), torch.zeros((1, 1, 8), device="cuda")
    A, D, zc = torch.zeros((C, 8), device="cuda"), torch.ones(C, device="cuda"), z.view(1, 1, C).cuda()
    y, _, _ = gdr2_ssm_scan(one, one, A, zero + 1.0, zero, D, zc)
    g = gdr2_ssm_scan_backward(one, one, A, zero + 1.0, zero, one, D, zc)
    gdr2_sync_status()
    r = np64(z)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-r))
    limit = (2 * np.minimum(np.abs(r), 130) + 12) * U * s * (1 + np.abs(r)) + 96 * SMALLEST
    assert np.all(np.abs(np64(y[0, 0]) - r * s) <= limit)
    assert np.all(np.abs(np64(g["dz"][0, 0]) - s * (1 + r * (1 - s))) <= limit)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("step", [-89.0, -1e4, "lowest", -float("inf")])
@pytest.mark.parametrize("N", [16, 64])
def test_masked_steps_among_ordinary_ones(dtype, step, N):
    """A step of softplus(-large) = 0 leaves the state, and no gradient of it is anything but a number."""
    T, C = 70, 40
    v = make((2, T), C, N, dtype, 400, states=2)
    value = torch.finfo(dtype).min if step == "lowest" else step
    for b, t in ((0, 0), (0, 17), (0, 18), (1, 33), (1, T - 1)):
        v["dt"][b, t] = value
    dy = torch.randn((2, T, C), generator=torch.Generator().manual_seed(41)).to(dtype)
    dS = torch.randn((2, C, N), generator=torch.Generator().manual_seed(42))
    y, S_T, _ = gdr2_ssm_scan(**cuda(v))
    g = backward(v, dy, dS)
    gdr2_sync_status()
    for k in g:
        assert g[k].isfinite().all(), k
    check_scan(v, y, S_T, [((b,), b, T) for b in range(2)])
    check_gradients(v, dy, dS, g, T)
    for b, t in ((0, 17), (1, T - 1)):
        assert not g["ddt"][b, t].any()


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_growth_over_a_segment_leaves_zero(N):
    """A > 0: 32 steps grow by e^256, which fp32 does not hold. The state is zero until the last three tokens, and the
    state's gradient zero after the first three, so that nothing that is there grows: all is finite, as token by token."""
    T, C = 2000, 33
    v = make((1, T), C, N, torch.float32, 410, z=False, bias=False)
    v.update(A=torch.full((C, N), 8.0), dt=torch.ones((1, T, C)))
    v["x"][:, :-3] = 0.0
    dy = torch.randn((1, T, C), generator=torch.Generator().manual_seed(43))
    dy[:, 3:] = 0.0
    y, S_T, _ = gdr2_ssm_scan(**cuda(v), softplus=False)
    g = backward(v, dy, softplus=False)
    gdr2_sync_status()
    for name, t in (("y", y), ("S_T", S_T), *g.items()):
        assert t is None or t.isfinite().all(), name
    check_scan(v, y, S_T, [((0,), 0, T)], with_softplus=False)
    check_gradients(v, dy, None, g, T, with_softplus=False)
    assert not g["dS0"][..., 0].eq(0).all()


@pytest.mark.parametrize("sign", [1, -1])
def test_a_factor_beyond_fp32_whose_product_is_not(sign):
    """Exponents that sum to 130 (of 2) over 32 tokens in the middle, and steps of zero elsewhere: the state of 2^-125
    ends at 32, the one of 2^125 at 2^-5, wherever the segments' borders fall. The same for the state's gradient.

    One step: 2^x 4 U, its exponent 4 (2 U) and the product 1 U; the tokens' 32 steps, or one factor's four parts."""
    T, C, N = 2048, 40, 16
    A = torch.full((C, N), sign * 130 / 32 * 0.6931471805599453, device="cuda")
    n, x = torch.zeros((1, T, N), device="cuda"), torch.zeros((1, T, C), device="cuda")
    dt = torch.zeros((1, T, C), device="cuda")
    dt[:, T // 2:T // 2 + 32] = 1.0
    S0 = torch.full((1, C, N), 2.0 ** (-125 * sign), device="cuda")
    _, S_T, _ = gdr2_ssm_scan(x, dt, A, n, n, S0=S0, softplus=False)
    g = gdr2_ssm_scan_backward(x, dt, A, n, n, x, S0=torch.zeros_like(S0), dS_T=S0, softplus=False)
    gdr2_sync_status()
    want = np.exp(np64(A)[None] * 32) * np64(S0)
    for got in (S_T, g["dS0"]):
        assert np.all(np.abs(np64(got) - want) <= 32 * 16 * U * want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 16, 41, 64, 1500])
def test_states_that_forget_at_every_step(dtype, T):
    """An A of minus infinity: h_t = s_t B_t x_t alone, whether the last tile is full or not, and no gradient passes a
    token or reaches A. A finite one of the same effect gives the same."""
    C, N = 40, 16
    v = make((2, T), C, N, dtype, 420 + T, states=2)
    v["A"][:, ::3] = -float("inf")
    w = {**v, "A": v["A"].nan_to_num(neginf=-1e6)}
    dy = torch.randn((2, T, C), generator=torch.Generator().manual_seed(44)).to(dtype)
    dS = torch.randn((2, C, N), generator=torch.Generator().manual_seed(45))
    y, S_T, saved = gdr2_ssm_scan(**cuda(v), save_states=True)
    g, h = backward(v, dy, dS, saved_states=saved), backward(w, dy, dS)
    y2, S2, _ = gdr2_ssm_scan(**cuda(w))
    gdr2_sync_status()
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    assert all(torch.equal(g[k], h[k]) for k in g)
    check_scan(w, y, S_T, [((b,), b, T) for b in range(2)])
    check_gradients(w, dy, dS, g, T)
    S = v["S0"].cuda()
    d = cuda({k: t[:, 0].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in v.items() if k != "S0"})
    gdr2_ssm_step(**d, S=S)
    gdr2_sync_status()
    step = (torch.nn.functional.softplus(d["dt"].double() + d["dt_bias"].double()) * d["x"].double())[..., None]
    want = (step * d["Bm"].double()[:, None, :])[..., ::3]
    assert ((S[..., ::3].double() - want).abs() <= 96 * U * want.abs()).all()
