"""Precision of the scan beyond what bounds that grow with the length can show: the elementwise laws with bounds that do
not grow with their argument, decays without a mean error, and errors over a long memory beside those of the
elementary fp32 form; and the scan without softplus where every value is compared."""
import numpy as np
import pytest
import torch

from gated_delta_rule_wy_b200 import gdr2_ssm_scan, gdr2_ssm_scan_backward, gdr2_ssm_step, gdr2_sync_status
from layer_bounds import U, np64
from oracle import layers as OL
from test_gpu_ssm import backward, check_gradients, check_scan, cuda, make

pytestmark = pytest.mark.gpu


def test_step_sizes_at_every_size():
    """Below zero: e = e^v 5 U (2^x 4, and 1 of the product that puts its argument's rounding back), e / (2 + e) 5.7 U more
    (the sum a third of 5 and 1, the quotient 2, a product 1), the polynomial 2.3 U, a product 1 U: 14 U. Above zero v
    itself is added, and the terms only shrink."""
    v = torch.cat([torch.linspace(-120, 120, 8001), torch.tensor([0.0, 1e-6, -1e-6, 1e-30, -1e-30, 3e38, -3e38])])
    C = v.numel()
    x, n = torch.ones((1, 1, C), device="cuda"), torch.ones((1, 1, 8), device="cuda")
    A = torch.zeros((C, 8), device="cuda")
    _, S, _ = gdr2_ssm_scan(x, v.view(1, 1, C).cuda(), A, n, n)
    S1 = torch.zeros((1, C, 8), device="cuda")
    gdr2_ssm_step(x[0], v.view(1, C).cuda(), A, n[0], n[0], S1)
    gdr2_sync_status()
    ref = OL.softplus(np64(v))
    for got in (S[0, :, 3], S1[0, :, 7]):
        assert np.all(np.abs(np64(got) - ref) <= 16 * U * ref + 2.0 ** -126)


@pytest.mark.parametrize("lo,hi", [(0.01, 0.1), (0.1, 0.5)])
def test_decays_have_no_mean_error(lo, hi):
    """The special-function unit's own mean is 0.35 U low, which a long memory adds up. Half a million decays: the mean
    of errors of 0.7 U at most has a deviation of 0.001 U, and less than half of the unit's own may be left."""
    C, N = 1 << 15, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.rand(s, device="cuda", generator=g)  # noqa: E731
    A = -torch.exp(rand(C, N) * 2)
    d = (lo + (hi - lo) * rand(1, C)) / 3
    S, z, n = torch.ones((1, C, N), device="cuda"), torch.zeros((1, C), device="cuda"), torch.zeros((1, N), device="cuda")
    gdr2_ssm_step(z, d, A, n, n, S, softplus=False)
    gdr2_sync_status()
    ref = torch.exp(d[0, :, None].double() * A.double())
    assert abs(((S[0].double() - ref) / ref).mean().item()) <= 0.15 * U


def elementary(x, d, A, B, C, dy, dS, dtype):
    """The recurrence and its gradients by elementary operations in `dtype`, token by token: one sequence."""
    x, d, A, B, C, dy, e = (t.to(dtype) for t in (x, d, A, B, C, dy, dS))
    h, before, ys = torch.zeros_like(A), [], []
    for t in range(x.shape[0]):
        before.append(h)
        h = torch.exp(d[t][:, None] * A) * h + (d[t] * x[t])[:, None] * B[t][None]
        ys.append((h * C[t][None]).sum(1))
    dA, S_T = torch.zeros_like(A), h
    for t in reversed(range(x.shape[0])):
        e = torch.exp(d[t][:, None] * A) * (e + dy[t][:, None] * C[t][None])
        dA = dA + d[t][:, None] * (e * before[t])
    return {"y": torch.stack(ys), "S_T": S_T, "dA": dA, "dS0": e}


def test_errors_over_a_long_memory_are_those_of_fp32():
    """4000 tokens, decays of 0.01 to 0.08 (a memory of 12 to 100 tokens) and nothing that cancels. Both forms round
    a decay by half a unit or a little more and the state once or twice per token; the kernel may have half as much
    again as the elementary one, and 2 U. (A mean error of 0.35 U per decay would be ten times that.)"""
    T, C, N = 4000, 64, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.rand(s, device="cuda", generator=g)  # noqa: E731
    x, d, Bm, Cm, dy = rand(T, C) + 0.5, 0.01 + 0.01 * rand(T, C), rand(T, N) + 0.5, rand(T, N) + 0.5, rand(T, C) + 0.5
    A, dS = -(1 + 3 * rand(C, N)), rand(C, N) + 0.5
    one = elementary(x, d, A, Bm, Cm, dy, dS, torch.float32)
    ref = elementary(x, d, A, Bm, Cm, dy, dS, torch.float64)
    b = lambda t: t[None].contiguous()  # noqa: E731
    y, S_T, saved = gdr2_ssm_scan(b(x), b(d), A, b(Bm), b(Cm), softplus=False, save_states=True)
    k = gdr2_ssm_scan_backward(b(x), b(d), A, b(Bm), b(Cm), b(dy), dS_T=b(dS), saved_states=saved, softplus=False)
    gdr2_sync_status()
    got = {"y": y[0], "S_T": S_T[0], "dA": k["dA"], "dS0": k["dS0"][0]}
    for name, want in ref.items():
        rms = [((v[name].double() - want) / want).pow(2).mean().sqrt().item() for v in (got, one)]
        assert rms[0] <= 1.5 * rms[1] + 2 * U, (name, rms[0] / U, rms[1] / U)


def all_held(v, dy, dS, **kw):
    """That no value is left out of a comparison: every scale below 1e30."""
    for i in range(dy.shape[0]):
        p = lambda k: None if v[k] is None else np64(v[k][i])  # noqa: E731,B023
        scale = OL.ssm_backward(p("x"), p("dt"), np64(v["A"]), p("Bm"), p("Cm"), np64(dy[i]), np64(v["D"]), p("z"),
                                np64(v["dt_bias"]), p("S0"), None if dS is None else np64(dS[i]), absolute=True, **kw)
        assert all(np.max(s) < 1e30 for s in scale.values())


@pytest.mark.parametrize("options", [dict(), dict(z=False), dict(skip=False), dict(bias=False), dict(states=None)])
@pytest.mark.parametrize("T,signs", [(70, False), (9, True)])
def test_without_softplus_every_value_is_compared(options, T, signs):
    """Steps above zero over a long sequence, and of either sign over a short one, which grows by e^10 at most."""
    v = make((2, T), 40, 16, torch.float32, 440 + T, **{"states": 2, **options}, rate=0.3 if signs else 0.75)
    if not signs:
        v["dt"] = v["dt"].abs()
    if v["dt_bias"] is not None:
        v["dt_bias"] = (v["dt_bias"] + 2.0).abs()
    dy = torch.randn((2, T, 40), generator=torch.Generator().manual_seed(46))
    dS = torch.randn((2, 40, 16), generator=torch.Generator().manual_seed(47))
    all_held(v, dy, dS, with_softplus=False)
    y, S_T, _ = gdr2_ssm_scan(**cuda(v), softplus=False)
    g = backward(v, dy, dS, softplus=False)
    gdr2_sync_status()
    check_scan(v, y, S_T, [((b,), b, T) for b in range(2)], with_softplus=False)
    check_gradients(v, dy, dS, g, T, with_softplus=False)
