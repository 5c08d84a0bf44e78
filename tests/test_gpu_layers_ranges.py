"""Ranges of the layers around the mixer: the elementwise laws over their whole domain, long
sequences in many segments, work splits that only large problems reach, values that are not finite."""
import numpy as np
import pytest
import torch

from gated_delta_rule_wy_b200 import (gdr2_head_norm_rope, gdr2_head_norm_rope_backward, gdr2_short_conv_silu_backward,
                                      gdr2_ssm_scan, gdr2_ssm_scan_backward, gdr2_ssm_step, gdr2_sync_status)
from gated_delta_rule_wy_b200 import inputs as I
from layer_bounds import U, np64
from oracle import layers as OL
from test_gpu_conv_backward import check as check_conv
from test_gpu_ssm import backward, check_gradients, check_scan, cuda, make

pytestmark = pytest.mark.gpu


def relative(got, ref):
    return np.abs(np64(got) - ref) / np.abs(ref)


def test_step_sizes_over_their_whole_range():
    """S_T of one token with x = B = 1 and no decay is the step size itself.

    With e = 2^(-|v| log2 e): the product and its constant round (2 |v| U of e), 2^x is off by 4 U; the quotient
    e / (2 + e) adds 4 U, the polynomial and its last product 6 U: below (2 |v| + 16) U of softplus."""
    v = torch.cat([torch.linspace(-80, 80, 4001), torch.tensor([0.0, 1e-6, -1e-6, 20.0, -20.0, 3e38])])
    C = v.numel()
    x, n = torch.ones((1, 1, C), device="cuda"), torch.ones((1, 1, 8), device="cuda")
    A = torch.zeros((C, 8), device="cuda")
    _, S, _ = gdr2_ssm_scan(x, v.view(1, 1, C).cuda(), A, n, n)
    S1 = torch.zeros((1, C, 8), device="cuda")
    gdr2_ssm_step(x[0], v.view(1, C).cuda(), A, n[0], n[0], S1)
    gdr2_sync_status()
    ref = OL.softplus(np64(v))
    for got in (S[0, :, 3], S1[0, :, 7]):
        assert np.all(relative(got, ref) <= (2 * np.minimum(np.abs(np64(v)), 90) + 16) * U)


def test_gates_and_slopes_over_their_whole_range():
    """y of one token with C = 0 and D = x = 1 is silu(z); its dz is the slope, and ddt the slope of softplus.

    1 / (1 + 2^(-z log2 e)): (2 |z| + 4) U of the exponential, 4 U of sum and quotient; the products add 2 U. The
    slope s (1 + z (1 - s)) has terms of size 1 + |z| that cancel."""
    z = torch.linspace(-80, 80, 4001)
    C = z.numel()
    one, zero = torch.ones((1, 1, C), device="cuda"), torch.zeros((1, 1, 8), device="cuda")
    A, D, n = torch.zeros((C, 8), device="cuda"), torch.ones(C, device="cuda"), torch.ones((1, 1, 8), device="cuda")
    zc = z.view(1, 1, C).cuda()
    y, _, _ = gdr2_ssm_scan(one, one, A, n, zero, D, zc)
    g = gdr2_ssm_scan_backward(one, one, A, n, zero, one, D, zc)
    # dS_T = 1 on the first state and x = 1: ddt = softplus'(dt)
    dS = torch.zeros((1, C, 8), device="cuda")
    dS[..., 0] = 1.0
    h = gdr2_ssm_scan_backward(one, zc, A, n, zero, torch.zeros_like(one), dS_T=dS)
    gdr2_sync_status()
    r = np64(z)
    limit = (2 * np.abs(r) + 12) * U
    # the quotients themselves: the oracle's (1 + tanh) / 2 has no value left below 1e-16, in 64 bits
    s, rest = 1 / (1 + np.exp(-r)), 1 / (1 + np.exp(r))
    assert np.all(np.abs(np64(y[0, 0]) - r * s) <= limit * np.abs(r * s) + 1e-37)
    assert np.all(np.abs(np64(g["dz"][0, 0]) - s * (1 + r * rest)) <= limit * s * (1 + np.abs(r)) + 1e-37)
    assert np.all(np.abs(np64(h["ddt"][0, 0]) - s) <= limit * s + 1e-37)


def test_a_step_of_zero_leaves_the_state():
    """Bit for bit: the tokens that fill up a tile are such steps."""
    v = cuda(make((2, 41), 50, 16, torch.float32, 30, states=2))
    v.update(dt=torch.zeros_like(v["dt"]), dt_bias=None)
    y, S_T, _ = gdr2_ssm_scan(**v, softplus=False)
    d = {k: t[:, 0].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in v.items()}
    S = d.pop("S0").clone()
    gdr2_ssm_step(**d, S=S, softplus=False)
    dS = torch.randn((2, 50, 16), generator=torch.Generator().manual_seed(9))
    g = backward({k: None if t is None else t.cpu() for k, t in v.items()}, torch.zeros((2, 41, 50)), dS, softplus=False)
    gdr2_sync_status()
    assert torch.equal(S_T, v["S0"]) and torch.equal(S, v["S0"]) and torch.equal(g["dS0"].cpu(), dS)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,C", [(16, 33), (8, 70), (32, 40)])
def test_long_sequences_in_many_segments(dtype, N, C):
    T = 1111
    v = make((1, T), C, N, dtype, 31, states=1)
    dy = torch.randn((1, T, C), generator=torch.Generator().manual_seed(3)).to(dtype)
    dS = torch.randn((1, C, N), generator=torch.Generator().manual_seed(4))
    y, S_T, saved = gdr2_ssm_scan(**cuda(v), save_states=True)
    g = backward(v, dy, dS, saved_states=saved)
    gdr2_sync_status()
    check_scan(v, y, S_T, [((0,), 0, T)])
    check_gradients(v, dy, dS, g, T)


@pytest.mark.parametrize("lens", [[1, 600, 0, 33, 477], [1111], [31, 1, 32, 32, 1, 1014]])
def test_long_packed_sequences_across_segments(lens):
    T, n = sum(lens), len(lens)
    v = make((T,), 65, 16, torch.float32, 32, states=n)
    ends = np.concatenate([[0], np.cumsum(lens)])
    y, S_T, _ = gdr2_ssm_scan(**cuda(v), cu_seqlens=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    gdr2_sync_status()
    check_scan(v, y, S_T, [(slice(ends[i], ends[i + 1]), i, lens[i]) for i in range(n) if lens[i]])


@pytest.mark.parametrize("states", [True, False])
def test_many_empty_sequences_keep_their_states(states):
    """Among tokens, behind the last one, and alone."""
    C, N = 45, 8
    for lens in ([0] * 37 + [3] + [0] * 50 + [40, 0, 0], [0] * 5):
        T, n = sum(lens), len(lens)
        v = make((T,), C, N, torch.float32, 40, states=n)
        if not states:
            v["S0"] = None
        ends = np.concatenate([[0], np.cumsum(lens)])
        y, S_T, _ = gdr2_ssm_scan(**cuda(v), cu_seqlens=torch.tensor(ends, dtype=torch.int32, device="cuda"))
        gdr2_sync_status()
        check_scan(v, y, S_T, [(slice(ends[i], ends[i + 1]), i, lens[i]) for i in range(n) if lens[i]])
        for i in range(n):
            if not lens[i]:
                assert torch.equal(S_T[i].cpu(), v["S0"][i] if states else torch.zeros(C, N))


def test_what_is_not_finite_stays_in_its_sequence():
    """A NaN or an infinity in one packed sequence, or one batch entry, reaches no other; the last
    token's, which padded tiles read again, reaches no earlier token."""
    lens = [50, 200, 37]
    ends = np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    v = make((sum(lens),), 40, 16, torch.float32, 33, states=3)
    clean = gdr2_ssm_scan(**cuda(v), cu_seqlens=cu)
    for key, value in (("x", float("nan")), ("dt", float("inf")), ("Bm", float("inf")), ("z", float("nan"))):
        w = {k: t.clone() for k, t in v.items()}
        w[key][ends[1] + 60] = value
        y, S_T, _ = gdr2_ssm_scan(**cuda(w), cu_seqlens=cu)
        gdr2_sync_status()
        for i in (0, 2):
            assert torch.equal(y[ends[i]:ends[i + 1]], clean[0][ends[i]:ends[i + 1]])
            assert torch.equal(S_T[i], clean[1][i])
        assert torch.equal(y[:ends[1] + 60], clean[0][:ends[1] + 60])
    v = make((2, 45), 40, 16, torch.float32, 34, states=2)
    dy = torch.randn((2, 45, 40), generator=torch.Generator().manual_seed(5))
    y0, S0, _ = gdr2_ssm_scan(**cuda(v))
    g0 = backward(v, dy)
    for key in ("x", "dt", "Bm", "Cm", "z"):
        w = {k: t.clone() for k, t in v.items()}
        w[key][0, 44] = float("inf")
        y, S, _ = gdr2_ssm_scan(**cuda(w))
        g = backward(w, dy)
        gdr2_sync_status()
        assert torch.equal(y[1], y0[1]) and torch.equal(S[1], S0[1]) and torch.equal(y[0, :44], y0[0, :44])
        for k in ("dx", "ddt", "dBm", "dCm", "dz", "dS0"):
            assert torch.equal(g[k][1], g0[k][1]), (key, k)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_single_tokens_of_many_sequences_are_those_of_few(dtype, N):
    """403 sequences are stepped several to a thread, a few one to a thread: the same operations on each."""
    B, C = 403, 520
    v = make((B,), C, N, dtype, 35, states=B)
    d = cuda(v)
    S = d.pop("S0")
    few = S.clone()
    y = gdr2_ssm_step(**d, S=S)
    gdr2_sync_status()
    for a in (0, 197, 398):
        part = {k: t[a:a + 5] if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
        Sp = few[a:a + 5].contiguous()
        assert torch.equal(gdr2_ssm_step(**part, S=Sp), y[a:a + 5])
        assert torch.equal(Sp, S[a:a + 5])


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_convolution_gradients_in_longer_runs(dtype, d):
    x, w, st = I.make_conv_inputs((3, 331, 40, d), 4, dtype, seed=36)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(6)).to(dtype)
    g = gdr2_short_conv_silu_backward(x.cuda(), w.cuda(), dy.cuda(), st.cuda(), l2norm=True)
    gdr2_sync_status()
    check_conv(x, w, dy, st, None, g, True)


def test_norm_of_huge_and_tiny_rows_and_zero_eps():
    """Squares stay in fp32: rows up to 1e17 keep their norm; with eps = 0 a row of zeros has none (NaN, as the
    formula's 0 / 0), and reaches no other row, in the weights' gradient either where its own is not asked."""
    q = torch.randn((1, 3, 2, 64), generator=torch.Generator().manual_seed(7)).cuda()
    q[0, 0] *= 1e17
    q[0, 1] *= 1e-17
    out, _ = gdr2_head_norm_rope(q, norm="rms", eps=0.0)
    ref = q.double() / q.double().pow(2).mean(-1, keepdim=True).sqrt()
    gdr2_sync_status()
    assert ((out.double() - ref).abs() <= 64 * U * ref.abs()).all()
    q[0, 1, 0] = 0.0
    again, _ = gdr2_head_norm_rope(q, norm="rms", eps=0.0)
    g = gdr2_head_norm_rope_backward(q, None, torch.ones_like(q), norm="rms", eps=0.0)
    gdr2_sync_status()
    assert again[0, 1, 0].isnan().all() and torch.equal(again[0, 0], out[0, 0]) and torch.equal(again[0, 1, 1], out[0, 1, 1])
    assert g["dq"][0, 1, 0].isnan().all() and g["dq"][0, 0].isfinite().all() and g["dq"][0, 2].isfinite().all()


@pytest.mark.parametrize("l2", [True, False])
def test_an_infinite_input_stays_within_the_convolutions_width(l2):
    """W = 2: u_j and u_{j+1} take x_j, so dx changes at j - 1, j and j + 1 only (with the norm, of its head only)."""
    N, T, H, d, W, j = 1, 40, 2, 64, 2, 20
    x, w, _ = I.make_conv_inputs((N, T, H, d), W, torch.float32, seed=38)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(10)).cuda()
    clean = gdr2_short_conv_silu_backward(x.cuda(), w.cuda(), dy, l2norm=l2)
    for at in (j, T - 1):
        bad = x.clone()
        bad[0, at, 1, 5] = float("inf")
        g = gdr2_short_conv_silu_backward(bad.cuda(), w.cuda(), dy, l2norm=l2)
        gdr2_sync_status()
        same = [t for t in range(T) if t not in (at - 1, at, at + 1)]
        assert torch.equal(g["dx"][0, same], clean["dx"][0, same])
        assert torch.equal(g["dx"][0, :, 0], clean["dx"][0, :, 0])
        assert torch.equal(g["dweight"][:d], clean["dweight"][:d])


def test_an_infinite_head_stays_in_its_channels_gradient():
    """Without a norm the weight's gradient takes x itself: infinite in that channel, the same elsewhere. 17
    heads leave tasks that read a head again, and few tokens groups that read a token again."""
    q = torch.randn((1, 3, 17, 64), generator=torch.Generator().manual_seed(11)).cuda()
    w, dy = torch.ones(64, device="cuda"), torch.rand_like(q) + 0.5
    clean = gdr2_head_norm_rope_backward(q, None, dy, q_weight=w, norm=None)
    q[0, 2, 16, 7] = float("inf")
    g = gdr2_head_norm_rope_backward(q, None, dy, q_weight=w, norm=None)
    gdr2_sync_status()
    rest = [i for i in range(64) if i != 7]
    assert g["dq_weight"][7] == float("inf") and torch.equal(g["dq_weight"][rest], clean["dq_weight"][rest])


def test_a_given_stream_owns_what_the_call_allocates():
    v = cuda(make((2, 300), 64, 16, torch.float32, 39, states=2))
    want = gdr2_ssm_scan(**v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # scratch of one call, freed at its end, is not handed to the current stream's tensors
        got = gdr2_ssm_scan(**v, stream=s)
        junk = torch.full((1 << 18,), float("nan"), device="cuda")
    s.synchronize()
    torch.cuda.synchronize()
    gdr2_sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and junk.isnan().all()


def test_two_streams_at_once():
    """Calls on two streams with buffers of their own do not touch each other."""
    v = cuda(make((1, 500), 96, 16, torch.bfloat16, 37, states=1))
    q = torch.randn((2, 300, 5, 128), generator=torch.Generator().manual_seed(8)).cuda().bfloat16()
    y0, S0, _ = gdr2_ssm_scan(**v)
    r0, _ = gdr2_head_norm_rope(q)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(a):
            got.append(gdr2_ssm_scan(**v)[:2])
        with torch.cuda.stream(b):
            got.append((gdr2_head_norm_rope(q)[0],))
            got.append(gdr2_ssm_scan(**v, stream=b)[:2])
    torch.cuda.synchronize()
    gdr2_sync_status()
    for r in got:
        assert torch.equal(r[0], r0 if len(r) == 1 else y0) and (len(r) == 1 or torch.equal(r[1], S0))
