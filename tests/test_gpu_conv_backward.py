"""GPU parity of the short convolution's gradients against the fp64 oracle."""
import pytest
import torch

from gated_delta_rule_wy_b200 import gdr2_short_conv_silu, gdr2_short_conv_silu_backward, gdr2_sync_status
from gated_delta_rule_wy_b200 import inputs as I
from layer_bounds import assert_bound, np64
from oracle import layers as OL

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def check(x, w, dy, st, dso, g, l2, eps=1e-6):
    """Per output: W products, silu and its slope (16 roundings, fast quotients 4 each) and, with the
    norm, two sums over d and a reciprocal root; sums over the tokens for the taps."""
    N, T, H, d = x.shape
    W = w.shape[-1]
    dw, dws = 0.0, 0.0
    for n in range(N):
        args = (np64(x[n]), np64(w), np64(dy[n]), None if st is None else np64(st[n]), None if dso is None else np64(dso[n]))
        ref = OL.conv_backward(*args, l2norm=l2, eps=eps)
        scale = OL.conv_backward(*args, l2norm=l2, eps=eps, absolute=True)
        r = 64 + 8 * W + (4 * d if l2 else 0)
        # u itself is off by W roundings of |w| |x|, which its slope passes on: |u| <= 8 here
        assert_bound(g["dx"][n], ref["dx"], scale["dx"] * 4, r, f"dx[{n}]")
        if g["dstate"] is not None:
            assert_bound(g["dstate"][n], ref["dstate"], scale["dstate"] * 4, r, f"dstate[{n}]")
        dw, dws = dw + ref["dweight"], dws + scale["dweight"]
    assert_bound(g["dweight"], dw, dws * 4, 128 + 4 * d + N * T, "dweight")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("l2", [True, False])
@pytest.mark.parametrize("T", [1, 2, 3, 63, 64, 65, 150])
def test_gradients_match_the_oracle(dtype, d, W, l2, T):
    N, H = 2, 3
    x, w, st = I.make_conv_inputs((N, T, H, d), W, dtype, seed=T)
    gen = torch.Generator().manual_seed(W)
    dy = torch.randn(x.shape, generator=gen).to(dtype)
    dso = torch.randn(st.shape, generator=gen).to(dtype)
    g = gdr2_short_conv_silu_backward(x.cuda(), w.cuda(), dy.cuda(), st.cuda(), dso.cuda(), l2norm=l2)
    gdr2_sync_status()
    check(x, w, dy, st, dso, g, l2)
    g = gdr2_short_conv_silu_backward(x.cuda(), w.cuda(), dy.cuda(), l2norm=l2)
    gdr2_sync_status()
    check(x, w, dy, None, None, g, l2)
    assert g["dstate"] is None


def test_state_gradient_without_a_state_and_conv1d_weight():
    x, w, _ = I.make_conv_inputs((1, 9, 2, 64), 4, torch.float32, seed=5)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(6))
    g = gdr2_short_conv_silu_backward(x.cuda(), w[:, None, :].cuda(), dy.cuda(), want_dstate=True)
    gdr2_sync_status()
    assert g["dweight"].shape == (128, 1, 4)
    check(x, w, dy, None, None, {**g, "dweight": g["dweight"][:, 0]}, False)


def test_no_tokens_pass_the_state_gradient_through():
    dso = torch.randn((2, 3, 2, 64), generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    x = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((128, 4), device="cuda")
    g = gdr2_short_conv_silu_backward(x, w, x, dso, dso)
    gdr2_sync_status()
    assert torch.equal(g["dstate"], dso) and not g["dweight"].any()


def test_zero_rows_have_no_gradient_through_the_norm():
    """x = 0: y = 0, r = sqrt(eps) and the gradient is dy / (2 r) through the taps, finite."""
    x = torch.zeros((1, 20, 2, 128))
    w = torch.full((256, 4), 0.5)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(8))
    g = gdr2_short_conv_silu_backward(x.cuda(), w.cuda(), dy.cuda(), l2norm=True)
    gdr2_sync_status()
    check(x, w, dy, None, None, g, True)


def test_gradients_follow_autograd_through_two_calls():
    """A sequence cut in two calls, the state's gradient carried back, gives the whole one's."""
    x, w, st = I.make_conv_inputs((1, 40, 2, 64), 4, torch.float32, seed=9)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(10))
    c = lambda t: t.contiguous().cuda()  # noqa: E731
    whole = gdr2_short_conv_silu_backward(c(x), c(w), c(dy), c(st), l2norm=True)
    _, mid = gdr2_short_conv_silu(c(x[:, :23]), c(w), c(st), l2norm=True, final_state=True)
    right = gdr2_short_conv_silu_backward(c(x[:, 23:]), c(w), c(dy[:, 23:]), mid, l2norm=True)
    left = gdr2_short_conv_silu_backward(c(x[:, :23]), c(w), c(dy[:, :23]), c(st), right["dstate"], l2norm=True)
    gdr2_sync_status()
    joined = {"dx": torch.cat([left["dx"], right["dx"]], 1), "dstate": left["dstate"],
              "dweight": left["dweight"] + right["dweight"]}
    check(x, w, dy, st, None, joined, True)
    check(x, w, dy, st, None, whole, True)


def test_same_bits_captured_and_on_another_stream():
    x, w, st = I.make_conv_inputs((2, 130, 2, 128), 4, torch.bfloat16, seed=11)
    x, w, st = x.cuda(), w.cuda(), st.cuda()
    dy = torch.randn_like(x)
    run = lambda: gdr2_short_conv_silu_backward(x, w, dy, st, l2norm=True)  # noqa: E731
    ref = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    for v in cap.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], other[k]) and torch.equal(ref[k], cap[k])
