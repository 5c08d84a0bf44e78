"""GPU parity of the per-head norm with rotation and its gradients against the fp64 oracle."""
import numpy as np
import pytest
import torch

from gated_delta_rule_wy_b200 import (GDR2Error, gdr2_head_norm_rope, gdr2_head_norm_rope_backward, gdr2_sync_status)
from layer_bounds import assert_bound, np64
from oracle import layers as OL

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def table(P, R):
    ang = torch.arange(P).double()[:, None] * 10000.0 ** (-torch.arange(0, R, 2).double() / R)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def make(B, T, Hq, Hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return rn(B, T, (Hq + 2 * Hk) * d).to(dtype), rn(d), rn(d), rn(B, T, Hq, d).to(dtype), rn(B, T, Hk, d).to(dtype)


def check(x, out, w, cs, pos, dy=None, dx=None, dw=None, *, norm, interleaved, eps=1e-6):
    """Forward: a sum over d, a reciprocal root (4), two products and a turn: d + 16 roundings.
    Backward: two sums over d more; the weights' gradient sums over all rows."""
    d = x.shape[-1]
    kw = dict(norm=norm, eps=eps, interleaved=interleaved, cos_sin=None if cs is None else np64(cs), positions=pos)
    ref = OL.head_norm_rope(np64(x), np64(w), **kw)
    scale = OL.head_norm_rope(np64(x), np64(w), absolute=True, **kw)
    assert_bound(out, ref, scale, d + 16, "rotated")
    if dx is not None:
        ref, rw = OL.head_norm_rope_backward(np64(x), np64(dy), np64(w), **kw)
        scale, sw = OL.head_norm_rope_backward(np64(x), np64(dy), np64(w), absolute=True, **kw)
        assert_bound(dx, ref, scale, 4 * d + 32, "dx")
        if dw is not None:
            assert_bound(dw, rw, sw, 4 * d + 32 + x.numel() // d, "dweight")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,R", [(64, 64), (64, 32), (128, 128), (128, 48), (256, 256), (256, 16), (128, 0)])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("interleaved", [True, False])
def test_matches_the_oracle(dtype, d, R, norm, interleaved):
    B, T, Hq, Hk = 2, 19, 5, 2
    qkv, wq, wk, dq, dk = make(B, T, Hq, Hk, d, dtype, d + R)
    fused = qkv.cuda()
    q, k = fused[..., :Hq * d].unflatten(-1, (Hq, d)), fused[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    cs = table(50, R) if R else None
    pos = torch.randint(0, 50, (B, T), generator=torch.Generator().manual_seed(1))
    kw = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), norm=norm, interleaved=interleaved,
              cos_sin=None if cs is None else cs.cuda(), positions=pos.to(torch.int32).cuda())
    qo, ko = gdr2_head_norm_rope(q, k, **kw)
    g = gdr2_head_norm_rope_backward(q, k, dq.cuda(), dk.cuda(), **kw)
    gdr2_sync_status()
    for x, o, w, dy, n in ((q, qo, wq, dq, "q"), (k, ko, wk, dk, "k")):
        check(x, o, w, cs, pos.numpy(), dy, g["d" + n], g[f"d{n}_weight"], norm=norm, interleaved=interleaved)


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 0), (1, 1, 1, 1), (3, 1, 16, 2), (1, 7, 17, 0), (2, 300, 4, 4), (1, 2000, 1, 3)])
def test_head_counts_lengths_and_implied_positions(B, T, Hq, Hk):
    d = 128
    qkv, wq, wk, dq, dk = make(B, T, Hq, Hk, d, torch.bfloat16, T)
    q = qkv[..., :Hq * d].unflatten(-1, (Hq, d)).contiguous().cuda()
    k = qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)).contiguous().cuda() if Hk else None
    cs = table(T + 9, d)
    kw = dict(q_weight=wq.cuda(), cos_sin=cs.cuda(), first_position=9)
    qo, ko = gdr2_head_norm_rope(q, k, **kw)
    g = gdr2_head_norm_rope_backward(q, k, dq.cuda(), dk.cuda() if Hk else None, **kw)
    gdr2_sync_status()
    pos = np.broadcast_to(np.arange(T) + 9, (B, T))
    check(q, qo, wq, cs, pos, dq, g["dq"], g["dq_weight"], norm="rms", interleaved=False)
    assert g["dk_weight"] is None and (ko is None) == (Hk == 0)
    if Hk:
        check(k, ko, None, cs, pos, dk, g["dk"], None, norm="rms", interleaved=False)


def test_far_positions_turn_by_the_tables_angles():
    P, d = 1 << 20, 64
    cs = table(P, d)
    qkv, wq, wk, _, _ = make(1, 3, 2, 1, d, torch.float32, 3)
    q = qkv[..., :2 * d].unflatten(-1, (2, d)).contiguous()
    pos = torch.tensor([[P - 1, 0, 777777]])
    qo, _ = gdr2_head_norm_rope(q.cuda(), None, wq.cuda(), None, cs.cuda(), pos.to(torch.int32).cuda())
    gdr2_sync_status()
    check(q, qo, wq, cs, pos.numpy(), norm="rms", interleaved=False)


def test_positions_outside_the_table_are_reported():
    d = 64
    qkv, wq, _, _, _ = make(1, 4, 1, 0, d, torch.float32, 4)
    q, cs = qkv.view(1, 4, 1, d).cuda(), table(10, d).cuda()
    pos = torch.tensor([[3, 10, -1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    gdr2_sync_status()
    out, _ = gdr2_head_norm_rope(q, None, wq.cuda(), None, cs, pos)
    with pytest.raises(GDR2Error, match="position"):
        gdr2_sync_status()
    gdr2_sync_status()  # reported once
    check(q[:, :1], out[:, :1], wq, cs.cpu(), np.array([[3]]), norm="rms", interleaved=False)
    check(q[:, 1:], out[:, 1:], wq, None, None, norm="rms", interleaved=False)  # normed, not turned


def test_zero_rows_and_no_tokens():
    q = torch.zeros((1, 3, 2, 128), device="cuda")
    out, _ = gdr2_head_norm_rope(q, None, None, None, table(3, 128).cuda())
    assert not out.any()
    e = torch.empty((2, 0, 2, 128), device="cuda")
    w = torch.ones(128, device="cuda")
    g = gdr2_head_norm_rope_backward(e, e, e, e, w, w, table(3, 128).cuda())
    gdr2_sync_status()
    assert not g["dq_weight"].any() and not g["dk_weight"].any() and g["dq"].shape == e.shape


def test_same_bits_captured_and_on_another_stream():
    B, T, Hq, Hk, d = 2, 64, 6, 2, 128
    qkv, wq, wk, dq, dk = make(B, T, Hq, Hk, d, torch.bfloat16, 12)
    f = qkv.cuda()
    q, k = f[..., :Hq * d].unflatten(-1, (Hq, d)), f[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    cs, dq, dk, wq, wk = table(T, d).cuda(), dq.cuda(), dk.cuda(), wq.cuda(), wk.cuda()

    def run():
        a, b = gdr2_head_norm_rope(q, k, wq, wk, cs)
        return {"q": a, "k": b, **gdr2_head_norm_rope_backward(q, k, dq, dk, wq, wk, cs)}

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
    for key in ref:
        assert torch.equal(ref[key], other[key]) and torch.equal(ref[key], cap[key])
