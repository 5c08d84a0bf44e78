"""GPU parity of the selective state-space scan, its single-token step and its gradients
against the fp64 oracle, with bounds derived in layer_bounds."""
import numpy as np
import pytest
import torch

from gated_delta_rule_wy_b200 import (gdr2_short_conv_silu, gdr2_short_conv_silu_backward, gdr2_ssm_scan,
                                      gdr2_ssm_scan_backward, gdr2_ssm_step, gdr2_sync_status)
from layer_bounds import assert_bound, np64, recurrence
from oracle import layers as OL

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def make(lead, C, N, dtype, seed, *, z=True, skip=True, bias=True, states=None, rate=1.0):
    """Inputs of a scan on the CPU: step sizes softplus(0.5 N(0, 1) - 2), decays -rate (1 .. N)."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    v = dict(x=rn(*lead, C).to(dtype), dt=(0.5 * rn(*lead, C)).to(dtype),
             A=-rate * torch.arange(1, N + 1).float() / N ** 0.5 * torch.exp(0.1 * rn(C, N)),
             Bm=rn(*lead, N).to(dtype), Cm=rn(*lead, N).to(dtype), D=rn(C) if skip else None,
             z=rn(*lead, C).to(dtype) if z else None, dt_bias=rn(C) * 0.1 - 2.0 if bias else None,
             S0=None if states is None else rn(states, C, N))
    return v


def cuda(v):
    return {k: t.cuda() if torch.is_tensor(t) else t for k, t in v.items()}


def oracle_scan(v, rows, seq, **kw):
    """The oracle on rows (an index of the leading dimensions) with state `seq`."""
    pick = lambda k: None if v[k] is None else np64(v[k][rows])  # noqa: E731
    return OL.ssm_scan(pick("x"), pick("dt"), np64(v["A"]), pick("Bm"), pick("Cm"), np64(v["D"]), pick("z"),
                       np64(v["dt_bias"]), None if v["S0"] is None else np64(v["S0"][seq]), **kw)


def check_scan(v, y, S_T, sequences, **kw):
    """sequences: (rows of the token tensors, index of the state, tokens)."""
    N = v["A"].shape[1]
    for rows, seq, T in sequences:
        y_ref, S_ref, _ = oracle_scan(v, rows, seq, **kw)
        y_abs, S_abs, _ = oracle_scan(v, rows, seq, absolute=True, **kw)
        assert_bound(y[rows], y_ref, y_abs, recurrence(T, N), f"y of sequence {seq}")
        if S_T is not None:
            assert_bound(S_T[seq], S_ref, S_abs, recurrence(T), f"S_T of sequence {seq}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T,C", [(1, 1), (5, 130), (31, 64), (32, 7), (33, 256), (77, 96), (200, 72)])
def test_dense_scan_matches_the_oracle(dtype, N, T, C):
    v = make((2, T), C, N, dtype, 1000 + T + N, states=2)
    y, S_T, saved = gdr2_ssm_scan(**cuda(v), save_states=True)
    gdr2_sync_status()
    check_scan(v, y, S_T, [((b,), b, T) for b in range(2)])
    for b in range(2):
        _, _, h = oracle_scan(v, (b,), b)
        _, _, ha = oracle_scan(v, (b,), b, absolute=True)
        at = np.arange(0, T, 16)
        assert_bound(saved[b], h[at], ha[at], recurrence(T), "saved states")


@pytest.mark.parametrize("options", [dict(z=False), dict(skip=False), dict(bias=False), dict(states=None),
                                     dict(z=False, skip=False, bias=False, states=None)])
def test_options_of_the_scan(options):
    v = make((2, 70), 40, 16, torch.float32, 7, **{"states": 2, **options})
    y, S_T, _ = gdr2_ssm_scan(**cuda(v))
    gdr2_sync_status()
    check_scan(v, y, S_T, [((b,), b, 70) for b in range(2)])
    y2, none, _ = gdr2_ssm_scan(**cuda(v), final_state=False)
    assert none is None and torch.equal(y2, y)


def test_without_softplus_steps_of_either_sign():
    v = make((1, 50), 24, 16, torch.float32, 8, bias=False, rate=0.3)
    y, S_T, _ = gdr2_ssm_scan(**cuda(v), softplus=False)
    gdr2_sync_status()
    check_scan(v, y, S_T, [((0,), 0, 50)], with_softplus=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,C", [(16, 100), (8, 129), (64, 40)])
@pytest.mark.parametrize("lens", [[0, 5, 1, 70, 2, 0, 140, 0], [300], [1, 1, 1], [64, 64, 63, 65], [0, 0, 9]])
def test_packed_sequences_scan_on_their_own(dtype, N, C, lens):
    T, n = sum(lens), len(lens)
    v = make((T,), C, N, dtype, 11 + T, states=n)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    y, S_T, _ = gdr2_ssm_scan(**cuda(v), cu_seqlens=cu)
    gdr2_sync_status()
    ends = np.concatenate([[0], np.cumsum(lens)])
    check_scan(v, y, S_T, [(slice(ends[i], ends[i + 1]), i, lens[i]) for i in range(n) if lens[i]])
    for i in range(n):
        if not lens[i]:
            assert torch.equal(S_T[i].cpu(), v["S0"][i])  # a sequence without tokens keeps its state
    y0, S0, _ = gdr2_ssm_scan(**{**cuda(v), "S0": None}, cu_seqlens=cu)
    gdr2_sync_status()
    w = {**v, "S0": None}
    check_scan(w, y0, S0, [(slice(ends[i], ends[i + 1]), i, lens[i]) for i in range(n) if lens[i]])
    for i in range(n):
        if not lens[i]:
            assert not S0[i].any()


def test_strided_views_give_the_same_bits():
    """Row strides of fused projections, odd element offsets and a reversed order of batch entries'
    memory (contiguous copies give the same values through either load path)."""
    B, T, C, N = 2, 75, 136, 16
    v = cuda(make((B, T), C, N, torch.bfloat16, 21, states=B))
    y, S_T, _ = gdr2_ssm_scan(**v)

    def widened(t, before, after):
        w = torch.full((*t.shape[:-1], before + t.shape[-1] + after), float("nan"), dtype=t.dtype, device="cuda")
        w[..., before:before + t.shape[-1]] = t
        return w[..., before:before + t.shape[-1]]

    for before, after in ((8, 16), (3, 2), (1, 0)):
        w = {**v, **{k: widened(v[k], before, after) for k in ("x", "dt", "z", "Bm", "Cm")}}
        y2, S2, _ = gdr2_ssm_scan(**w)
        assert torch.equal(y2, y) and torch.equal(S2, S_T)
    flat = torch.zeros(v["x"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:]
    flat.copy_(v["x"].flatten())
    y2, S2, _ = gdr2_ssm_scan(**{**v, "x": flat.view(B, T, C)})  # base off by one element
    gdr2_sync_status()
    assert torch.equal(y2, y) and torch.equal(S2, S_T)


@pytest.mark.parametrize("dtype", TYPES)
def test_split_prompt_and_single_tokens_continue_the_state(dtype):
    B, T, C, N = 3, 90, 70, 16
    host = make((B, T), C, N, dtype, 31, states=B)
    v = cuda(host)
    tok = ("x", "dt", "Bm", "Cm", "z")
    y1, S, _ = gdr2_ssm_scan(**{**v, **{k: v[k][:, :37].contiguous() for k in tok}})
    ys = [y1]
    one = {k: t for k, t in v.items() if k != "S0"}
    for t in range(37, T):
        ys.append(gdr2_ssm_step(**{**one, **{k: v[k][:, t] for k in tok}}, S=S)[:, None])  # rows of a longer tensor
    gdr2_sync_status()
    check_scan(host, torch.cat(ys, 1), S, [((b,), b, T) for b in range(B)])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 130), (2, 1000)])
def test_single_token_matches_the_oracle(dtype, N, B, C):
    v = make((B, 1), C, N, dtype, 41, states=B)
    d = cuda({k: (t[:, 0] if k in ("x", "dt", "Bm", "Cm", "z") else t) for k, t in v.items()})
    S = d.pop("S0").clone()
    y = gdr2_ssm_step(**d, S=S)
    gdr2_sync_status()
    check_scan(v, y[:, None], S, [((b,), b, 1) for b in range(B)])
    d.update(z=None, D=None, dt_bias=None)
    w = {**v, "z": None, "D": None, "dt_bias": None}
    S = w["S0"].cuda()
    y = gdr2_ssm_step(**d, S=S)
    gdr2_sync_status()
    check_scan(w, y[:, None], S, [((b,), b, 1) for b in range(B)])


def test_extreme_decays_stay_finite_and_forget():
    """Steps of size 60 underflow to a decay of 0: each token forgets the past; A = 0 never forgets."""
    T, C, N = 40, 33, 16
    v = make((1, T), C, N, torch.float32, 51, bias=False, z=False, skip=False, states=1)
    v["dt"] = torch.full((1, T, C), 60.0)
    v["A"] = torch.full((C, N), -20.0)
    y, S_T, _ = gdr2_ssm_scan(**cuda(v))
    gdr2_sync_status()
    ref = 60.0 * np64(v["x"])[0, -1][:, None] * np64(v["Bm"])[0, -1][None, :]
    assert_bound(S_T[0], ref, np.abs(ref), 96, "state of the last token alone")
    v["dt"] = torch.full((1, T, C), -3.0)
    v["A"] = torch.zeros(C, N)
    y, S_T, _ = gdr2_ssm_scan(**cuda(v))
    gdr2_sync_status()
    check_scan(v, y, S_T, [((0,), 0, T)])


def test_empty_problems():
    v = cuda(make((2, 0), 20, 16, torch.bfloat16, 61, states=2))
    y, S_T, _ = gdr2_ssm_scan(**v)
    assert y.shape == (2, 0, 20) and torch.equal(S_T, v["S0"])
    _, S_T, _ = gdr2_ssm_scan(**{**v, "S0": None})
    assert not S_T.any()
    g = gdr2_ssm_scan_backward(*(v[k] for k in ("x", "dt", "A", "Bm", "Cm")), torch.empty_like(v["x"]), v["D"], v["z"],
                               v["dt_bias"], v["S0"], v["S0"] * 2)
    gdr2_sync_status()
    assert torch.equal(g["dS0"], v["S0"] * 2) and not g["dA"].any() and not g["dD"].any() and not g["ddt_bias"].any()
    w = cuda(make((0, 5), 20, 16, torch.bfloat16, 62))
    y, S_T, _ = gdr2_ssm_scan(**w)
    assert y.shape == (0, 5, 20) and S_T.shape == (0, 20, 16)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")  # two empty packed sequences
    p = cuda(make((0,), 20, 16, torch.bfloat16, 63, states=2))
    _, S_T, _ = gdr2_ssm_scan(**p, cu_seqlens=cu)
    gdr2_sync_status()
    assert torch.equal(S_T, p["S0"])


# ---------------------------------------------------------------- gradients


def check_gradients(v, dy, dS_T, g, T, **kw):
    N, C = v["A"].shape[1], v["A"].shape[0]
    B = dy.shape[0]
    sums = {k: 0.0 for k in ("dA", "dD", "ddt_bias")}
    scales = dict(sums)
    for b in range(B):
        p = lambda k: None if v[k] is None else np64(v[k][b])  # noqa: E731,B023
        args = (p("x"), p("dt"), np64(v["A"]), p("Bm"), p("Cm"), np64(dy[b]), np64(v["D"]), p("z"), np64(v["dt_bias"]),
                p("S0"), None if dS_T is None else np64(dS_T[b]))
        ref, scale = OL.ssm_backward(*args, **kw), OL.ssm_backward(*args, absolute=True, **kw)
        r = 2 * recurrence(T, N)  # two recurrences: the states and their gradient
        for k in ("dx", "ddt", "dz"):
            if k in ref:
                assert_bound(g[k][b], ref[k], scale[k], r, f"{k}[{b}]")
        for k in ("dBm", "dCm"):
            assert_bound(g[k][b], ref[k], scale[k], r + C, f"{k}[{b}]")
        assert_bound(g["dS0"][b], ref["dS0"], scale["dS0"], r, f"dS0[{b}]")
        for k in sums:
            if k in ref:
                sums[k], scales[k] = sums[k] + ref[k], scales[k] + scale[k]
    for k in sums:
        if np.ndim(sums[k]):
            assert_bound(g[k], sums[k], scales[k], 2 * recurrence(T, N) + B * T, k)


def backward(v, dy, dS_T=None, **kw):
    d = cuda(v)
    return gdr2_ssm_scan_backward(*(d[k] for k in ("x", "dt", "A", "Bm", "Cm")), dy.cuda(), d["D"], d["z"], d["dt_bias"],
                                  d["S0"], None if dS_T is None else dS_T.cuda(), **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T,C", [(1, 1), (15, 130), (17, 64), (33, 7), (77, 96), (200, 72)])
def test_gradients_match_the_oracle(dtype, N, T, C):
    v = make((2, T), C, N, dtype, 2000 + T + N, states=2)
    gen = torch.Generator().manual_seed(T)
    dy, dS = torch.randn((2, T, C), generator=gen).to(dtype), torch.randn((2, C, N), generator=gen)
    g = backward(v, dy, dS)
    gdr2_sync_status()
    check_gradients(v, dy, dS, g, T)
    _, _, saved = gdr2_ssm_scan(**cuda(v), save_states=True)
    again = backward(v, dy, dS, saved_states=saved)
    gdr2_sync_status()
    for k in g:
        assert torch.equal(g[k], again[k]), f"{k}: saved states and states formed again"


@pytest.mark.parametrize("options", [dict(z=False), dict(skip=False), dict(bias=False), dict(states=None)])
@pytest.mark.parametrize("softplus", [True, False])
def test_gradients_of_the_options(options, softplus):
    v = make((2, 70), 40, 16, torch.float32, 71, **{"states": 2, **options})
    if not softplus:
        v["dt"] = v["dt"].abs()
    dy = torch.randn((2, 70, 40), generator=torch.Generator().manual_seed(5))
    g = backward(v, dy, softplus=softplus)
    gdr2_sync_status()
    check_gradients(v, dy, None, g, 70, with_softplus=softplus)
    assert (g["dz"] is None) == (v["z"] is None) and (g["dD"] is None) == (v["D"] is None)
    assert backward(v, dy, softplus=softplus, want_dS0=False)["dS0"] is None


def test_gradients_are_differences_of_the_kernel():
    """Directional differences of the fp32 forward: a step of 2^-8 along unit directions, so the
    second-order term cancels, the third is below 2^-16 of the gradient's size, and rounding adds
    T U |y| / 2^-8."""
    T, C, N = 24, 12, 16
    v = make((1, T), C, N, torch.float32, 81, states=1)
    gen = torch.Generator().manual_seed(9)
    dy = torch.randn((1, T, C), generator=gen)
    g = backward(v, dy)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dBm", "Cm": "dCm", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
             "S0": "dS0"}
    for k, gk in names.items():
        u = torch.randn(v[k].shape, generator=gen)
        u /= u.norm()
        loss = []
        for s in (2.0 ** -8, -2.0 ** -8):
            y, _, _ = gdr2_ssm_scan(**cuda({**v, k: v[k] + s * u}))
            loss.append((np64(y) * np64(dy)).sum())
        want, got = (loss[0] - loss[1]) * 2.0 ** 7, (np64(g[gk]) * np64(u)).sum()
        size = np.linalg.norm(np64(g[gk])) + 1.0
        rounding = 2.0 ** -24 * 24 * T * np.abs(np64(y)).max() * np.linalg.norm(np64(dy)) * 2.0 ** 8
        assert abs(want - got) <= 2.0 ** -10 * size + rounding, (k, want, got)
    gdr2_sync_status()


def test_same_bits_each_time_and_on_another_stream():
    v = make((2, 300), 130, 16, torch.bfloat16, 91, states=2)
    dy = torch.randn((2, 300, 130), generator=torch.Generator().manual_seed(1)).bfloat16()
    d = cuda(v)
    ref, ref_g = gdr2_ssm_scan(**d), backward(v, dy)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:  # two calls at once, each with a workspace of its own
        with torch.cuda.stream(s):
            outs.append((gdr2_ssm_scan(**d), backward(v, dy)))
    explicit = gdr2_ssm_scan(**d, stream=streams[0])
    torch.cuda.synchronize()
    for (y, S, _), g in outs:
        assert torch.equal(y, ref[0]) and torch.equal(S, ref[1])
        assert all(torch.equal(g[k], ref_g[k]) for k in g)
    assert torch.equal(explicit[0], ref[0])


def test_captured_and_replayed():
    B, T, C, N = 1, 160, 96, 16
    v = cuda(make((B, T), C, N, torch.bfloat16, 101, states=B))
    dy = torch.randn((B, T, C), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    opt = dict(D=v["D"], z=v["z"], dt_bias=v["dt_bias"], S0=v["S0"])

    def step():
        y, S, saved = gdr2_ssm_scan(*args, **opt, save_states=True)
        return y, S, gdr2_ssm_scan_backward(*args, dy, **opt, saved_states=saved)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, S, g = step()
    new = cuda(make((B, T), C, N, torch.bfloat16, 102, states=B))
    for k in ("x", "dt", "Bm", "Cm", "z", "S0"):
        v[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    y2, S2, g2 = step()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(S, S2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_convolution_and_scan_as_one_layer():
    """The layer as it is used: short convolution, scan and gate for a prompt, then token by token
    from its states; and the chain of gradients back to the convolution's input."""
    B, T, H, d, N, W = 2, 50, 2, 64, 16, 4
    C = H * d
    v = cuda(make((B, T), C, N, torch.float32, 111))
    v.pop("S0")
    gen = torch.Generator().manual_seed(3)
    w = ((torch.rand((C, W), generator=gen) * 2 - 1) / 2).cuda()
    u = v.pop("x").view(B, T, H, d)
    x, conv = gdr2_short_conv_silu(u, w, final_state=True)
    y, S, _ = gdr2_ssm_scan(x.flatten(-2), **v)
    x1, conv1 = gdr2_short_conv_silu(u[:, :30].contiguous(), w, final_state=True)
    pre = {k: (t[:, :30].contiguous() if k in ("dt", "Bm", "Cm", "z") else t) for k, t in v.items()}
    _, S1, _ = gdr2_ssm_scan(x1.flatten(-2), **pre)
    for t in range(30, T):
        xt, _ = gdr2_short_conv_silu(u[:, t:t + 1].contiguous(), w, conv1, state_out=conv1)
        one = {k: (a[:, t] if k in ("dt", "Bm", "Cm", "z") else a) for k, a in v.items()}
        yt = gdr2_ssm_step(xt.view(B, C), S=S1, **one)
        assert_bound(yt, np64(y[:, t]), np.abs(np64(y[:, t])) + 8.0, 2 * recurrence(T, N), f"token {t}")
    assert torch.equal(conv1, conv)
    dy = torch.randn((B, T, C), generator=gen).cuda()
    g = gdr2_ssm_scan_backward(x.flatten(-2), *(v[k] for k in ("dt", "A", "Bm", "Cm")), dy, v["D"], v["z"], v["dt_bias"])
    gc = gdr2_short_conv_silu_backward(u, w, g["dx"].view(B, T, H, d))
    gdr2_sync_status()
    for b in range(B):
        ref = OL.conv_backward(np64(u[b]), np64(w), np64(g["dx"][b]).reshape(T, H, d))
        scale = OL.conv_backward(np64(u[b]), np64(w), np64(g["dx"][b]).reshape(T, H, d), absolute=True)
        assert_bound(gc["dx"][b], ref["dx"], scale["dx"], 96, "dx of the layer")
