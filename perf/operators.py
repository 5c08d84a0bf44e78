"""Measured cases of the layers around the mixer: the selective state-space scan (prompts, single
tokens, training), the short convolution's backward and the per-head norm with rotation.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end) where ``own`` is false, and calls the library where it is true.
Token tensors are token-major; views of a fused projection keep its row stride, as a
user's program has them in hand. Channel counts and lengths follow the 1.3B-layer
workloads (16 heads of 128 channels = 2048, T = 4096, 256 decoding sequences) and generic
ragged sizes around them.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # a short odd prompt of one user: few channels' worth of work, latency counts
        dict(name="scan_prompt_short", op="scan", B=1, T=37, D=2048, N=16, dtype="bf16", z=True, S0=True, lens=""),
        # the prefill of a layer with a 1.3B-layer batch
        dict(name="scan_prompt_b4", op="scan", B=4, T=4096, D=2048, N=16, dtype="bf16", z=True, S0=False, lens=""),
        # one long document: the time axis has to give the parallel work
        dict(name="scan_prompt_long", op="scan", B=1, T=32768, D=2048, N=16, dtype="bf16", z=True, S0=True, lens=""),
        # mixed requests packed in one stream, odd channel count, fp32, no gate
        dict(name="scan_packed_fp32", op="scan", B=1, T=4500, D=1000, N=16, dtype="fp32", z=False, S0=True,
             lens="1,700,0,33,1530,64,2,1201,969"),
        # one token for 256 decoding sequences, and for one
        dict(name="step_256", op="step", B=256, D=2048, N=16, dtype="bf16", z=True),
        dict(name="step_1", op="step", B=1, D=1000, N=16, dtype="fp32", z=True),
        # a training step of the scan: forward and all gradients
        dict(name="train_b2", op="train", B=2, T=4096, D=2048, N=16, dtype="bf16", z=True, S0=False),
        # a small ragged fp32 one with an initial state
        dict(name="train_small_fp32", op="train", B=1, T=203, D=520, N=16, dtype="fp32", z=False, S0=True),
        # gradients of the query/key branch of the block prologue at the 1.3B layer's size
        dict(name="conv_backward_b4", op="conv", B=4, T=4096, H=16, d=128, W=4, dtype="bf16", l2=True, state=False),
        # and of a small value branch continued from a state
        dict(name="conv_backward_small", op="conv", B=1, T=77, H=3, d=64, W=4, dtype="fp32", l2=False, state=True),
        # queries and keys of an attention layer in training: forward and gradients
        dict(name="rope_train_b4", op="rope_train", B=4, T=4096, Hq=16, Hk=2, d=128, R=128, P=4096, norm="rms",
             interleaved=False, dtype="bf16"),
        # and for one token of 256 sequences at far positions
        dict(name="rope_step_256", op="rope", B=256, T=1, Hq=16, Hk=2, d=128, R=64, P=131072, norm="rms",
             interleaved=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "train", "conv", "rope_train", "rope"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("scan", "train"):
        D, N = _log_int(rng, 64, 4096), rng.choice([8, 16, 16, 32])
        most = min(1 << 30, (1 << 25) * N) if op == "scan" else min(1 << 27, (1 << 23) * N)
        most //= D * N  # tokens: the plain form's tensors, and the bytes of a pass
        T = _log_int(rng, 1, min(32768, most))
        B = rng.randint(1, max(1, min(4, most // T)))
        case = dict(op=op, B=B, T=T, D=D, N=N, dtype=dtype, z=rng.random() < 0.7, S0=rng.random() < 0.5)
        if op == "scan":
            case["lens"] = ""
            if rng.random() < 0.4:  # packed: B sequences' tokens cut at random places, empty ones among them
                cuts = sorted(rng.randint(0, B * T) for _ in range(rng.randint(1, 12)))
                ends = [0] + cuts + [B * T]
                case.update(B=1, T=B * T, lens=",".join(str(b - a) for a, b in zip(ends, ends[1:])))
        return case
    if op == "step":
        D, N = _log_int(rng, 64, 4096), rng.choice([8, 16, 16, 32])
        return dict(op=op, B=_log_int(rng, 1, min(512, (1 << 25) // (D * N))), D=D, N=N, dtype=dtype,
                    z=rng.random() < 0.7)
    if op == "conv":
        return dict(op=op, B=rng.randint(1, 4), T=_log_int(rng, 1, 4096), H=rng.randint(1, 16), d=rng.choice([64, 128]),
                    W=rng.choice([2, 3, 4, 4]), dtype=dtype, l2=rng.random() < 0.5, state=rng.random() < 0.5)
    d = rng.choice([64, 128])
    T = _log_int(rng, 1, 4096)
    B = rng.randint(1, max(1, min(4, 8192 // T))) if T > 1 else _log_int(rng, 1, 512)
    return dict(op=op, B=B, T=T, Hq=rng.randint(1, 16), Hk=rng.randint(1, 4), d=d,
                R=rng.choice([d, d, d // 2]), P=_log_int(rng, 4096, 131072), norm=rng.choice(["rms", "rms", "l2"]),
                interleaved=rng.random() < 0.5, dtype=dtype)


def work(case):
    e = SIZE[case["dtype"]]
    op, B = case["op"], case["B"]
    if op in ("scan", "step", "train"):
        T, D, N = case.get("T", 1), case["D"], case["N"]
        tc, z = B * T * D, 1 if case["z"] else 0
        par = 4 * D * (N + 2)
        if op == "step":  # the state read and written, then the token's own values
            return {"bytes": tc * e * (3 + z) + 2 * B * T * N * e + 8 * B * D * N + par, "flops": tc * (7 * N + 12)}
        seqs = len(case["lens"].split(",")) if case.get("lens") else B
        st = 4 * seqs * D * N * (2 if case["S0"] else 1)
        if op == "scan":
            return {"bytes": tc * e * (3 + z) + 2 * B * T * N * e + st + par, "flops": tc * (7 * N + 12)}
        # training: x, dt, z, dy in; y, dx, ddt, dz out; B, C in and their gradients out
        return {"bytes": tc * e * (6 + 2 * z) + 4 * B * T * N * e + 2 * st + 2 * par, "flops": tc * (26 * N + 30)}
    if op == "conv":
        n, W = B * case["T"] * case["H"] * case["d"], case["W"]
        return {"bytes": 3 * n * e + 8 * case["H"] * case["d"] * W, "flops": n * (6 * W + 20)}
    rows = B * case["T"] * (case["Hq"] + case["Hk"])
    n, tab = rows * case["d"], 4 * min(B * case["T"], case["P"]) * case["R"]
    if op == "rope":
        return {"bytes": 2 * n * e + tab, "flops": 8 * n}
    return {"bytes": 4 * n * e + tab, "flops": 24 * n}  # x, dy in; y, dx out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    op, B = case["op"], case["B"]
    s = {"case": case}
    if op in ("scan", "step", "train"):
        T, D, N = case.get("T", 1), case["D"], case["N"]
        lens = [int(v) for v in case["lens"].split(",")] if case.get("lens") else None
        lead = (B,) if op == "step" else (T,) if lens else (B, T)
        s["x"] = torch.nn.functional.silu(rn(*lead, D)).to(t)  # the convolution's output
        if case["z"]:
            s["z"] = rn(*lead, 2 * D).to(t)[..., D:]  # the second half of the input projection
        s["dt"] = (0.5 * rn(*lead, D)).to(t)
        R = -(-D // 16)  # rank of the step-size projection: B and C are the columns after it
        proj = rn(*lead, R + 2 * N).to(t)
        s["Bm"], s["Cm"] = proj[..., R:R + N], proj[..., R + N:]
        # decays -1 .. -N with a spread, step sizes between 1e-3 and 1e-1: the usual initialisation
        s["A"] = -torch.arange(1, N + 1, device="cuda").float() * torch.exp(0.1 * rn(D, N))
        step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1.0 + 0.1 * rn(D)
        seqs = len(lens) if lens else B
        if op == "step":
            s["S"] = rn(B, D, N) * 0.3
        elif case["S0"]:
            s["S0"] = rn(seqs, D, N) * 0.3
        if lens:
            s["cu_seqlens"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        if op == "train":
            s["dy"] = rn(*lead, D).to(t)
        return s
    if op == "conv":
        T, H, d, W = case["T"], case["H"], case["d"], case["W"]
        s["x"] = rn(B, T, H, d).to(t)
        s["dy"] = rn(B, T, H, d).to(t)
        s["weight"] = (torch.rand(H * d, W, generator=g, device="cuda") * 2 - 1) / W ** 0.5
        if case["state"]:
            s["state"] = rn(B, W - 1, H, d).to(t)
        return s
    T, Hq, Hk, d, R, P = (case[k] for k in ("T", "Hq", "Hk", "d", "R", "P"))
    qkv = rn(B, T, (Hq + 2 * Hk) * d).to(t)  # a fused projection; the queries and keys are views of it
    s["q"] = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
    s["k"] = qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    s["q_weight"], s["k_weight"] = 1.0 + 0.1 * rn(d), 1.0 + 0.1 * rn(d)
    # the rotation's table, which a program keeps: angles in 64 bits
    ang = torch.arange(P, device="cuda").double()[:, None] * (
        10000.0 ** (-torch.arange(0, R, 2, device="cuda").double() / R))
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    if T == 1:
        s["positions"] = torch.randint(0, P, (B, T), generator=g, device="cuda").to(torch.int32)
    else:
        first = torch.randint(0, max(1, P - T), (B, 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(T, device="cuda")).remainder(P).to(torch.int32)
    if op == "rope_train":
        s["dq"], s["dk"] = rn(B, T, Hq, d).to(t), rn(B, T, Hk, d).to(t)
    return s


# ------------------------------------------------------------------ plain forms


def _scan(a, b, dim):
    """h_t = a_t h_{t-1} + b_t along `dim` by doubling: log2(T) passes over whole tensors."""
    T, s = a.shape[dim], 1
    while s < T:
        lo = lambda v: v.narrow(dim, 0, T - s)  # noqa: E731
        hi = lambda v: v.narrow(dim, s, T - s)  # noqa: E731
        hi(b).add_(hi(a) * lo(b))
        hi(a).copy_(hi(a) * lo(a))
        s *= 2
    return b


def _softplus(v):
    return torch.where(v > 0, v, 0.0) + torch.log1p(torch.exp(-v.abs()))


def _sequences(case, s):
    """Row of every sequence's first and last token in the [rows, D] matrix, and its length."""
    B, T = case["B"], case["T"]
    if "cu_seqlens" in s:
        cu = s["cu_seqlens"].long()
        return cu[:-1], cu[1:] - 1, cu[1:] - cu[:-1]
    first = torch.arange(B, device="cuda") * T
    return first, first + T - 1, torch.full((B,), T, device="cuda")


def _plain_scan(s):
    case = s["case"]
    D, N, t = case["D"], case["N"], s["x"].dtype
    x, dt, Bm, Cm = (s[k].reshape(-1, s[k].shape[-1]).float() for k in ("x", "dt", "Bm", "Cm"))
    delta = _softplus(dt + s["dt_bias"])
    a = torch.exp(delta[:, :, None] * s["A"])
    b = (delta * x)[:, :, None] * Bm[:, None, :]
    first, last, length = _sequences(case, s)
    some = length > 0
    S0 = s["S0"] if "S0" in s else torch.zeros((len(length), D, N), device="cuda")
    start = first[some]
    b[start] += a[start] * S0[some]
    a[start] = 0.0
    keep = a.clone() if case["op"] == "train" else None
    h = _scan(a, b, 0)
    S_T = S0.clone()
    S_T[some] = h[last[some]]
    pre = (h * Cm[:, None, :]).sum(-1) + s["D"] * x
    y = pre
    if case["z"]:
        z = s["z"].reshape(-1, D).float()
        y = pre * (z * torch.sigmoid(z))
    return y.to(t).reshape(s["x"].shape), S_T, (x, dt, Bm, Cm, delta, keep, h, pre)


def _plain_train(s):
    case = s["case"]
    B, T, D, N, t = case["B"], case["T"], case["D"], case["N"], s["x"].dtype
    y, S_T, (x, dt, Bm, Cm, delta, a, h, pre) = _plain_scan(s)
    g = s["dy"].reshape(-1, D).float()
    out = {"y": y, "S_T": S_T}
    if case["z"]:
        z = s["z"].reshape(-1, D).float()
        sg = torch.sigmoid(z)
        out["dz"] = (g * pre * (sg * (1 + z * (1 - sg)))).to(t).reshape(s["x"].shape)
        g = g * (z * sg)
    # dh_t = C_t g_t + a_{t+1} dh_{t+1}: the same scan on the reversed axis; the factor of a
    # sequence's last token is that of the next sequence's first, which is 0 here
    r = torch.roll(a, -1, 0).flip(0)
    dh = _scan(r, (g[:, :, None] * Cm[:, None, :]).flip(0), 0).flip(0)
    out["dCm"] = (h * g[:, :, None]).sum(1).to(t).reshape(s["Cm"].shape)
    out["dBm"] = (dh * (delta * x)[:, :, None]).sum(1).to(t).reshape(s["Bm"].shape)
    du = (dh * Bm[:, None, :]).sum(-1)
    out["dx"] = (delta * du + s["D"] * g).to(t).reshape(s["x"].shape)
    out["dD"] = (g * x).sum(0)
    first = torch.arange(B, device="cuda") * T
    full = torch.exp(delta[:, :, None] * s["A"])
    out["dS0"] = full[first] * dh[first]
    back = torch.roll(h, 1, 0)
    back[first] = s["S0"] if "S0" in s else 0.0
    q = dh * full * back  # gradient of the exponent
    ddelta = x * du + (q * s["A"]).sum(-1)
    out["dA"] = (q * delta[:, :, None]).sum(0)
    ddt = ddelta * torch.sigmoid(dt + s["dt_bias"])
    out["ddt"] = ddt.to(t).reshape(s["x"].shape)
    out["ddt_bias"] = ddt.sum(0)
    return out


def _plain_step(s):
    case, t = s["case"], s["x"].dtype
    x, dt, Bm, Cm = (s[k].float() for k in ("x", "dt", "Bm", "Cm"))
    delta = _softplus(dt + s["dt_bias"])
    S = torch.exp(delta[:, :, None] * s["A"]) * s["S"] + (delta * x)[:, :, None] * Bm[:, None, :]
    y = (S * Cm[:, None, :]).sum(-1) + s["D"] * x
    if case["z"]:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["S"].copy_(S)  # the state is updated in place
    return {"y": y.to(t), "S": s["S"]}


def _plain_conv(s):
    case = s["case"]
    B, T, H, d, W, t = (*(case[k] for k in ("B", "T", "H", "d", "W")), s["x"].dtype)
    past = s["state"].float() if case["state"] else torch.zeros((B, W - 1, H, d), device="cuda")
    x = torch.cat([past, s["x"].float()], 1).reshape(B, T + W - 1, H * d)
    w = s["weight"]
    taps = x.unfold(1, W, 1)  # [B, T, C, W]: the inputs that the taps meet
    u = (taps * w).sum(-1)
    sg = torch.sigmoid(u)
    y, dy = u * sg, s["dy"].float().reshape(B, T, H * d)
    ds = dy
    if case["l2"]:
        yh, gh = y.unflatten(-1, (H, d)), dy.unflatten(-1, (H, d))
        r = torch.sqrt((yh * yh).sum(-1, keepdim=True) + EPS)
        yh = yh / r
        ds = ((gh - yh * (gh * yh).sum(-1, keepdim=True)) / r).flatten(-2)
    du = ds * (sg * (1 + u * (1 - sg)))
    dw = (taps * du[..., None]).sum((0, 1))
    pad = torch.nn.functional.pad(du, (0, 0, W - 1, W - 1))  # du is 0 outside the sequence
    dx = (pad.unfold(1, W, 1) * w.flip(-1)).sum(-1).to(t).reshape(B, T + W - 1, H, d)
    out = {"dx": dx[:, W - 1:].contiguous(), "dweight": dw}
    if case["state"]:
        out["dstate"] = dx[:, :W - 1].contiguous()
    return out


def _rotate(v, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    a, b = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([turned, v[..., R:]], -1)


def _plain_rope(s, name):
    case, x = s["case"], s[name]
    t, R, w, l2 = x.dtype, case["R"], s[name + "_weight"], case["norm"] == "l2"
    row = s["cos_sin"][s["positions"].long()][:, :, None, :]
    cos, sin = row[..., :R // 2], row[..., R // 2:]
    v = x.float()
    sq = (v * v).sum(-1, keepdim=True)
    r = torch.sqrt((sq if l2 else sq / case["d"]) + EPS)
    xh = v / r
    y = _rotate(xh * w, cos, sin, case["interleaved"]).to(t)
    if case["op"] == "rope":
        return y, None, None
    dv = _rotate(s["d" + name].float(), cos, -sin, case["interleaved"])
    dw = (dv * xh).sum((0, 1, 2))
    dh = dv * w
    dot = (dh * xh).sum(-1, keepdim=True)
    dx = (dh - xh * (dot if l2 else dot / case["d"])) / r
    return y, dx.to(t), dw


def _run_plain(s):
    op = s["case"]["op"]
    if op == "scan":
        y, S_T, _ = _plain_scan(s)
        return {"y": y, "S_T": S_T}
    if op == "train":
        return _plain_train(s)
    if op == "step":
        return _plain_step(s)
    if op == "conv":
        return _plain_conv(s)
    qo, dq, dqw = _plain_rope(s, "q")
    ko, dk, dkw = _plain_rope(s, "k")
    out = {"q": qo, "k": ko}
    if op == "rope_train":
        out.update(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    return out


# ------------------------------------------------------------------ the library's calls


def _run_own(s):
    import gated_delta_rule_wy_b200 as gdr2

    case = s["case"]
    op = case["op"]
    if op in ("scan", "step", "train"):
        args = [s[k] for k in ("x", "dt", "A", "Bm", "Cm")]
        par = dict(D=s["D"], z=s.get("z"), dt_bias=s["dt_bias"])
        if op == "step":
            return {"y": gdr2.gdr2_ssm_step(*args, s["S"], **par), "S": s["S"]}
        y, S_T, saved = gdr2.gdr2_ssm_scan(*args, S0=s.get("S0"), cu_seqlens=s.get("cu_seqlens"),
                                           save_states=op == "train", **par)
        out = {"y": y, "S_T": S_T}
        if op == "train":
            grads = gdr2.gdr2_ssm_scan_backward(*args, s["dy"], S0=s.get("S0"), saved_states=saved, **par)
            out.update({k: v for k, v in grads.items() if v is not None})
        return out
    if op == "conv":
        g = gdr2.gdr2_short_conv_silu_backward(s["x"], s["weight"], s["dy"], s.get("state"), l2norm=case["l2"], eps=EPS)
        return {k: v for k, v in g.items() if v is not None}
    par = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], cos_sin=s["cos_sin"], positions=s["positions"],
               norm=case["norm"], eps=EPS, interleaved=case["interleaved"])
    qo, ko = gdr2.gdr2_head_norm_rope(s["q"], s["k"], **par)
    out = {"q": qo, "k": ko}
    if op == "rope_train":
        out.update(gdr2.gdr2_head_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], **par))
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_scan(case, s):
    """The recurrence token by token (all batch entries at once), then its reverse."""
    op, B, T, D = case["op"], case["B"], case.get("T", 1), case["D"]
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    rows = lambda k: f[k].reshape(B, T, -1).transpose(0, 1)  # noqa: E731
    x, Bm, Cm = rows("x"), rows("Bm"), rows("Cm")
    delta = torch.logaddexp(rows("dt") + f["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    lens = s["cu_seqlens"].diff().tolist() if "cu_seqlens" in s else None
    first = "S" if op == "step" else "S0"
    S0 = f[first] if first in f else torch.zeros((len(lens) if lens else B, D, case["N"]), dtype=torch.float64,
                                                 device="cuda")
    starts, ends, at = {0: None}, {}, 0
    if lens:
        starts = {}
        for i, n in enumerate(lens):
            if n:
                starts[at], ends[at + n - 1] = i, i
            at += n
    h, S_T, kept = S0, S0.clone(), []
    pre = torch.empty((T, B, D), dtype=torch.float64, device="cuda")
    for t in range(T):
        if t in starts and lens:
            h = S0[starts[t]][None]
        if op == "train":
            kept.append(h)
        h = torch.exp(delta[t][..., None] * f["A"]) * h + (delta[t] * x[t])[..., None] * Bm[t][:, None, :]
        pre[t] = torch.einsum("bcn,bn->bc", h, Cm[t])
        if t in ends:
            S_T[ends[t]] = h[0]
    if not lens:
        S_T = h
    pre += f["D"] * x
    back = lambda v: v.transpose(0, 1).reshape(s["x"].shape[:-1] + v.shape[-1:])  # noqa: E731
    y, z = pre, rows("z") if case["z"] else None
    if case["z"]:
        y = pre * z / (1 + torch.exp(-z))
    if op != "train":
        return {"y": back(y), "S" if op == "step" else "S_T": S_T}
    out = {"y": back(y), "S_T": S_T}
    g = rows("dy")
    if case["z"]:
        sg = 1 / (1 + torch.exp(-z))
        out["dz"] = back(g * pre * (sg + z * sg * (1 - sg)))
        g = g * z * sg
    dA, dD = torch.zeros_like(f["A"]), (g * x).sum((0, 1))
    dx, ddt = torch.empty_like(x), torch.empty_like(delta)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    e = torch.zeros_like(S0)  # a_{t+1} dh_{t+1}
    for t in reversed(range(T)):
        a = torch.exp(delta[t][..., None] * f["A"])
        hp = kept[t]
        dh = e + g[t][..., None] * Cm[t][:, None, :]
        ht = a * hp + (delta[t] * x[t])[..., None] * Bm[t][:, None, :]
        dC[t] = (ht * g[t][..., None]).sum(1)
        dB[t] = (dh * (delta[t] * x[t])[..., None]).sum(1)
        du = (dh * Bm[t][:, None, :]).sum(-1)
        dx[t] = delta[t] * du + f["D"] * g[t]
        m = dh * a * hp
        dA += (m * delta[t][..., None]).sum(0)
        ddt[t] = (x[t] * du + (m * f["A"]).sum(-1)) * (1 - torch.exp(-delta[t]))  # sigmoid = 1 - e^-softplus
        e = a * dh
    out.update(dx=back(dx), ddt=back(ddt), dBm=back(dB), dCm=back(dC), dA=dA, dD=dD, ddt_bias=ddt.sum((0, 1)), dS0=e)
    return out


def _exact_conv(case, s):
    B, T, H, d, W = (case[k] for k in ("B", "T", "H", "d", "W"))
    x, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double().reshape(H, d, W)
    past = s["state"].double() if case["state"] else x.new_zeros((B, W - 1, H, d))
    xp = torch.cat([past, x], 1)
    u = sum(w[..., i] * xp[:, i:i + T] for i in range(W))
    sg = 1 / (1 + torch.exp(-u))
    v = u * sg
    ds = dy
    if case["l2"]:
        n2 = (v * v).sum(-1, keepdim=True) + EPS
        ds = dy * n2 ** -0.5 - v * (dy * v).sum(-1, keepdim=True) * n2 ** -1.5
    du = ds * (sg + u * sg * (1 - sg))
    dw = torch.stack([(du * xp[:, i:i + T]).sum((0, 1)) for i in range(W)], -1).reshape(H * d, W)
    dxp = torch.zeros_like(xp)
    for i in range(W):
        dxp[:, i:i + T] += w[..., i] * du
    out = {"dx": dxp[:, W - 1:], "dweight": dw}
    if case["state"]:
        out["dstate"] = dxp[:, :W - 1]
    return out


def _exact_rope(case, s):
    out, R, d = {}, case["R"], case["d"]
    row = s["cos_sin"].double()[s["positions"].long()][:, :, None, :]
    turn = torch.complex(row[..., :R // 2], row[..., R // 2:])
    l2 = case["norm"] == "l2"

    def rotated(v, by):
        if case["interleaved"]:
            p = torch.view_as_complex(v[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * by
            front = torch.view_as_real(p).flatten(-2)
        else:
            p = torch.complex(v[..., :R // 2].contiguous(), v[..., R // 2:R].contiguous()) * by
            front = torch.cat([p.real, p.imag], -1)
        return torch.cat([front, v[..., R:]], -1)

    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"].double()
        m = ((x * x).sum(-1, keepdim=True) if l2 else (x * x).mean(-1, keepdim=True)) + EPS
        out[n] = rotated(x * m ** -0.5 * w, turn)
        if case["op"] == "rope_train":
            dv = rotated(s["d" + n].double(), turn.conj())
            out["d" + n + "_weight"] = (dv * x * m ** -0.5).sum((0, 1, 2))
            dot = (dv * w * x).sum(-1, keepdim=True)
            out["d" + n] = dv * w * m ** -0.5 - x * dot * m ** -1.5 / (1 if l2 else d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "step", "train"):
        return _exact_scan(case, s)
    return _exact_conv(case, s) if op == "conv" else _exact_rope(case, s)


if __name__ == "__main__":
    rng = random.Random(0)
    for c in listed() + [draw(rng) for _ in range(8)]:
        print(c, work(c))
