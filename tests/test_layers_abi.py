"""Refusals of the layer entry points, on the host before any launch (no GPU needed)."""
import ctypes

import pytest

import gated_delta_rule_wy_b200 as g
from gated_delta_rule_wy_b200 import binding as b

P, Q, S = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000))
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_wy_b200 import build

    build.build()
    return g.load_library()


def scan(lib, B=1, T=8, D=16, N=16, dt=1, soft=1, cu=None, x=P, ldx=16, step=P, lds=16, A=P, Bm=P, ldb=16, Cm=P, ldc=16,
         skip=None, z=None, ldz=0, bias=None, S0=None, y=Q, S_T=S, saved=None, ws=P, nws=1 << 40):
    return lib.gdr2_ssm_scan(B, T, D, N, dt, soft, cu, x, ldx, step, lds, A, Bm, ldb, Cm, ldc, skip, z, ldz, bias, S0, y,
                             S_T, saved, ws, ctypes.c_size_t(nws), None)


@pytest.mark.parametrize("bad,word", [
    (dict(dt=3), b"dtype"), (dict(B=-1), b"negative"), (dict(T=-1), b"negative"), (dict(D=-1), b"negative"),
    (dict(soft=2), b"softplus"), (dict(x=None), b"x is NULL"), (dict(step=None), b"step is NULL"),
    (dict(A=None), b"A is NULL"), (dict(Bm=None), b"Bm is NULL"), (dict(Cm=None), b"Cm is NULL"),
    (dict(y=None), b"y is NULL"), (dict(x=ODD), b"x is not 2-byte"), (dict(ldx=15), b"rows of x"),
    (dict(ldb=15), b"rows of Bm"), (dict(z=P, ldz=3), b"rows of z"), (dict(A=ctypes.c_void_p(0x10008)), b"A is not 16"),
    (dict(S0=S), b"S_T must not be S0"), (dict(y=P), b"y must not be x"), (dict(skip=ODD), b"Dskip"),
    (dict(bias=ODD), b"step_bias"), (dict(cu=ODD), b"cu_seqlens"), (dict(T=1 << 20, B=1 << 12, D=1 << 12), b"too large"),
    (dict(T=4096, nws=16), b"workspace"), (dict(T=4096, ws=None), b"workspace"),
])
def test_scan_refuses(lib, bad, word):
    assert scan(lib, **bad) == b.GDR2_ERR_INVALID_ARG and word in lib.gdr2_last_error()


def test_scan_sizes_not_supported_and_nothing_to_do(lib):
    for N in (0, 4, 12, 128, -8):
        assert scan(lib, N=N) == b.GDR2_ERR_UNSUPPORTED
    assert scan(lib, cu=Q, saved=P) == b.GDR2_ERR_UNSUPPORTED and b"dense" in lib.gdr2_last_error()
    nothing = dict(x=None, step=None, A=None, Bm=None, Cm=None, y=None, S_T=None, ws=None, nws=0)
    assert scan(lib, B=0, **nothing) == b.GDR2_OK and scan(lib, D=0, **nothing) == b.GDR2_OK
    assert scan(lib, T=0, **nothing) == b.GDR2_OK
    assert scan(lib, B=0, cu=Q) == b.GDR2_ERR_INVALID_ARG  # tokens without sequences


def test_workspace_queries(lib):
    assert lib.gdr2_ssm_scan_workspace_bytes(8, 4096, 65536, 16) == 0  # the channels fill the GPU
    n = lib.gdr2_ssm_scan_workspace_bytes(1, 4096, 2048, 16)
    assert n > 0 and n % 256 == 0
    assert lib.gdr2_ssm_scan_workspace_bytes(1, 4096, 2048, 12) == 0
    a, c = (lib.gdr2_ssm_scan_backward_workspace_bytes(2, 100, 64, 16, h) for h in (1, 0))
    assert c >= a + 2 * 7 * 64 * 16 * 4 and a % 256 == 0
    assert lib.gdr2_short_conv_silu_backward_workspace_bytes(2, 100, 3, 64, 4) >= 2 * 3 * 64 * 4 * 4
    assert lib.gdr2_short_conv_silu_backward_workspace_bytes(2, 100, 3, 96, 4) == 0
    assert lib.gdr2_head_norm_rope_backward_workspace_bytes(128) > 0
    assert lib.gdr2_head_norm_rope_backward_workspace_bytes(96) == 0


def test_step_refuses(lib):
    def step(B=1, D=16, N=16, dt=1, soft=1, x=P, st=S, y=Q, A=P):
        return lib.gdr2_ssm_step(B, D, N, dt, soft, x, 16, P, 16, A, P, 16, P, 16, None, None, 0, None, st, y, None)

    assert step(N=24) == b.GDR2_ERR_UNSUPPORTED
    assert step(st=None) == b.GDR2_ERR_INVALID_ARG and b"S is NULL" in lib.gdr2_last_error()
    assert step(y=P) == b.GDR2_ERR_INVALID_ARG
    assert step(st=ctypes.c_void_p(0x30004)) == b.GDR2_ERR_INVALID_ARG
    assert step(B=-1) == b.GDR2_ERR_INVALID_ARG
    assert step(B=0, x=None, st=None, y=None, A=None) == b.GDR2_OK


def test_scan_backward_refuses(lib):
    def bwd(B=1, T=8, D=16, N=16, dt=1, x=P, z=None, dy=P, dS_T=None, saved=P, dx=Q, dA=Q, dz=None, dS0=None, ws=P,
            nws=1 << 40):
        return lib.gdr2_ssm_scan_backward(B, T, D, N, dt, 1, x, 16, P, 16, P, P, 16, P, 16, None, z, 16, None, None, dy,
                                          dS_T, saved, dx, Q, dA, Q, Q, None, dz, None, dS0, ws, ctypes.c_size_t(nws),
                                          None)

    for bad, word in ((dict(dy=None), b"dy"), (dict(dx=None), b"dx"), (dict(dA=None), b"dA"), (dict(z=P), b"dz"),
                      (dict(dS_T=S, dS0=S), b"dS0"), (dict(nws=16), b"workspace"), (dict(ws=ctypes.c_void_p(0x10010)),
                                                                                  b"workspace"), (dict(dt=9), b"dtype"),
                      (dict(saved=ODD), b"saved_states"), (dict(T=-2), b"negative")):
        assert bwd(**bad) == b.GDR2_ERR_INVALID_ARG and word in lib.gdr2_last_error(), bad
    assert bwd(N=20) == b.GDR2_ERR_UNSUPPORTED


def test_conv_backward_refuses(lib):
    def conv(N=1, T=8, H=2, d=64, dt=1, W=4, l2=0, eps=1e-6, x=P, w=P, st=None, dy=P, dso=None, dx=Q, dw=Q, ds=None,
             ws=P, nws=1 << 40):
        return lib.gdr2_short_conv_silu_backward(N, T, H, d, dt, W, l2, ctypes.c_float(eps), x, w, st, dy, dso, dx, dw,
                                                 ds, ws, ctypes.c_size_t(nws), None)

    for bad, word in ((dict(x=None), b"x is NULL"), (dict(dy=None), b"dy"), (dict(dx=P), b"dx must not"),
                      (dict(w=None), b"weight"), (dict(dw=None), b"dweight"), (dict(nws=3), b"workspace"),
                      (dict(eps=-1.0), b"l2_eps"), (dict(eps=float("nan")), b"l2_eps"), (dict(l2=2), b"l2norm"),
                      (dict(st=S, ds=S), b"dstate_in"), (dict(N=-1), b"negative"), (dict(x=ctypes.c_void_p(0x10008)), b"x")):
        assert conv(**bad) == b.GDR2_ERR_INVALID_ARG and word in lib.gdr2_last_error(), bad
    assert conv(W=5) == b.GDR2_ERR_UNSUPPORTED and conv(W=0) == b.GDR2_ERR_UNSUPPORTED and conv(d=96) == b.GDR2_ERR_UNSUPPORTED
    assert conv(N=0, x=None, w=None, dy=None, dx=None, dw=None, ws=None) == b.GDR2_OK


def rope(lib, B=1, T=4, Hq=2, Hk=1, d=64, dt=1, norm=1, eps=1e-6, q=P, ldq=128, k=P, ldk=64, wq=None, wk=None, R=64, il=0,
         cs=P, n=16, pos=None, first=0, qo=Q, ko=S):
    return lib.gdr2_head_norm_rope(B, T, Hq, Hk, d, dt, norm, ctypes.c_float(eps), q, ldq, k, ldk, wq, wk, R, il, cs, n,
                                   pos, first, qo, ko, None)


@pytest.mark.parametrize("bad,word", [
    (dict(dt=4), b"dtype"), (dict(B=-1), b"negative"), (dict(Hq=-1), b"negative"), (dict(norm=3), b"norm"),
    (dict(norm=-1), b"norm"), (dict(eps=-1.0), b"eps"), (dict(il=2), b"interleaved"), (dict(q=None), b"q is NULL"),
    (dict(k=None), b"k is NULL"), (dict(ldq=127), b"rows of q"), (dict(ldq=129), b"16 bytes"), (dict(wq=ODD), b"q_weight"),
    (dict(cs=None), b"cos_sin"), (dict(n=3), b"outside"), (dict(first=13), b"outside"), (dict(first=-1), b"negative"),
    (dict(pos=ODD), b"positions"), (dict(qo=None), b"q_out"), (dict(ko=None), b"k_out"), (dict(qo=P), b"must not be"),
    (dict(first=2 ** 31 - 1), b"outside"),
])
def test_head_norm_rope_refuses(lib, bad, word):
    assert rope(lib, **bad) == b.GDR2_ERR_INVALID_ARG and word in lib.gdr2_last_error()


def test_head_norm_rope_sizes(lib):
    for bad in (dict(d=96), dict(R=24), dict(R=80), dict(R=-16)):
        assert rope(lib, **bad) == b.GDR2_ERR_UNSUPPORTED
    assert rope(lib, T=0, q=None, k=None, cs=None, qo=None, ko=None) == b.GDR2_OK
    assert rope(lib, Hq=0, Hk=0, q=None, k=None, cs=None, qo=None, ko=None) == b.GDR2_OK


def test_bindings_check_before_calling():
    import torch

    x, n = torch.zeros(1, 8, 16), torch.zeros(1, 8, 16)
    A = torch.zeros(16, 16)
    with pytest.raises(ValueError, match="CUDA"):
        g.gdr2_ssm_scan(x, x, A, n, n)
    with pytest.raises(ValueError, match=r"\[B, T, C\]"):
        g.gdr2_ssm_scan(x[0], x[0], A, n[0], n[0])
    with pytest.raises(ValueError, match=r"\[B, T, C\]"):
        g.gdr2_ssm_scan_backward(x[0], x[0], A, n[0], n[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        g.gdr2_ssm_step(x[0], x[0], A, n[0], n[0], torch.zeros(8, 16, 16))
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        g.gdr2_head_norm_rope(q)
    with pytest.raises(ValueError, match="norm must be"):
        g.gdr2_head_norm_rope(q, norm="layer")
    with pytest.raises(ValueError, match="CUDA"):
        g.gdr2_short_conv_silu_backward(q, torch.zeros(128, 4), q)
    with pytest.raises(ValueError, match="one CUDA device"):
        g.gdr2_ssm_scan(x, x, A, n, torch.zeros(1, 8, 16, device="meta"))


def test_row_strides_of_views():
    """The distance between rows, or a refusal, from shapes and strides alone (a stand-in for a
    CUDA tensor: the check reads metadata only)."""
    import torch

    class Fake:
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    rows = lambda t, lead, w: b._rows(Fake(t), "x", lead, w, torch.float32)  # noqa: E731
    base = torch.zeros(2, 6, 40)
    assert rows(base, (2, 6), 40) == 40
    assert rows(base[..., 7:23], (2, 6), 16) == 40
    assert rows(base[:, 3], (2,), 40) == 240          # one token of each sequence
    assert rows(base[:1, :, :5], (1, 6), 5) == 40
    assert rows(base[:, :1, :5], (2, 1), 5) == 240
    assert rows(base[:1, :1], (1, 1), 40) == 40
    for bad, lead, w in ((base[:, :4], (2, 4), 40), (base[..., ::2], (2, 6), 20), (base.transpose(0, 1), (6, 2), 40),
                         (base[:, :1].expand(2, 6, 40), (2, 6), 40)):
        with pytest.raises(ValueError):
            rows(bad, lead, w)


def test_norm_and_rotation_refuse_what_their_counters_cannot_hold(lib):
    assert rope(lib, B=40000, T=40000, n=40000) == b.GDR2_ERR_INVALID_ARG and b"large" in lib.gdr2_last_error()
