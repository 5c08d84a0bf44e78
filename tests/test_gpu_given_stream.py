"""Calls on a given stream: what they allocate, and who reads it."""
import pytest
import torch

from gated_delta_rule_wy_b200 import gdr2_forward_segmented, gdr2_ssm_scan, gdr2_sync_status
from gated_delta_rule_wy_b200 import inputs as I
from test_gpu_ssm import cuda, make

pytestmark = pytest.mark.gpu


def test_outputs_of_a_given_stream_outlive_their_readers():
    """Outputs read on the caller's stream, late, and let go: the given stream's next calls must not be handed their
    memory before that read."""
    v, w = (cuda(make((2, 300), 64, 16, torch.float32, seed, states=2)) for seed in (430, 431))
    want = gdr2_ssm_scan(**v)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        y, S_T, _ = gdr2_ssm_scan(**v, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(50_000_000)
        kept = y.clone(), S_T.clone()
        del y, S_T
        for _ in range(4):
            gdr2_ssm_scan(**w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(kept[0], want[0]) and torch.equal(kept[1], want[1])
    gdr2_sync_status()


def test_a_given_stream_inside_a_capture():
    """A side stream forked and joined inside a capture: replays give the eager call's bits for new inputs."""
    v, w = (cuda(make((2, 300), 64, 16, torch.bfloat16, seed, states=2)) for seed in (432, 433))
    want = gdr2_ssm_scan(**w)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        y, S_T, _ = gdr2_ssm_scan(**v, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        y2 = y + 0
        S2 = S_T + 0
        del y, S_T
        s.wait_stream(torch.cuda.current_stream())
        again = gdr2_ssm_scan(**v, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for k in v:
        if torch.is_tensor(v[k]):
            v[k].copy_(w[k])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, want[0]) and torch.equal(S2, want[1])
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_segmented_forward_makes_its_own_inputs_on_the_given_stream():
    """The zero and identity inputs of the segments' transitions are made where they are read: not behind what the
    caller's stream still has to do, and not in memory that its tensors get back."""
    x = I.make_forward_inputs(B=1, H=2, T=512, dk=128, dv=128, dtype=torch.bfloat16, decay_shift=2.0, seed=145,
                              with_S0=True).to("cuda")
    args = (x.q, x.k, x.v, x.log_alpha, x.b, x.w, x.S0)
    want = gdr2_forward_segmented(*args, segments=4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(50_000_000)
        o, S_T = gdr2_forward_segmented(*args, segments=4, stream=s)
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 15, 1 << 17, 1 << 20)]
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(S_T, want[1])
    torch.cuda.synchronize()
    gdr2_sync_status()
    assert all(t.isnan().all() for t in junk)
