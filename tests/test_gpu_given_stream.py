"""Calls on a given stream: what they allocate, and who reads it."""
import pytest
import torch

from gated_delta_rule_wy_b200 import gdr2_ssm_scan, gdr2_sync_status
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
