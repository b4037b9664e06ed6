"""MuonStepPlan(mx_forms=True) on other streams than the one it was made on."""
import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu

SHAPES = [(768, 768), (768, 3072), (3072, 768)]


def make(shapes=SHAPES):
    g = torch.Generator().manual_seed(3)
    W = [(0.02 * torch.randn(s, generator=g)).cuda() for s in shapes]
    G = [(1e-2 * torch.randn(s, generator=g)).bfloat16().cuda() for s in shapes]
    return W, G, [torch.zeros_like(w) for w in W]


def check(plan, W, V):
    torch.cuda.synchronize()
    for w, v, pair in zip(W, V, plan.mx_forms):
        assert torch.equal(w, v)
        for got, want in zip(pair, nsb.muon_mx_quantize(v, rows=True, cols=True)):
            assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("way", ["call", "capture", "replay"])
def test_made_on_one_stream_and_run_on_another(way, handle):
    """The filling is held up on its stream; the step on the other one comes after it all the same."""
    W, G, M = make()
    V, N = [w.clone() for w in W], [m.clone() for m in M]
    nsb.muon_step(V, G, N)
    if way != "call":
        nsb.muon_step(V, G, N)
    torch.cuda.synchronize()
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    with torch.cuda.stream(a):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        plan = nsb.MuonStepPlan(W, G, M, mx_forms=True)
    if way == "call":
        plan(stream=b.cuda_stream if handle else b)
    elif way == "capture":  # one step by capture itself, one by the replay
        with torch.cuda.stream(c):
            plan.capture(b)
            plan.replay()
    else:
        with torch.cuda.stream(a):
            plan.capture(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(c):
            plan.replay()
    check(plan, W, V)


def test_memory_of_a_dropped_plan_is_not_given_away_while_its_call_runs():
    W, G, M = make()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    plan = nsb.MuonStepPlan(W, G, M, mx_forms=True)
    plan(s)  # the workspace of that stream
    torch.cuda.synchronize()
    buffer = plan.mx_forms[0][0]._buffer
    at, size = buffer.data_ptr(), buffer.numel()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    plan(s)
    del plan, buffer
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert not s.query()
    assert other.data_ptr() + size <= at or at + size <= other.data_ptr()
    torch.cuda.synchronize()
