"""Workspaces of the operators around the routed experts: one that other calls have used, one of
uninitialised memory, and the scratch that calls without a workspace share."""
import ctypes
import threading

import pytest
import torch

import block_reference as R
from helpers import run_fused
from mixture_experts_forward_moe_gb300 import binding as B
from mixture_experts_forward_moe_gb300 import inputs

pytestmark = pytest.mark.gpu


def router_case(T, E, k, lens, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g)
    ids = x.topk(k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, generator=g) < 0.05] = -1
    off = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return x.cuda(), ids.cuda(), None if off is None else off.cuda()


def balance_bytes(T, E, k, n_seq):
    p = B.make_problem(T, 8, E, 8, k)
    return int(B.lib().moe_balance_loss_workspace_size(ctypes.byref(p), n_seq))


def assert_balance(got, x, ids, off, scoring):
    T = x.shape[0]
    loss, counts, live, sums, coef = R.balance64(x.cpu().double(), ids.cpu(), 0.25, scoring, off)
    assert torch.equal(got["counts"].cpu(), counts)
    assert torch.equal(got["live_tokens"].cpu(), live)
    rel = (64 + T) * R.F32  # 64 roundings of a probability, and the sum over tokens
    R.assert_within(got["prob_sum"], sums, rel * sums + 1e-37, "prob_sum")
    R.assert_within(got["coef"], coef, 16 * R.F32 * coef, "coef")
    R.assert_within(got["loss"], loss.view(1), (rel + 32 * R.F32) * loss.view(1), "loss")


# T, E, k, lengths, scoring: the loss is joined by several CTAs
SHARED = [
    (1024, 256, 8, None, "softmax"),
    (1500, 256, 8, [37] * 40 + [20], "sigmoid"),
    (0, 256, 8, [0] * 700, "softmax"),
]


@pytest.mark.parametrize("T,E,k,lens,scoring", SHARED)
def test_balance_loss_on_the_workspace_of_the_fused_forward(T, E, k, lens, scoring, cuda_device):
    w = inputs.Workload("shared-workspace", T=512, H=256, E=64, F=128, top_k=4)
    d = inputs.generate(w, seed=1, device=cuda_device)
    prob = B.make_problem(w.T, w.H, w.E, w.F, w.top_k)
    n_seq = 1 if lens is None else len(lens)
    ws = B.new_workspace(max(B.workspace_size(prob), balance_bytes(T, E, k, n_seq)))
    x, ids, off = router_case(T, E, k, lens, seed=2)
    want = None
    for _ in range(2):
        out = run_fused(w, d, workspace=ws)
        want = out.clone() if want is None else want
        assert torch.equal(out, want)
        # what an output that is not written would show
        poison = torch.full((3 * n_seq * E + n_seq + 64,), float("nan"), device=cuda_device)
        del poison
        got = B.moe_balance_loss(x, ids, 0.25, scoring, seq_offsets=off, workspace=ws)
        assert B.get_device_status(ws) == B.MOE_OK
        assert_balance(got, x, ids, off, scoring)


@pytest.mark.parametrize("T,E,k,lens,scoring", SHARED)
def test_balance_loss_needs_no_more_than_a_clear_status_word(T, E, k, lens, scoring, cuda_device):
    n_seq = 1 if lens is None else len(lens)
    ws = torch.full((balance_bytes(T, E, k, n_seq),), 0x5b, dtype=torch.uint8, device=cuda_device)
    ws[:4] = 0
    x, ids, off = router_case(T, E, k, lens, seed=3)
    for _ in range(2):
        got = B.moe_balance_loss(x, ids, 0.25, scoring, seq_offsets=off, workspace=ws)
        assert B.get_device_status(ws) == B.MOE_OK
        assert_balance(got, x, ids, off, scoring)


def test_threads_share_the_scratch_of_a_stream(cuda_device):
    x = torch.randn(64, 512, device=cuda_device).to(torch.bfloat16)
    y = torch.randn(200, 2048, device=cuda_device).to(torch.bfloat16)
    g = torch.randn_like(y)
    want = B.moe_linear(x, x)
    B.moe_block_norm_bwd(g, g, y)
    where = B.call_workspace().data_ptr()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    seen, failures = [], []

    def work():
        try:
            out = B.moe_linear(x, x)
            B.moe_block_norm_bwd(g, g, y)
            seen.append(B.call_workspace().data_ptr())
            assert torch.equal(out, want)
        except BaseException as e:  # reported by the test's own thread
            failures.append(e)

    for _ in range(4):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failures
    assert seen == [where] * 4
    assert torch.cuda.memory_allocated() == before


def test_a_larger_scratch_keeps_what_was_reported(cuda_device):
    x, ids, _ = router_case(70, 32, 4, None, seed=4)
    ids[5, 1] = 32
    B.moe_balance_loss(x, ids, 1.0)
    held = B.call_workspace()
    # a call that needs twice the scratch
    grown = B._call("scratch", None, (2 * held.numel(), torch.cuda.current_device()))
    assert grown.numel() >= 2 * held.numel()
    assert B.get_device_status(B.call_workspace()) == B.MOE_ERR_BAD_EXPERT_ID
    assert B.get_device_status(B.call_workspace()) == B.MOE_OK


def test_a_workspace_on_another_device_is_refused(cuda_device):
    x = torch.randn(8, 64, device=cuda_device).to(torch.bfloat16)
    # none but the first GPU is used here: a host buffer stands for one elsewhere
    with pytest.raises(ValueError, match="workspace"):
        B.moe_linear(x, x, workspace=torch.zeros(256, dtype=torch.uint8))
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError, match="workspace is on another device"):
            B.moe_linear(x, x, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda:1"))
