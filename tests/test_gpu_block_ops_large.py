"""The operators around the routed experts at sizes that reach their kernels for many rows: several
rows per persistent CTA, every gate, rows too long for the per-channel vectors in shared memory,
ragged tiles of the products, long records of the balance loss.  References in 64 bits on the GPU."""
import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, norm_inputs, rand, status

pytestmark = pytest.mark.gpu

# T, N, K, dtype, act, bias, residual, f32
LINEAR = [
    (2, 4096, 4160, BF, "none", True, False, True),       # few rows, large product
    (4, 2056, 8192, HF, "silu", False, True, False),
    (12, 7168, 7168, BF, "none", False, False, True),
    (48, 1536, 2048, BF, "gelu_tanh", True, True, False),
    (96, 300, 7168, BF, "none", True, True, True),        # K split over pairs, f32 sums
    (300, 4096, 4104, HF, "relu2", True, False, False),
    (512, 4096, 1024, BF, "none", False, True, True),     # f32, no split
    (1000, 5000, 1032, BF, "silu", True, True, False),    # 256-column tiles, ragged everywhere
    (1300, 6152, 520, HF, "none", True, True, False),
    (4100, 2049, 264, BF, "gelu_tanh", True, True, False),
    (4100, 2048, 2056, BF, "none", False, True, True),
]


# few output columns (at most one 128-row slab of weights) and many rows, on both sides of the edge
NARROW = [
    (4096, 128, 2048, BF, "none", True, False, True),
    (4097, 100, 7168, HF, "gelu_tanh", True, True, False),
    (2048, 127, 18432, BF, "none", False, False, True),
    (9001, 64, 1032, BF, "silu", True, True, False),
    (20000, 1, 2048, HF, "none", True, False, True),
    (16384, 128, 7168, BF, "none", True, True, True),
    (2500, 129, 7168, BF, "relu2", True, True, False),
    (4096, 128, 7168, BF, "none", True, False, True),     # f32: two tiles on an SM, K in four parts
    (64, 7168, 7168, BF, "none", False, True, True),
    (40, 9728, 7168, HF, "none", False, False, True),
]


@pytest.mark.parametrize("T,N,K,dtype,act,bias,res,f32", LINEAR + NARROW)
def test_linear(T, N, K, dtype, act, bias, res, f32, cuda_device):
    odt = torch.float32 if f32 else dtype
    x = rand(T, K, seed=1, dtype=dtype)
    w = rand(N, K, seed=2, std=K ** -0.5, dtype=dtype)
    b = rand(N, seed=3, dtype=dtype) if bias else None
    r = rand(T, N, seed=4, dtype=odt) if res else None
    kw = dict(bias=b, activation=act, residual=r, out_dtype=torch.float32 if f32 else None)
    out, again = B.moe_linear(x, w, **kw), B.moe_linear(x, w, **kw)
    assert out.dtype == odt and status(cuda_device) == B.MOE_OK
    assert torch.equal(out, again)
    z, mag = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    off = (K / 16 + 16) * 2 * R.F32 * mag
    a = R.act64(z, act)
    slope = {"none": 1.0, "silu": 1.2, "gelu_tanh": 1.2}.get(act)
    err = off * (2 * (z.abs() + off) if slope is None else slope) + 2.0 ** -20 * a.abs()
    if res:
        a = a + r.double()
        err = err + 2 * R.F32 * (a.abs() + r.double().abs())
    over = (out.double() - a).abs() - err - R.half_step(a, odt) * (1 + 2.0 ** -7)
    assert float(over.max()) <= 0, float(over.max())


# The f32 sums' error in norms: an accumulator meets at most eight 64-k blocks, 32 additions, and
# each may truncate by a step (2^-23) of a partial sum that in norms is at most the result.  The
# truncations of one accumulator go one way, so they add: 32 * 2^-23, and half of it on average
# (a truncation loses half a step).  The sums of accumulators and parts add a few roundings.
@pytest.mark.parametrize("T,N,K", [(4096, 128, 2048), (4096, 128, 7168), (2048, 128, 18432),
                                   (64, 7168, 7168), (300, 128, 32768), (96, 300, 18432)])
def test_linear_f32_sums_stay_short(T, N, K, cuda_device):
    x, w = rand(T, K, seed=5, dtype=BF), rand(N, K, seed=6, std=K ** -0.5, dtype=BF)
    guard = 1 << 12
    buf = torch.full((T * N + 2 * guard,), -77.0, device=cuda_device)
    out = buf[guard:guard + T * N].view(T, N)
    B.moe_linear(x, w, out_dtype=torch.float32, out=out)
    z = x.double() @ w.double().T
    assert float((out.double() - z).norm() / z.norm()) <= 16 * 2.0 ** -23
    assert bool((buf[:guard] == -77).all()) and bool((buf[guard + T * N:] == -77).all())


# T, H, dtype, gate, post, pre, a, o, residual
NORM = [
    (1500, 7168, BF, "channel", True, True, 0.7, 0.0, True),
    (1300, 7168, HF, "element", True, True, 1.0, 1.0, True),
    (1400, 4096, BF, "token", True, True, 1.0, 0.0, True),
    (2500, 2056, BF, "none", True, True, 0.5, 1.0, True),
    (9000, 256, HF, "channel", True, True, 1.0, 0.0, False),
    (9001, 520, BF, "token", False, True, 1.0, 1.0, True),
    (700, 8192, BF, "channel", True, True, 0.7, 0.0, True),
    (650, 16384, BF, "element", True, True, 1.0, 0.0, True),
    (640, 12296, HF, "token", True, False, 1.0, 1.0, True),
    (650, 14336, BF, "none", False, True, 1.0, 0.0, True),
    (1000, 7176, BF, "channel", False, False, 2.0, 0.0, True),
]


def args64(d, post, pre, a, o, eps):
    c = {k: None if v is None else v.double() for k, v in d.items()}
    g = 1.0 if c["gate"] is None else c["gate"].expand(*c["branch"].shape)
    return (c["branch"], c["residual"], g, c["post_weight"], c["pre_weight"], post, pre, a, o, eps)


def within(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert float(over.max()) <= 0, (what, float(over.max()))


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,a,o,residual", NORM)
def test_block_norm_and_gradients(T, H, dtype, gate, post, pre, a, o, residual, cuda_device):
    d = norm_inputs(T, H, dtype, gate, post, pre, o, residual)
    kw = dict(post_norm=post, pre_norm=pre, residual_scale=a, weight_offset=o, eps=1e-5)
    s, h = B.moe_block_norm(**d, **kw)
    args = args64(d, post, pre, a, o, 1e-5)
    rs, rh = R.norm64(*args)
    bs, bh = R.norm_bounds(*args, dtype)
    within(s, rs, bs, "stream")
    if pre:
        within(h, rh, bh, "normed")
    dr = rand(T, H, seed=6, std=0.5, dtype=dtype)
    dh = rand(T, H, seed=7, std=0.5, dtype=dtype) if pre else None
    got = B.moe_block_norm_bwd(dr, dh, **d, **kw)
    ref, mag = R.norm_bwd64(dr.double(), None if dh is None else dh.double(), *args)
    for k, n in (("d_branch", "branch"), ("d_residual", "residual"), ("d_gate", "gate"),
                 ("d_post_weight", "post"), ("d_pre_weight", "pre")):
        if k not in got:
            continue
        r, m, terms = ref[n], mag[n], 1
        if n in ("post", "pre") or (n == "gate" and gate == "channel"):
            r, m, terms = r.sum(0), m.sum(0), T
        elif n == "gate" and gate == "token":
            r, m = r.sum(1, keepdim=True), m.sum(1, keepdim=True)
        within(got[k], r, R.grad_bound(r, m, dtype, terms), k)
    again = B.moe_block_norm_bwd(dr, dh, **d, **kw)
    assert all(torch.equal(again[k], got[k]) for k in got)


def test_block_norm_bwd_in_place(cuda_device):
    """d_residual over d_stream and d_branch over d_normed, through the C entry."""
    import ctypes
    T, H = 700, 2048
    d = norm_inputs(T, H, BF, "channel", True, True, 0.0, True)
    dr, dh = rand(T, H, seed=6, dtype=BF), rand(T, H, seed=7, dtype=BF)
    want = B.moe_block_norm_bwd(dr, dh, **d)
    p = B.BlockNorm(T, H, B.MOE_BF16, 1, 1, 1, 1.0, 0.0, 1e-6)
    L = B.lib()
    n = L.moe_block_norm_bwd_workspace_size(ctypes.byref(p))
    ws = B.new_workspace(n)
    outs = [torch.empty(H, dtype=BF, device="cuda") for _ in range(3)]
    rc = L.moe_block_norm_bwd(
        ctypes.byref(p), dr.data_ptr(), dh.data_ptr(), d["branch"].data_ptr(),
        d["residual"].data_ptr(), d["gate"].data_ptr(), d["post_weight"].data_ptr(),
        d["pre_weight"].data_ptr(), dh.data_ptr(), dr.data_ptr(), *[o.data_ptr() for o in outs],
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == B.MOE_OK
    assert torch.equal(dr, want["d_residual"]) and torch.equal(dh, want["d_branch"])
    for o, k in zip(outs, ("d_gate", "d_post_weight", "d_pre_weight")):
        assert torch.equal(o, want[k]), k


# T, E, k, scoring, lengths, pad
BALANCE = [
    (20000, 384, 8, "sigmoid", [3000, 0, 9000, 1, 7999], 0.05),
    (20000, 130, 6, "softmax", None, 0.05),
    (9000, 1000, 4, "softmax", [1] * 100 + [8900], 0.0),
    (5000, 7, 2, "sigmoid", [10] * 500, 0.3),
    (33000, 64, 8, "softmax", [33000], 0.0),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scoring,lens,pad", BALANCE)
def test_router_training(T, E, k, scoring, lens, pad, renorm, cuda_device):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn(T, E, generator=g, device="cuda")
    ids = x.topk(k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, generator=g, device="cuda") < pad] = -1
    off = None if lens is None else torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    n = 1 if lens is None else len(lens)
    got = B.moe_balance_loss(x, ids, 0.25, scoring, seq_offsets=off)
    assert status(cuda_device) == B.MOE_OK
    # the definition, in 64 bits, by one-hot sums
    seq = torch.zeros(T, dtype=torch.int64, device="cuda")
    if off is not None:
        seq = (torch.arange(T, device="cuda")[:, None] >= off[1:-1][None]).sum(1)
    live = (ids >= 0).any(1)
    member = ((seq[None] == torch.arange(n, device="cuda")[:, None]) & live[None]).double()
    x64 = x.double().requires_grad_(True)
    p = R.probs64(x64, scoring)
    hot = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
    hot.scatter_add_(1, torch.where(ids >= 0, ids, E).long(), torch.ones(T, k, device="cuda").double())
    counts, T_s = member @ hot[:, :E], member.sum(1)
    coef = 0.25 * E * counts / (k * max(1, int((T_s > 0).sum())) * T_s.clamp(min=1)[:, None] ** 2)
    sums = (member @ p).detach()
    assert torch.equal(got["counts"].double(), counts)
    assert torch.equal(got["live_tokens"].double(), T_s)
    rel = (64 + T ** 0.5) * R.F32  # 64 roundings of a term, chunk by chunk sums of them
    within(got["prob_sum"], sums, rel * sums + 1e-37, "prob_sum")
    within(got["coef"], coef, 16 * R.F32 * coef, "coef")
    loss = (coef * sums).sum()
    within(got["loss"], loss.view(1), (rel + 32 * R.F32) * loss.view(1), "loss")
    # both gradients by automatic differentiation
    dw = torch.randn(T, k, generator=g, device="cuda")
    c2 = torch.rand(n, E, generator=g, device="cuda")
    grad = B.moe_router_bwd(x, ids, dw, c2, None, off, scoring, renorm, 1.5)
    on = (ids >= 0).all(1)
    score = p if scoring == "softmax" else torch.sigmoid(x64)
    w = score[on].gather(1, ids[on].long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    total = (member.T @ c2.double() * p).sum() + 1.5 * (w * dw.double()[on]).sum()
    ref = torch.autograd.grad(total, x64)[0]
    mag = p.detach() * c2.double().max()
    big = 2 * 1.5 * dw.double().abs().amax(1, keepdim=True) * k
    mag = mag + big * (hot[:, :E] + (p.detach() if scoring == "softmax" and not renorm else 0))
    within(grad, ref, 128 * R.F32 * mag + 1e-36, "d_gating_output")
