"""Gradients of the dense feed-forward block with over 2^31 elements in rows, shared launches in f16,
and 4-bit weights against many rows.  References in 64 bits, on the GPU where every row goes into them."""
import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, rand, status
from test_gpu_dense_block import d64, weights4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def given_back():
    """Many gigabytes of scratch."""
    yield
    B.release_call_workspaces()


def normal(*shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=BF, device="cuda").normal_(std=std, generator=g)


def sampled(n, count, seed):
    rows = torch.randint(0, n, (count,), generator=torch.Generator().manual_seed(seed))
    rows[0], rows[-1] = 0, n - 1
    return rows.cuda()


def chunks(T, step=16384):
    return (slice(i, min(i + step, T)) for i in range(0, T, step))


def over_rows(T, a, b):
    """(sum_t a(t)^T b(t), sum of its terms' squares), from functions of a slice of rows."""
    total = squares = 0.0
    for rows in chunks(T):
        p, q = a(rows).double(), b(rows).double()
        total, squares = total + p.T @ q, squares + p.square().T @ q.square()
    return total.cpu(), squares.cpu()


def spread(T, squares):
    """What truncation may take off a sum over T rows of terms of either sign: at most a step (2^-23) of
    a running sum per four terms, which stays within six deviations of 8192 terms."""
    return T / 4 * 2.0 ** -23 * 6 * (8192 / T * squares).sqrt()


# T, H, F: x and d_x, then d_out, d_gate and d_up, of more than 2^31 elements
@pytest.mark.parametrize("T,H,F", [(270000, 8192, 8), (135000, 16, 16392)])
@pytest.mark.parametrize("saved", [False, True])
def test_gated_gradients_past_2_31_elements(T, H, F, saved, cuda_device):
    x, w = normal(T, H, seed=1), normal(2 * F, H, seed=2, std=H ** -0.5)
    dh = normal(T, F, seed=3, std=0.5)
    if saved:
        x8 = B.moe_checkpoint(x)
        out, gate, up = B.moe_gated_linear(x, w, save=True)
        del out
        got = B.moe_gated_linear_bwd(dh, x8, w, gate=gate, up=up, want_out=True)
        x = B.moe_checkpoint_restore(x8, BF)

        def pre(rows, cols):  # gate and up
            return [D.restore64(c.codes[rows], c.scale[rows], F).cuda()[:, cols] for c in (gate, up)]
    else:
        got = B.moe_gated_linear_bwd(dh, x, w, want_out=True)

        def pre(rows, cols):
            v = x[rows].double()
            return [v @ w[cols].double().T, v @ w[F + cols].double().T]
    rows, cols, wide = sampled(T, 24, 4), sampled(F, min(F, 8), 5), sampled(H, min(H, 64), 6)
    every = torch.arange(F, device="cuda")

    def d_pre(rows, cols):
        g, u = pre(rows, cols)
        d = dh[rows][:, cols].double()
        return torch.cat([d * u * D.slope64(g, "silu"), d * R.act64(g, "silu")], dim=1)

    # d_gate and d_up are rounded, half a step each with a sign of its own: six deviations of the sum
    even = 6 * 2.0 ** -8
    g, u = pre(rows, every)
    h = (R.act64(g, "silu") * u).cpu()
    _, err, *_ = D.gated64(d64(x[rows]), d64(w), "silu")
    R.assert_within(got["out"][rows], h, D.rounded(h, D.EVAL * h.abs() if saved else err, BF), "out")
    d, v = d_pre(rows, every), torch.cat([w[:F], w[F:]])[:, wide].double()
    ref, squares = (d @ v).cpu(), (d.square() @ v.square()).cpu()
    R.assert_within(got["d_x"][rows][:, wide], ref,
                    even * squares.sqrt() + spread(2 * F, squares) + R.half_step(ref, BF), "d_x")
    ref, squares = over_rows(T, lambda r: d_pre(r, cols), lambda r: x[r][:, wide])
    R.assert_within(got["d_w"][torch.cat([cols, F + cols])][:, wide], ref,
                    even * squares.sqrt() + spread(T, squares) + R.half_step(ref, BF), "d_w")


def test_odd_rows_past_2_31_elements(cuda_device):
    """d_out whose rows start anywhere: copied, added and multiplied past 2^31 elements."""
    T, N, K = 530000, 4099, 8
    dy, w, x = normal(T, N, seed=1, std=0.5), normal(N, K, seed=2), normal(T, K, seed=3)
    rows, cols = sampled(T, 40, 4), sampled(N, 64, 5)
    d_w, squares = over_rows(T, lambda r: dy[r][:, cols], lambda r: x[r])
    d_b = sum(dy[r].double().sum(0) for r in chunks(T)).cpu()
    d_x, off = D.product64(d64(dy[rows]), d64(w).T.contiguous())
    for bias in (True, False):  # the copy is made in the bias's pass, or in one of its own
        got = B.moe_linear_bwd(dy, x, w, want_bias=bias)
        R.assert_within(got["d_x"][rows], d_x, D.rounded(d_x, off, BF), "d_x")
        R.assert_within(got["d_w"][cols], d_w, spread(T, squares) + R.half_step(d_w, BF), "d_w")
        if bias:
            # 256 sums of T / 256 values each, rounded to half a step of what six deviations reach
            err = T * R.F32 * 6 * (T / 256) ** 0.5 * 0.5
            R.assert_within(got["d_bias"], d_b, err + R.half_step(d_b, BF), "d_bias")


# Shared launches of f16, x from a checkpoint or not
@pytest.mark.parametrize("T,N,K", [(2584, 4310, 48), (2506, 2255, 672), (777, 2333, 2568),
                                   (6943, 12360, 680)])
@pytest.mark.parametrize("saved", [False, True])
def test_linear_bwd_shares_pairs_in_f16(T, N, K, saved, cuda_device):
    x = rand(T, K, seed=1, dtype=HF)
    w = rand(N, K, seed=2, std=K ** -0.5, dtype=HF)
    dy = rand(T, N, seed=3, std=0.5, dtype=HF)
    given = B.moe_checkpoint(x) if saved else x
    got = B.moe_linear_bwd(dy, given, w, want_bias=True)
    x64 = D.restore64(given.codes, given.scale, K) if saved else d64(x)
    rows, cols = sampled(T, 300, 4).cpu(), sampled(N, 300, 5).cpu()
    assert status(cuda_device) == B.MOE_OK
    want, off = D.product64(d64(dy)[rows], d64(w).T.contiguous())
    R.assert_within(got["d_x"].cpu()[rows], want, D.rounded(want, off, HF), "d_x")
    want, off = D.product64(d64(dy)[:, cols].T.contiguous(), x64.T.contiguous())
    R.assert_within(got["d_w"].cpu()[cols], want, D.rounded(want, off, HF), "d_w")
    want = d64(dy).sum(0)
    R.assert_within(got["d_bias"], want,
                    D.rounded(want, (T / 32 + 40) * R.F32 * d64(dy).abs().sum(0), HF), "d_bias")


# Prompts: several tiles of 128 rows, the last one's end
@pytest.mark.parametrize("T,F,K,dtype", [(300, 70, 992, BF), (1000, 130, 160, HF), (4096, 64, 2080, BF),
                                         (4099, 20, 96, HF)])
def test_4_bit_weights_of_many_rows(T, F, K, dtype, cuda_device):
    x = rand(T, K, seed=1, dtype=dtype)
    codes, scales, alpha = weights4(2 * F, K, seed=2)
    alpha = alpha / (K ** 0.5 * 8)
    w = D.weights64(codes, scales, alpha.cpu())
    for act in ("silu", "gelu_tanh"):
        out = B.moe_gated_linear_w4a16(x, codes, scales, alpha, activation=act)
        R.assert_within(out, *D.w4_gated64(x, w, act), act)
    b, r = rand(2 * F, seed=3, dtype=dtype), rand(T, 2 * F, seed=4, dtype=dtype)
    out = B.moe_linear_w4a16(x, codes, scales, alpha, bias=b, activation="gelu_tanh", residual=r)
    R.assert_within(out, *D.w4_linear64(x, w, b, "gelu_tanh", r), "linear")
    assert status(cuda_device) == B.MOE_OK


def test_tensors_that_require_gradients(cuda_device):
    """The calls are no part of torch's graph: their outputs require no gradient, their inputs get none."""
    x, w = rand(40, 64, seed=1, dtype=BF).requires_grad_(), rand(80, 64, seed=2, dtype=BF).requires_grad_()
    out, gate, up = B.moe_gated_linear(x, w, save=True)
    back = B.moe_gated_linear_bwd(out, x, w, gate=gate, up=up)
    for t in (out, gate.codes, up.scale, *back.values(), B.moe_checkpoint(x).codes):
        assert not t.requires_grad and t.grad_fn is None
    assert x.grad is None and w.grad is None and x.requires_grad
