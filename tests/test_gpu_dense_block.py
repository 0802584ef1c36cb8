"""The dense feed-forward block on the GPU against its plain 64-bit forms: the gated product and its
gradients, the gradients of a dense product, 8-bit checkpoints and 4-bit weights."""
import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, rand, status

pytestmark = pytest.mark.gpu


def d64(t):
    return t.detach().cpu().double()


def check_saved(saved, ref, off, what):
    """A checkpoint of values that are `off` from `ref` at most: its scales, and its values within
    half a step of E4M3."""
    want, got = D.scales64(ref), saved.scale.cpu().double()
    # the scale may be the next one where the largest value lies within `off` of a border
    edge = ((D.scales64(ref.abs() + off) != want) |
            (D.scales64((ref.abs() - off).clamp(min=0)) != want))
    assert torch.equal(got[~edge], want[~edge]), what
    assert bool(((got == want) | (got == 2 * want) | (got == want / 2)).all()), what
    v = D.restore64(saved.codes, saved.scale, ref.shape[1])
    s = got.repeat_interleave(D.GROUP, dim=1)[:, :ref.shape[1]]
    # half a step: 2^-4 of a normal value, 2^-10 scales of a subnormal one
    R.assert_within(v, ref, off + torch.maximum(2.0 ** -4 * (ref.abs() + off), 2.0 ** -10 * s), what)
    pad = saved.codes[:, ref.shape[1]:]
    assert not bool(pad.any()), what


# T, H, F: streamed rows and their edges, K split, several tiles, ragged ends
GATED = [
    (1, 8, 8, BF, "silu"), (1, 2048, 768, HF, "gelu_tanh"), (1, 7168, 2048, BF, "silu"),
    (3, 72, 40, HF, "silu"),
    (8, 264, 128, BF, "gelu_tanh"), (9, 1032, 136, BF, "silu"), (16, 520, 264, HF, "gelu_tanh"),
    (17, 136, 264, BF, "silu"), (33, 2056, 1544, HF, "gelu_tanh"), (64, 4096, 1536, BF, "silu"),
    (128, 512, 128, HF, "silu"), (257, 520, 136, BF, "gelu_tanh"), (300, 1032, 520, HF, "silu"),
    (513, 200, 4104, BF, "silu"), (2300, 72, 1160, HF, "gelu_tanh"), (1000, 2048, 1288, BF, "silu"),
]


@pytest.mark.parametrize("T,H,F,dtype,act", GATED)
@pytest.mark.parametrize("save", [False, True])
def test_gated_linear(T, H, F, dtype, act, save, cuda_device):
    x = rand(T, H, seed=1, dtype=dtype)
    w = rand(2 * F, H, seed=2, std=1.5 * H ** -0.5, dtype=dtype)
    ref, err, g, u, og, ou = D.gated64(d64(x), d64(w), act)
    out = B.moe_gated_linear(x, w, activation=act, save=save)
    again = B.moe_gated_linear(x, w, activation=act, save=save)
    if save:
        out, gate, up = out
        check_saved(gate, g, og, "gate")
        check_saved(up, u, ou, "up")
        assert torch.equal(gate.codes, again[1].codes) and torch.equal(up.scale, again[2].scale)
        again = again[0]
    assert out.dtype == dtype and torch.equal(out, again)
    assert status(cuda_device) == B.MOE_OK
    R.assert_within(out, ref, D.rounded(ref, err, dtype), "out")


@pytest.mark.parametrize("T,H,F,dtype,act", GATED)
@pytest.mark.parametrize("saved", [False, True])
def test_gated_linear_bwd(T, H, F, dtype, act, saved, cuda_device):
    x = rand(T, H, seed=1, dtype=dtype)
    w = rand(2 * F, H, seed=2, std=1.5 * H ** -0.5, dtype=dtype)
    dh = rand(T, F, seed=3, std=0.5, dtype=dtype)
    if saved:
        g, u = rand(T, F, seed=4, std=1.5, dtype=dtype), rand(T, F, seed=5, dtype=dtype)
        xs, gs, us = B.moe_checkpoint(x), B.moe_checkpoint(g), B.moe_checkpoint(u)
        got = B.moe_gated_linear_bwd(dh, xs, w, act, gate=gs, up=us, want_out=True)
        again = B.moe_gated_linear_bwd(dh, xs, w, act, gate=gs, up=us, want_out=True)
        x64, g64, u64 = (D.restore64(c.codes, c.scale, c.C) for c in (xs, gs, us))
        zero = torch.zeros_like(g64)
        ref = D.gated_bwd64(d64(dh), x64, d64(w), g64, u64, zero, zero, act, dtype)
    else:
        got = B.moe_gated_linear_bwd(dh, x, w, act, want_out=True)
        again = B.moe_gated_linear_bwd(dh, x, w, act, want_out=True)
        _, _, g, u, og, ou = D.gated64(d64(x), d64(w), act)
        ref = D.gated_bwd64(d64(dh), d64(x), d64(w), g, u, og, ou, act, dtype)
    assert status(cuda_device) == B.MOE_OK
    assert sorted(got) == ["d_w", "d_x", "out"]
    for k, (want, bound) in ref.items():
        assert got[k].dtype == dtype and torch.equal(got[k], again[k])
        R.assert_within(got[k], want, bound, k)


# Up to 128 rows of x: tiles of 16, 32, 64 and 128 of them, outputs that end inside a tile, K of one block
# and of several parts, more tiles than SMs, and both sides of the rule on the weights' size.
@pytest.mark.parametrize("T,H,F,dtype,act", [
    (2, 8, 8, BF, "silu"), (2, 7168, 72, HF, "silu"), (16, 64, 20000, BF, "gelu_tanh"),
    (31, 5000, 136, BF, "silu"), (32, 4096, 4096, HF, "silu"), (48, 2056, 1000, BF, "silu"),
    (64, 4096, 4088, HF, "gelu_tanh"), (64, 4096, 4096, BF, "silu"), (65, 1032, 3080, BF, "silu"),
    (127, 96, 64, HF, "silu"), (128, 7168, 520, BF, "gelu_tanh"),
])
def test_gated_linear_of_few_rows(T, H, F, dtype, act, cuda_device):
    x = rand(T, H, seed=1, dtype=dtype)
    w = rand(2 * F, H, seed=2, std=1.5 * H ** -0.5, dtype=dtype)
    ref, err, *_ = D.gated64(d64(x), d64(w), act)
    out = B.moe_gated_linear(x, w, activation=act)
    assert out.dtype == dtype and torch.equal(out, B.moe_gated_linear(x, w, activation=act))
    assert status(cuda_device) == B.MOE_OK
    R.assert_within(out, ref, D.rounded(ref, err, dtype), "out")


# T, N, K
LINEAR_BWD = [
    (1, 8, 8, BF), (1, 4099, 264, HF), (5, 3, 16, BF), (64, 2048, 768, BF), (100, 4099, 520, HF),
    (129, 1, 136, HF), (257, 130, 264, BF), (300, 513, 1032, HF), (512, 256, 2048, BF),
    (1000, 8, 8, HF), (2056, 264, 72, BF), (40, 72, 5000, BF), (7000, 40, 24, BF),
]


@pytest.mark.parametrize("T,N,K,dtype", LINEAR_BWD)
@pytest.mark.parametrize("saved", [False, True])
def test_linear_bwd(T, N, K, dtype, saved, cuda_device):
    x = rand(T, K, seed=1, dtype=dtype)
    w = rand(N, K, seed=2, std=K ** -0.5, dtype=dtype)
    dy = rand(T, N, seed=3, std=0.5, dtype=dtype)
    given = B.moe_checkpoint(x) if saved else x
    got = B.moe_linear_bwd(dy, given, w, want_bias=True)
    again = B.moe_linear_bwd(dy, given, w, want_bias=True)
    x64 = D.restore64(given.codes, given.scale, K) if saved else d64(x)
    assert status(cuda_device) == B.MOE_OK
    assert sorted(got) == ["d_bias", "d_w", "d_x"]
    for k, (want, bound) in D.linear_bwd64(d64(dy), x64, d64(w), dtype).items():
        assert got[k].dtype == dtype and torch.equal(got[k], again[k])
        R.assert_within(got[k], want, bound, k)


# The two products of one launch: both split along K with the longer parts first or second, one split,
# neither; more tiles than pairs, so that pairs take tiles of both; and a launch for each.
@pytest.mark.parametrize("T,N,K", [
    (2584, 4310, 48), (4878, 2119, 72), (2586, 4440, 488), (2506, 2255, 672), (1500, 12000, 264),
    (777, 2333, 2568), (2333, 900, 3080), (4099, 4097, 72),
    (6943, 12360, 680),
])
def test_linear_bwd_shares_pairs(T, N, K, cuda_device):
    x = rand(T, K, seed=1, dtype=BF)
    w = rand(N, K, seed=2, std=K ** -0.5, dtype=BF)
    dy = rand(T, N, seed=3, std=0.5, dtype=BF)
    got = B.moe_linear_bwd(dy, x, w)
    again = B.moe_linear_bwd(dy, x, w)
    assert status(cuda_device) == B.MOE_OK and sorted(got) == ["d_w", "d_x"]
    ref = D.linear_bwd64(d64(dy), d64(x), d64(w), BF)
    for k in got:
        assert torch.equal(got[k], again[k])
        R.assert_within(got[k], *ref[k], k)
    # alone, each is the same within its bound
    R.assert_within(B.moe_linear_bwd(dy, x, w, want_w=False)["d_x"], *ref["d_x"], "d_x")
    R.assert_within(B.moe_linear_bwd(dy, x, w, want_x=False)["d_w"], *ref["d_w"], "d_w")


# T, C
CHECKPOINT = [(1, 8), (1, 128), (2, 136), (3, 7168), (33, 2056), (300, 1000), (5000, 72), (2, 40000)]


@pytest.mark.parametrize("T,C", CHECKPOINT)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_checkpoint(T, C, dtype, cuda_device):
    x = rand(T, C, seed=1, dtype=dtype)
    x[:, ::7] *= 40  # far values
    x[0, : C // 2] = 0  # groups of zeros
    saved = B.moe_checkpoint(x)
    want, scale = D.checkpoint64(d64(x))
    assert saved.shape == (T, C) and saved.codes.shape == (T, (C + 127) // 128 * 128)
    assert torch.equal(saved.scale.cpu().double(), scale)
    assert torch.equal(D.restore64(saved.codes, saved.scale, C), want)
    assert not bool(saved.codes[:, C:].any())
    # half a step of E4M3, whose normal values go down to 2^-6 of the scale
    s = scale.repeat_interleave(D.GROUP, dim=1)[:, :C]
    assert bool(((want - d64(x)).abs() <= torch.maximum(2.0 ** -4 * d64(x).abs(), 2.0 ** -10 * s)).all())
    for to in (BF, HF):
        back = B.moe_checkpoint_restore(saved, to)
        assert back.dtype == to and torch.equal(d64(back), want)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_checkpoint_of_extreme_values(dtype, cuda_device):
    fi = torch.finfo(dtype)
    rows = [[fi.max, -fi.max, 1.0, 0.0], [fi.smallest_normal, -fi.smallest_normal, 0.0, 0.0],
            [fi.smallest_normal * fi.eps, 0.0, 0.0, 0.0], [448.0, -448.0, 240.0, 0.4],
            [449.0 if dtype is HF else 450.0, 17.0, 19.0, 21.0],
            [float("inf"), 2.0, -3.0, 0.1], [float("nan"), -float("inf"), 5.0, 0.0],
            [float("inf"), float("nan"), -float("inf"), 0.0]]
    x = torch.zeros(len(rows), 136)
    x[:, :4] = torch.tensor(rows)
    x[:, 130] = torch.tensor([r[1] for r in rows])
    x = x.to(dtype).cuda()
    saved = B.moe_checkpoint(x)
    want, scale = D.checkpoint64(d64(x))
    assert torch.equal(saved.scale.cpu().double(), scale)
    got = D.restore64(saved.codes, saved.scale, 136)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    back = d64(B.moe_checkpoint_restore(saved, dtype))
    # rounded past the largest value: that one
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.nan_to_num(), want.nan_to_num().clamp(-fi.max, fi.max))


def weights4(rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    # every finite E4M3 value of either sign
    scales = torch.randint(0, 254, (rows, K // 16), generator=g, dtype=torch.int32)
    scales = torch.where(scales >= 127, scales + 1, scales).to(torch.uint8)
    return codes.cuda(), scales.cuda(), torch.tensor([0.013], device="cuda")


# T, N, K
W4 = [
    (1, 1, 32, BF, "none", False, False), (1, 7168, 2048, BF, "none", False, True),
    (1, 300, 18432, HF, "relu2", True, True), (2, 5, 64, HF, "silu", True, False),
    (7, 4099, 160, BF, "gelu_tanh", False, True), (8, 16, 4096, BF, "none", True, False),
    (9, 17, 96, HF, "none", False, False), (16, 1000, 1056, BF, "silu", True, True),
    (17, 33, 32, HF, "gelu_tanh", True, True), (32, 4099, 4128, HF, "gelu_tanh", True, True),
    (33, 64, 352, BF, "none", False, True), (100, 130, 224, HF, "relu2", False, False),
]


@pytest.mark.parametrize("T,N,K,dtype,act,bias,res", W4)
def test_linear_w4(T, N, K, dtype, act, bias, res, cuda_device):
    x = rand(T, K, seed=1, dtype=dtype)
    x[0, : K // 2] *= 2.0 ** -12  # small values
    codes, scales, alpha = weights4(N, K, seed=2)
    alpha = alpha / (K ** 0.5 * 8)
    b = rand(N, seed=3, dtype=dtype) if bias else None
    r = rand(T, N, seed=4, dtype=dtype) if res else None
    kw = dict(bias=b, activation=act, residual=r)
    out = B.moe_linear_w4a16(x, codes, scales, alpha, **kw)
    assert torch.equal(out, B.moe_linear_w4a16(x, codes, scales, alpha, **kw))
    assert out.dtype == dtype and status(cuda_device) == B.MOE_OK
    ref, bound = D.w4_linear64(x, D.weights64(codes, scales, alpha.cpu()), b, act, r)
    R.assert_within(out, ref, bound, "out")


# Past sixteen rows: tiles of 32, 64 and 128 of them, of one and several blocks and parts of K, more
# tiles than SMs, K that ends inside a block.
W4_TILES = [
    (17, 1, 32, BF), (17, 4099, 7168, BF), (31, 130, 2080, HF), (32, 129, 256, BF), (33, 20000, 288, HF),
    (64, 257, 4128, BF), (65, 1000, 96, BF), (128, 2048, 2048, HF), (129, 40, 5152, BF),
    (300, 1000, 992, BF),
]


@pytest.mark.parametrize("T,N,K,dtype", W4_TILES)
def test_w4_tiles(T, N, K, dtype, cuda_device):
    x = rand(T, K, seed=1, dtype=dtype)
    x[0, : K // 2] *= 2.0 ** -12  # small values
    codes, scales, alpha = weights4(2 * N, K, seed=2)
    alpha = alpha / (K ** 0.5 * 8)
    w = D.weights64(codes, scales, alpha.cpu())
    b, r = rand(N, seed=3, dtype=dtype), rand(T, N, seed=4, dtype=dtype)
    c1, s1 = codes[:N].contiguous(), scales[:N].contiguous()
    for kw in (dict(bias=b, activation="silu", residual=r), {}):
        out = B.moe_linear_w4a16(x, c1, s1, alpha, **kw)
        assert torch.equal(out, B.moe_linear_w4a16(x, c1, s1, alpha, **kw))
        ref, bound = D.w4_linear64(x, w[:N], kw.get("bias"), kw.get("activation", "none"),
                                   kw.get("residual"))
        R.assert_within(out, ref, bound, "out")
    out = B.moe_gated_linear_w4a16(x, codes, scales, alpha)
    assert torch.equal(out, B.moe_gated_linear_w4a16(x, codes, scales, alpha))
    assert out.dtype == dtype and status(cuda_device) == B.MOE_OK
    R.assert_within(out, *D.w4_gated64(x, w, "silu"), "gated")


@pytest.mark.parametrize("T,F,K,dtype,act", [
    (1, 1, 32, HF, "silu"), (1, 2048, 7168, BF, "silu"), (3, 20, 96, BF, "gelu_tanh"),
    (8, 771, 544, HF, "gelu_tanh"), (11, 9, 2048, BF, "silu"), (32, 1536, 4096, BF, "silu"),
    (40, 100, 64, HF, "silu"),
])
def test_gated_linear_w4(T, F, K, dtype, act, cuda_device):
    x = rand(T, K, seed=1, dtype=dtype)
    codes, scales, alpha = weights4(2 * F, K, seed=2)
    alpha = alpha / (K ** 0.5 * 8)
    out = B.moe_gated_linear_w4a16(x, codes, scales, alpha, activation=act)
    assert torch.equal(out, B.moe_gated_linear_w4a16(x, codes, scales, alpha, activation=act))
    assert out.dtype == dtype and status(cuda_device) == B.MOE_OK
    ref, bound = D.w4_gated64(x, D.weights64(codes, scales, alpha.cpu()), act)
    R.assert_within(out, ref, bound, "out")
