"""Sums of the dense feed-forward block: checkpoints as close to those of 64 bits as an f32 product's."""
import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def neighbours(z, want):
    """Values of the checkpoint of `z` (64 bits) that are not those of `want`."""
    return int((D.checkpoint64(z)[0] != want).sum())


# T, H, F: K of a few blocks to many; the last one's tiles are all split along K
@pytest.mark.parametrize("T,H,F,dtype", [
    (65536, 136, 640, BF), (32768, 264, 1280, HF), (16384, 512, 2560, BF), (8192, 2056, 2560, BF),
    (4096, 7168, 2048, BF), (512, 7168, 2304, HF),
])
def test_saved_values_next_to_a_border(T, H, F, dtype, cuda_device):
    """A sum that is a little off falls on the other side of a border between E4M3 values now and
    then.  That may happen as often as to the sums of an f32 product, within three standard deviations
    of the difference of two such counts (each has the root of itself)."""
    x, w = randn(T, H, seed=1, dtype=dtype), randn(2 * F, H, seed=2, std=H ** -0.5, dtype=dtype)
    _, gate, up = B.moe_gated_linear(x, w, save=True)
    mine = plain = 0
    for part, saved in ((w[:F], gate), (w[F:], up)):
        for i in range(0, T, 4096):
            rows = slice(i, min(i + 4096, T))
            want = D.checkpoint64(x[rows].double() @ part.double().T)[0]
            got = B.moe_checkpoint_restore(B.Fp8Checkpoint(saved.codes[rows], saved.scale[rows], F),
                                           BF).double()
            mine += int((got != want).sum())
            plain += neighbours((x[rows].float() @ part.float().T).double(), want)
    assert mine <= plain + 3 * (2 * plain) ** 0.5, (mine, plain)


# --------------------------------------------------------------------------- sums of a long K
# The tensor cores add with truncation, always toward zero.  Of terms of one sign each addition takes at
# most a step (2^-23), half of one on average, off a running sum that is half the last one on average.
# Four products at a time and 8192 of them in an accumulator are 2048 additions: 2^-13 of the result at
# most, 2^-14 on average, whatever K is.
CHAIN = 2.0 ** -13


def positive(*shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((0.5 + 0.5 * torch.rand(shape, generator=g, device="cuda")) * scale).to(dtype)


def check_long(got, ref, dtype, what, times=1):
    """`times` sums go into a value.  Each value, and their mean, which has no share of the rounding to
    16 bits: that is even, with a deviation of a step / sqrt(12) each."""
    got, ref = got.double().cpu(), ref.double().cpu()
    R.assert_within(got, ref, R.half_step(ref, dtype) + times * CHAIN * ref, what)
    off = float(((got - ref) / ref).mean())
    even = 6 * torch.finfo(dtype).eps / (12 * ref.numel()) ** 0.5
    assert abs(off) <= times * CHAIN / 2 + even, (what, off)


def sampled(n, count, seed):
    rows = torch.randint(0, n, (count,), generator=torch.Generator().manual_seed(seed))
    rows[-1] = n - 1
    return rows.cuda()


# T, N, K: d_w of many rows alone in its tiles' accumulators; both gradients of a long N
@pytest.mark.parametrize("T,N,K", [(262144, 2312, 2312), (2600, 40000, 2312)])
def test_gradients_of_long_sums(T, N, K, cuda_device):
    dy = positive(T, N, seed=1, dtype=HF, scale=2.0 ** -5)
    x, w = positive(T, K, seed=2, dtype=HF), positive(N, K, seed=3, dtype=HF, scale=2.0 ** -3)
    got = B.moe_linear_bwd(dy, x, w)
    rows, cols, some = sampled(N, 64, 4), sampled(K, 64, 5), sampled(T, 64, 6)
    check_long(got["d_w"][rows][:, cols], dy[:, rows].double().T @ x[:, cols].double(), HF, "d_w")
    check_long(got["d_x"][some][:, cols], dy[some].double() @ w[:, cols].double(), HF, "d_x")
    alone = B.moe_linear_bwd(dy, x, w, want_x=False)["d_w"]
    check_long(alone[rows][:, cols], dy[:, rows].double().T @ x[:, cols].double(), HF, "d_w alone")


# T, H, F: tiles of 256 rows; a few rows, whose parts of K take several accumulators
@pytest.mark.parametrize("T,H,F", [(2304, 61448, 1104), (40, 262144, 64), (17, 200008, 72)])
def test_gated_products_of_long_sums(T, H, F, cuda_device):
    x = positive(T, H, seed=1, dtype=HF, scale=H ** -0.5)
    w = positive(2 * F, H, seed=2, dtype=HF, scale=8 * H ** -0.5)
    rows, cols = sampled(T, min(T, 64), 3), sampled(F, 64, 4)
    gate = x[rows].double() @ w[cols].double().T
    up = x[rows].double() @ w[F + cols].double().T
    # act(g) = g s(g), whose slope is at most 1.1 of act(g) / g here (g around 4.5)
    ref = gate * torch.sigmoid(gate) * up
    check_long(B.moe_gated_linear(x, w)[rows][:, cols], ref, HF, "out", times=2.1)
    if T > 128:
        dh = positive(T, F, seed=5, dtype=HF)
        got = B.moe_gated_linear_bwd(dh, x, w, want_x=False, want_w=False, want_out=True)["out"]
        check_long(got[rows][:, cols], ref, HF, "out of the gradient", times=2.1)


# The last one's parts of K are longer than four accumulators take: 20480 of it each.
@pytest.mark.parametrize("T,K,times", [(16, 655360, 1), (40, 262144, 1), (40, 655360, 2.5)])
def test_4_bit_products_of_long_sums(T, K, times, cuda_device):
    N = 64
    g = torch.Generator().manual_seed(1)
    low, high = (torch.randint(1, 8, (N, K // 2), generator=g, dtype=torch.uint8) for _ in range(2))
    codes = (low | (high << 4)).cuda()
    scales = torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    alpha = torch.tensor([2.0 ** -11], device="cuda")
    x = positive(T, K, seed=2, dtype=HF)
    ref = x.cpu().double() @ D.weights64(codes, scales, alpha.cpu()).T
    check_long(B.moe_linear_w4a16(x, codes, scales, alpha), ref, HF, "out", times)
