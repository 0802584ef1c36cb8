"""The operators around the routed experts on the GPU against their plain 64-bit forms: the dense
product with its epilogue, the norm between two blocks and its gradients, the balance loss and the
gradient of the router logits."""
import pytest
import torch

import block_reference as R
from mixture_experts_forward_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def rand(*shape, seed, std=1.0, mean=0.0, dtype=torch.float32, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(device)


def status(device):
    return B.get_device_status(B.call_workspace(device))


# ------------------------------------------------------------------------------------- linear
LINEAR = [
    # T, N, K, dtype, act, bias, residual, f32: each row count class and its edges, ragged N and K
    (1, 256, 7168, BF, "none", False, False, True),
    (1, 1, 8, HF, "silu", True, True, False),
    (2, 10, 72, BF, "gelu_tanh", True, True, True),
    (3, 4099, 264, HF, "relu2", False, True, False),
    (4, 130, 2048, BF, "none", True, False, False),
    (5, 128, 64, BF, "none", False, False, True),
    (16, 129, 4096, HF, "gelu_tanh", True, True, False),
    (17, 40, 520, BF, "silu", True, False, True),
    (32, 2048, 768, BF, "relu2", True, True, False),
    (33, 4099, 2056, HF, "gelu_tanh", True, True, False),
    (64, 7, 8, BF, "none", True, True, True),
    (65, 384, 7168, BF, "none", True, False, True),
    (200, 1000, 1160, HF, "silu", False, True, False),
    (513, 255, 1032, BF, "none", True, True, False),
    (700, 5000, 328, BF, "gelu_tanh", True, True, False),
    (4096, 128, 136, HF, "none", False, False, True),
    (2048, 2560, 192, BF, "silu", True, True, False),
    (2500, 2600, 72, HF, "relu2", True, False, False),
]


@pytest.mark.parametrize("T,N,K,dtype,act,bias,res,f32", LINEAR)
def test_linear(T, N, K, dtype, act, bias, res, f32, cuda_device):
    odt = torch.float32 if f32 else dtype
    x = rand(T, K, seed=1, dtype=dtype)
    w = rand(N, K, seed=2, std=K ** -0.5, dtype=dtype)
    b = rand(N, seed=3, dtype=dtype) if bias else None
    r = rand(T, N, seed=4, dtype=odt) if res else None
    out = B.moe_linear(x, w, bias=b, activation=act, residual=r,
                       out_dtype=torch.float32 if f32 else None)
    again = B.moe_linear(x, w, bias=b, activation=act, residual=r,
                         out_dtype=torch.float32 if f32 else None)
    assert out.dtype == odt and status(cuda_device) == B.MOE_OK
    assert torch.equal(out, again)
    ref, bound = R.linear64(x, w, b, act, r, odt)
    R.assert_within(out, ref, bound, "linear")
    if f32 and act == "none":
        # over a whole output the truncations average out: half a step per addition
        err = (out.cpu().double() - ref).norm() / ref.norm()
        assert err <= R.F32 * (K / 16 + 16), float(err)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_writes_over_its_residual(T, cuda_device):
    x, w = rand(T, 512, seed=5, dtype=BF), rand(384, 512, seed=6, std=0.05, dtype=BF)
    r = rand(T, 384, seed=7, dtype=BF)
    want = B.moe_linear(x, w, residual=r)
    assert torch.equal(B.moe_linear(x, w, residual=r, out=r), want)
    assert r.data_ptr() and torch.equal(r, want)


@pytest.mark.parametrize("T", [1, 12, 150])
def test_linear_keeps_what_is_not_finite_in_its_row(T, cuda_device):
    x, w = rand(T, 256, seed=8, dtype=BF), rand(136, 256, seed=9, std=0.06, dtype=BF)
    x[0, 3] = float("nan")
    out = B.moe_linear(x, w, activation="relu2")
    assert out[0].isnan().all() and out[1:].isfinite().all()


def test_linear_touches_nothing_past_its_output(cuda_device):
    for T, N in ((3, 5), (20, 131), (70, 129), (300, 127)):
        flat = torch.full((T * N + 64,), 7.0, dtype=BF, device=cuda_device)
        out = flat[: T * N].view(T, N)
        B.moe_linear(rand(T, 64, seed=T, dtype=BF), rand(N, 64, seed=N, dtype=BF), out=out)
        assert (flat[T * N:] == 7).all()


def test_linear_wait_that_gives_up_is_reported(cuda_device):
    x, w = rand(40, 4096, seed=10, dtype=BF), rand(512, 4096, seed=11, std=0.02, dtype=BF)
    want = B.moe_linear(x, w)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        B.moe_linear(x, w)
        got = status(cuda_device)
    finally:
        B.set_wait_limit_ns(old)
    assert got == B.MOE_ERR_TIMEOUT
    assert torch.equal(B.moe_linear(x, w), want) and status(cuda_device) == B.MOE_OK


# ----------------------------------------------------------------------------------- the norm
NORM = [
    # T, H, dtype, gate, post, pre, a, o, residual
    (1, 7168, BF, "channel", True, True, 1.0, 0.0, True),
    (1, 8, HF, "none", False, True, 1.0, 0.0, False),
    (3, 2056, BF, "element", True, True, 0.7, 1.0, True),
    (300, 256, HF, "token", True, True, 0.7, 1.0, True),
    (37, 8192, BF, "channel", False, True, 1.0, 1.0, True),
    (5, 16384, BF, "channel", True, True, 0.5, 0.0, True),
    (200, 4096, HF, "none", True, False, 1.0, 0.0, True),
    (33, 2048, BF, "token", False, False, 2.0, 0.0, True),
    (400, 520, BF, "channel", True, True, 1.0, 0.0, False),
    (64, 12296, HF, "element", True, True, 1.0, 0.0, True),
]


def norm_inputs(T, H, dtype, gate, post, pre, o, residual):
    d = dict(branch=rand(T, H, seed=1, std=0.8, dtype=dtype),
             residual=rand(T, H, seed=2, std=1.5, dtype=dtype) if residual else None,
             post_weight=rand(H, seed=4, std=0.1, mean=1 - o, dtype=dtype) if post else None,
             pre_weight=rand(H, seed=5, std=0.1, mean=1 - o, dtype=dtype) if pre else None)
    shape = dict(none=None, channel=(H,), token=(T, 1), element=(T, H))[gate]
    d["gate"] = None if shape is None else rand(*shape, seed=3, std=0.3, mean=0.6, dtype=dtype)
    return d


def norm64_args(d, post, pre, a, o, eps):
    c = {k: None if v is None else v.cpu().double() for k, v in d.items()}
    g = 1.0 if c["gate"] is None else c["gate"].expand(*c["branch"].shape)
    return (c["branch"], c["residual"], g, c["post_weight"], c["pre_weight"], post, pre, a, o, eps)


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,a,o,residual", NORM)
def test_block_norm(T, H, dtype, gate, post, pre, a, o, residual, cuda_device):
    d = norm_inputs(T, H, dtype, gate, post, pre, o, residual)
    kw = dict(post_norm=post, pre_norm=pre, residual_scale=a, weight_offset=o, eps=1e-5)
    s, h = B.moe_block_norm(**d, **kw)
    args = norm64_args(d, post, pre, a, o, 1e-5)
    rs, rh = R.norm64(*args)
    bs, bh = R.norm_bounds(*args, dtype)
    R.assert_within(s, rs, bs, "stream")
    if pre:
        R.assert_within(h, rh, bh, "normed")
        none, h2 = B.moe_block_norm(**d, **kw, want_stream=False)
        assert none is None and torch.equal(h, h2)
    else:
        assert h is None
    if residual:  # in place of the residual
        x = d["residual"].clone()
        s2, h2 = B.moe_block_norm(**{**d, "residual": x}, **kw, stream_out=x)
        assert torch.equal(s2, s) and (h is None or torch.equal(h2, h))


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,a,o,residual", NORM)
def test_block_norm_gradients(T, H, dtype, gate, post, pre, a, o, residual, cuda_device):
    d = norm_inputs(T, H, dtype, gate, post, pre, o, residual)
    kw = dict(post_norm=post, pre_norm=pre, residual_scale=a, weight_offset=o, eps=1e-5)
    dr = rand(T, H, seed=6, std=0.5, dtype=dtype)
    dh = rand(T, H, seed=7, std=0.5, dtype=dtype) if pre else None
    got = B.moe_block_norm_bwd(dr, dh, **d, **kw)
    again = B.moe_block_norm_bwd(dr, dh, **d, **kw)
    ref, mag = R.norm_bwd64(dr.cpu().double(), None if dh is None else dh.cpu().double(),
                            *norm64_args(d, post, pre, a, o, 1e-5))
    want = {"d_branch": "branch"}
    if residual:
        want["d_residual"] = "residual"
    if gate != "none":
        want["d_gate"] = "gate"
    if post:
        want["d_post_weight"] = "post"
    if pre:
        want["d_pre_weight"] = "pre"
    assert set(got) == set(want)
    for k, n in want.items():
        r, m, terms = ref[n], mag[n], 1
        if n in ("post", "pre") or (n == "gate" and gate == "channel"):
            r, m, terms = r.sum(0), m.sum(0), T
        elif n == "gate" and gate == "token":
            r, m = r.sum(1, keepdim=True), m.sum(1, keepdim=True)
        R.assert_within(got[k], r, R.grad_bound(r, m, dtype, terms), k)
        assert torch.equal(got[k], again[k]), k


def test_block_norm_gradients_in_place_and_without_stream(cuda_device):
    d = norm_inputs(50, 512, BF, "channel", True, True, 0.0, True)
    dr, dh = rand(50, 512, seed=6, dtype=BF), rand(50, 512, seed=7, dtype=BF)
    want = B.moe_block_norm_bwd(torch.zeros_like(dr), dh, **d)
    got = B.moe_block_norm_bwd(None, dh, **d)
    for k in want:
        assert torch.equal(want[k], got[k]), k


def test_block_norm_of_no_rows(cuda_device):
    d = norm_inputs(0, 64, BF, "channel", True, True, 0.0, True)
    s, h = B.moe_block_norm(**d)
    assert s.shape == h.shape == (0, 64)
    g = B.moe_block_norm_bwd(torch.empty_like(s), torch.empty_like(s), **d)
    for k in ("d_gate", "d_post_weight", "d_pre_weight"):
        assert (g[k] == 0).all(), k


def test_block_norm_zero_rows_and_rows_that_are_not_finite(cuda_device):
    d = norm_inputs(4, 256, BF, "none", True, True, 0.0, False)
    d["branch"][0] = 0
    d["branch"][2, 5] = float("nan")
    s, h = B.moe_block_norm(**d)
    assert (s[0] == 0).all() and (h[0] == 0).all()
    assert s[2].isnan().all() and h[2].isnan().all()
    assert s[[1, 3]].isfinite().all() and h[[1, 3]].isfinite().all()


# --------------------------------------------------------------------------------- the router
ROUTER = [
    # T, E, k, scoring, offsets (None, or lengths), pad, kind of logits
    (1, 8, 2, "softmax", None, 0.0, "plain"),
    (1, 1, 1, "sigmoid", None, 0.0, "plain"),
    (64, 128, 8, "softmax", None, 0.0, "plain"),
    (130, 256, 8, "sigmoid", [0, 63, 1, 0, 2, 64], 0.2, "plain"),
    (77, 40, 3, "softmax", [70, 7], 0.3, "plain"),
    (65, 1024, 32, "sigmoid", [64, 1], 0.0, "plain"),
    (200, 33, 1, "softmax", [1] * 200, 0.1, "plain"),
    (50, 384, 8, "sigmoid", [0, 0, 50, 0], 1.0, "plain"),   # every token is padding
    (40, 64, 6, "sigmoid", None, 0.0, "far"),               # logits of +-120
    (40, 64, 6, "softmax", None, 0.0, "far"),
    (40, 64, 6, "softmax", None, 0.0, "masked"),            # some experts at -inf, a row of -inf
    (40, 64, 6, "sigmoid", None, 0.0, "masked"),
    (150, 500, 8, "softmax", [149, 1], 0.05, "plain"),
]


def router_inputs(T, E, k, lens, pad, kind, device="cuda"):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = torch.randn(T, E, generator=g) + 0.4 * torch.randn(E, generator=g)
    ids = x.topk(k, dim=1).indices.to(torch.int32)
    if kind == "far":
        x = x * 60
        x[1] = -115 - x[1].abs() / 60  # every sigmoid underflows
    if kind == "masked":
        x[:, ::3] = float("-inf")
        ids = x.topk(k, dim=1).indices.to(torch.int32)
        x[2] = float("-inf")
    ids[torch.rand(T, generator=g) < pad] = -1
    if T > 4 and pad:
        ids[3, : k // 2] = -1  # dropped routes of a live token
    off = None
    if lens is not None:
        off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    dw = torch.randn(T, k, generator=g)
    return (x.to(device), ids.to(device), None if off is None else off.to(device),
            dw.to(device))


@pytest.mark.parametrize("T,E,k,scoring,lens,pad,kind", ROUTER)
def test_balance_loss(T, E, k, scoring, lens, pad, kind, cuda_device):
    x, ids, off, _ = router_inputs(T, E, k, lens, pad, kind)
    got = B.moe_balance_loss(x, ids, 0.25, scoring, seq_offsets=off)
    again = B.moe_balance_loss(x, ids, 0.25, scoring, seq_offsets=off)
    assert status(cuda_device) == B.MOE_OK
    loss, counts, live, sums, coef = R.balance64(x.cpu().double(), ids.cpu(), 0.25, scoring, off)
    assert torch.equal(got["counts"].cpu(), counts)
    assert torch.equal(got["live_tokens"].cpu(), live)
    # positive terms: 64 roundings of a probability (two exponentials of arguments up to 120 in
    # steps of 2^-17, their sum, a quotient), and the sum over tokens
    far = 120 * R.F32 * 2 if kind == "far" else 0.0
    rel = (64 + T) * R.F32 + far
    R.assert_within(got["prob_sum"], sums, rel * sums + 1e-37, "prob_sum")
    R.assert_within(got["coef"], coef, 16 * R.F32 * coef, "coef")
    R.assert_within(got["loss"], loss.view(1), (rel + 32 * R.F32) * loss.view(1) + 1e-37, "loss")
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scoring,lens,pad,kind", ROUTER)
def test_router_gradient(T, E, k, scoring, lens, pad, kind, renorm, cuda_device):
    x, ids, off, dw = router_inputs(T, E, k, lens, pad, kind)
    n = 1 if off is None else off.numel() - 1
    coef = rand(n, E, seed=3).abs()
    d_loss = torch.tensor([0.5], device=cuda_device)
    got = B.moe_router_bwd(x, ids, dw, coef, d_loss, off, scoring, renorm, 2.5)
    assert torch.equal(got, B.moe_router_bwd(x, ids, dw, coef, d_loss, off, scoring, renorm, 2.5))
    x64 = x.cpu().double()
    if kind == "masked":
        # a row of -inf alone has no route weights to speak of; the others' are finite
        x64[2] = 0
        keep = torch.arange(T) != 2
        assert torch.isfinite(got[2]).all()
    else:
        keep = torch.ones(T, dtype=torch.bool)
    x64 = torch.where(torch.isinf(x64), torch.full_like(x64, -1e4), x64).requires_grad_(True)
    total = R.router_loss64(x64, ids.cpu(), dw.cpu().double(), coef.cpu().double(), off, scoring,
                            renorm, 2.5, 0.5)
    ref = torch.autograd.grad(total, x64)[0] if total.requires_grad else torch.zeros_like(x64)
    # a term is a probability times a difference of averages: their magnitudes are at most
    # p (max coef + sum coef p) / 2 for the loss and 2 * 2.5 max|dw| for the weights (those of the
    # selected experts alone unless softmax is over all)
    far = 120 * R.F32 * 2 if kind == "far" else 0.0
    p = R.probs64(x64.detach(), scoring)
    mag = p * coef.cpu().double().max() + torch.zeros_like(p)
    big = 2 * 2.5 * dw.cpu().double().abs().amax(dim=1, keepdim=True) * k
    sel = torch.zeros_like(p)
    on = ids.cpu() >= 0
    t, j = on.nonzero(as_tuple=True)
    sel[t, ids.cpu()[t, j].long()] = 1.0
    mag = mag + big * (sel + (p if scoring == "softmax" and not renorm else 0))
    bound = (128 * R.F32 + far) * mag + 1e-36
    R.assert_within(got[keep.to(got.device)], ref[keep], bound[keep], "d_gating_output")


def test_router_gradient_of_one_term_alone(cuda_device):
    x, ids, off, dw = router_inputs(90, 128, 8, [40, 50], 0.2, "plain")
    coef = rand(2, 128, seed=3).abs()
    both = B.moe_router_bwd(x, ids, dw, coef, None, off, "softmax").double()
    a = B.moe_router_bwd(x, ids, dw, None, None, off, "softmax").double()
    b = B.moe_router_bwd(x, ids, None, coef, None, off, "softmax").double()
    assert torch.allclose(both, a + b, rtol=0, atol=1e-5)
    assert (B.moe_router_bwd(x, ids, None, None, None, off) == 0).all()
    y = x.clone()
    assert torch.equal(B.moe_router_bwd(y, ids, dw, coef, None, off, "softmax", out=y),
                       both.float())


def test_router_gradient_of_an_expert_named_twice(cuda_device):
    x = rand(3, 16, seed=1)
    ids = torch.tensor([[4, 4, 2], [1, 0, 1], [7, 7, 7]], dtype=torch.int32, device=cuda_device)
    dw = rand(3, 3, seed=2)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = B.moe_router_bwd(x, ids, dw, scoring_func=scoring, renormalize=renorm)
            x64 = x.cpu().double().requires_grad_(True)
            ref = torch.autograd.grad(
                R.router_loss64(x64, ids.cpu(), dw.cpu().double(), None, None, scoring, renorm,
                                1.0, 1.0), x64)[0]
            R.assert_within(got, ref, 128 * R.F32 * 6 * dw.abs().max().item()
                            * torch.ones_like(ref), scoring)


def test_router_gradient_is_zero_outside_the_sequences(cuda_device):
    x, ids, _, _ = router_inputs(30, 32, 4, None, 0.0, "plain")
    off = torch.tensor([5, 12, 20], dtype=torch.int32, device=cuda_device)
    loss = B.moe_balance_loss(x, ids, 1.0, seq_offsets=off)
    assert loss["live_tokens"].tolist() == [7, 8]
    g = B.moe_router_bwd(x, ids, coef=loss["coef"], seq_offsets=off)
    assert (g[:5] == 0).all() and (g[20:] == 0).all() and (g[5:20] != 0).any(dim=1).all()


def test_balance_loss_gradient_against_differences(cuda_device):
    x, ids, off, _ = router_inputs(24, 16, 2, [10, 14], 0.2, "plain")
    for scoring in ("softmax", "sigmoid"):
        got = B.moe_balance_loss(x, ids, 1.0, scoring, seq_offsets=off)
        grad = B.moe_router_bwd(x, ids, coef=got["coef"], seq_offsets=off, scoring_func=scoring)
        x64, h = x.cpu().double(), 1e-6
        for t, e in ((0, 1), (9, 15), (10, 0), (23, 7)):
            d = torch.zeros_like(x64)
            d[t, e] = h
            up, down = (R.balance64(x64 + s * d, ids.cpu(), 1.0, scoring, off)[0] for s in (1, -1))
            # a central difference of step h: h^2 of the third derivative, 2^-52 / h of rounding
            want = (up - down) / (2 * h)
            assert abs(float(grad[t, e]) - float(want)) <= 1e-8, (scoring, t, e)


def test_balance_loss_reports_bad_ids_and_offsets(cuda_device):
    x, ids, off, _ = router_inputs(70, 32, 4, [30, 40], 0.0, "plain")
    bad = ids.clone()
    bad[5, 1], bad[66, 0] = 32, -2
    got = B.moe_balance_loss(x, bad, 1.0, seq_offsets=off)
    assert status(cuda_device) == B.MOE_ERR_BAD_EXPERT_ID
    clean = ids.clone()
    clean[5, 1], clean[66, 0] = -1, -1
    want = B.moe_balance_loss(x, clean, 1.0, seq_offsets=off)
    assert status(cuda_device) == B.MOE_OK
    for n in want:
        assert torch.equal(got[n], want[n]), n
    for o in ([0, 80], [-3, 70], [0, 50, 20, 70]):
        B.moe_balance_loss(x, ids, 1.0, seq_offsets=torch.tensor(o, dtype=torch.int32,
                                                                device=cuda_device))
        assert status(cuda_device) == B.MOE_ERR_INVALID_ARG, o


def test_balance_loss_of_no_tokens(cuda_device):
    x = torch.empty(0, 16, device=cuda_device)
    ids = torch.empty(0, 2, dtype=torch.int32, device=cuda_device)
    got = B.moe_balance_loss(x, ids, 1.0)
    assert float(got["loss"]) == 0 and (got["counts"] == 0).all() and (got["coef"] == 0).all()
    assert B.moe_router_bwd(x, ids, coef=got["coef"]).shape == (0, 16)


# ------------------------------------------------------------------------- streams and graphs
def all_calls(t):
    out = [B.moe_linear(t["x"], t["w"], out_dtype=torch.float32)]
    s, h = B.moe_block_norm(t["x"], t["res"], post_weight=t["wq"], pre_weight=t["wp"])
    g = B.moe_block_norm_bwd(s, h, t["x"], t["res"], post_weight=t["wq"], pre_weight=t["wp"])
    b = B.moe_balance_loss(out[0], t["ids"], 0.1)
    d = B.moe_router_bwd(out[0], t["ids"], t["dw"], b["coef"])
    return out + [s, h, d] + [g[k] for k in sorted(g)] + [b[k] for k in sorted(b)]


def call_inputs(seed):
    T, K, N = 96, 512, 64
    x = rand(T, K, seed=seed, dtype=BF)
    return dict(x=x, w=rand(N, K, seed=seed + 1, std=0.04, dtype=BF),
                res=rand(T, K, seed=seed + 2, dtype=BF), wq=rand(K, seed=seed + 3, dtype=BF),
                wp=rand(K, seed=seed + 4, dtype=BF), dw=rand(T, 4, seed=seed + 5),
                ids=rand(T, N, seed=seed + 6).topk(4, dim=1).indices.to(torch.int32))


def test_calls_on_two_streams_at_a_time(cuda_device):
    ins = [call_inputs(10), call_inputs(20)]
    want = [all_calls(t) for t in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for t, s in zip(ins, streams):
            with torch.cuda.stream(s):
                got.append(all_calls(t))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_calls_captured_into_a_graph(cuda_device):
    t = call_inputs(30)
    all_calls(t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = all_calls(t)
    other = call_inputs(40)
    want = [v.clone() for v in all_calls(other)]
    for k in t:
        t[k].copy_(other[k])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
