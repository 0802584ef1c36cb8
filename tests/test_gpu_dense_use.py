"""How the dense feed-forward block is used: captured graphs, streams and threads, caller's workspaces
and outputs, no rows, values that are not finite, waits that give up, tensors past 2^31 elements."""
import ctypes
import threading

import pytest
import torch

import block_reference as R
import dense_reference as D
from mixture_experts_forward_moe_gb300 import binding as B
from test_gpu_block_ops import BF, HF, rand
from test_gpu_dense_block import d64, weights4

pytestmark = pytest.mark.gpu


def block(T, H, F, dtype, seed=1):
    return (rand(T, H, seed=seed, dtype=dtype),
            rand(2 * F, H, seed=seed + 1, std=H ** -0.5, dtype=dtype),
            rand(T, F, seed=seed + 2, std=0.5, dtype=dtype))


def same(a, b):
    if isinstance(a, dict):
        return sorted(a) == sorted(b) and all(same(a[k], b[k]) for k in a)
    if isinstance(a, tuple):
        return all(same(x, y) for x, y in zip(a, b))
    if isinstance(a, B.Fp8Checkpoint):
        return torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)
    return torch.equal(a, b)


def every_call(seed, dtype=BF, **kw):
    """Each operator once, on inputs of `seed`: calls without arguments."""
    x, w, dh = block(70, 520, 264, dtype, seed)
    g8, u8 = B.moe_checkpoint(rand(70, 264, seed=seed + 5, dtype=dtype)), B.moe_checkpoint(dh)
    x8 = B.moe_checkpoint(x)
    dy = rand(70, 13, seed=seed + 6, dtype=dtype)
    w13 = rand(13, 520, seed=seed + 7, dtype=dtype)
    few = rand(3, 544, seed=seed + 8, dtype=dtype)
    codes, scales, alpha = weights4(66, 544, seed)
    alpha = alpha / 64
    torch.cuda.synchronize()
    return [
        lambda: B.moe_gated_linear(x, w, **kw),
        lambda: B.moe_gated_linear(x[:1].contiguous(), w, **kw),
        lambda: B.moe_gated_linear(x[:5].contiguous(), w, **kw),
        lambda: B.moe_gated_linear(x, w, save=True, **kw),
        lambda: B.moe_gated_linear_bwd(dh, x, w, want_out=True, **kw),
        lambda: B.moe_gated_linear_bwd(dh, x8, w, gate=g8, up=u8, **kw),
        lambda: B.moe_linear_bwd(dy, x8, w13, want_bias=True, **kw),
        lambda: B.moe_linear_w4a16(few, codes, scales, alpha, **kw),
        lambda: B.moe_gated_linear_w4a16(few, codes, scales, alpha, **kw),
    ]


def test_calls_captured_into_a_graph(cuda_device):
    """A captured run of all calls, replayed on other inputs and beside eager calls."""
    calls = every_call(1)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same calls, alive at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [c() for c in calls]
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            g.replay()
        eager = [c() for c in calls]
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(same(a, b) for a, b in zip(out, want))
    assert all(same(a, b) for a, b in zip(eager, want))


def test_streams_and_threads(cuda_device):
    """The same calls on streams of their own at the same time, from two host threads."""
    sets = [every_call(s) for s in (1, 30)]
    want = [[c() for c in calls] for calls in sets]
    torch.cuda.synchronize()
    got, wrong = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got[i] = [c() for c in sets[i]]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for i in range(2):
        assert all(same(a, b) for a, b in zip(got[i], want[i]))


def test_a_given_stream(cuda_device):
    s = torch.cuda.Stream()
    want = [c() for c in every_call(3)]
    calls = every_call(3, stream=s)
    got = [c() for c in calls]
    s.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))


def gated_bytes(T, H, F, fn="moe_gated_linear"):
    p = B.GatedLinear(T, H, F, 0, 0)
    return int(getattr(B.lib(), fn + "_workspace_size")(ctypes.byref(p)))


@pytest.mark.parametrize("T,H,F", [(40, 2048, 264), (300, 1032, 520), (4, 64, 48)])
def test_a_callers_workspace_of_any_contents(T, H, F, cuda_device):
    x, w, dh = block(T, H, F, BF)
    want = (B.moe_gated_linear(x, w, save=True), B.moe_gated_linear_bwd(dh, x, w, want_out=True))
    sizes = [gated_bytes(T, H, F), gated_bytes(T, H, F, "moe_gated_linear_bwd")]
    for n in sizes:
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        if n == sizes[0]:
            assert same(B.moe_gated_linear(x, w, save=True, workspace=ws), want[0])
        if n == sizes[1]:
            assert same(B.moe_gated_linear_bwd(dh, x, w, want_out=True, workspace=ws), want[1])
        assert B.get_device_status(ws) == B.MOE_OK
    short = B.new_workspace(sizes[1] - 256)
    with pytest.raises(B.MoeError, match="workspace"):
        B.moe_gated_linear_bwd(dh, x, w, workspace=short)
    with pytest.raises(ValueError, match="workspace"):
        B.moe_gated_linear(x, w, workspace=torch.zeros(1 << 20))


@pytest.mark.parametrize("T,H,F", [(1, 64, 40), (5, 520, 72), (40, 2048, 264), (300, 520, 136),
                                   (600, 200, 1160)])
def test_nothing_is_written_beside_the_outputs(T, H, F, cuda_device):
    x, w, dh = block(T, H, F, HF)
    guard = 4096
    mark = 0xA5

    def room(nbytes):
        t = torch.full((guard + nbytes + guard,), mark, dtype=torch.uint8, device="cuda")
        return t, t[guard:guard + nbytes]

    groups = (F + 127) // 128
    sizes = dict(out=T * F * 2, gc=T * groups * 128, gs=T * groups * 4, uc=T * groups * 128,
                 us=T * groups * 4)
    bufs = {k: room(n) for k, n in sizes.items()}
    L, p = B.lib(), B.GatedLinear(T, H, F, B.MOE_F16, 0)
    ws = B.new_workspace(gated_bytes(T, H, F, "moe_gated_linear_bwd"))
    stream = torch.cuda.current_stream().cuda_stream
    rc = L.moe_gated_linear(ctypes.byref(p), x.data_ptr(), w.data_ptr(),
                            *(bufs[k][1].data_ptr() for k in sizes), ws.data_ptr(), ws.numel(),
                            stream)
    assert rc == B.MOE_OK
    grads = {k: room(n) for k, n in dict(dx=T * H * 2, dw=2 * F * H * 2, h=T * F * 2).items()}
    rc = L.moe_gated_linear_bwd(ctypes.byref(p), dh.data_ptr(), x.data_ptr(), None, None,
                                w.data_ptr(), None, None, None, None,
                                *(g[1].data_ptr() for g in grads.values()), ws.data_ptr(),
                                ws.numel(), stream)
    assert rc == B.MOE_OK
    torch.cuda.synchronize()
    for whole, _ in list(bufs.values()) + list(grads.values()):
        assert bool((whole[:guard] == mark).all()) and bool((whole[-guard:] == mark).all())
    want = B.moe_gated_linear(x, w, save=True)
    assert torch.equal(bufs["out"][1].view(HF).view(T, F), want[0])
    assert torch.equal(bufs["gc"][1].view(T, -1), want[1].codes)
    assert torch.equal(bufs["us"][1].view(torch.float32).view(T, -1), want[2].scale)
    back = B.moe_gated_linear_bwd(dh, x, w, want_out=True)
    assert torch.equal(grads["dw"][1].view(HF).view(2 * F, H), back["d_w"])
    assert torch.equal(grads["h"][1].view(HF).view(T, F), back["out"])


def test_what_is_wanted(cuda_device):
    x, w, dh = block(70, 264, 136, BF)
    full = B.moe_gated_linear_bwd(dh, x, w, want_out=True)
    for kw, keys in ((dict(want_w=False), ["d_x"]), (dict(want_x=False), ["d_w"]),
                     (dict(want_x=False, want_w=False, want_out=True), ["out"]),
                     (dict(want_x=False, want_w=False), [])):
        got = B.moe_gated_linear_bwd(dh, x, w, **kw)
        assert sorted(got) == keys and all(torch.equal(got[k], full[k]) for k in keys)
    g8, u8 = B.moe_checkpoint(dh), B.moe_checkpoint(dh)
    got = B.moe_gated_linear_bwd(dh, None, w, gate=g8, up=u8, want_w=False)
    want = B.moe_gated_linear_bwd(dh, x, w, gate=g8, up=u8)
    assert sorted(got) == ["d_x"] and torch.equal(got["d_x"], want["d_x"])
    with pytest.raises(ValueError, match="needed"):
        B.moe_gated_linear_bwd(dh, None, w, gate=g8, up=u8)
    with pytest.raises(ValueError, match="needed"):
        B.moe_linear_bwd(dh, None, rand(136, 64, seed=1, dtype=BF))
    lin = rand(136, 64, seed=1, dtype=BF)
    assert sorted(B.moe_linear_bwd(dh, None, lin, want_w=False)) == ["d_x"]
    assert sorted(B.moe_linear_bwd(dh, None, lin, want_w=False, want_x=False,
                                   want_bias=True)) == ["d_bias"]


def test_outputs_in_place_of_inputs(cuda_device):
    x, w, dh = block(300, 264, 136, BF)
    # `out` may be d_out, and the 4-bit product's out its residual
    L, p = B.lib(), B.GatedLinear(300, 264, 136, B.MOE_BF16, 0)
    for saved in (False, True):
        g8, u8 = B.moe_checkpoint(dh), B.moe_checkpoint(-dh)
        kw = dict(gate=g8, up=u8) if saved else {}
        want = B.moe_gated_linear_bwd(dh, x, w, want_out=True, **kw)
        ws = B.new_workspace(gated_bytes(300, 264, 136, "moe_gated_linear_bwd"))
        mine, dw = dh.clone(), torch.empty_like(w)
        ck = [t.data_ptr() for t in (g8.codes, g8.scale, u8.codes, u8.scale)] if saved else [None] * 4
        rc = L.moe_gated_linear_bwd(ctypes.byref(p), mine.data_ptr(), x.data_ptr(), None, None,
                                    w.data_ptr(), *ck, None, dw.data_ptr(), mine.data_ptr(),
                                    ws.data_ptr(), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream)
        assert rc == B.MOE_OK
        assert torch.equal(mine, want["out"]) and torch.equal(dw, want["d_w"])
    codes, scales, alpha = weights4(70, 256, 1)
    few, res = rand(9, 256, seed=2, dtype=BF), rand(9, 70, seed=3, dtype=BF)
    want = B.moe_linear_w4a16(few, codes, scales, alpha / 99, residual=res)
    assert torch.equal(B.moe_linear_w4a16(few, codes, scales, alpha / 99, residual=res, out=res), want)


def test_no_rows(cuda_device):
    w = rand(2 * 40, 64, seed=1, dtype=BF)
    x, dh = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 40, dtype=BF, device="cuda")
    out, gate, up = B.moe_gated_linear(x, w, save=True)
    assert out.shape == (0, 40) and gate.shape == (0, 40) and up.scale.shape == (0, 1)
    assert B.moe_gated_linear(x, w).shape == (0, 40)
    for kw in ({}, dict(gate=gate, up=up)):
        got = B.moe_gated_linear_bwd(dh, x, w, want_out=True, **kw)
        assert got["d_x"].shape == (0, 64) and got["out"].shape == (0, 40)
        assert got["d_w"].shape == w.shape and not bool(got["d_w"].any())
    got = B.moe_linear_bwd(dh, B.moe_checkpoint(x), rand(40, 64, seed=2, dtype=BF), want_bias=True)
    assert not bool(got["d_w"].any()) and not bool(got["d_bias"].any())
    assert got["d_x"].shape == (0, 64)
    assert B.moe_checkpoint_restore(B.moe_checkpoint(x)).shape == (0, 64)
    codes, scales, alpha = weights4(40, 64, 1)
    assert B.moe_linear_w4a16(x, codes, scales, alpha).shape == (0, 40)
    assert B.moe_gated_linear_w4a16(x, codes, scales, alpha).shape == (0, 20)


@pytest.mark.parametrize("T", [1, 2, 9, 40, 300])
def test_values_that_are_not_finite_stay_in_their_row(T, cuda_device):
    x, w, dh = block(T, 520, 136, BF)
    row = T // 2
    bad = x.clone()
    bad[row, 3] = float("nan")
    bad[row, 100] = float("inf")
    clean, gate, up = B.moe_gated_linear(x, w, save=True)
    out, gate2, up2 = B.moe_gated_linear(bad, w, save=True)
    keep = torch.arange(T, device="cuda") != row
    for a, b in ((out, clean), (gate2.codes, gate.codes), (up2.scale, up.scale),
                 (B.moe_gated_linear(bad, w), B.moe_gated_linear(x, w))):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(out[row]).all()) and bool(torch.isnan(B.moe_checkpoint_restore(gate2)[row]).all())
    got, ref = B.moe_gated_linear_bwd(dh, bad, w), B.moe_gated_linear_bwd(dh, x, w)
    assert torch.equal(got["d_x"][keep], ref["d_x"][keep])
    assert bool(torch.isnan(got["d_x"][row]).all()) and bool(torch.isnan(got["d_w"]).all())


def test_far_activations(cuda_device):
    """Gates far out on either side: the activation's flat and steep ends, and its slope there."""
    T, H, F = 64, 64, 64
    x = torch.zeros(T, H)
    x[:, 0] = torch.linspace(-120, 120, T)
    w = torch.zeros(2 * F, H)
    w[:, 0] = 1.0
    x, w = x.to(BF).cuda(), w.to(BF).cuda()
    dh = rand(T, F, seed=1, dtype=BF)
    for act in ("silu", "gelu_tanh"):
        ref, err, g, u, og, ou = D.gated64(d64(x), d64(w), act)
        for out in (B.moe_gated_linear(x, w, activation=act),
                    torch.cat([B.moe_gated_linear(x[i:i + 1], w, activation=act) for i in range(T)])):
            # e^-v of a large v is a subnormal that may be 0
            R.assert_within(out, ref, D.rounded(ref, err, BF) + 2.0 ** -100, act)
        got = B.moe_gated_linear_bwd(dh, x, w, act, want_out=True)
        for k, (want, bound) in D.gated_bwd64(d64(dh), d64(x), d64(w), g, u, og, ou, act, BF).items():
            R.assert_within(got[k], want, bound + 2.0 ** -40, k)


def test_w4_x_past_the_f16_range(cuda_device):
    codes, scales, alpha = weights4(40, 64, 1)
    ws = B.new_workspace(256)
    x = rand(5, 64, seed=1, dtype=BF)
    B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws)
    B.moe_gated_linear_w4a16(x, codes, scales, alpha, workspace=ws)
    assert B.get_device_status(ws) == B.MOE_OK
    x[4, 63] = 65536.0
    B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws)
    assert B.get_device_status(ws) == B.MOE_ERR_F16_RANGE
    B.moe_gated_linear_w4a16(x, codes, scales, alpha, workspace=ws)
    assert B.get_device_status(ws) == B.MOE_ERR_F16_RANGE
    B.moe_linear_w4a16(x.to(HF), codes, scales, alpha, workspace=ws)  # f16 is taken as it is
    assert B.get_device_status(ws) == B.MOE_OK


def test_w4_scales_behind_a_row_are_not_used(cuda_device):
    """K ends inside a block: the next row's scales, NaN here, lie behind it."""
    codes, scales, alpha = weights4(41, 96, 1)
    scales[1::2] = 0x7F  # NaN
    out = B.moe_linear_w4a16(rand(3, 96, seed=1, dtype=HF), codes, scales, alpha)
    assert bool(torch.isfinite(out[:, 0::2]).all()) and bool(torch.isnan(out[:, 1::2]).all())


def w4_bytes(T, N, K, dtype):
    g = B.Linear(T, N, K, B.MOE_BF16 if dtype is BF else B.MOE_F16, 0, 0)
    return int(B.lib().moe_linear_w4a16_workspace_size(ctypes.byref(g)))


@pytest.mark.parametrize("T", [20, 70])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_w4_tiles_in_a_callers_workspace(T, dtype, cuda_device):
    """Any contents, canaries behind it, a captured graph, and one that is too small."""
    N, K = 200, 608
    codes, scales, alpha = weights4(N, K, 1)
    x = rand(T, K, seed=1, dtype=dtype)
    want = B.moe_linear_w4a16(x, codes, scales, alpha)
    n = w4_bytes(T, N, K, dtype)
    assert n % 256 == 0 and n >= 256 + (T * K * 2 if dtype is BF else 0)
    whole = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = whole[:n]
    ws[:256] = 0
    assert torch.equal(B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws), want)
    assert bool((whole[n:] == 0xFF).all())
    if dtype is BF:
        with pytest.raises(B.MoeError, match="workspace"):
            B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws[:n - 256])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        B.moe_linear_w4a16(x, codes, scales, alpha)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.moe_linear_w4a16(x, codes, scales, alpha)
    x2 = rand(T, K, seed=2, dtype=dtype)
    want2 = B.moe_linear_w4a16(x2, codes, scales, alpha)
    x.copy_(x2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want2)


def test_w4_tiles_report_values_past_the_f16_range(cuda_device):
    codes, scales, alpha = weights4(40, 64, 1)
    ws = B.new_workspace(w4_bytes(20, 40, 64, BF))
    x = rand(20, 64, seed=1, dtype=BF)
    for call in (B.moe_linear_w4a16, B.moe_gated_linear_w4a16):
        x[19, 63] = 1.0
        call(x, codes, scales, alpha, workspace=ws)
        assert B.get_device_status(ws) == B.MOE_OK
        x[19, 63] = 65536.0
        call(x, codes, scales, alpha, workspace=ws)
        assert B.get_device_status(ws) == B.MOE_ERR_F16_RANGE


def test_w4_tiles_leave_out_scales_behind_a_row(cuda_device):
    codes, scales, alpha = weights4(41, 96, 1)
    scales[1::2] = 0x7F  # NaN
    x = rand(40, 96, seed=1, dtype=HF)
    x[7] = float("nan")  # and a row of NaN stays in its row
    out = B.moe_linear_w4a16(x, codes, scales, alpha)
    assert bool(torch.isnan(out[7]).all()) and bool(torch.isnan(out[:, 1::2]).all())
    out = torch.cat([out[:7], out[8:]])
    assert bool(torch.isfinite(out[:, 0::2]).all())


@pytest.mark.parametrize("T,N,K", [(20, 500, 4096), (100, 300, 1000 // 32 * 32), (200, 24000, 256)])
def test_a_wait_of_w4_tiles_that_gives_up(T, N, K, cuda_device):
    """As test_a_wait_that_gives_up."""
    codes, scales, alpha = weights4(N, K, 1)
    x = rand(T, K, seed=1, dtype=BF)
    ws = B.new_workspace(w4_bytes(T, N, K, BF))
    want = B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        for _ in range(2):
            B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws)
            assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT
    finally:
        B.set_wait_limit_ns(old)
    assert torch.equal(B.moe_linear_w4a16(x, codes, scales, alpha, workspace=ws), want)
    assert B.get_device_status(ws) == B.MOE_OK


def test_w4_rows_agree_with_the_experts(cuda_device):
    """The 4-bit product is the grouped 4-bit product of one expert, whose weights are packed."""
    codes, scales, alpha = weights4(256, 512, 5)
    alpha = alpha / 64
    x = rand(4, 512, seed=1, dtype=BF)
    w = B.pack_nvfp4_weights(codes[None], scales[None], alpha)
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    s = B.moe_align_sort(ids, 1)
    act = B.moe_gemm1_w4a16(x, s["sorted_ids"], s["offsets"], w, 1)
    out = B.moe_gated_linear_w4a16(x, codes, scales, alpha)
    ref, bound = D.w4_gated64(x, D.weights64(codes, scales, alpha.cpu()), "silu")
    R.assert_within(out, ref, bound, "rows")
    # their results are one rounding to f16 apart from the sums
    R.assert_within(act[:4], ref, bound, "experts")


def test_checkpoints_are_the_rows_of_the_fp8_grouped_product(cuda_device):
    x = rand(96, 256, seed=1, dtype=BF)
    b = torch.randint(0, 120, (1, 128, 256), generator=torch.Generator().manual_seed(2),
                      dtype=torch.uint8).cuda()
    bs = torch.full((1, 1, 2), 2.0 ** -6, device="cuda")
    c = B.moe_checkpoint(x)
    rows = torch.tensor([96], dtype=torch.int32, device="cuda")
    out = B.moe_grouped_gemm_fp8(c.codes, c.scale, b, bs, rows)
    wide = D.restore64(b[0], bs[0].expand(128, 2), 256)
    ref, off = D.product64(D.restore64(c.codes, c.scale, 256), wide)
    # f32 sums of 128-k blocks, each scaled once and rounded
    R.assert_within(out, ref, D.rounded(ref, 2 * off, BF), "fp8")


@pytest.mark.parametrize("T,H,F", [(7, 4096, 136), (30, 520, 20000), (100, 1032, 3080)])
def test_a_wait_of_few_rows_that_gives_up(T, H, F, cuda_device):
    """As test_a_wait_that_gives_up; and a captured graph with a row of NaN in its second input."""
    x, w, _ = block(T, H, F, HF)
    ws = B.new_workspace(gated_bytes(T, H, F, "moe_gated_linear"))
    want = B.moe_gated_linear(x, w, workspace=ws)
    torch.cuda.synchronize()
    old = B.set_wait_limit_ns(0)
    try:
        for _ in range(2):
            B.moe_gated_linear(x, w, workspace=ws)
            assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT
    finally:
        B.set_wait_limit_ns(old)
    assert torch.equal(B.moe_gated_linear(x, w, workspace=ws), want)
    assert B.get_device_status(ws) == B.MOE_OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.moe_gated_linear(x, w)
    x[2] = float("nan")
    graph.replay()
    torch.cuda.synchronize()
    rest = [i for i in range(T) if i != 2]
    assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[2]).all())


# T, H, F: each form of the tiles (narrow and wide, split or not), its epilogues and both operand orders
@pytest.mark.parametrize("T,H,F", [(40, 4096, 136), (300, 520, 136), (1000, 1032, 3080)])
def test_a_wait_that_gives_up(T, H, F, cuda_device):
    """The wait limit is 0, so that the first look that finds nothing landed gives up; nothing hangs."""
    x, w, dh = block(T, H, F, BF)
    ws = B.new_workspace(gated_bytes(T, H, F, "moe_gated_linear_bwd"))
    calls = [lambda: B.moe_gated_linear(x, w, workspace=ws),
             lambda: B.moe_gated_linear(x, w, save=True, workspace=ws),
             lambda: B.moe_gated_linear_bwd(dh, x, w, want_out=True, workspace=ws)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for c, right in zip(calls, want):
        old = B.set_wait_limit_ns(0)
        try:
            for _ in range(2):
                c()
                assert B.get_device_status(ws) == B.MOE_ERR_TIMEOUT  # synchronises, clears
        finally:
            B.set_wait_limit_ns(old)
        assert same(c(), right) and B.get_device_status(ws) == B.MOE_OK


def some(n, count, seed):
    return torch.randint(0, n, (count,), generator=torch.Generator().manual_seed(seed))


def test_gradients_past_2_31_elements(cuda_device):
    """d_w of 46400 x 46400: over 2^31 elements, and d_x from as many weights."""
    N = K = 46400
    T = 9
    dy, x = rand(T, N, seed=1, dtype=BF), rand(T, K, seed=2, dtype=BF)
    w = torch.empty(N, K, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(0, N, 4640):
        w[i:i + 4640] = (torch.randn(4640, K, generator=g, device="cuda") * 0.005).to(BF)
    got = B.moe_linear_bwd(dy, x, w, want_bias=True)
    rows, cols = some(N, 64, 4), some(K, 64, 5)
    rows[-1], cols[-1] = N - 1, K - 1
    want, off = D.product64(d64(dy)[:, rows].T, d64(x)[:, cols].T)
    R.assert_within(got["d_w"][rows.cuda()][:, cols.cuda()], want, D.rounded(want, off, BF), "d_w")
    want, off = D.product64(d64(dy), d64(w[:, cols.cuda()]).T)
    R.assert_within(got["d_x"][:, cols.cuda()], want, D.rounded(want, off, BF), "d_x")


def test_rows_past_2_31_elements(cuda_device):
    """x, its checkpoint and the gated product's gradients with over 2^31 elements in rows."""
    T, C = 270000, 8192
    x = torch.empty(T, C, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(0, T, 27000):
        x[i:i + 27000] = torch.randn(27000, C, generator=g, device="cuda").to(BF)
    saved = B.moe_checkpoint(x)
    back = B.moe_checkpoint_restore(saved, BF)
    rows = some(T, 40, 4)
    rows[-1] = T - 1
    want, scale = D.checkpoint64(d64(x[rows.cuda()]))
    assert torch.equal(d64(back[rows.cuda()]), want)
    assert torch.equal(saved.scale[rows.cuda()].cpu().double(), scale)
    del back
    w = rand(2 * 8, C, seed=5, std=C ** -0.5, dtype=BF)
    out = B.moe_gated_linear(x, w)
    ref, err = D.gated64(d64(x[rows.cuda()]), d64(w), "silu")[:2]
    R.assert_within(out[rows.cuda()], ref, D.rounded(ref, err, BF), "out")


def test_4_bit_weights_past_2_31_bytes(cuda_device):
    N, K = 70016, 65536
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda",
                          generator=torch.Generator(device="cuda").manual_seed(1))
    scales = torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    scales[:, 7] = 0x40  # 2.0
    alpha = torch.tensor([2.0 ** -10], device="cuda")
    x = rand(2, K, seed=2, dtype=BF)
    rows = some(N, 24, 3)
    rows[-1] = N - 1
    out = B.moe_linear_w4a16(x, codes, scales, alpha)
    w = D.weights64(codes[rows.cuda()], scales[rows.cuda()], alpha.cpu())
    ref, bound = D.w4_linear64(x, w, None, "none", None)
    R.assert_within(out[:, rows.cuda()], ref, bound, "out")
