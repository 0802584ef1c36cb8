"""The dense feed-forward block beside the routed experts, as it is measured: training with 8-bit
checkpoints, and decoding with 4-bit weights.  The cases, their inputs, one pass of each in plain
torch operations (``own`` false) or through the library (``own`` true), and the same from the
definitions in 64 bits (``exact``).

  gated       h = act(x Wg^T) * (x Wu^T), and its pre-activations as an 8-bit checkpoint
  gated_bwd   the gradients of gated; the pre-activations recomputed, or from the checkpoint
  linear_bwd  the gradients of x w^T + bias; x in 16 bits or from a checkpoint
  checkpoint  E4M3 values with one power of two per 128 channels: saved and restored
  w4          x w^T of 4-bit weights with a scale per 16 (NVFP4): act, bias, residual, or gated

Sizes are those of the workloads in ``mixture_experts_forward_moe_gb300.inputs`` (hidden 2048,
4096 and 7168; intermediate 768, 1536, 2048 and 18432; 32, 512 and 4096 tokens), and odd ones.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_GROUP = 128  # channels that share a scale of a checkpoint
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token through a shared expert's first half
        dict(name="gated-t1", op="gated", T=1, H=7168, F=2048, dtype="bf16", act="silu",
             save=False),
        # a ragged batch of a small model, nothing saved
        dict(name="gated-ragged-t333", op="gated", T=333, H=2056, F=1544, dtype="f16",
             act="gelu_tanh", save=False),
        # a training step's forward that saves 8 bits per pre-activation
        dict(name="gated-t4096-save", op="gated", T=4096, H=7168, F=2048, dtype="bf16",
             act="silu", save=True),
        # a ragged batch's gradients with nothing saved but the input
        dict(name="gated-bwd-ragged-t517", op="gated_bwd", T=517, H=2056, F=1544, dtype="f16",
             act="gelu_tanh", saved=False),
        # the gradients of gated-t4096-save, from 8-bit checkpoints alone
        dict(name="gated-bwd-t4096-saved", op="gated_bwd", T=4096, H=7168, F=2048, dtype="bf16",
             act="silu", saved=True),
        # a small projection with a bias and an odd width
        dict(name="linear-bwd-ragged-t100", op="linear_bwd", T=100, N=4099, K=2056, dtype="f16",
             bias=True, saved=False),
        # a dense down projection's gradients in a training step: the largest products
        dict(name="linear-bwd-t4096", op="linear_bwd", T=4096, N=7168, K=18432, dtype="bf16",
             bias=False, saved=True),
        # the checkpoint of a small batch, channels that end inside a group
        dict(name="checkpoint-t33", op="checkpoint", T=33, C=2056, dtype="f16"),
        # the checkpoint of a packed training batch
        dict(name="checkpoint-t32768", op="checkpoint", T=32768, C=7168, dtype="bf16"),
        # one decoded token, 4-bit weights: a down projection with the residual, a gated half
        dict(name="w4-down-t1", op="w4", T=1, N=7168, K=18432, dtype="bf16", act="none",
             gated=False, bias=False, residual=True),
        dict(name="w4-gated-t1", op="w4", T=1, N=2048, K=7168, dtype="bf16", act="silu",
             gated=True, bias=False, residual=False),
        # a decode batch with everything in the epilogue and an odd width
        dict(name="w4-ragged-t32", op="w4", T=32, N=4099, K=4128, dtype="f16", act="gelu_tanh",
             gated=False, bias=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_bwd", "linear_bwd", "checkpoint", "w4", "w4"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "checkpoint":
        C = 8 * _log_int(rng, 8, 2304)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 32768 * 7168 // C)), C=C, dtype=dtype)
    if op == "w4":
        gated = rng.random() < 0.4
        return dict(op=op, T=_log_int(rng, 1, 64), N=_log_int(rng, 8, 8192),
                    K=32 * _log_int(rng, 2, 576), dtype=dtype, gated=gated,
                    act=rng.choice(["silu", "gelu_tanh"] if gated else
                                   ["none", "silu", "gelu_tanh", "relu2"]),
                    bias=not gated and rng.random() < 0.4,
                    residual=not gated and rng.random() < 0.4)
    if op == "linear_bwd":
        return dict(op=op, T=_log_int(rng, 1, 4096), N=_log_int(rng, 8, 8192),
                    K=8 * _log_int(rng, 8, 1024), dtype=dtype, bias=rng.random() < 0.5,
                    saved=rng.random() < 0.5)
    c = dict(op=op, T=_log_int(rng, 1, 4096), H=8 * _log_int(rng, 8, 1024),
             F=8 * _log_int(rng, 8, 512), dtype=dtype, act=rng.choice(["silu", "gelu_tanh"]))
    c["save" if op == "gated" else "saved"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------------- inputs
def _groups(v):
    """[T, C] as [T, groups, 128], zeros behind the last channel."""
    pad = -v.shape[1] % _GROUP
    return torch.nn.functional.pad(v, (0, pad)).view(v.shape[0], -1, _GROUP)


def _save(v):
    """The 8-bit checkpoint of [T, C]: codes [T, C up to 128] as bytes and scales [T, groups]: the
    smallest power of two that brings the group's largest value to 448 or less, 1 for zeros."""
    b = _groups(v.float())
    top = b.abs().amax(dim=2)
    mantissa, exponent = torch.frexp(top)
    k = exponent - 9 + (mantissa > 0.875)  # 448 = 0.875 * 2^9
    scale = torch.where(top > 0, torch.exp2(k.clamp(-118, 120).float()), torch.ones_like(top))
    codes = (b / scale[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(v.shape[0], -1), scale


def _restore(saved, C, dtype):
    codes, scale = saved
    v = codes.view(torch.float8_e4m3fn).float().view(*scale.shape, _GROUP) * scale[:, :, None]
    v = v.view(scale.shape[0], -1)[:, :C]
    top = torch.finfo(dtype).max
    return v.clamp(-top, top).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (t * std).to(dtype)

    s = dict(case)
    op, T, dt = case["op"], case["T"], _DTYPES[case["dtype"]]
    if op in ("gated", "gated_bwd"):
        H, F = case["H"], case["F"]
        s["x"] = randn(T, H, dtype=dt)
        s["w"] = randn(2 * F, H, std=1.0 / math.sqrt(H), dtype=dt)
        if op == "gated_bwd":
            s["dh"] = randn(T, F, std=0.5, dtype=dt)
            if case["saved"]:  # the checkpoints of the forward, which keeps nothing else
                s["x8"] = _save(s.pop("x"))
                s["gate8"], s["up8"] = _save(randn(T, F)), _save(randn(T, F))
    elif op == "linear_bwd":
        N, K = case["N"], case["K"]
        s["x"] = randn(T, K, dtype=dt)
        s["w"] = randn(N, K, std=1.0 / math.sqrt(K), dtype=dt)
        s["dy"] = randn(T, N, std=0.5, dtype=dt)
        if case["saved"]:
            s["x8"] = _save(s.pop("x"))
    elif op == "checkpoint":
        # a few channels of large values, as hidden states have them
        C = case["C"]
        wide = torch.rand(C, generator=g, device="cuda") < 0.01
        s["x"] = (randn(T, C) * torch.where(wide, 30.0, 1.0)).to(dt)
    else:
        N, K = case["N"], case["K"]
        rows = 2 * N if case["gated"] else N
        s["x"] = randn(T, K, dtype=dt)
        s["codes"] = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda",
                                   dtype=torch.uint8)
        # scales of blocks of normal weights: E4M3 values around 448 / 2
        block = 120.0 + 300.0 * torch.rand(rows, K // 16, generator=g, device="cuda")
        s["scales"] = block.to(torch.float8_e4m3fn).view(torch.uint8)
        s["alpha"] = torch.full((1,), 1.0 / (280.0 * 3.0 * math.sqrt(K)), device="cuda")
        s["b"] = randn(N, std=0.5, dtype=dt) if case["bias"] else None
        s["res"] = randn(T, N, dtype=dt) if case["residual"] else None
    return s


# ------------------------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu2":
        return z.clamp(min=0) ** 2
    return z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _gated(s):
    dt = s["x"].dtype
    gate, up = (s["x"].float() @ s["w"].float().t()).chunk(2, dim=1)
    out = dict(out=(_act(gate, s["act"]) * up).to(dt))
    if s["save"]:
        out["gate"] = _restore(_save(gate), s["F"], dt)
        out["up"] = _restore(_save(up), s["F"], dt)
    return out


def _gated_bwd(s):
    dt, w = s["w"].dtype, s["w"].float()
    if s["saved"]:
        x = _restore(s["x8"], s["H"], dt).float()
        gate = _restore(s["gate8"], s["F"], torch.float32)
        up = _restore(s["up8"], s["F"], torch.float32)
    else:
        x = s["x"].float()
        gate, up = (x @ w.t()).chunk(2, dim=1)
    dh = s["dh"].float()
    a = _act(gate, s["act"])
    d = torch.cat([dh * up * _act_slope(gate, s["act"]), dh * a], dim=1)
    return dict(d_x=(d @ w).to(dt), d_w=(d.t() @ x).to(dt), out=(a * up).to(dt))


def _linear_bwd(s):
    dt, dy = s["w"].dtype, s["dy"].float()
    x = _restore(s["x8"], s["K"], dt) if s["saved"] else s["x"]
    out = dict(d_x=(dy @ s["w"].float()).to(dt), d_w=(dy.t() @ x.float()).to(dt))
    if s["bias"]:
        out["d_bias"] = dy.sum(dim=0).to(dt)
    return out


def _checkpoint(s):
    codes, scale = _save(s["x"])
    return dict(values=_restore((codes, scale), s["C"], s["x"].dtype), scale=scale)


def _w4(s):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda")
    codes = s["codes"]
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=2)
    scales = s["scales"].view(torch.float8_e4m3fn).float()
    w = v.view(codes.shape[0], -1, 16) * scales[:, :, None]
    z = (s["x"].float() @ w.view(codes.shape[0], -1).t()) * s["alpha"]
    if s["gated"]:
        gate, up = z.chunk(2, dim=1)
        return (_act(gate, s["act"]) * up).to(s["x"].dtype)
    if s["b"] is not None:
        z = z + s["b"].float()
    z = _act(z, s["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return z.to(s["x"].dtype)


_PLAIN = {"gated": _gated, "gated_bwd": _gated_bwd, "linear_bwd": _linear_bwd,
          "checkpoint": _checkpoint, "w4": _w4}


def _library(s):
    from mixture_experts_forward_moe_gb300 import binding as B

    op = s["op"]
    if op == "gated":
        if not s["save"]:
            return dict(out=B.moe_gated_linear(s["x"], s["w"], activation=s["act"]))
        out, gate, up = B.moe_gated_linear(s["x"], s["w"], activation=s["act"], save=True)
        return dict(out=out, gate=B.moe_checkpoint_restore(gate, s["x"].dtype),
                    up=B.moe_checkpoint_restore(up, s["x"].dtype))
    if op == "gated_bwd":
        x, saved = s.get("x"), {}
        if s["saved"]:
            x = B.Fp8Checkpoint(*s["x8"], s["H"])
            saved = dict(gate=B.Fp8Checkpoint(*s["gate8"], s["F"]),
                         up=B.Fp8Checkpoint(*s["up8"], s["F"]))
        return B.moe_gated_linear_bwd(s["dh"], x, s["w"], activation=s["act"], want_out=True,
                                      **saved)
    if op == "linear_bwd":
        x = B.Fp8Checkpoint(*s["x8"], s["K"]) if s["saved"] else s["x"]
        return B.moe_linear_bwd(s["dy"], x, s["w"], want_bias=s["bias"])
    if op == "checkpoint":
        saved = B.moe_checkpoint(s["x"])
        return dict(values=B.moe_checkpoint_restore(saved, s["x"].dtype), scale=saved.scale)
    if s["gated"]:
        return B.moe_gated_linear_w4a16(s["x"], s["codes"], s["scales"], s["alpha"],
                                        activation=s["act"])
    return B.moe_linear_w4a16(s["x"], s["codes"], s["scales"], s["alpha"], bias=s["b"],
                              activation=s["act"], residual=s["res"])


def run(state):
    return _library(state) if own else _PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["T"]

    def saved_bytes(C):
        groups = -(-C // _GROUP)
        return T * groups * (_GROUP + 4)

    if op == "gated":
        H, F = case["H"], case["F"]
        b = 2 * (T * H + 2 * F * H + T * F)
        if case["save"]:  # written, and read back into 16 bits
            b += 2 * (2 * saved_bytes(F) + 2 * T * F)
        return {"bytes": b, "flops": 4 * T * F * H}
    if op == "gated_bwd":
        H, F = case["H"], case["F"]
        x = saved_bytes(H) + 2 * saved_bytes(F) if case["saved"] else 2 * T * H
        b = x + 2 * (2 * F * H + T * F + T * H + 2 * F * H + T * F)
        return {"bytes": b, "flops": (8 if case["saved"] else 12) * T * F * H}
    if op == "linear_bwd":
        N, K = case["N"], case["K"]
        x = saved_bytes(K) if case["saved"] else 2 * T * K
        b = x + 2 * (2 * N * K + T * N + T * K + (N if case["bias"] else 0))
        return {"bytes": b, "flops": 4 * T * N * K}
    if op == "checkpoint":
        C = case["C"]
        return {"bytes": 4 * T * C + 2 * saved_bytes(C), "flops": 4 * T * C}
    N, K = case["N"], case["K"]
    rows = 2 * N if case["gated"] else N
    b = rows * K // 2 + rows * K // 16 + 2 * T * (K + N)
    b += (2 * N if case["bias"] else 0) + (2 * T * N if case["residual"] else 0)
    return {"bytes": b, "flops": 2 * T * rows * K}


# ------------------------------------------------------------------------- the 64-bit oracle
def _exact_restore(saved, C, dtype=None):
    """What a checkpoint stands for: E4M3 bits taken apart, times the group's scale."""
    codes, scale = saved
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    v = torch.where(c >= 128, -mag, mag) * scale.double().repeat_interleave(_GROUP, dim=1)
    v = v[:, :C]
    if dtype is torch.float16:
        v = v.clamp(-65504.0, 65504.0)
    return v


def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return torch.nn.functional.gelu(z, approximate="tanh")
    if act == "relu2":
        return torch.relu(z).square()
    return z


def _exact_e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.exp2((e.clamp(min=-5) - 4).double())
    return torch.round(v / step) * step


def _exact_checkpoint(v, C):
    b = _groups(v)
    top = b.abs().amax(dim=2)
    k = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    k = k + (torch.exp2(k) * 448 < top).double() - (torch.exp2(k - 1) * 448 >= top).double()
    scale = torch.where(top > 0, torch.exp2(k.clamp(-118, 120)), torch.ones_like(top))
    q = _exact_e4m3(b / scale[:, :, None]) * scale[:, :, None]
    return q.reshape(v.shape[0], -1)[:, :C], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        z = torch.nn.functional.linear(s["x"].double(), s["w"].double())
        gate, up = z[:, :case["F"]], z[:, case["F"]:]
        out = dict(out=_exact_act(gate, case["act"]) * up)
        if case["save"]:
            out["gate"] = _exact_checkpoint(gate, case["F"])[0]
            out["up"] = _exact_checkpoint(up, case["F"])[0]
        return out
    if op == "gated_bwd":
        H, F, dt = case["H"], case["F"], s["w"].dtype
        w = s["w"].double()
        if case["saved"]:
            x = _exact_restore(s["x8"], H, dt)
            gate, up = _exact_restore(s["gate8"], F), _exact_restore(s["up8"], F)
        else:
            x = s["x"].double()
            z = torch.nn.functional.linear(x, w)
            gate, up = z[:, :F], z[:, F:]
        gate, up = gate.clone().requires_grad_(True), up.clone().requires_grad_(True)
        h = _exact_act(gate, case["act"]) * up
        dg, du = torch.autograd.grad(h, [gate, up], s["dh"].double())
        return dict(d_x=dg @ w[:F] + du @ w[F:], d_w=torch.cat([dg.t() @ x, du.t() @ x]),
                    out=h.detach())
    if op == "linear_bwd":
        x = (_exact_restore(s["x8"], case["K"], s["w"].dtype) if case["saved"]
             else s["x"].double())
        dy = s["dy"].double()
        out = dict(d_x=torch.einsum("tn,nk->tk", dy, s["w"].double()),
                   d_w=torch.einsum("tn,tk->nk", dy, x))
        if case["bias"]:
            out["d_bias"] = torch.einsum("tn->n", dy)
        return out
    if op == "checkpoint":
        v, scale = _exact_checkpoint(s["x"].double(), case["C"])
        if s["x"].dtype is torch.float16:
            v = v.clamp(-65504.0, 65504.0)
        return dict(values=v, scale=scale)
    c = s["codes"].to(torch.int64)
    nibble = torch.empty(c.shape[0], 2 * c.shape[1], dtype=torch.int64, device="cuda")
    nibble[:, 0::2], nibble[:, 1::2] = c % 16, c // 16
    e, m = (nibble // 2) % 4, (nibble % 2).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
    v = torch.where(nibble >= 8, -v, v)
    sc = s["scales"].to(torch.int32)
    se, sm = (sc >> 3) & 15, (sc & 7).double()
    scale = torch.where(se > 0, (1 + sm / 8) * torch.exp2((se - 7).double()), sm * 2.0 ** -9)
    w = v * scale.repeat_interleave(16, dim=1) * s["alpha"].double()
    z = torch.nn.functional.linear(s["x"].double(), w, None if s["b"] is None else s["b"].double())
    if case["gated"]:
        return _exact_act(z[:, :case["N"]], case["act"]) * z[:, case["N"]:]
    z = _exact_act(z, case["act"])
    return z if s["res"] is None else z + s["res"].double()
