"""The operators around the routed experts, as they are measured: the cases, their inputs, one
pass of each in plain torch operations (``own`` false) or through the library (``own`` true), and
the same from the definitions in 64 bits (``exact``).

  linear      out = act(x w^T + bias) + residual; 16-bit operands, out in their type or f32
  norm        stream = a residual + gate * norm(branch); normed = norm(stream)
  norm_bwd    the gradients of norm
  balance     per-expert counts and the balance loss over ragged sequences
  router_bwd  the gradient of the router logits: balance loss and route weights

Sizes are those of the workloads in ``mixture_experts_forward_moe_gb300.inputs`` (hidden 2048,
4096 and 7168; 128, 256 and 384 experts, top-8; 32, 512 and 4096 tokens; a dense intermediate
size of 18432), and odd ones.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6


def listed():
    return [
        # the router's projection of one decoded token: a call's latency
        dict(name="router-proj-t1", op="linear", T=1, N=256, K=7168, dtype="bf16", act="none",
             bias=False, residual=False, out_f32=True),
        # the same at prefill: f32 logits with a bias
        dict(name="router-proj-t4096", op="linear", T=4096, N=256, K=7168, dtype="bf16",
             act="none", bias=True, residual=False, out_f32=True),
        # a ragged decode batch through a dense projection with everything in its epilogue
        dict(name="dense-ragged-t33", op="linear", T=33, N=4099, K=2056, dtype="f16",
             act="gelu_tanh", bias=True, residual=True, out_f32=False),
        # a dense down projection of a prefill with the residual: the largest product
        dict(name="dense-down-t4096", op="linear", T=4096, N=7168, K=18432, dtype="bf16",
             act="none", bias=False, residual=True, out_f32=False),
        # one decoded token between two blocks
        dict(name="norm-t1", op="norm", T=1, H=7168, dtype="bf16", gate="channel", post=True,
             pre=True, scale=1.0, offset=0.0),
        # a prefill between two blocks
        dict(name="norm-t4096", op="norm", T=4096, H=7168, dtype="bf16", gate="channel",
             post=True, pre=True, scale=0.7, offset=0.0),
        # training: a ragged batch with a gate per element, zero-centred norm weights
        dict(name="norm-bwd-ragged-t517", op="norm_bwd", T=517, H=2056, dtype="f16",
             gate="element", post=True, pre=True, scale=1.0, offset=1.0),
        # training: the gradients of norm-t4096
        dict(name="norm-bwd-t4096", op="norm_bwd", T=4096, H=7168, dtype="bf16", gate="channel",
             post=True, pre=True, scale=0.7, offset=0.0),
        # a small step's loss over the whole batch
        dict(name="balance-t512", op="balance", T=512, E=128, k=8, n_seq=1, scoring="softmax",
             pad=0.0),
        # packed sequences of a training step, some tokens padding
        dict(name="balance-t32768-seqs", op="balance", T=32768, E=256, k=8, n_seq=11,
             scoring="sigmoid", pad=0.03),
        # the gradient of a small step: renormalised softmax weights
        dict(name="router-bwd-t512", op="router_bwd", T=512, E=128, k=8, n_seq=1,
             scoring="softmax", renorm=True, pad=0.0),
        # the gradient of the packed sequences
        dict(name="router-bwd-t32768-seqs", op="router_bwd", T=32768, E=384, k=8, n_seq=11,
             scoring="sigmoid", renorm=True, pad=0.03),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm_bwd", "balance", "router_bwd"])
    if op == "linear":
        out_f32 = rng.random() < 0.4
        return dict(op=op, T=_log_int(rng, 1, 4096), N=_log_int(rng, 8, 8192),
                    K=8 * _log_int(rng, 8, 1024), dtype=rng.choice(["bf16", "f16"]),
                    act=rng.choice(["none", "silu", "gelu_tanh", "relu2"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, out_f32=out_f32)
    if op in ("norm", "norm_bwd"):
        H = 8 * _log_int(rng, 8, 1024)
        return dict(op=op, T=_log_int(rng, 1, min(16384, 4096 * 7168 // H)), H=H,
                    dtype=rng.choice(["bf16", "f16"]),
                    gate=rng.choice(["none", "channel", "token", "element"]),
                    post=rng.random() < 0.7, pre=rng.random() < 0.8,
                    scale=rng.choice([1.0, 0.7]), offset=rng.choice([0.0, 1.0]))
    E = _log_int(rng, 8, 512)
    T = _log_int(rng, 1, min(32768, 32768 * 256 // E))
    c = dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), n_seq=_log_int(rng, 1, 40),
             scoring=rng.choice(["softmax", "sigmoid"]), pad=rng.choice([0.0, 0.05]))
    if op == "router_bwd":
        c["renorm"] = rng.random() < 0.6
    return c


# ---------------------------------------------------------------------------------- inputs
def _ragged(T, n_seq, g):
    """[n_seq + 1] int32 offsets of random lengths that add up to T (some may be empty)."""
    cuts = torch.randint(0, T + 1, (n_seq - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (t * std + mean).to(dtype)

    s = dict(case)
    op = case["op"]
    if op == "linear":
        T, N, K, dt = case["T"], case["N"], case["K"], _DTYPES[case["dtype"]]
        odt = torch.float32 if case["out_f32"] else dt
        s["x"] = randn(T, K, dtype=dt)
        s["w"] = randn(N, K, std=1.0 / math.sqrt(K), dtype=dt)
        s["b"] = randn(N, std=0.5, dtype=dt) if case["bias"] else None
        s["res"] = randn(T, N, dtype=odt) if case["residual"] else None
    elif op in ("norm", "norm_bwd"):
        T, H, dt = case["T"], case["H"], _DTYPES[case["dtype"]]
        mean = 1.0 - case["offset"]
        s["y"] = randn(T, H, std=0.8, dtype=dt)
        s["x"] = randn(T, H, std=1.5, dtype=dt)
        shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[case["gate"]]
        s["g"] = None if shape is None else randn(*shape, std=0.3, mean=0.6, dtype=dt)
        s["wq"] = randn(H, std=0.1, mean=mean, dtype=dt) if case["post"] else None
        s["wp"] = randn(H, std=0.1, mean=mean, dtype=dt) if case["pre"] else None
        if op == "norm_bwd":
            s["dr"] = randn(T, H, std=0.5, dtype=dt)
            s["dh"] = randn(T, H, std=0.5, dtype=dt) if case["pre"] else None
    else:
        T, E, k, n_seq = case["T"], case["E"], case["k"], case["n_seq"]
        # logits of a router whose experts are not equally popular
        s["logits"] = randn(T, E) + randn(E, std=0.4)
        ids = s["logits"].topk(k, dim=1).indices.to(torch.int32)
        if case["pad"]:
            dead = torch.rand(T, generator=g, device="cuda") < case["pad"]
            ids = torch.where(dead[:, None], torch.full_like(ids, -1), ids)
        s["ids"] = ids
        s["offsets"] = _ragged(T, n_seq, g) if n_seq > 1 else None
        s["coeff"] = 0.01
        if op == "router_bwd":
            # gradients of a mean over the tokens
            s["dw"] = randn(T, k, std=0.02 / T)
            s["d_loss"] = torch.ones(1, device="cuda")
            s["coef"] = _coef(s)
            s["factor"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
    return s


def _live(s):
    """Each token's sequence, and which tokens are not padding."""
    T = s["T"]
    live = (s["ids"] >= 0).any(dim=1)
    if s["offsets"] is None:
        return torch.zeros(T, dtype=torch.int64, device="cuda"), live
    tok = torch.arange(T, device="cuda")
    return (tok[:, None] >= s["offsets"][None, 1:-1]).sum(dim=1), live


def _tables(s):
    """Routes and live tokens of each sequence: counts [n_seq, E], live [n_seq]."""
    n, E = s["n_seq"], s["E"]
    seq, live = _live(s)
    slot = torch.where(s["ids"] >= 0, seq[:, None] * E + s["ids"], n * E).reshape(-1)
    counts = torch.zeros(n * E + 1, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    tokens.scatter_add_(0, seq, live.to(torch.int32))
    return counts[: n * E].view(n, E), tokens


def _coef(s):
    """coeff E count / (n_live k T_s^2): what each token's probabilities are weighted with."""
    counts, tokens = _tables(s)
    n_live = (tokens > 0).sum().clamp(min=1)
    per = tokens.clamp(min=1).double()[:, None]
    return (s["coeff"] * s["E"] * counts / (n_live * s["k"] * per * per)).float()


# ------------------------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu2":
        return z.clamp(min=0) ** 2
    return z


def _linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    z = _act(z, s["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return z if s["out_f32"] else z.to(s["x"].dtype)


def _rstd(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS)


def _gate(s):
    if s["g"] is None:
        return 1.0
    g = s["g"].float()
    return g[:, None] if s["gate"] == "token" else g


def _norm(s):
    dt = s["y"].dtype
    u = s["y"].float()
    if s["post"]:
        u = u * _rstd(u) * (s["offset"] + s["wq"].float())
    r = s["scale"] * s["x"].float() + _gate(s) * u
    h = (r * _rstd(r) * (s["offset"] + s["wp"].float())).to(dt) if s["pre"] else None
    return dict(stream=r.to(dt), normed=h)


def _norm_bwd(s):
    dt = s["y"].dtype
    y, x, g = s["y"].float(), s["x"].float(), _gate(s)
    u = y
    if s["post"]:
        ry = _rstd(y)
        yh = y * ry
        wq = s["offset"] + s["wq"].float()
        u = yh * wq
    d = s["dr"].float()
    out = {}
    if s["pre"]:
        r = s["scale"] * x + g * u
        rr = _rstd(r)
        rh = r * rr
        dh = s["dh"].float()
        dn = dh * (s["offset"] + s["wp"].float())
        out["d_pre_weight"] = (dh * rh).sum(dim=0).to(dt)
        d = d + rr * (dn - rh * (dn * rh).mean(dim=1, keepdim=True))
    out["d_residual"] = (s["scale"] * d).to(dt)
    if s["g"] is not None:
        dg = d * u
        if s["gate"] == "channel":
            dg = dg.sum(dim=0)
        elif s["gate"] == "token":
            dg = dg.sum(dim=1)
        out["d_gate"] = dg.to(dt)
    du = d * g
    if s["post"]:
        out["d_post_weight"] = (du * yh).sum(dim=0).to(dt)
        dn = du * wq
        du = ry * (dn - yh * (dn * yh).mean(dim=1, keepdim=True))
    out["d_branch"] = du.to(dt)
    return out


def _probs(logits, scoring):
    if scoring == "softmax":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    else:
        e = 1 / (1 + torch.exp(-logits))
    return e, e / e.sum(dim=1, keepdim=True)


def _balance(s):
    counts, tokens = _tables(s)
    coef = _coef(s)
    seq, live = _live(s)
    _, p = _probs(s["logits"], s["scoring"])
    member = (seq[None, :] == torch.arange(s["n_seq"], device="cuda")[:, None]) & live[None, :]
    sums = member.float() @ p
    return dict(loss=(coef.double() * sums).sum().float().view(1), counts=counts,
                live_tokens=tokens, prob_sum=sums, coef=coef)


def _router_bwd(s):
    x, k = s["logits"], s["k"]
    seq, live = _live(s)
    e, p = _probs(x, s["scoring"])
    c = s["coef"][seq] * s["d_loss"]
    d = p * (c - (c * p).sum(dim=1, keepdim=True))
    # the route weights: f times the selected scores, over their sum when renormalised
    on = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    dw = torch.where(on, s["dw"], torch.zeros_like(s["dw"])) * s["factor"]
    if s["renorm"]:
        w = torch.where(on, e.gather(1, ids), torch.zeros_like(dw))
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-30)
        q = w * (dw - (dw * w).sum(dim=1, keepdim=True))
        d = d.scatter_add(1, ids, q)
    elif s["scoring"] == "softmax":
        w = p.gather(1, ids)
        d = d.scatter_add(1, ids, w * dw) - p * (w * dw).sum(dim=1, keepdim=True)
    else:
        d = d.scatter_add(1, ids, e.gather(1, ids) * dw)
    if s["scoring"] == "sigmoid":
        d = d * (1 - e)
    return torch.where(live[:, None], d, torch.zeros_like(d))


_PLAIN = {"linear": _linear, "norm": _norm, "norm_bwd": _norm_bwd, "balance": _balance,
          "router_bwd": _router_bwd}


def _library(s):
    from mixture_experts_forward_moe_gb300 import binding as B

    op = s["op"]
    # a gate's length does not tell its kind in a batch of as many rows as channels
    kind = {}
    if op in ("norm", "norm_bwd") and s["g"] is not None and s["T"] == s["H"]:
        kind["gate_kind"] = s["gate"]
    if op == "linear":
        return B.moe_linear(s["x"], s["w"], bias=s["b"], activation=s["act"], residual=s["res"],
                            out_dtype=torch.float32 if s["out_f32"] else None)
    if op == "norm":
        stream, normed = B.moe_block_norm(
            s["y"], s["x"], gate=s["g"], post_weight=s["wq"], pre_weight=s["wp"],
            post_norm=s["post"], pre_norm=s["pre"], residual_scale=s["scale"],
            weight_offset=s["offset"], eps=_EPS, **kind)
        return dict(stream=stream, normed=normed)
    if op == "norm_bwd":
        return B.moe_block_norm_bwd(
            s["dr"], s["dh"], s["y"], s["x"], gate=s["g"], post_weight=s["wq"],
            pre_weight=s["wp"], post_norm=s["post"], pre_norm=s["pre"],
            residual_scale=s["scale"], weight_offset=s["offset"], eps=_EPS, **kind)
    if op == "balance":
        return B.moe_balance_loss(s["logits"], s["ids"], s["coeff"], scoring_func=s["scoring"],
                                  seq_offsets=s["offsets"])
    return B.moe_router_bwd(s["logits"], s["ids"], d_topk_weights=s["dw"], coef=s["coef"],
                            d_loss=s["d_loss"], seq_offsets=s["offsets"],
                            scoring_func=s["scoring"], renormalize=s["renorm"],
                            routed_scaling_factor=s["factor"])


def run(state):
    return _library(state) if own else _PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        o = 4 if case["out_f32"] else 2
        b = 2 * (T * K + N * K) + o * T * N
        b += (o * T * N if case["residual"] else 0) + (2 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * N * K}
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        gate = {"none": 0, "channel": H, "token": T, "element": T * H}[case["gate"]]
        weights = H * (case["post"] + case["pre"])
        if op == "norm":
            b = 2 * ((3 + case["pre"]) * T * H + gate + weights)
            return {"bytes": b, "flops": T * H * (4 + 3 * case["post"] + 4 * case["pre"])}
        # without a pre norm and a gate the residual is not needed: dx = a dr
        reads = 1 + case["pre"] + (case["post"] or case["pre"] or case["gate"] != "none")
        reads += case["pre"]
        b = 2 * ((reads + 2) * T * H + 2 * gate + 2 * weights)
        return {"bytes": b, "flops": T * H * (6 + 8 * case["post"] + 10 * case["pre"])}
    T, E, k, n = case["T"], case["E"], case["k"], case["n_seq"]
    offsets = 4 * (n + 1) if n > 1 else 0
    if op == "balance":
        return {"bytes": 4 * T * (E + k) + offsets + 4 * n * (3 * E + 1) + 4, "flops": 5 * T * E}
    return {"bytes": 4 * T * (2 * E + 2 * k) + offsets + 4 * n * E + 4, "flops": 9 * T * E}


# ------------------------------------------------------------------------- the 64-bit oracle
def _exact_linear(s):
    z = torch.nn.functional.linear(s["x"].double(), s["w"].double(),
                                   None if s["b"] is None else s["b"].double())
    if s["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif s["act"] == "gelu_tanh":
        z = torch.nn.functional.gelu(z, approximate="tanh")
    elif s["act"] == "relu2":
        z = torch.relu(z).square()
    return z if s["res"] is None else z + s["res"].double()


def _exact_norm(case, s, grads):
    """The forward in 64 bits, and its gradients by automatic differentiation."""
    names = ["y", "x", "g", "wq", "wp"]
    v = {n: None if s[n] is None else s[n].double().requires_grad_(grads) for n in names}

    def norm(t, w):
        return t / (t.square().sum(1, keepdim=True) / t.shape[1] + _EPS).sqrt() * (
            w + case["offset"])

    u = norm(v["y"], v["wq"]) if case["post"] else v["y"]
    if v["g"] is not None:
        u = torch.einsum("t,th->th", v["g"], u) if case["gate"] == "token" else u * v["g"]
    r = torch.add(u, v["x"], alpha=case["scale"])
    h = norm(r, v["wp"]) if case["pre"] else None
    if not grads:
        return dict(stream=r, normed=h)
    total = (r * s["dr"].double()).sum()
    if h is not None:
        total = total + (h * s["dh"].double()).sum()
    out = {"y": "d_branch", "x": "d_residual", "g": "d_gate", "wq": "d_post_weight",
           "wp": "d_pre_weight"}
    have = [n for n in names if v[n] is not None]
    return {out[n]: d for n, d in zip(have, torch.autograd.grad(total, [v[n] for n in have]))}


def _exact_loss(case, s, logits):
    """(loss, counts, live, probability sums, weights) from the definition, sequence by sequence."""
    E, k, n = case["E"], case["k"], case["n_seq"]
    off = [0, case["T"]] if s["offsets"] is None else s["offsets"].tolist()
    if case["scoring"] == "softmax":
        p = torch.softmax(logits, dim=1)
    else:
        sg = torch.sigmoid(logits)
        p = sg / sg.sum(1, keepdim=True)
    counts, live, sums, loads = [], [], [], []
    for a, b in zip(off, off[1:]):
        ids = s["ids"][a:b].long()
        keep = (ids >= 0).any(1)
        counts.append(torch.bincount(ids[ids >= 0], minlength=E))
        live.append(int(keep.sum()))
        sums.append((p[a:b] * keep[:, None]).sum(0))
        T_s = max(live[-1], 1)
        loads.append(counts[-1].double() * E / (k * T_s) / T_s)
    seqs = max(1, sum(t > 0 for t in live))
    coef = torch.stack(loads) * (s["coeff"] / seqs)
    sums = torch.stack(sums)
    assert len(live) == n
    return (coef * sums).sum(), torch.stack(counts), torch.tensor(live, device="cuda"), sums, coef


def _exact_router_bwd(case, s):
    x = s["logits"].double().requires_grad_(True)
    loss = _exact_loss(case, s, x)[0]
    ids = s["ids"].long()
    # padding tokens have no route weights; elsewhere every id is an expert
    keep = (ids >= 0).all(1)
    score = (torch.softmax if case["scoring"] == "softmax" else lambda t, _: torch.sigmoid(t))(x, 1)
    w = score[keep].gather(1, ids[keep])
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    loss = loss + (s["factor"] * w * s["dw"].double()[keep]).sum()
    return torch.autograd.grad(loss, x)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(s)
    if op in ("norm", "norm_bwd"):
        return _exact_norm(case, s, op == "norm_bwd")
    if op == "balance":
        loss, counts, live, sums, coef = _exact_loss(case, s, s["logits"].double())
        return dict(loss=loss.view(1), counts=counts.to(torch.int32),
                    live_tokens=live.to(torch.int32), prob_sum=sums, coef=coef)
    return _exact_router_bwd(case, s)
