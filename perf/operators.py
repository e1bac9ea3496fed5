"""The training-side operators around the mixture-of-experts layer, as measured cases.

Three operators, in each direction that they have:

* the gated feed-forward block (``ffn_forward``, ``ffn_backward``): the dense expert that runs
  beside the routed ones, ``Y = (silu(X Wg^T) * (X Wu^T)) Wd^T (+ residual)``;
* softmax cross entropy over a vocabulary straight from the hidden rows (``ce_forward``,
  ``ce_backward``): ``loss = logsumexp(X W^T) - (X W^T)[target]``;
* the global gradient norm over many tensors and clipping by it (``clip``).

Each has a plain form in elementary torch operations (32 bits inside, rounded once), the call a
user makes of the library (``own``), and its definition in 64 bits (``exact``).
"""

import math
import random

import torch

own = False

IGNORE = -100
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# The largest listed work of each operator; a drawn case stays at or below it.
_FFN_MOST = 4096 * 2048 * 8192
_CE_MOST = 4096 * 2048 * 151936
_CLIP_MOST = 1_200_000_000


def listed():
    return [
        # one token of a served model through a dense expert of OLMoE's expert size: latency counts
        {"name": "ffn token", "op": "ffn_forward", "T": 1, "H": 2048, "I": 1024, "dtype": "bf16",
         "residual": False, "save": False},
        # a decode batch; the routed experts' fp32 output is added in the same pass
        {"name": "ffn decode batch", "op": "ffn_forward", "T": 32, "H": 4096, "I": 8192,
         "dtype": "bf16", "residual": True, "save": False},
        # a ragged fp16 batch whose sizes fill no tile, keeping what the backward pass needs
        {"name": "ffn ragged", "op": "ffn_forward", "T": 517, "H": 1000, "I": 2744,
         "dtype": "fp16", "residual": True, "save": True},
        # a training batch, forward
        {"name": "ffn train", "op": "ffn_forward", "T": 4096, "H": 2048, "I": 8192,
         "dtype": "bf16", "residual": False, "save": True},
        # the backward pass of a ragged fp16 batch
        {"name": "ffn backward ragged", "op": "ffn_backward", "T": 333, "H": 1024, "I": 2816,
         "dtype": "fp16", "weights": True},
        # the training batch, backward
        {"name": "ffn backward train", "op": "ffn_backward", "T": 4096, "H": 2048, "I": 8192,
         "dtype": "bf16", "weights": True},
        # scoring a short continuation
        {"name": "ce short", "op": "ce_forward", "T": 40, "H": 2048, "V": 50304, "dtype": "bf16",
         "ignored": 0.0},
        # a training batch over a large vocabulary
        {"name": "ce train", "op": "ce_forward", "T": 4096, "H": 2048, "V": 151936,
         "dtype": "bf16", "ignored": 0.0},
        # backward of a ragged fp16 batch with an odd vocabulary; half of the rows are prompt
        {"name": "ce backward ragged", "op": "ce_backward", "T": 1000, "H": 1024, "V": 32003,
         "dtype": "fp16", "ignored": 0.5, "head": True},
        # backward of the training batch, some rows padding, the head trained too
        {"name": "ce backward train", "op": "ce_backward", "T": 4096, "H": 2048, "V": 151936,
         "dtype": "bf16", "ignored": 0.25, "head": True},
        # the gradients of low-rank adapters: many small fp32 tensors
        {"name": "clip adapters", "op": "clip", "tensors": 224, "mean": 24576, "ragged": False,
         "dtype": "fp32", "packed": False, "clipped": True, "layout": 1},
        # the gradients of a whole 16-bit model: a few hundred large ragged tensors
        {"name": "clip model", "op": "clip", "tensors": 290, "mean": 4_000_000, "ragged": True,
         "dtype": "bf16", "packed": True, "clipped": True, "layout": 2},
    ]


def _spread(rng, lo, hi, step=1):
    """An integer between ``lo`` and ``hi``, spread over its logarithm, a multiple of ``step``."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_backward", "ce_forward", "ce_backward", "clip"])
    if op == "clip":
        n = _spread(rng, 1, 900)
        return {"op": op, "tensors": n,
                "mean": _spread(rng, 16, min(40_000_000, _CLIP_MOST // (2 * n))),
                "ragged": rng.random() < 0.7, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "packed": rng.random() < 0.5, "clipped": rng.random() < 0.7,
                "layout": rng.randrange(1 << 20)}
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    T = _spread(rng, 1, 4096)
    H = _spread(rng, 256, 4096, 8)
    if op.startswith("ffn"):
        I = _spread(rng, 256, min(8192, max(256, _FFN_MOST // (T * H))), 8)
        if op == "ffn_forward":
            return {"op": op, "T": T, "H": H, "I": I, "dtype": dtype,
                    "residual": rng.random() < 0.5, "save": rng.random() < 0.5}
        return {"op": op, "T": T, "H": H, "I": I, "dtype": dtype, "weights": rng.random() < 0.8}
    V = _spread(rng, 1000, min(151936, max(1000, _CE_MOST // (T * H))))
    c = {"op": op, "T": T, "H": H, "V": V, "dtype": dtype,
         "ignored": rng.choice([0.0, 0.0, 0.25, 0.5, 0.9])}
    if op == "ce_backward":
        c["head"] = rng.random() < 0.7
    return c


# ------------------------------------------------------------------ inputs


def _clip_sizes(case):
    """The element counts of the tensors, from the case alone."""
    rng, mean = random.Random(case["layout"]), case["mean"]
    if not case["ragged"]:
        return [mean] * case["tensors"]
    return [max(1, int(mean * rng.choice([0.01, 0.3, 1.0, 1.0, 2.0]) * rng.uniform(0.5, 1.5)))
            for _ in range(case["tensors"])]


def _clip_views(case, flat):
    """Each tensor's part of the flat gradient buffer; aligned to 16 bytes unless packed."""
    step = 1 if case["packed"] else 16 // flat.element_size()
    views, at = [], 0
    for n in _clip_sizes(case):
        views.append(flat[at:at + n])
        at += (n + step - 1) // step * step
    return views


def _clip_numel(case):
    step = 1 if case["packed"] else 16 // TYPES[case["dtype"]].itemsize
    return sum((n + step - 1) // step * step for n in _clip_sizes(case))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=g)

    s = {"case": case}
    if case["op"] == "clip":
        # zeros between the tensors, where the flat buffer aligns them
        flat = torch.zeros(_clip_numel(case), dtype=dt, device="cuda")
        sigma = 1e-2 if dt == torch.float16 else 1e-3
        for v in _clip_views(case, flat):
            v.normal_(0.0, sigma, generator=g)
        out = torch.zeros_like(flat)
        limit = sigma * math.sqrt(sum(_clip_sizes(case))) * (0.3 if case["clipped"] else 4.0)
        s.update(flat=flat, out=out, max_norm=limit)
        if own:
            import bit_mixture_experts_route_b200 as moe
            s["grads"] = moe.grad_list(_clip_views(case, flat), _clip_views(case, out))
        return s
    T, H = case["T"], case["H"]
    if case["op"].startswith("ffn"):
        I = case["I"]
        s["X"] = normal(T, H)
        s["W_gu"] = normal(2 * I, H, sigma=1.0 / math.sqrt(H))
        s["W_d"] = normal(H, I, sigma=1.0 / math.sqrt(I))
        if case["op"] == "ffn_forward":
            s["residual"] = normal(T, H, dtype=torch.float32) if case["residual"] else None
        else:
            s["dY"] = normal(T, H, sigma=0.05)
            s["gu"] = (s["X"].float() @ s["W_gu"].float().t()).to(dt)  # kept by the forward pass
        return s
    V = case["V"]
    s["W"] = normal(V, H, sigma=1.0 / math.sqrt(H))
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    # rows of a model that has learned something: the target's logit is raised by 0 to 12
    lift = torch.rand((T, 1), device="cuda", generator=g) * 12.0
    s["X"] = (normal(T, H, dtype=torch.float32) + lift * s["W"][y].float()).to(dt)
    gone = torch.rand((T,), device="cuda", generator=g) < case["ignored"]
    s["targets"] = torch.where(gone, torch.full_like(y, IGNORE), y).int()
    if case["op"] == "ce_backward":
        keep = ~gone
        # the mean over the rows that count, with the loss scale of an fp16 run
        scale = 1024.0 if dt == torch.float16 else 1.0
        s["dloss"] = keep.float() * (scale / keep.sum().clamp(min=1).float())
        l = s["X"].float() @ s["W"].float().t()
        s["lse"] = torch.where(keep, torch.logsumexp(l.double(), 1), 0.0).float()
        del l
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    dt = TYPES[c["dtype"]]
    if c["op"] == "clip":
        flat = state["flat"]
        norm = flat.float().square().sum(dtype=torch.float64).sqrt()
        coef = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
        state["out"].copy_(flat.float() * coef.float())
        return {"norm": norm.float().reshape(1), "grads": state["out"]}
    if c["op"] == "ffn_forward":
        gu = state["X"].float() @ state["W_gu"].float().t()
        g, u = gu[:, :c["I"]], gu[:, c["I"]:]
        y = (g / (1.0 + torch.exp(-g)) * u) @ state["W_d"].float().t()
        if state["residual"] is not None:
            y = y + state["residual"]
        return {"Y": y.to(dt), "gu": gu.to(dt)} if c["save"] else {"Y": y.to(dt)}
    if c["op"] == "ffn_backward":
        g, u = state["gu"][:, :c["I"]].float(), state["gu"][:, c["I"]:].float()
        dy = state["dY"].float()
        s = 1.0 / (1.0 + torch.exp(-g))
        dh = dy @ state["W_d"].float()
        dgu = torch.cat([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], 1)
        r = {"dX": (dgu @ state["W_gu"].float()).to(dt)}
        if c["weights"]:
            r["dW_gu"] = (dgu.t() @ state["X"].float()).to(dt)
            r["dW_d"] = (dy.t() @ (g * s * u)).to(dt)
        return r
    y = state["targets"].long()
    keep = y != IGNORE
    rows, at = torch.arange(c["T"], device=y.device), torch.where(keep, y, 0)
    l = state["X"].float() @ state["W"].float().t()
    if c["op"] == "ce_forward":
        m = l.amax(1)
        lse = m + torch.log(torch.exp(l - m[:, None]).sum(1))
        return {"loss": torch.where(keep, lse - l[rows, at], 0.0),
                "lse": torch.where(keep, lse, 0.0)}
    p = torch.exp(l - state["lse"][:, None])
    p[rows, at] -= 1.0
    dl = torch.where(keep[:, None], p * state["dloss"][:, None], 0.0)
    r = {"dX": (dl @ state["W"].float()).to(dt)}
    if c["head"]:
        r["dW"] = (dl.t() @ state["X"].float()).to(dt)
    return r


def _run_own(c, s):
    import bit_mixture_experts_route_b200 as moe
    if c["op"] == "clip":
        return {"norm": moe.grad_norm_clip(s["grads"], s["max_norm"]), "grads": s["out"]}
    if c["op"] == "ffn_forward":
        r = moe.gated_ffn_forward(s["X"], s["W_gu"], s["W_d"], residual=s["residual"],
                                  save_gu=c["save"])
        return {"Y": r[0], "gu": r[1]} if c["save"] else {"Y": r}
    if c["op"] == "ffn_backward":
        dx, dwgu, dwd = moe.gated_ffn_backward(s["dY"], s["X"], s["gu"], s["W_gu"], s["W_d"],
                                               need_dw=c["weights"])
        return {"dX": dx, "dW_gu": dwgu, "dW_d": dwd} if c["weights"] else {"dX": dx}
    if c["op"] == "ce_forward":
        loss, lse = moe.linear_ce_forward(s["X"], s["W"], s["targets"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    dx, dw = moe.linear_ce_backward(s["dloss"], s["X"], s["W"], s["targets"], s["lse"],
                                    ignore_index=IGNORE, need_dw=c["head"])
    return {"dX": dx, "dW": dw} if c["head"] else {"dX": dx}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = TYPES[case["dtype"]].itemsize
    if case["op"] == "clip":
        n = sum(_clip_sizes(case))
        return {"bytes": 2 * n * b, "flops": 3 * n}  # read once, written once
    T, H = case["T"], case["H"]
    if case["op"].startswith("ffn"):
        I = case["I"]
        if case["op"] == "ffn_forward":
            n = 2 * T * H * b + 3 * H * I * b
            n += 4 * T * H if case["residual"] else 0
            n += 2 * T * I * b if case["save"] else 0
            return {"bytes": n, "flops": 6 * T * H * I}
        n = 2 * T * H * b + 2 * T * I * b + 3 * H * I * b
        if not case["weights"]:
            return {"bytes": n, "flops": 6 * T * H * I}
        return {"bytes": n + T * H * b + 3 * H * I * b, "flops": 12 * T * H * I}
    V, rows = case["V"], T * (1.0 - case["ignored"])  # ignored rows need no logits
    if case["op"] == "ce_forward":
        return {"bytes": rows * H * b + V * H * b + 12 * T, "flops": 2 * rows * H * V}
    n = rows * H * b + T * H * b + V * H * b + 12 * T
    if not case["head"]:
        return {"bytes": n, "flops": 4 * rows * H * V}
    return {"bytes": n + V * H * b, "flops": 6 * rows * H * V}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g)
        f = s["max_norm"] / (norm.item() + 1e-6)
        return {"norm": norm.reshape(1), "grads": g.mul_(f) if f < 1.0 else g}
    X = s["X"].double()
    if case["op"] == "ffn_forward":
        gate, up = (torch.einsum("th,ih->ti", X, w.double()) for w in s["W_gu"].chunk(2))
        Y = torch.einsum("ti,hi->th", gate.mul(torch.sigmoid(gate)).mul(up), s["W_d"].double())
        if s["residual"] is not None:
            Y += s["residual"].double()
        return {"Y": Y, "gu": torch.cat([gate, up], 1)} if case["save"] else {"Y": Y}
    if case["op"] == "ffn_backward":
        gate, up = (v.double() for v in s["gu"].chunk(2, dim=1))
        dY, sig = s["dY"].double(), torch.sigmoid(gate)
        dh = torch.einsum("th,hi->ti", dY, s["W_d"].double())
        d_gate = dh * up * (sig + gate * sig * torch.sigmoid(-gate))
        d_up = dh * gate * sig
        wg, wu = (w.double() for w in s["W_gu"].chunk(2))
        r = {"dX": torch.einsum("ti,ih->th", d_gate, wg) + torch.einsum("ti,ih->th", d_up, wu)}
        if case["weights"]:
            r["dW_gu"] = torch.cat([torch.einsum("ti,th->ih", d, X) for d in (d_gate, d_up)])
            r["dW_d"] = torch.einsum("th,ti->hi", dY, gate * sig * up)
        return r
    y = s["targets"].long()
    keep = (y != IGNORE).double()
    onehot_at = y.clamp(min=0)[:, None]
    W = s["W"].double()
    logits = torch.einsum("th,vh->tv", X, W)
    if case["op"] == "ce_forward":
        logp = torch.log_softmax(logits, 1)
        return {"loss": -logp.gather(1, onehot_at)[:, 0] * keep,
                "lse": torch.logsumexp(logits, 1) * keep}
    d = logits.sub_(s["lse"].double()[:, None]).exp_()
    d.scatter_add_(1, onehot_at, torch.full_like(onehot_at, -1, dtype=torch.float64))
    d *= (keep * s["dloss"].double())[:, None]
    r = {"dX": torch.einsum("tv,vh->th", d, W)}
    if case["head"]:
        r["dW"] = torch.einsum("tv,th->vh", d, X)
    return r
