"""What is measured of a differential decoder's operators.

Six calls of the framework: the difference of two attention softmax maps with a
learned weight per head (forward and backward), the norms after and before a
block fused with the block's gate and residual scale (forward and backward),
and the softmax cross entropy taken from the hidden states and the vocabulary
matrix without keeping the logits (forward and backward).  ``run`` computes
each in its plain form from elementary torch operations, or, where ``own`` is
true, calls the framework.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_INF = float("inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _diff(op, name, dtype, B, H, Tq, Tk, causal, scale, mask, shortest, pairs, shared):
    return {"op": op, "name": name, "dtype": dtype, "B": B, "H": H, "Tq": Tq, "Tk": Tk,
            "causal": causal, "scale": scale, "mask": mask, "shortest": shortest, "pairs": pairs,
            "shared": shared}


def _block(op, name, dtype, rows, hidden, kind, post, gate, sequence, residual_scale):
    return {"op": op, "name": name, "dtype": dtype, "rows": rows, "hidden": hidden, "kind": kind,
            "post": post, "gate": gate, "sequence": sequence, "residual_scale": residual_scale}


def _loss(op, name, dtype, rows, hidden, vocab, ignored):
    return {"op": op, "name": name, "dtype": dtype, "rows": rows, "hidden": hidden, "vocab": vocab,
            "ignored": ignored}


def listed():
    return [
        # one decoding step of a batch: a single query row per head over a cache of odd length
        _diff("diff_fw", "diff_fw step", "bf16", 16, 16, 1, 1001, True, 0.125, "inf", 0.3, False,
              False),
        # the Transformer-big layer's 16 maps as 8 differential heads, padded sentences
        _diff("diff_fw", "diff_fw encoder", "bf16", 32, 8, 512, 512, False, 0.125, "inf", 0.5,
              True, False),
        # its backward
        _diff("diff_bw", "diff_bw encoder", "bf16", 32, 8, 512, 512, False, 0.125, "inf", 0.5,
              True, False),
        # backward of a causal decoder on sentences of an odd length, one weight for all heads
        _diff("diff_bw", "diff_bw odd", "f16", 8, 6, 777, 777, True, 0.125, "none", 1.0, False,
              True),
        # one decoding step of 16 sequences: latency counts
        _block("block_fw", "block_fw step", "bf16", 16, 1024, "rms", True, "none", 1, 1.0),
        # the Transformer-big layer, LayerNorm after and before the block, a learned gate
        _block("block_fw", "block_fw train", "bf16", 16384, 1024, "layer", True, "one", 512, 1.0),
        # its backward
        _block("block_bw", "block_bw train", "bf16", 16384, 1024, "layer", True, "one", 512, 1.0),
        # a wide layer with a gate per sequence, odd row count, a scaled residual stream
        _block("block_bw", "block_bw wide", "f16", 4095, 4096, "rms", True, "sequence", 455, 1.5),
        # scoring a short continuation
        _loss("loss_fw", "loss_fw score", "f16", 33, 768, 32000, 0.0),
        # a training step's tokens on the GPT-2 vocabulary, a tenth of them padding
        _loss("loss_fw", "loss_fw train", "bf16", 8192, 1024, 50257, 0.1),
        # its backward
        _loss("loss_bw", "loss_bw train", "bf16", 8192, 1024, 50257, 0.1),
        # fp32 with odd sizes throughout, half of the tokens a prompt that does not count
        _loss("loss_bw", "loss_bw odd", "f32", 1001, 333, 10007, 0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["diff_fw", "diff_bw", "block_fw", "block_bw", "loss_fw", "loss_bw"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op.startswith("diff"):
        most = 1 << (25 if dtype != "f32" else 24)
        Tk = _log_int(rng, 2, 4000)
        Tk = Tk // 8 * 8 if rng.random() < 0.4 and Tk >= 8 else Tk
        Tq = rng.choice([1, Tk, Tk, _log_int(rng, 1, Tk)])
        H = rng.choice([1, 3, 4, 6, 8, 12, 16])
        B = _log_int(rng, 1, 64)
        while B * H * Tq * Tk > most and B > 1:
            B //= 2
        while B * H * Tq * Tk > most and H > 1:
            H //= 2
        return {"op": op, "dtype": dtype, "B": B, "H": H, "Tq": Tq, "Tk": Tk,
                "causal": rng.random() < 0.5,
                "scale": round(rng.choice([1.0, 0.125, rng.uniform(0.05, 1.5)]), 4),
                "mask": rng.choice(["none", "inf", "inf", "lowest"]),
                "shortest": rng.choice([0.0, 0.3, 0.6]), "pairs": rng.random() < 0.5,
                "shared": rng.random() < 0.3}
    if op.startswith("block"):
        hidden = rng.choice([256, 512, 768, 1024, 1024, 2048, 4096, 8192, _log_int(rng, 16, 9000)])
        rows = _log_int(rng, 1, 32768)
        sequence = _log_int(rng, 1, 1024)
        while rows * hidden * _BYTES[dtype] > 1 << 25:
            rows = rows // 2 + 1
        gate = rng.choice(["none", "one", "sequence", "token"])
        if gate == "sequence":  # whole sequences
            sequence = min(sequence, rows)
            rows = rows // sequence * sequence
        return {"op": op, "dtype": dtype, "rows": rows, "hidden": hidden,
                "kind": rng.choice(["rms", "layer"]), "post": rng.random() < 0.7, "gate": gate,
                "sequence": sequence,
                "residual_scale": round(rng.choice([1.0, 1.0, rng.uniform(0.5, 3.0)]), 3)}
    hidden = rng.choice([64, 256, 512, 768, 1024, 2048, _log_int(rng, 8, 2000)])
    vocab = rng.choice([65, 32000, 50257, 50304, _log_int(rng, 50, 60000)])
    rows = _log_int(rng, 1, 8192)
    while rows * hidden * vocab * (1 if dtype != "f32" else 8) > 8192 * 1024 * 50257:
        rows = rows // 2 + 1
    return {"op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "vocab": vocab,
            "ignored": rng.choice([0.0, 0.1, 0.5, 0.9])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _normal(shape, std, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _diff_state(case, seed):
    dt, gen = _DTYPES[case["dtype"]], _generator(seed, 1)
    B, H, Tq, Tk = case["B"], case["H"], case["Tq"], case["Tk"]
    state = dict(case)
    # both maps of a layer lie in one tensor of scores [B, 2H, Tq, Tk]: neighbouring heads are
    # a pair, or the first half of the heads is the first map of each
    s = _normal((B, 2 * H, Tq, Tk), 2.0 / case["scale"], dt, gen)
    state["s1"], state["s2"] = (s[:, 0::2], s[:, 1::2]) if case["pairs"] else (s[:, :H], s[:, H:])
    state["lam"] = torch.rand(1 if case["shared"] else H, generator=gen, device="cuda") * 0.6 + 0.2
    state["add"] = None
    if case["mask"] != "none":  # a valid length per batch entry; 0: nothing is left of its rows
        n = torch.rand(B, generator=gen, device="cuda") * (1 - case["shortest"]) + case["shortest"]
        n = (n * (Tk + 1)).floor().clamp(max=Tk)
        if case["mask"] == "lowest":
            n = n.clamp(min=1)
        fill = -_INF if case["mask"] == "inf" else torch.finfo(dt).min
        hidden = torch.arange(Tk, device="cuda")[None, :] >= n[:, None]
        state["add"] = torch.zeros(B, Tk, device="cuda").masked_fill_(hidden, fill).to(dt)
    if case["op"] == "diff_bw":  # the row statistics, as a training step has saved them
        stats = [t for s_ in (state["s1"], state["s2"]) for t in _plain_map(s_, state)[1:]]
        state["stats"] = torch.cat(stats, -1).contiguous()
        state["dout"] = _normal((B, H, Tq, Tk), 1.0, dt, gen)
    return state


def _block_state(case, seed):
    dt, gen = _DTYPES[case["dtype"]], _generator(seed, 2)
    rows, hidden = case["rows"], case["hidden"]
    layer = case["kind"] == "layer"
    state = dict(case)

    def parameters(name):
        state["g_" + name] = _normal((hidden,), 0.2, torch.float32, gen).add_(1.0).to(dt)
        state["b_" + name] = _normal((hidden,), 0.1, dt, gen) if layer else None

    parameters("pre")
    state["g_post"] = state["b_post"] = state["gate_by"] = None
    if case["post"]:
        parameters("post")
    groups = {"none": 0, "one": 1, "sequence": rows // max(case["sequence"], 1), "token": rows}
    if case["gate"] != "none":
        state["gate_by"] = _normal((groups[case["gate"]], hidden), 0.5, torch.float32,
                                   gen).add_(0.5).to(dt)
    state["x"] = _normal((rows, hidden), 1.5, torch.float32, gen).add_(0.3).to(dt)
    state["r"] = _normal((rows, hidden), 2.0, dt, gen)
    if case["op"] == "block_bw":
        out = _plain_block_fw(state)
        state["h"], state["stats"] = out["h"], out["stats"]
        state["dy"] = _normal((rows, hidden), 1.0, dt, gen)
        state["dh"] = _normal((rows, hidden), 1.0, dt, gen)
    return state


def _loss_state(case, seed):
    dt, gen = _DTYPES[case["dtype"]], _generator(seed, 3)
    rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
    state = dict(case)
    std = 2.5 / math.sqrt(hidden)  # logits of a standard deviation of about 2.5
    w = _normal((vocab, hidden), std, torch.float32, gen)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    # a model that has learned something: a token's own logit lies higher
    x = _normal((rows, hidden), 1.0, torch.float32, gen).add_(w[t], alpha=6.0 / (std * std * hidden))
    skip = torch.rand(rows, generator=gen, device="cuda") < case["ignored"]
    state["x"], state["w"] = x.to(dt), w.to(dt)
    state["t"] = t.masked_fill(skip, -1).to(torch.int32)
    if case["op"] == "loss_bw":
        state["lse"] = _plain_loss_fw(state)["lse"]
        count = (state["t"] >= 0).sum().clamp(min=1).float()
        state["dloss"] = (state["t"] >= 0).float() / count
    return state


def prepare(case, seed):
    if case["op"].startswith("diff"):
        return _diff_state(case, seed)
    if case["op"].startswith("block"):
        return _block_state(case, seed)
    return _loss_state(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_map(scores, s):
    """Weights of one map, with each row's largest z and the inverse of its sum."""
    z = scores.float() * s["scale"]
    if s["add"] is not None:
        z = z + s["add"].float()[:, None, None, :]
    if s["causal"]:
        i = torch.arange(s["Tq"], device="cuda")[:, None] + (s["Tk"] - s["Tq"])
        z = z.masked_fill(torch.arange(s["Tk"], device="cuda")[None, :] > i, -_INF)
    m = z.amax(-1, keepdim=True)
    m = m.masked_fill(m == -_INF, 0.0)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    inv = torch.where(total == 0, torch.zeros_like(total), 1.0 / total)
    return e * inv, m, inv


def _lam(s):
    return s["lam"].expand(s["H"])[None, :, None, None]


def _plain_diff_fw(s):
    p1, m1, i1 = _plain_map(s["s1"], s)
    p2, m2, i2 = _plain_map(s["s2"], s)
    return {"y": (p1 - _lam(s) * p2).to(s["s1"].dtype), "stats": torch.cat((m1, i1, m2, i2), -1)}


def _plain_diff_bw(s):
    g = s["dout"].float()
    p1, p2 = _plain_map(s["s1"], s)[0], _plain_map(s["s2"], s)[0]
    d1 = (p1 * g).sum(-1, keepdim=True)
    d2 = (p2 * g).sum(-1, keepdim=True)
    dlam = -d2.double().sum((0, 2, 3))
    if s["shared"]:
        dlam = dlam.sum(0, keepdim=True)
    dt = s["s1"].dtype
    return {"ds1": (s["scale"] * p1 * (g - d1)).to(dt),
            "ds2": (-s["scale"] * _lam(s) * p2 * (g - d2)).to(dt), "dlam": dlam.float()}


def _plain_stats(v, s):
    mean = v.mean(-1) if s["kind"] == "layer" else torch.zeros_like(v[:, 0])
    return mean, ((v - mean[:, None]).square().mean(-1) + 1e-6).rsqrt()


def _gate_rows(s):
    """The gate of every row, or 1."""
    if s["gate_by"] is None:
        return 1.0
    g = s["gate_by"].float()
    return g.repeat_interleave(s["rows"] // g.shape[0], 0)


def _plain_block_fw(s):
    n = s["x"].float()
    mean1, rstd1 = torch.zeros_like(n[:, 0]), torch.ones_like(n[:, 0])
    if s["g_post"] is not None:
        mean1, rstd1 = _plain_stats(n, s)
        n = (n - mean1[:, None]) * rstd1[:, None] * s["g_post"].float()
        if s["b_post"] is not None:
            n = n + s["b_post"].float()
    h = s["residual_scale"] * s["r"].float() + _gate_rows(s) * n
    mean2, rstd2 = _plain_stats(h, s)
    y = (h - mean2[:, None]) * rstd2[:, None] * s["g_pre"].float()
    if s["b_pre"] is not None:
        y = y + s["b_pre"].float()
    dt = s["x"].dtype
    return {"h": h.to(dt), "y": y.to(dt), "stats": torch.stack((mean1, rstd1, mean2, rstd2))}


def _plain_norm_bw(dy, v, mean, rstd, gamma, s):
    """(dv, dgamma, dbeta) of one norm"""
    vhat = (v - mean[:, None]) * rstd[:, None]
    g = dy * gamma.float()
    back = g - vhat * (g * vhat).mean(-1, keepdim=True)
    if s["kind"] == "layer":
        back = back - g.mean(-1, keepdim=True)
    return rstd[:, None] * back, _column_sum(dy * vhat), _column_sum(dy)


def _column_sum(v):
    return v.sum(0, dtype=torch.float64).float()


def _plain_block_bw(s):
    mean1, rstd1, mean2, rstd2 = s["stats"]
    layer = s["kind"] == "layer"
    out = {}
    dh, out["dg_pre"], db = _plain_norm_bw(s["dy"].float(), s["h"].float(), mean2, rstd2,
                                           s["g_pre"], s)
    if layer:
        out["db_pre"] = db
    dh = dh + s["dh"].float()
    x = s["x"].float()
    dn = dh * _gate_rows(s)
    dx, n = dn, x
    if s["g_post"] is not None:
        dx, out["dg_post"], db = _plain_norm_bw(dn, x, mean1, rstd1, s["g_post"], s)
        n = (x - mean1[:, None]) * rstd1[:, None] * s["g_post"].float()
        if layer:
            out["db_post"] = db
            n = n + s["b_post"].float()
    if s["gate_by"] is not None:
        groups = s["gate_by"].shape[0]
        out["dgate"] = (dh * n).view(groups, -1, s["hidden"]).sum(1, dtype=torch.float64).float()
    out["dx"] = dx.to(s["x"].dtype)
    out["dr"] = (s["residual_scale"] * dh).to(s["x"].dtype)
    return out


def _plain_loss_fw(s):
    t = s["t"].long()
    skip = t < 0
    z = s["x"].float() @ s["w"].float().T
    m = z.amax(-1)
    lse = m + torch.exp(z - m[:, None]).sum(-1).log()
    loss = lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return {"loss": loss.masked_fill(skip, 0.0), "lse": lse.masked_fill(skip, 0.0)}


def _plain_loss_bw(s):
    t = s["t"].long()
    skip = (t < 0)[:, None]
    x, w = s["x"].float().masked_fill(skip, 0.0), s["w"].float()
    p = torch.exp(x @ w.T - s["lse"][:, None])
    p[torch.arange(s["rows"], device="cuda"), t.clamp(min=0)] -= 1.0
    p = (p * s["dloss"][:, None]).masked_fill_(skip, 0.0)
    return {"dx": (p @ w).to(s["x"].dtype), "dw": (p.T @ x).to(s["w"].dtype)}


_PLAIN = {"diff_fw": _plain_diff_fw, "diff_bw": _plain_diff_bw, "block_fw": _plain_block_fw,
          "block_bw": _plain_block_bw, "loss_fw": _plain_loss_fw, "loss_bw": _plain_loss_bw}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import transformer_reduce_gb300 as L
    if s["op"] == "diff_fw":
        y, stats = L.softmax_fw_diff(s["s1"], s["s2"], s["lam"], s["add"], causal=s["causal"],
                                     scale=s["scale"])
        return {"y": y, "stats": stats}
    if s["op"] == "diff_bw":
        ds1, ds2, dlam = L.softmax_bw_diff(s["dout"], s["s1"], s["s2"], s["lam"], s["stats"],
                                           s["add"], causal=s["causal"], scale=s["scale"])
        return {"ds1": ds1, "ds2": ds2, "dlam": dlam}
    if s["op"] == "block_fw":
        h, y, stats = L.block_norm_fw(s["x"], s["r"], gamma_pre=s["g_pre"], beta_pre=s["b_pre"],
                                      gamma_post=s["g_post"], beta_post=s["b_post"],
                                      gate=s["gate_by"], residual_scale=s["residual_scale"],
                                      kind=s["kind"], eps=1e-6)
        return {"h": h, "y": y, "stats": stats}
    if s["op"] == "block_bw":
        grads = L.block_norm_bw(s["dy"], s["dh"], s["x"], s["h"], s["stats"],
                                gamma_pre=s["g_pre"], gamma_post=s["g_post"],
                                beta_post=s["b_post"], gate=s["gate_by"],
                                residual_scale=s["residual_scale"], kind=s["kind"])
        names = ("dx", "dr", "dg_pre", "db_pre", "dg_post", "db_post", "dgate")
        return {k: v for k, v in zip(names, grads) if v is not None}
    if s["op"] == "loss_fw":
        loss, lse = L.linear_cross_entropy_fw(s["x"], s["w"], s["t"])
        return {"loss": loss, "lse": lse}
    dx, dw = L.linear_cross_entropy_bw(s["x"], s["w"], s["t"], s["lse"], s["dloss"])
    return {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = _BYTES[case["dtype"]]
    if case["op"].startswith("diff"):
        B, H, Tq, Tk = case["B"], case["H"], case["Tq"], case["Tk"]
        pairs = float(B * H * Tq * Tk)
        seen = (Tk - (Tq - 1) / 2) / Tk if case["causal"] and Tq <= Tk else 1.0
        if case["mask"] == "inf":  # -inf keys need not be read
            seen *= (1 + case["shortest"]) / 2
        small = 16.0 * B * H * Tq + 4 * H + (0 if case["mask"] == "none" else B * Tk * es)
        if case["op"] == "diff_fw":
            return {"bytes": pairs * es * (2 * seen + 1) + small, "flops": 14 * pairs * seen}
        return {"bytes": pairs * es * (3 * seen + 2) + small, "flops": 20 * pairs * seen}
    if case["op"].startswith("block"):
        n = float(case["rows"] * case["hidden"])
        groups = {"none": 0, "one": 1, "sequence": case["rows"] // max(case["sequence"], 1),
                  "token": case["rows"]}[case["gate"]]
        sides = 1 + case["post"]
        small = 4.0 * case["rows"] * sides * (2 if case["kind"] == "layer" else 1)
        vectors = sides * (2 if case["kind"] == "layer" else 1) + groups
        if case["op"] == "block_fw":
            return {"bytes": 4 * n * es + small + vectors * case["hidden"] * es,
                    "flops": n * (14 if case["post"] else 8)}
        reads = 4 if case["post"] or groups else 3
        return {"bytes": (reads + 2) * n * es + small + vectors * case["hidden"] * (es + 4),
                "flops": n * (26 if case["post"] else 14)}
    n, D, V = float(case["rows"]) * (1 - case["ignored"]), case["hidden"], case["vocab"]
    if case["op"] == "loss_fw":
        return {"bytes": (n + V) * D * es + 12.0 * case["rows"], "flops": 2 * n * D * V}
    return {"bytes": 2 * (n + V) * D * es + (case["rows"] - n) * D * es + 12.0 * case["rows"],
            "flops": 6 * n * D * V}


# ---------------------------------------------------------------------------
# 64-bit answers
# ---------------------------------------------------------------------------
def _exact_weights(scores, s, b):
    """(p, largest z, 1 / sum) of batch entry b in 64 bits"""
    Tq, Tk = s["Tq"], s["Tk"]
    see = torch.ones(1, Tq, Tk, dtype=torch.bool, device="cuda")
    if s["causal"]:
        see = see.tril(Tk - Tq)
    z = scores[b].double() * s["scale"]
    if s["add"] is not None:
        extra = s["add"][b].double()
        see = see & ~torch.isneginf(extra)
        z = z + extra.clamp(min=-1e300)
    see = see.expand_as(z)
    z = torch.where(see, z, torch.full_like(z, -_INF))
    top = z.max(-1, keepdim=True).values
    top = torch.where(see.any(-1, keepdim=True), top, torch.zeros_like(top))
    w = torch.where(see, (z - top).exp(), torch.zeros_like(z))
    total = w.sum(-1, keepdim=True)
    inv = torch.where(total > 0, total.clamp(min=1e-300).reciprocal(), torch.zeros_like(total))
    return w * inv, top, inv


def _exact_diff(case, s):
    weight = s["lam"].double().repeat(s["H"] // s["lam"].numel()).view(-1, 1, 1)
    parts, stats, slopes = [], [], []
    for b in range(s["B"]):
        p1, m1, i1 = _exact_weights(s["s1"], s, b)
        p2, m2, i2 = _exact_weights(s["s2"], s, b)
        if case["op"] == "diff_fw":
            parts.append(p1 - weight * p2)
            stats.append(torch.cat((m1, i1, m2, i2), -1))
            continue
        g = s["dout"][b].double()
        a1, a2 = torch.einsum("hij,hij->hi", p1, g), torch.einsum("hij,hij->hi", p2, g)
        parts.append(torch.stack((p1 * g - p1 * a1[..., None],
                                  weight * p2 * a2[..., None] - weight * p2 * g)) * s["scale"])
        slopes.append(-a2.sum(-1))
    if case["op"] == "diff_fw":
        return {"y": torch.stack(parts), "stats": torch.stack(stats)}
    both, dlam = torch.stack(parts, 1), torch.stack(slopes).sum(0)
    return {"ds1": both[0], "ds2": both[1],
            "dlam": dlam.sum().reshape(1) if case["shared"] else dlam}


def _exact_hat(v, s, column):
    """Centred and scaled rows by the saved statistics ``column`` and the next."""
    return (v - s["stats"][column].double().unsqueeze(1)) * s["stats"][column + 1].double().unsqueeze(1)


def _exact_block(case, s):
    x = s["x"].double()
    rows, hidden = x.shape
    gate = torch.ones(1, hidden, dtype=torch.float64, device="cuda")
    if s["gate_by"] is not None:
        gate = s["gate_by"].double()
    which = torch.arange(rows, device="cuda") // (rows // gate.shape[0])
    zero = torch.zeros(hidden, dtype=torch.float64, device="cuda")
    wide = {k: zero if s[k] is None else s[k].double() for k in ("g_pre", "b_pre", "g_post",
                                                                 "b_post")}
    centred = 1.0 if case["kind"] == "layer" else 0.0
    if case["op"] == "block_fw":
        def normed(v):
            mean = v.sum(-1, keepdim=True) / hidden * centred
            rstd = 1.0 / torch.sqrt(((v - mean) ** 2).sum(-1, keepdim=True) / hidden + 1e-6)
            return (v - mean) * rstd, mean.squeeze(-1), rstd.squeeze(-1)

        first = (torch.zeros(rows, dtype=torch.float64, device="cuda"),
                 torch.ones(rows, dtype=torch.float64, device="cuda"))
        n = x
        if s["g_post"] is not None:
            n, *first = normed(x)
            n = n * wide["g_post"] + wide["b_post"]
        h = s["r"].double() * s["residual_scale"] + n * gate[which]
        hhat, *second = normed(h)
        return {"h": h, "y": hhat * wide["g_pre"] + wide["b_pre"],
                "stats": torch.stack((*first, *second))}

    def back(up, hat, gamma, rstd):
        g = up * gamma
        inner = (g * hat).sum(-1, keepdim=True) / hidden
        shift = g.sum(-1, keepdim=True) / hidden * centred
        return (g - shift - hat * inner) * rstd.double().unsqueeze(1)

    dy, hhat = s["dy"].double(), _exact_hat(s["h"].double(), s, 2)
    dh = s["dh"].double() + back(dy, hhat, wide["g_pre"], s["stats"][3])
    out = {"dg_pre": torch.einsum("rc,rc->c", dy, hhat), "dr": dh * s["residual_scale"]}
    if centred:
        out["db_pre"] = dy.sum(0)
    dn, n = dh * gate[which], x
    out["dx"] = dn
    if s["g_post"] is not None:
        xhat = _exact_hat(x, s, 0)
        n = xhat * wide["g_post"] + wide["b_post"]
        out["dx"] = back(dn, xhat, wide["g_post"], s["stats"][1])
        out["dg_post"] = torch.einsum("rc,rc->c", dn, xhat)
        if centred:
            out["db_post"] = dn.sum(0)
    if s["gate_by"] is not None:
        out["dgate"] = torch.zeros_like(gate).index_add_(0, which, dh * n)
    return out


def _exact_loss(case, s):
    live = (s["t"] >= 0).nonzero().squeeze(1)
    x, w, t = s["x"].double()[live], s["w"].double(), s["t"][live].long()
    if case["op"] == "loss_fw":
        z = torch.einsum("nd,vd->nv", x, w)
        lse = torch.logsumexp(z, -1)
        wide = torch.zeros(2, s["rows"], dtype=torch.float64, device="cuda")
        wide[0, live], wide[1, live] = lse - (x * w[t]).sum(-1), lse
        return {"loss": wide[0], "lse": wide[1]}
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for part in torch.arange(len(live), device="cuda").split(2048):
        z = torch.einsum("nd,vd->nv", x[part], w)
        up = s["dloss"].double()[live[part]].unsqueeze(1)
        p = z.sub_(s["lse"].double()[live[part]].unsqueeze(1)).exp_().mul_(up)
        p.scatter_add_(1, t[part].unsqueeze(1), -up)
        dx[live[part]] = torch.einsum("nv,vd->nd", p, w)
        dw += torch.einsum("nv,nd->vd", p, x[part])
    return {"dx": dx, "dw": dw}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("diff"):
        return _exact_diff(case, s)
    if case["op"].startswith("block"):
        return _exact_block(case, s)
    return _exact_loss(case, s)
