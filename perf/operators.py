"""What is measured of the attention layer's position operators and of gradient clipping.

Five calls of the framework: the attention softmax with a learned relative
position bias by buckets (forward and backward), the per-head norm of queries
and keys with the position rotation (forward and backward), and the global
gradient norm with clipping.  ``run`` computes each in its plain form from
elementary torch operations, or, where ``own`` is true, calls the framework.
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
def _softmax(op, name, dtype, B, H, Tq, Tk, buckets, distance, causal, scale, mask, shortest):
    return {"op": op, "name": name, "dtype": dtype, "B": B, "H": H, "Tq": Tq, "Tk": Tk,
            "buckets": buckets, "distance": distance, "causal": causal, "scale": scale,
            "mask": mask, "shortest": shortest}


def _qk(op, name, dtype, tokens, Hq, Hk, D, rot, interleaved, packed, sequence):
    return {"op": op, "name": name, "dtype": dtype, "tokens": tokens, "Hq": Hq, "Hk": Hk, "D": D,
            "rot": rot, "interleaved": interleaved, "packed": packed, "sequence": sequence}


def _clip(name, kind, layers, hidden, count, largest, dtype, clipped):
    return {"op": "clip", "name": name, "kind": kind, "layers": layers, "hidden": hidden,
            "count": count, "largest": largest, "dtype": dtype, "clipped": clipped}


def listed():
    return [
        # one decoding step of a batch: a single query row per head over a cache of odd length
        _softmax("softmax_fw", "softmax_fw step", "bf16", 16, 16, 1, 1001, 32, 128, True, 1.0,
                 "inf", 0.3),
        # the Transformer-big encoder layer with padded sentences
        _softmax("softmax_fw", "softmax_fw encoder", "bf16", 32, 16, 512, 512, 32, 128, False, 1.0,
                 "inf", 0.5),
        # the last queries of a long context in fp32, padding marked by the type's lowest value
        _softmax("softmax_fw", "softmax_fw ragged", "f32", 4, 8, 333, 777, 20, 50, True, 0.125,
                 "lowest", 0.2),
        # backward of the encoder layer
        _softmax("softmax_bw", "softmax_bw encoder", "bf16", 32, 16, 512, 512, 32, 128, False, 1.0,
                 "inf", 0.5),
        # backward of a causal decoder on sentences of an odd length, no padding
        _softmax("softmax_bw", "softmax_bw odd", "f16", 8, 12, 777, 777, 32, 128, True, 0.125,
                 "none", 1.0),
        # one decoding step with shared key heads
        _qk("qk_fw", "qk_fw step", "bf16", 16, 32, 8, 128, 128, False, True, 1),
        # a training step of the Transformer-big layer (16 heads of 64), packed projections
        _qk("qk_fw", "qk_fw train", "bf16", 16384, 16, 16, 64, 64, False, True, 512),
        # its backward
        _qk("qk_bw", "qk_bw train", "bf16", 16384, 16, 16, 64, 64, False, True, 512),
        # shared key heads, a rotation of half the head in neighbouring pairs, odd token count
        _qk("qk_bw", "qk_bw shared", "f16", 5003, 24, 6, 128, 64, True, False, 1000),
        # the gradients of one small decoder layer: latency counts
        _clip("clip small", "layers", 1, 256, 0, 0, "f16", True),
        # the gradients of twelve Transformer-big layers: 16-bit matrices, fp32 norm parameters
        _clip("clip model", "layers", 12, 1024, 0, 0, "bf16", True),
        # many tensors of odd sizes and mixed types
        _clip("clip odd", "mixed", 0, 0, 150, 300000, "mixed", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["softmax_fw", "softmax_bw", "qk_fw", "qk_bw", "clip"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op.startswith("softmax"):
        most = 1 << (26 if dtype != "f32" else 25)
        Tk = _log_int(rng, 2, 4000)
        Tk = Tk // 8 * 8 if rng.random() < 0.4 and Tk >= 8 else Tk
        causal = rng.random() < 0.5
        Tq = rng.choice([1, Tk, Tk, _log_int(rng, 1, Tk)])
        H = rng.choice([1, 3, 4, 5, 8, 12, 16, 20])
        B = _log_int(rng, 1, 64)
        while B * H * Tq * Tk > most and B > 1:
            B //= 2
        while B * H * Tq * Tk > most and H > 1:
            H //= 2
        buckets = rng.choice([8, 12, 16, 32, 32, 48, 64])
        return {"op": op, "dtype": dtype, "B": B, "H": H, "Tq": Tq, "Tk": Tk, "buckets": buckets,
                "distance": rng.randint(buckets, 300), "causal": causal,
                "scale": round(rng.choice([1.0, 1.0, 0.125, rng.uniform(0.05, 1.5)]), 4),
                "mask": rng.choice(["none", "inf", "inf", "lowest"]),
                "shortest": rng.choice([0.0, 0.3, 0.6])}
    if op.startswith("qk"):
        D = rng.choice([32, 48, 64, 64, 72, 80, 96, 128, 128, 160, 256, rng.randint(8, 256)])
        rot = rng.choice([D // 2 * 2, D // 2 * 2, D // 4 * 2, 0])
        Hq, Hk = rng.choice([(8, 8), (16, 16), (32, 8), (12, 12), (9, 3), (24, 2), (5, 1)])
        tokens = _log_int(rng, 1, 16384)
        while tokens * (Hq + Hk) * D * _BYTES[dtype] > 1 << 26:
            tokens = tokens // 2 + 1
        return {"op": op, "dtype": dtype, "tokens": tokens, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
                "interleaved": rng.random() < 0.4, "packed": rng.random() < 0.5,
                "sequence": _log_int(rng, 1, 4096)}
    if rng.random() < 0.5:
        return {"op": "clip", "kind": "layers", "layers": rng.randint(1, 6),
                "hidden": rng.choice([128, 256, 384, 520, 768, 1024]), "count": 0, "largest": 0,
                "dtype": dtype, "clipped": rng.random() < 0.7}
    return {"op": "clip", "kind": "mixed", "layers": 0, "hidden": 0, "count": _log_int(rng, 1, 200),
            "largest": _log_int(rng, 10, 400000), "dtype": rng.choice([dtype, "mixed"]),
            "clipped": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _bucket_map(buckets, distance):
    """Bucket of each clipped distance -distance..distance: half the buckets for each
    direction, the near distances one by one and the far ones in ratios, found with
    whole numbers (log(n/e) / log(d/e) * k >= t  <=>  n^k e^t >= d^t e^k)."""
    half = buckets // 2
    exact = max(1, half // 2)
    k = half - exact
    ids = []
    for r in range(-distance, distance + 1):
        n, b = abs(r), half if r > 0 else 0
        if n < exact:
            ids.append(b + n)
            continue
        t = 0
        while t + 1 < k and n ** k * exact ** (t + 1) >= distance ** (t + 1) * exact ** k:
            t += 1
        ids.append(b + min(half - 1, exact + t))
    return ids


def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _normal(shape, std, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _softmax_state(case, seed):
    dt, gen = _DTYPES[case["dtype"]], _generator(seed, 1)
    B, H, Tq, Tk = case["B"], case["H"], case["Tq"], case["Tk"]
    state = dict(case)
    state["table"] = _normal((case["buckets"], H), 0.7, dt, gen)
    state["ids"] = torch.tensor(_bucket_map(case["buckets"], case["distance"]), dtype=torch.int32,
                                device="cuda")
    state["add"] = None
    if case["mask"] != "none":  # a valid length per batch entry; 0: nothing is left of its rows
        n = torch.rand(B, generator=gen, device="cuda") * (1 - case["shortest"]) + case["shortest"]
        n = (n * (Tk + 1)).floor().clamp(max=Tk)
        if case["mask"] == "lowest":
            n = n.clamp(min=1)
        fill = -_INF if case["mask"] == "inf" else torch.finfo(dt).min
        hidden = torch.arange(Tk, device="cuda")[None, :] >= n[:, None]
        state["add"] = torch.zeros(B, Tk, device="cuda").masked_fill_(hidden, fill).to(dt)
    scores = _normal((B, H, Tq, Tk), 2.0 / case["scale"], dt, gen)
    if case["op"] == "softmax_fw":
        state["scores"] = scores
    else:  # the forward's output, as a training step has saved it
        state["y"] = _plain_softmax_fw(dict(state, scores=scores))
        state["dout"] = _normal((B, H, Tq, Tk), 1.0, dt, gen)
    return state


def _qk_state(case, seed):
    dt, gen = _DTYPES[case["dtype"]], _generator(seed, 2)
    n, Hq, Hk, D, rot = case["tokens"], case["Hq"], case["Hk"], case["D"], case["rot"]

    def pair(std):
        if case["packed"]:  # queries and keys are views of one projection [tokens, q | k | v]
            qkv = _normal((n, (Hq + 2 * Hk) * D), std, dt, gen)
            return (qkv[:, :Hq * D].view(n, Hq, D),
                    qkv[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D))
        return _normal((n, Hq, D), std, dt, gen), _normal((n, Hk, D), std, dt, gen)

    state = dict(case)
    state["q"], state["k"] = pair(1.5)
    state["gq"] = _normal((D,), 0.2, torch.float32, gen).add_(1.0).to(dt)
    state["gk"] = _normal((D,), 0.2, torch.float32, gen).add_(1.0).to(dt)
    state["cos"] = state["sin"] = state["pos"] = None
    if rot:
        length = max(case["sequence"], 1)
        if length == 1:  # a step: every sequence stands somewhere else
            length = 2048
            state["pos"] = torch.randint(0, length, (n,), generator=gen, device="cuda",
                                         dtype=torch.int32)
        else:
            state["pos"] = (torch.arange(n, device="cuda") % length).to(torch.int32)
        turn = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * turn[None, :]
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    if case["op"] == "qk_bw":
        state["dq"], state["dk"] = pair(1.0)
        state["rq"] = (state["q"].float().square().mean(-1) + 1e-6).rsqrt()
        state["rk"] = (state["k"].float().square().mean(-1) + 1e-6).rsqrt()
    return state


def _clip_shapes(case, rnd):
    if case["kind"] == "layers":  # projections, the inner layer, their biases, two norms
        h = case["hidden"]
        one = [(3 * h, h), (3 * h,), (h, h), (h,), (4 * h, h), (4 * h,), (h, 4 * h), (h,)]
        norms = [(h,), (h,), (h,), (h,)]
        wide = case["dtype"]
        return [(s, wide) for _ in range(case["layers"]) for s in one] + \
               [(s, "f32") for _ in range(case["layers"]) for s in norms]
    top = math.log(case["largest"])
    sizes = [max(1, int(math.exp(u * top))) for u in rnd[:case["count"]].tolist()]
    types = ["f32", "f16", "bf16"]
    return [((n,), types[i % 3] if case["dtype"] == "mixed" else case["dtype"])
            for i, n in enumerate(sizes)]


def _clip_state(case, seed):
    gen = _generator(seed, 3)
    rnd = torch.rand(256, generator=torch.Generator().manual_seed(case["count"] + 7))
    shapes = _clip_shapes(case, rnd)
    total = sum(math.prod(s) for s, _ in shapes)
    std = 2.0 / math.sqrt(total)  # a norm of about 2
    state = dict(case)
    # the gradients of one type lie end to end in one buffer, as in buckets for their exchange,
    # and so do the clipped ones
    grads, flat = {}, {}
    for d in sorted({d for _, d in shapes}):
        sizes = [math.prod(s) for s, e in shapes if e == d]
        whole = _normal((sum(sizes),), std * (64.0 if d == "f16" else 1.0), _DTYPES[d], gen)
        flat[str(whole.dtype)] = torch.empty_like(whole)
        grads[d] = list(zip(whole.split(sizes), flat[str(whole.dtype)].split(sizes)))
    pairs = [grads[d].pop(0) + (s,) for s, d in shapes]
    state["grads"] = [g.view(s) for g, _, s in pairs]
    state["out"] = [o.view(s) for _, o, s in pairs]
    state["flat"] = flat
    state["max_norm"] = 1.0 if case["clipped"] else 1000.0
    return state


def prepare(case, seed):
    if case["op"].startswith("softmax"):
        return _softmax_state(case, seed)
    if case["op"].startswith("qk"):
        return _qk_state(case, seed)
    return _clip_state(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _ids_of(s):
    """Bucket of every (query, key) pair [Tq, Tk], and which keys lie in the query's future."""
    i = torch.arange(s["Tq"], device="cuda")[:, None] + (s["Tk"] - s["Tq"])
    r = torch.arange(s["Tk"], device="cuda")[None, :] - i
    return s["ids"].long()[r.clamp(-s["distance"], s["distance"]) + s["distance"]], r > 0


def _plain_softmax_fw(s):
    ids, future = _ids_of(s)
    z = s["scores"].float() * s["scale"] + s["table"].float()[ids].permute(2, 0, 1)
    if s["add"] is not None:
        z = z + s["add"].float()[:, None, None, :]
    if s["causal"]:
        z = z.masked_fill(future, -_INF)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m.masked_fill(m == -_INF, 0.0))
    t = e.sum(-1, keepdim=True)
    return (e / t.masked_fill(t == 0, 1.0)).to(s["table"].dtype)


def _plain_softmax_bw(s):
    ids, future = _ids_of(s)
    y, g = s["y"].float(), s["dout"].float()
    if s["add"] is not None:
        y = y.masked_fill((s["add"] == -_INF)[:, None, None, :], 0.0)
    if s["causal"]:
        y = y.masked_fill(future, 0.0)
    dz = y * (g - (y * g).sum(-1, keepdim=True))
    flat = dz.sum(0, dtype=torch.float64).permute(1, 2, 0).reshape(-1, s["H"])
    dtable = torch.zeros(s["buckets"], s["H"], dtype=torch.float64, device="cuda")
    dtable.index_add_(0, ids.reshape(-1), flat)
    return (dz * s["scale"]).to(s["y"].dtype), dtable.float()


def _angles(s):
    p = s["pos"].long()
    return s["cos"][p][:, None, :], s["sin"][p][:, None, :]


def _turn(x, s, back):
    """x with its first rot features rotated (``back``: by the opposite angles)."""
    rot = s["rot"]
    if not rot:
        return x
    c, w = _angles(s)
    w = -w if back else w
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * w, b * c + a * w), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * w, b * c + a * w), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_norm(x, gamma, s):
    f = x.float()
    r = (f.square().mean(-1) + 1e-6).rsqrt()
    return _turn(f * r[..., None] * gamma.float(), s, False).to(x.dtype), r


def _plain_norm_bw(dout, x, gamma, r, s):
    dn = _turn(dout.float(), s, True)
    xhat = x.float() * r[..., None]
    g = dn * gamma.float()
    dx = r[..., None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dn * xhat).sum((0, 1), dtype=torch.float64).float()


def _plain_clip(s):
    sums = [g.float().square().sum(dtype=torch.float64) for g in s["grads"]]
    norm = torch.stack(sums).sum().sqrt().float()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * factor) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm.reshape(1), **s["flat"]}


def _run_plain(s):
    if s["op"] == "softmax_fw":
        return {"y": _plain_softmax_fw(s)}
    if s["op"] == "softmax_bw":
        dinp, dtable = _plain_softmax_bw(s)
        return {"dinp": dinp, "dtable": dtable}
    if s["op"] == "qk_fw":
        q, rq = _plain_norm(s["q"], s["gq"], s)
        k, rk = _plain_norm(s["k"], s["gk"], s)
        return {"q": q, "k": k, "rq": rq, "rk": rk}
    if s["op"] == "qk_bw":
        dq, dgq = _plain_norm_bw(s["dq"], s["q"], s["gq"], s["rq"], s)
        dk, dgk = _plain_norm_bw(s["dk"], s["k"], s["gk"], s["rk"], s)
        return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}
    return _plain_clip(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import transformer_reduce_gb300 as L
    if s["op"] == "softmax_fw":
        return {"y": L.softmax_fw_relpos(s["scores"], s["table"], s["ids"], s["add"],
                                         causal=s["causal"], scale=s["scale"])}
    if s["op"] == "softmax_bw":
        dinp, dtable = L.softmax_bw_relpos(s["dout"], s["y"], s["ids"], s["buckets"], s["add"],
                                           causal=s["causal"], scale=s["scale"])
        return {"dinp": dinp, "dtable": dtable}
    if s["op"] == "qk_fw":
        q, k, rq, rk = L.qk_norm_rope_fw(s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"],
                                         s["pos"], interleaved=s["interleaved"], eps=1e-6)
        return {"q": q, "k": k, "rq": rq, "rk": rk}
    if s["op"] == "qk_bw":
        dq, dk, dgq, dgk = L.qk_norm_rope_bw(s["dq"], s["dk"], s["q"], s["k"], s["gq"], s["gk"],
                                             s["rq"], s["rk"], s["cos"], s["sin"], s["pos"],
                                             interleaved=s["interleaved"])
        return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}
    _, norm = L.grad_clip(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, **s["flat"]}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("softmax"):
        es, H, Tq, Tk = _BYTES[case["dtype"]], case["H"], case["Tq"], case["Tk"]
        pairs = float(case["B"] * H * Tq * Tk)
        seen = 1.0
        if case["causal"]:
            seen = (Tk - (Tq - 1) / 2) / Tk
        if case["mask"] == "inf":  # -inf keys need not be read
            seen *= (1 + case["shortest"]) / 2
        small = case["buckets"] * H * es + (0 if case["mask"] == "none" else case["B"] * Tk * es)
        if case["op"] == "softmax_fw":
            return {"bytes": pairs * es * (seen + 1) + small, "flops": 8 * pairs * seen}
        return {"bytes": pairs * es * (2 * seen + 1) + small + 4 * case["buckets"] * H,
                "flops": 6 * pairs * seen}
    if case["op"].startswith("qk"):
        es, rows = _BYTES[case["dtype"]], float(case["tokens"] * (case["Hq"] + case["Hk"]))
        angles = 4.0 * case["rot"] * min(case["tokens"], max(case["sequence"], 1))
        if case["sequence"] == 1:
            angles = 4.0 * case["rot"] * min(case["tokens"], 2048)
        n = rows * case["D"]
        moved = 2 if case["op"] == "qk_fw" else 3
        return {"bytes": n * es * moved + 4 * rows + angles + 4 * case["tokens"],
                "flops": n * (8 if moved == 2 else 14)}
    rnd = torch.rand(256, generator=torch.Generator().manual_seed(case["count"] + 7))
    moved = sum(math.prod(s) * _BYTES[d] for s, d in _clip_shapes(case, rnd))
    values = sum(math.prod(s) for s, _ in _clip_shapes(case, rnd))
    return {"bytes": 2.0 * moved, "flops": 3.0 * values}


# ---------------------------------------------------------------------------
# 64-bit answers
# ---------------------------------------------------------------------------
def _exact_bias(s):
    """[H, Tq, Tk] of the bias, from the distance of each pair."""
    Tq, Tk, R = s["Tq"], s["Tk"], s["distance"]
    reach = torch.arange(Tk, device="cuda").unsqueeze(0) - torch.arange(Tk - Tq, Tk,
                                                                        device="cuda").unsqueeze(1)
    ids = torch.take(s["ids"].long(), torch.minimum(torch.maximum(reach, reach * 0 - R),
                                                    reach * 0 + R) + R)
    return reach, ids


def _exact_visible(s, reach, b):
    see = torch.ones(1, s["Tq"], s["Tk"], dtype=torch.bool, device="cuda")
    if s["causal"]:
        see = see & (reach <= 0)[None]
    if s["add"] is not None:
        see = see & ~torch.isneginf(s["add"][b].double())[None, None, :]
    return see


def _exact_softmax(case, s):
    reach, ids = _exact_bias(s)
    parts, total = [], torch.zeros(case["buckets"], s["H"], dtype=torch.float64, device="cuda")
    table = None if case["op"] == "softmax_bw" else s["table"].double().T[:, ids]
    for b in range(s["B"]):
        see = _exact_visible(s, reach, b)
        if case["op"] == "softmax_fw":
            z = s["scores"][b].double() * s["scale"] + table
            if s["add"] is not None:
                z = z + s["add"][b].double()
            z = torch.where(see, z, torch.full_like(z, -_INF))
            top = z.max(-1, keepdim=True).values
            w = torch.where(see, (z - top).exp(), torch.zeros_like(z))
            norm = w.sum(-1, keepdim=True)
            parts.append(torch.where(norm > 0, w / norm, torch.zeros_like(w)))
        else:
            y = torch.where(see, s["y"][b].double(), torch.zeros((), dtype=torch.float64,
                                                                 device="cuda"))
            g = s["dout"][b].double()
            d = y * g - y * (y * g).sum(-1, keepdim=True)
            parts.append((s["scale"] * d).float())
            for h in range(s["H"]):
                total[:, h] += torch.bincount(ids.reshape(-1), weights=d[h].reshape(-1),
                                              minlength=case["buckets"])
    if case["op"] == "softmax_fw":
        return {"y": torch.stack(parts)}
    return {"dinp": torch.stack(parts).double(), "dtable": total}


def _exact_turn(x, s, sign):
    """The rotation as a product of complex numbers."""
    rot = s["rot"]
    if rot == 0:
        return x
    p = s["pos"].long()
    unit = torch.complex(s["cos"].double()[p], sign * s["sin"].double()[p]).unsqueeze(1)
    head = x[..., :rot]
    if s["interleaved"]:
        v = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * unit
        head = torch.view_as_real(v).reshape(head.shape)
    else:
        v = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * unit
        head = torch.cat((v.real, v.imag), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _exact_qk(case, s):
    out = {}
    for side, x, gamma in (("q", s["q"], s["gq"]), ("k", s["k"], s["gk"])):
        x, gamma = x.double(), gamma.double()
        if case["op"] == "qk_fw":
            r = 1.0 / torch.sqrt((x * x).sum(-1) / x.shape[-1] + 1e-6)
            out["r" + side] = r
            out[side] = _exact_turn(x * gamma * r.unsqueeze(-1), s, 1.0)
        else:
            r = s["r" + side].double().unsqueeze(-1)
            dn = _exact_turn(s["d" + side].double(), s, -1.0)
            mean = (dn * gamma * x).sum(-1, keepdim=True) * r / x.shape[-1]
            out["d" + side] = r * dn * gamma - r * r * x * mean
            out["dg" + side] = (dn * x * r).flatten(0, 1).sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("softmax"):
        return _exact_softmax(case, s)
    if case["op"].startswith("qk"):
        return _exact_qk(case, s)
    wide = [g.double() for g in s["grads"]]
    norm = math.sqrt(math.fsum(float(torch.dot(w.reshape(-1), w.reshape(-1))) for w in wide))
    factor = min(1.0, s["max_norm"] / (norm + 1e-6))
    joined = {}
    for g, w in zip(s["grads"], wide):
        joined.setdefault(str(g.dtype), []).append(w.reshape(-1) * factor)
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            **{k: torch.cat(v) for k, v in joined.items()}}
