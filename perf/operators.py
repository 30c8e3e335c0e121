"""Measured cases of the mixture-of-experts operators and of the int4 linear layer.

The operators, as a user reaches them through ``weight_quantized_linear_amd``:

* ``int4_gemm`` / ``int4_grouped_gemm``: products with 4-bit weights that carry
  one scale (and, asymmetric, one zero point) per group of consecutive k;
* ``moe_route`` / ``moe_route_backward``: the top-k softmax router;
* ``moe_sort``, ``moe_gather``, ``moe_combine`` / ``moe_combine_backward``: rows
  sorted by expert and back, with the router's weights applied;
* ``swiglu`` / ``swiglu_backward``: the experts' gated activation.

``run`` computes them with elementary torch operations in float32 (``own``
false) or through the library (``own`` true).
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _lib():
    import weight_quantized_linear_amd as q
    return q


def listed():
    return [
        # One token through a square projection: launch and latency count.
        {"name": "int4 m1 4096x4096", "kind": "int4", "m": 1, "n": 4096, "k": 4096, "group": 128, "zeros": True,
         "out": "bf16"},
        # One token through the output head over a 128256-word vocabulary: HBM counts.
        {"name": "int4 m1 head", "kind": "int4", "m": 1, "n": 128256, "k": 4096, "group": 128, "zeros": False,
         "out": "bf16"},
        # A prompt chunk through an up-projection, a ragged row count: the matrix cores count.
        {"name": "int4 m500 up", "kind": "int4", "m": 500, "n": 14336, "k": 4096, "group": 64, "zeros": True,
         "out": "bf16"},
        # Eight decoding sequences, eight experts each: 64 rows spread over 64 experts.
        {"name": "experts decode", "kind": "grouped", "rows": 64, "e": 64, "n": 1536, "k": 2048, "group": 128,
         "zeros": True, "skew": 0.5, "out": "bf16"},
        # The 64-expert workload of the library's benchmark: 4096 rows, Zipf 1.2, two groups switched off.
        {"name": "experts prefill", "kind": "grouped", "rows": 4096, "e": 64, "n": 1536, "k": 2048, "group": 128,
         "zeros": True, "skew": 1.2, "out": "bf16"},
        # Router of a decode step.
        {"name": "route decode", "kind": "route", "t": 8, "e": 64, "top_k": 8, "renorm": True, "masked": 0.0,
         "logits": "f32", "train": False},
        # Router of a training step with its gradient; a quarter of the experts masked away, some rows whole.
        {"name": "route train", "kind": "route", "t": 16384, "e": 256, "top_k": 8, "renorm": False, "masked": 0.25,
         "logits": "bf16", "train": True},
        # Rows to their experts and back in a decode step.
        {"name": "permute decode", "kind": "permute", "t": 8, "top_k": 8, "e": 64, "h": 2048, "dropped": 0.0,
         "io": "bf16", "train": False},
        # The same for a long prompt, a few slots dropped.
        {"name": "permute prefill", "kind": "permute", "t": 16384, "top_k": 8, "e": 256, "h": 2048, "dropped": 0.01,
         "io": "bf16", "train": False},
        # Gradients of the way there and of the weighted way back in a training step.
        {"name": "permute train", "kind": "permute", "t": 4099, "top_k": 6, "e": 64, "h": 4096, "dropped": 0.0,
         "io": "bf16", "train": True},
        # The experts' activation over the rows of a long prompt.
        {"name": "swiglu prefill", "kind": "swiglu", "t": 32768, "f": 1536, "io": "bf16", "train": False},
        # Its gradient at an odd width in float32.
        {"name": "swiglu train", "kind": "swiglu", "t": 4100, "f": 1535, "io": "f32", "train": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["int4", "int4", "grouped", "grouped", "route", "permute", "permute", "swiglu"])
    if kind == "int4":
        m = _log(rng, 1, 640)
        k = _log(rng, 64, 14336)
        k = k if rng.random() < 0.25 else max(64, k // 64 * 64)
        n = min(_log(rng, 64, 131072), 500 * 14336 * 4096 // (m * k))
        return {"kind": kind, "m": m, "n": n, "k": k, "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "out": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "grouped":
        e = _log(rng, 4, 128)
        k = _log(rng, 128, 4096)
        k = k if rng.random() < 0.2 else max(128, k // 64 * 64)
        n = min(_log(rng, 128, 4096), 64 * 1536 * 2048 // (e * k) + 128)
        return {"kind": kind, "rows": _log(rng, 1, 4096), "e": e, "n": n, "k": k, "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "skew": round(rng.uniform(0.0, 1.2), 2), "out": rng.choice(["bf16", "f32"])}
    if kind == "route":
        e = _log(rng, 4, 512)
        return {"kind": kind, "t": _log(rng, 1, 16384), "e": e, "top_k": rng.randint(1, min(e, 10)),
                "renorm": rng.random() < 0.5, "masked": rng.choice([0.0, 0.3, 0.9]), "logits": rng.choice(["bf16", "f32"]),
                "train": rng.random() < 0.5}
    if kind == "permute":
        e = _log(rng, 4, 512)
        top_k = rng.randint(1, min(e, 10))
        h = _log(rng, 64, 7168)
        t = min(_log(rng, 1, 16384), 16384 * 8 * 2048 // (top_k * h))
        return {"kind": kind, "t": t, "top_k": top_k, "e": e, "h": h, "dropped": rng.choice([0.0, 0.02, 0.5]),
                "io": rng.choice(["bf16", "bf16", "f32"]), "train": rng.random() < 0.5}
    f = _log(rng, 64, 8192)
    return {"kind": kind, "t": min(_log(rng, 1, 32768), 32768 * 1536 // f), "f": f, "io": rng.choice(["bf16", "f32"]),
            "train": rng.random() < 0.5}


def _groups(c):
    """Groups of a row of weights."""
    return -(-c["k"] // c["group"])


def _counts(c):
    """Rows of each group, largest first: Zipf shares of the rows, rounded by largest remainder (the seed only
    says which expert has which)."""
    shares = [(z + 1) ** -c["skew"] for z in range(c["e"])]
    shares = [c["rows"] * s / sum(shares) for s in shares]
    counts = [int(s) for s in shares]
    order = sorted(range(c["e"]), key=lambda z: (counts[z] - shares[z], z))
    for z in order[:c["rows"] - sum(counts)]:
        counts[z] += 1
    return counts


def _off(c):
    """How many of the groups are switched off (id -1): two of the middle ones where there are many."""
    return 2 if c["e"] >= 32 and c["rows"] >= 1024 else 0


def _weights(g, c, lead):
    """int4 codes, scales and zero points of Gaussian weights, as a quantiser leaves them."""
    n, k, groups = c["n"], c["k"], _groups(c)
    codes = torch.randn((2, *lead, n, (k + 1) // 2), generator=g, device=DEV).mul_(2.7).add_(7.5).round_().clamp_(0, 15)
    codes = codes.to(torch.uint8)
    packed = codes[0] | (codes[1] << 4)
    scale = ((0.5 + torch.rand((*lead, n, groups), generator=g, device=DEV)) * 0.005).to(torch.bfloat16)
    zero = None
    if c["zeros"]:
        zero = torch.randint(5, 12, (*lead, n, groups), generator=g, device=DEV, dtype=torch.uint8)
    return packed, scale, zero


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": c}
    if c["kind"] == "int4":
        s["w"], s["scale"], s["zero"] = _weights(g, c, ())
        s["x"] = _normal(g, (c["m"], c["k"]), torch.bfloat16)
    elif c["kind"] == "grouped":
        s["w"], s["scale"], s["zero"] = _weights(g, c, (c["e"],))
        s["x"] = _normal(g, (c["rows"], c["k"]), torch.bfloat16)
        counts = torch.tensor(_counts(c), device=DEV)
        perm = torch.randperm(c["e"], generator=g, device=DEV)
        counts = counts[perm]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        ids = torch.randperm(c["e"], generator=g, device=DEV).to(torch.int32)
        off, mid = _off(c), c["e"] // 2  # switched off by rank, so that the work does not hang on the seed
        ids[(perm >= mid) & (perm < mid + off)] = -1
        s["ids"] = ids
        s["most"] = max(_counts(c))
    elif c["kind"] == "route":
        logits = _normal(g, (c["t"], c["e"]), torch.float32, 2.0)
        if c["masked"] > 0.0:
            logits[torch.rand(logits.shape, generator=g, device=DEV) < c["masked"]] = -math.inf
            logits[torch.rand((c["t"],), generator=g, device=DEV) < 0.002] = -math.inf  # nothing is left of a few rows
        s["logits"] = logits.to(DTYPES[c["logits"]])
        s["dw"] = _normal(g, (c["t"], c["top_k"]), torch.float32)
    elif c["kind"] == "permute":
        t, k, h, dt = c["t"], c["top_k"], c["h"], DTYPES[c["io"]]
        pull = torch.linspace(0.0, 1.5, c["e"], device=DEV)  # some experts are more popular than others
        ids = (torch.randn((t, c["e"]), generator=g, device=DEV) + pull).topk(k, dim=1).indices.to(torch.int32)
        if c["dropped"] > 0.0:
            ids[torch.rand(ids.shape, generator=g, device=DEV) < c["dropped"]] = -1
        s["ids"] = ids
        w = torch.rand((t, k), generator=g, device=DEV) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["rows"] = _normal(g, (t * k, h), dt)       # what the experts returned, or a gradient of what they were given
        s["tokens"] = _normal(g, (t, h), dt)         # the tokens, or the gradient of the combined output
        if c["train"]:
            s["drows"] = _normal(g, (t * k, h), dt)
            s["slot_row"] = _sort_plain(ids, c["e"])[2]
    else:
        s["x"] = _normal(g, (c["t"], 2 * c["f"]), DTYPES[c["io"]], 1.5)
        if c["train"]:
            s["dy"] = _normal(g, (c["t"], c["f"]), DTYPES[c["io"]])
    return s


# ---------------------------------------------------------------- the plain forms


def _dequant_plain(s, c):
    """(code - zero) * scale in float32."""
    w, lead, k = s["w"], s["w"].shape[:-1], c["k"]
    codes = torch.stack([w & 15, w >> 4], dim=-1).reshape(*lead, -1)[..., :k].float()
    group = torch.arange(k, device=DEV) // c["group"]
    scale = s["scale"].float()[..., group]
    if s["zero"] is None:
        return (codes - 8.0) * scale
    return (codes - s["zero"].float()[..., group]) * scale


def _grouped_plain(s, c):
    """Every group padded to the largest one's rows, and one batched product."""
    w = _dequant_plain(s, c)
    offsets, ids = s["offsets"].long(), s["ids"].long()
    place = torch.arange(s["most"], device=DEV)
    row = offsets[:-1, None] + place                               # [groups, most]
    inside = row < offsets[1:, None]
    x = s["x"].float()[row.clamp(max=c["rows"] - 1)]
    y = torch.bmm(x, w[ids.clamp(min=0)].transpose(1, 2).contiguous())
    y = torch.where((ids >= 0)[:, None, None], y, 0.0)
    out = torch.zeros((c["rows"], c["n"]), device=DEV)
    out[row[inside]] = y[inside]
    return out


def _route_plain(s, c):
    logits = s["logits"].float()
    values, order = torch.sort(logits, dim=1, descending=True, stable=True)
    values, order = values[:, :c["top_k"]], order[:, :c["top_k"]]
    left = values > -math.inf
    ids = torch.where(left, order, -1).to(torch.int32)
    top = logits.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    chosen = torch.where(left, torch.exp(values - top), 0.0)
    every = torch.exp(logits - top)
    total = chosen.sum(1, keepdim=True) if c["renorm"] else every.sum(1, keepdim=True)
    total = torch.where(total > 0.0, total, 1.0)
    weights = chosen / total
    if not c["train"]:
        return {"ids": ids, "weights": weights}
    dw = torch.where(left, s["dw"], 0.0)
    mean = (weights * dw).sum(1, keepdim=True)
    spread = torch.zeros_like(logits) if c["renorm"] else -(every / total) * mean
    own_part = weights * (dw - mean) if c["renorm"] else weights * dw
    dlogits = spread.scatter_add(1, order, torch.where(left, own_part, 0.0))
    return {"ids": ids, "weights": weights, "dlogits": dlogits.to(s["logits"].dtype)}


def _sort_plain(ids, e):
    """Rows in expert order (equal experts in slot order), then the slots without an expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= e), e, flat)
    keys, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(keys, torch.arange(e + 1, device=DEV))
    active = keys < e
    row = torch.arange(flat.numel(), device=DEV)
    row_slot = torch.where(active, order, ~order).to(torch.int32)
    slot_row = torch.empty_like(row).scatter(0, order, torch.where(active, row, ~row)).to(torch.int32)
    return offsets.to(torch.int32), row_slot, slot_row.reshape(ids.shape)


def _permute_plain(s, c):
    offsets, row_slot, slot_row = _sort_plain(s["ids"], c["e"])
    token = torch.where(row_slot < 0, ~row_slot, row_slot).long() // c["top_k"]
    gathered = torch.where(row_slot[:, None] >= 0, s["tokens"][token], 0)
    return {"offsets": offsets, "row_slot": row_slot, "slot_row": slot_row, "gathered": gathered,
            "combined": _combine_plain(s["rows"], slot_row, s["weights"])}


def _combine_plain(rows, slot_row, weights):
    part = rows.float()[slot_row.clamp(min=0).long()]                        # [t, k, h]
    part = part if weights is None else part * weights[:, :, None]
    return torch.where(slot_row[:, :, None] >= 0, part, 0.0).sum(1).to(rows.dtype)


def _permute_train_plain(s, c):
    slot_row, dy, rows = s["slot_row"], s["tokens"].float(), s["rows"]
    on = slot_row >= 0
    place = torch.where(on, slot_row, ~slot_row).long()
    dweights = torch.where(on, (dy[:, None, :] * rows.float()[place]).sum(2), 0.0)
    spread = torch.where(on[:, :, None], dy[:, None, :] * s["weights"][:, :, None], 0.0)
    drows = torch.empty_like(rows)
    drows[place.reshape(-1)] = spread.reshape(-1, c["h"]).to(rows.dtype)
    return {"dtokens": _combine_plain(s["drows"], slot_row, None), "drows": drows, "dweights": dweights}


def _swiglu_plain(s, c):
    gate, up = s["x"].float().split(c["f"], dim=1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if not c["train"]:
        return (gate * sig * up).to(s["x"].dtype)
    dy = s["dy"].float()
    dgate = dy * up * sig * (1.0 + gate * (1.0 - sig))
    return torch.cat([dgate, dy * gate * sig], dim=1).to(s["x"].dtype)


def _plain(s, c):
    if c["kind"] == "int4":
        return (s["x"].float() @ _dequant_plain(s, c).t()).to(DTYPES[c["out"]])
    if c["kind"] == "grouped":
        return _grouped_plain(s, c).to(DTYPES[c["out"]])
    if c["kind"] == "route":
        return _route_plain(s, c)
    if c["kind"] == "permute":
        return _permute_train_plain(s, c) if c["train"] else _permute_plain(s, c)
    return _swiglu_plain(s, c)


# ---------------------------------------------------------------- the library's calls


def _calls(s, c):
    q = _lib()
    if c["kind"] == "int4":
        return q.int4_gemm(s["w"], s["scale"], s["x"], w_zero=s["zero"], group_size=c["group"],
                           out_dtype=DTYPES[c["out"]])
    if c["kind"] == "grouped":
        return q.int4_grouped_gemm(s["w"], s["scale"], s["x"], s["offsets"], s["ids"], w_zero=s["zero"],
                                   group_size=c["group"], out_dtype=DTYPES[c["out"]], max_tokens_per_group=s["most"])
    if c["kind"] == "route":
        ids, weights = q.moe_route(s["logits"], c["top_k"], renormalize=c["renorm"])
        if not c["train"]:
            return {"ids": ids, "weights": weights}
        return {"ids": ids, "weights": weights,
                "dlogits": q.moe_route_backward(s["logits"], ids, s["dw"], renormalize=c["renorm"])}
    if c["kind"] == "permute" and not c["train"]:
        offsets, row_slot, slot_row = q.moe_sort(s["ids"], c["e"])
        return {"offsets": offsets, "row_slot": row_slot, "slot_row": slot_row,
                "gathered": q.moe_gather(s["tokens"], slot_row), "combined": q.moe_combine(s["rows"], slot_row, s["weights"])}
    if c["kind"] == "permute":
        drows, dweights = q.moe_combine_backward(s["tokens"], s["rows"], s["slot_row"], s["weights"])
        return {"dtokens": q.moe_combine(s["drows"], s["slot_row"]), "drows": drows, "dweights": dweights}
    return q.swiglu_backward(s["dy"], s["x"]) if c["train"] else q.swiglu(s["x"])


def run(state):
    return _calls(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------- the work, and the definition in 64 bits


def work(case):
    c = case
    if c["kind"] == "int4":
        per = c["n"] * ((c["k"] + 1) // 2 + _groups(c) * (3 if c["zeros"] else 2))
        return {"bytes": per + 2 * c["m"] * c["k"] + BYTES[c["out"]] * c["m"] * c["n"],
                "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["kind"] == "grouped":
        counts, mid, off = _counts(c), c["e"] // 2, _off(c)
        live = [r for z, r in enumerate(counts) if r and not mid <= z < mid + off]
        per = c["n"] * ((c["k"] + 1) // 2 + _groups(c) * (3 if c["zeros"] else 2))
        return {"bytes": len(live) * per + 2 * sum(live) * c["k"] + BYTES[c["out"]] * c["rows"] * c["n"],
                "flops": 2 * sum(live) * c["n"] * c["k"]}
    if c["kind"] == "route":
        size, slots = c["t"] * c["e"], c["t"] * c["top_k"]
        ways = 2 if c["train"] else 1
        return {"bytes": ways * BYTES[c["logits"]] * size + 8 * slots + (4 * slots if c["train"] else 0),
                "flops": ways * 4 * size}
    if c["kind"] == "permute":
        slots, size, tok = c["t"] * c["top_k"], BYTES[c["io"]] * c["h"], c["t"]
        read = round(slots * (1.0 - c["dropped"]))  # rows that count; a dropped slot's row is only written, as zeros
        if c["train"]:  # drows in and out, rows in, tokens in and out, weights and their gradient, the places
            return {"bytes": (2 * read + slots + 2 * tok) * size + 12 * slots, "flops": 4 * read * c["h"]}
        return {"bytes": (read + slots + 2 * tok) * size + 16 * slots + 4 * (c["e"] + 1), "flops": 2 * read * c["h"]}
    size = c["t"] * c["f"] * BYTES[c["io"]]
    return {"bytes": (5 if c["train"] else 3) * size, "flops": (12 if c["train"] else 6) * c["t"] * c["f"]}


def _matrix64(packed, scale, zero, k, group):
    """One weight matrix by its definition in float64."""
    n = packed.shape[0]
    q = torch.empty((n, 2 * packed.shape[1]), dtype=torch.float64, device=DEV)
    q[:, 0::2] = (packed % 16).double()
    q[:, 1::2] = torch.div(packed, 16, rounding_mode="floor").double()
    q = q[:, :k]
    out = torch.empty_like(q)
    for b in range(scale.shape[1]):
        cut = slice(b * group, min(k, (b + 1) * group))
        z = 8.0 if zero is None else zero[:, b:b + 1].double()
        out[:, cut] = (q[:, cut] - z) * scale[:, b:b + 1].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] == "int4":
        step = 16384
        parts = []
        for n0 in range(0, c["n"], step):
            z = None if s["zero"] is None else s["zero"][n0:n0 + step]
            w = _matrix64(s["w"][n0:n0 + step], s["scale"][n0:n0 + step], z, c["k"], c["group"])
            parts.append(torch.mm(s["x"].double(), w.t()))
        return torch.cat(parts, dim=1)
    if c["kind"] == "grouped":
        out = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device=DEV)
        edges, ids = s["offsets"].tolist(), s["ids"].tolist()
        for z, e in enumerate(ids):
            if e >= 0 and edges[z + 1] > edges[z]:
                w = _matrix64(s["w"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e], c["k"], c["group"])
                out[edges[z]:edges[z + 1]] = torch.mm(s["x"][edges[z]:edges[z + 1]].double(), w.t())
        return out
    if c["kind"] == "route":
        a = s["logits"].double().cpu()
        t, k = c["t"], c["top_k"]
        ids = _route_plain({"logits": s["logits"], "dw": s["dw"]}, {**c, "train": False})["ids"].cpu().long()
        on = ids >= 0
        chosen = torch.zeros_like(a, dtype=torch.bool)
        rows = torch.arange(t)[:, None].expand(t, k)
        chosen[rows[on], ids[on]] = True
        pool = torch.where(chosen, a, -math.inf) if c["renorm"] else a
        p = torch.exp(pool - torch.logsumexp(pool, 1, keepdim=True))
        p = torch.nan_to_num(p, nan=0.0)  # rows of which nothing is left
        weights = torch.where(on, p.gather(1, ids.clamp(min=0)), 0.0)
        if not c["train"]:
            return {"ids": None, "weights": weights}
        dp = torch.zeros_like(a)
        dp[rows[on], ids[on]] = s["dw"].double().cpu()[on]
        return {"ids": None, "weights": weights, "dlogits": p * (dp - (p * dp).sum(1, keepdim=True))}
    if c["kind"] == "permute":
        t, k, h, e = c["t"], c["top_k"], c["h"], c["e"]
        ids = s["ids"].cpu().reshape(-1)
        place = torch.empty(t * k, dtype=torch.int64)  # the row of every slot, by counting
        at = 0
        for x in range(e + 1):
            mine = torch.nonzero(ids == x if x < e else (ids < 0) | (ids >= e)).reshape(-1)
            place[mine] = at + torch.arange(mine.numel())
            at += mine.numel()
        place, on = place.to(DEV), (ids >= 0).to(DEV)
        token = torch.arange(t, device=DEV).repeat_interleave(k)
        w = s["weights"].double().reshape(-1) * on
        tokens = s["tokens"].double()
        if not c["train"]:
            gathered = torch.zeros((t * k, h), dtype=torch.float64, device=DEV)
            gathered[place[on]] = tokens[token[on]]
            combined = torch.zeros((t, h), dtype=torch.float64, device=DEV)
            for j in range(k):
                combined += s["rows"][place[j::k]].double() * w[j::k, None]
            return {"offsets": None, "row_slot": None, "slot_row": None, "gathered": gathered, "combined": combined}
        dtokens = torch.zeros((t, h), dtype=torch.float64, device=DEV)
        drows = torch.zeros((t * k, h), dtype=torch.float64, device=DEV)
        dweights = torch.zeros((t, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            dtokens += s["drows"][place[j::k]].double() * on[j::k, None]
            drows[place[j::k]] = tokens * w[j::k, None]
            dweights[:, j] = (tokens * s["rows"][place[j::k]].double()).sum(1) * on[j::k]
        return {"dtokens": dtokens, "drows": drows, "dweights": dweights}
    x = s["x"].double()
    gate, up = x[:, :c["f"]], x[:, c["f"]:]
    if not c["train"]:
        return torch.sigmoid(gate) * gate * up
    dy, sig = s["dy"].double(), torch.sigmoid(gate)
    return torch.cat([dy * up * (sig + gate * sig * (1.0 - sig)), dy * sig * gate], dim=1)
