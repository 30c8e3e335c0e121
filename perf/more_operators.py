"""Measured cases of a feed-forward block's operators around the quantized projections.

The operators, as a user reaches them through ``weight_quantized_linear_amd``:

* ``gated_gemm`` / ``gated_gemm_backward``: gate and up projection, the activation and the
  product in one kernel, bf16 or FP8 weights, and the gradients of the bf16 one;
* ``lora_gemm`` / ``lora_gemm_backward``: low-rank adapters of many requests beside a shared
  projection, and their gradients;
* ``block_norm`` / ``block_norm_backward``: the norm behind a block with its gate and residual
  scale, fused with the norm in front of the next one.

``run`` computes them with elementary torch operations in float32 (``own`` false) or through
the library (``own`` true).
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
EPS = 1e-6


def _lib():
    import weight_quantized_linear_amd as q
    return q


def listed():
    return [
        # One token through a wide feed-forward layer with FP8 weights: HBM counts.
        {"name": "gated fp8 m1", "kind": "gated", "m": 1, "f": 14336, "k": 4096, "weight": "fp8", "act": "silu",
         "addend": False, "out": "bf16", "train": False},
        # Thirteen decoding sequences with adapters on the projections: their part comes in as an addend.
        {"name": "gated bf16 m13 addend", "kind": "gated", "m": 13, "f": 5504, "k": 2048, "weight": "bf16",
         "act": "silu", "addend": True, "out": "bf16", "train": False},
        # A prompt chunk of a ragged row count: the matrix cores count.
        {"name": "gated fp8 m500", "kind": "gated", "m": 500, "f": 14336, "k": 4096, "weight": "fp8", "act": "silu",
         "addend": False, "out": "bf16", "train": False},
        # A training step: the forward pass that keeps the pre-activations, and all gradients.
        {"name": "gated train", "kind": "gated", "m": 4096, "f": 5632, "k": 2048, "weight": "bf16", "act": "silu",
         "addend": False, "out": "bf16", "train": True},
        # The same where no size is a multiple of anything, with the tanh GELU.
        {"name": "gated train odd", "kind": "gated", "m": 515, "f": 1365, "k": 1023, "weight": "bf16",
         "act": "gelu_tanh", "addend": False, "out": "bf16", "train": True},
        # 64 decoding requests, each with one of 32 adapters, a few with none.
        {"name": "lora decode", "kind": "lora", "t": 64, "groups": 64, "adapters": 32, "r": 16, "k": 4096, "n": 4096,
         "skew": 0.0, "off": 2, "base": True, "out": "bf16", "train": False},
        # A batch of prompts of very different lengths, rank 64.
        {"name": "lora prefill", "kind": "lora", "t": 4096, "groups": 12, "adapters": 8, "r": 64, "k": 4096, "n": 14336,
         "skew": 1.0, "off": 1, "base": True, "out": "bf16", "train": False},
        # A training step of four adapters over five sequences beside a frozen projection.
        {"name": "lora train", "kind": "lora", "t": 4099, "groups": 5, "adapters": 4, "r": 16, "k": 2048, "n": 8192,
         "skew": 0.5, "off": 0, "base": True, "out": "bf16", "train": True},
        # Between two blocks in a decode step: launch and latency count.
        {"name": "norm decode", "kind": "norm", "t": 8, "h": 4096, "res": "bf16", "io": "bf16", "par": "bf16",
         "post": True, "gates": 1, "scale": 1.0, "train": False},
        # The same over the rows of a long prompt, the residual stream in float32: HBM counts.
        {"name": "norm prefill", "kind": "norm", "t": 16384, "h": 4096, "res": "f32", "io": "bf16", "par": "f32",
         "post": True, "gates": 1, "scale": 1.0, "train": False},
        # Gradients in a training step, one modulating gate per sequence of 1024 rows.
        {"name": "norm train", "kind": "norm", "t": 8192, "h": 2048, "res": "bf16", "io": "bf16", "par": "f32",
         "post": False, "gates": 8, "scale": 1.0, "train": True},
        # Gradients at an odd width in float32, both norms and a gate of channels.
        {"name": "norm train odd", "kind": "norm", "t": 4100, "h": 1535, "res": "f32", "io": "f32", "par": "f32",
         "post": True, "gates": 1, "scale": 0.5, "train": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """The same, three times of four a multiple of `step`."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(step, v // step * step)


def draw(rng):
    kind = rng.choice(["gated", "gated", "lora", "lora", "norm", "norm"])
    if kind == "gated":
        train = rng.random() < 0.4
        m, k = _log(rng, 1, 4096), _size(rng, 64, 4096, 64)
        f = min(_size(rng, 64, 14336, 64), max(64, 4096 * 5632 * 2048 // (m * k)) if train else
                max(64, 500 * 14336 * 4096 // (m * k)))
        return {"kind": kind, "m": m, "f": f, "k": k, "weight": "bf16" if train else rng.choice(["bf16", "fp8"]),
                "act": rng.choice(["silu", "silu", "gelu_tanh", "relu"]), "addend": not train and rng.random() < 0.3,
                "out": "bf16" if train else rng.choice(["bf16", "bf16", "f32"]), "train": train}
    if kind == "lora":
        train = rng.random() < 0.4
        groups = _log(rng, 1, 64)
        k, n = _size(rng, 128, 8192, 64), _size(rng, 128, 8192, 64)
        return {"kind": kind, "t": max(groups, _log(rng, 1, 4096)), "groups": groups, "adapters": _log(rng, 1, 32),
                "r": rng.choice([4, 8, 16, 16, 32, 64, 100, 128]), "k": k, "n": n, "skew": round(rng.uniform(0.0, 1.2), 2),
                "off": 1 if groups > 4 and rng.random() < 0.5 else 0, "base": rng.random() < 0.7,
                "out": rng.choice(["bf16", "bf16", "f32"]), "train": train}
    h = _size(rng, 64, 8192, 64)
    per = _log(rng, 1, 2048)  # rows of a gate
    t = _log(rng, 1, min(16384, 16384 * 4096 // h))
    gates = rng.choice([0, 1, max(1, t // per), t])
    res, io = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    return {"kind": kind, "t": t // gates * gates if gates else t, "h": h, "res": res, "io": io,
            "par": rng.choice(["bf16", "f32"]), "post": rng.random() < 0.6, "gates": gates,
            "scale": rng.choice([1.0, 1.0, 0.5]), "train": rng.random() < 0.5}


def _counts(c):
    """Rows of each group: Zipf shares, one row at least, rounded by largest remainder."""
    g, spare = c["groups"], c["t"] - c["groups"]
    shares = [(z + 1) ** -c["skew"] for z in range(g)]
    shares = [spare * s / sum(shares) for s in shares]
    counts = [int(s) for s in shares]
    order = sorted(range(g), key=lambda z: (counts[z] - shares[z], z))
    for z in order[:spare - sum(counts)]:
        counts[z] += 1
    return [n + 1 for n in counts]


def _ids(c):
    """Which adapter each group takes, in order of size; the last ones have none."""
    live = c["groups"] - c["off"]
    return [z % c["adapters"] for z in range(live)] + [-1] * c["off"]


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)
    s = {"case": c}
    if c["kind"] == "gated":
        m, f, k = c["m"], c["f"], c["k"]
        s["alpha"] = 1.0
        if c["weight"] == "fp8":  # codes of Gaussian weights, spread over E4M3's range by one scale
            s["alpha"] = k ** -0.5 / 64.0
            s["w"] = _normal(g, (2 * f, k), torch.float32, 64.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        else:
            s["w"] = _normal(g, (2 * f, k), torch.bfloat16, k ** -0.5)
        s["x"] = _normal(g, (m, k), torch.bfloat16)
        s["addend"] = _normal(g, (m, 2 * f), torch.bfloat16, 0.5) if c["addend"] else None
        if c["train"]:
            s["dy"] = _normal(g, (m, f), torch.bfloat16)
    elif c["kind"] == "lora":
        t, r, k, n = c["t"], c["r"], c["k"], c["n"]
        s["x"] = _normal(g, (t, k), torch.bfloat16)
        s["a"] = _normal(g, (c["adapters"], r, k), torch.bfloat16, k ** -0.5)
        s["b"] = _normal(g, (c["adapters"], n, r), torch.bfloat16, r ** -0.5)
        s["scale"] = torch.rand((c["adapters"],), generator=g, device=DEV) + 0.5
        counts = torch.tensor(_counts(c), device=DEV)
        perm = torch.randperm(c["groups"], generator=g, device=DEV)
        counts = counts[perm]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        names = torch.randperm(c["adapters"], generator=g, device=DEV)
        ids = torch.tensor(_ids(c), device=DEV)[perm]
        s["ids"] = torch.where(ids >= 0, names[ids.clamp(min=0)], ids).to(torch.int32)
        s["most"] = max(_counts(c))
        s["base"] = _normal(g, (t, n), DTYPES[c["out"]]) if c["base"] else None
        if c["train"]:
            s["dy"] = _normal(g, (t, n), torch.bfloat16)
            s["dx"] = _normal(g, (t, k), torch.bfloat16)  # what came back through the shared projection
    else:
        t, h, par = c["t"], c["h"], DTYPES[c["par"]]
        s["res"] = _normal(g, (t, h), DTYPES[c["res"]], 2.0)  # in training the residual as the forward pass left it
        s["block"] = _normal(g, (t, h), DTYPES[c["io"]])
        s["w"] = _normal(g, (h,), torch.float32, 0.2).add_(1.0).to(par)
        s["post"] = _normal(g, (h,), torch.float32, 0.2).add_(1.0).to(par) if c["post"] else None
        s["gate"] = _normal(g, (c["gates"], h), par, 0.7) if c["gates"] else None
        if c["train"]:
            s["dy"] = _normal(g, (t, h), DTYPES[c["io"]])
            s["dres"] = _normal(g, (t, h), DTYPES[c["res"]])
    return s


# ---------------------------------------------------------------- the plain forms


def _act_plain(v, act):
    """(act(v), act'(v))."""
    if act == "relu":
        return v.clamp(min=0.0), (v > 0.0).to(v.dtype)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return v * sig, sig * (1.0 + v * (1.0 - sig))
    rate = math.sqrt(2.0 / math.pi)
    sig = 1.0 / (1.0 + torch.exp(-2.0 * rate * (v + 0.044715 * v * v * v)))
    return v * sig, sig + v * sig * (1.0 - sig) * 2.0 * rate * (1.0 + 3.0 * 0.044715 * v * v)


def _gated_plain(s, c):
    w, x = s["w"].float(), s["x"].float()
    pre = (x @ w.t()) * s["alpha"]
    if s["addend"] is not None:
        pre = pre + s["addend"].float()
    gate, up = pre.split(c["f"], dim=1)
    val, slope = _act_plain(gate, c["act"])
    out = (val * up).to(DTYPES[c["out"]])
    if not c["train"]:
        return out
    dy = s["dy"].float()
    dpre = torch.cat([dy * up * slope, dy * val], dim=1)
    return {"out": out, "dpre": dpre.to(torch.bfloat16), "dx": (dpre @ w).to(torch.bfloat16),
            "dw": (dpre.t() @ x).to(torch.bfloat16)}


def _lora_plain(s, c):
    """Every group padded to the largest one's rows, and batched products."""
    t, k, n, dt = c["t"], c["k"], c["n"], DTYPES[c["out"]]
    offsets, ids = s["offsets"].long(), s["ids"].long()
    row = offsets[:-1, None] + torch.arange(s["most"], device=DEV)
    inside = (row < offsets[1:, None]) & (ids >= 0)[:, None]
    at = row.clamp(max=t - 1)
    a, b = s["a"].float()[ids.clamp(min=0)], s["b"].float()[ids.clamp(min=0)]
    scale = s["scale"][ids.clamp(min=0)][:, None, None]
    x = torch.where(inside[:, :, None], s["x"].float()[at], 0.0)
    z = torch.bmm(x, a.transpose(1, 2).contiguous())
    delta = torch.bmm(z, b.transpose(1, 2).contiguous()) * scale
    out = torch.zeros((t, n), device=DEV) if s["base"] is None else s["base"].float()
    out[row[inside]] += delta[inside]
    if not c["train"]:
        return out.to(dt)
    dy = torch.where(inside[:, :, None], s["dy"].float()[at], 0.0)
    dz = torch.bmm(dy, b) * scale
    dx = s["dx"].float()
    dx[row[inside]] += torch.bmm(dz, a)[inside]
    da = torch.zeros(s["a"].shape, device=DEV)
    da.index_add_(0, ids.clamp(min=0), torch.bmm(dz.transpose(1, 2).contiguous(), x))
    db = torch.zeros(s["b"].shape, device=DEV)
    db.index_add_(0, ids.clamp(min=0), torch.bmm(dy.transpose(1, 2).contiguous(), z) * scale)
    return {"out": out.to(dt), "dx": dx.to(torch.bfloat16), "da": da, "db": db}


def _inverse_rms(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _rows_of_gate(s, c):
    return s["gate"].float().repeat_interleave(c["t"] // c["gates"], 0) if c["gates"] else 1.0


def _norm_plain(s, c):
    block = s["block"].float()
    if c["post"]:
        block = block * _inverse_rms(block) * s["post"].float()
    res = (c["scale"] * s["res"].float() + _rows_of_gate(s, c) * block).to(DTYPES[c["res"]])
    r = res.float()
    return {"y": (r * _inverse_rms(r) * s["w"].float()).to(DTYPES[c["io"]]), "res": res}


def _norm_train_plain(s, c):
    r, o, dy, w = s["res"].float(), s["block"].float(), s["dy"].float(), s["w"].float()
    gate = _rows_of_gate(s, c)
    inv = _inverse_rms(r)
    unit, a = r * inv, dy * w
    d = s["dres"].float() + inv * (a - unit * (a * unit).mean(1, keepdim=True))
    out = {"dres": (c["scale"] * d).to(DTYPES[c["res"]]), "dw": (dy * unit).sum(0).to(DTYPES[c["par"]])}
    if c["post"]:
        inv_o = _inverse_rms(o)
        unit_o, post = o * inv_o, s["post"].float()
        b = d * gate * post
        out["dblock"] = (inv_o * (b - unit_o * (b * unit_o).mean(1, keepdim=True))).to(DTYPES[c["io"]])
        out["dpost"] = (d * gate * unit_o).sum(0).to(DTYPES[c["par"]])
        o = unit_o * post
    else:
        out["dblock"] = (d * gate).to(DTYPES[c["io"]])
    if c["gates"]:
        out["dgate"] = (d * o).reshape(c["gates"], -1, c["h"]).sum(1).to(DTYPES[c["par"]])
    return out


def _plain(s, c):
    if c["kind"] == "gated":
        return _gated_plain(s, c)
    if c["kind"] == "lora":
        return _lora_plain(s, c)
    return _norm_train_plain(s, c) if c["train"] else _norm_plain(s, c)


# ---------------------------------------------------------------- the library's calls


def _calls(s, c):
    q = _lib()
    if c["kind"] == "gated":
        if not c["train"]:
            return q.gated_gemm(s["w"], s["x"], alpha=s["alpha"], addend=s["addend"], activation=c["act"],
                                out_dtype=DTYPES[c["out"]])
        out, pre = q.gated_gemm(s["w"], s["x"], activation=c["act"], return_pre=True)
        dpre, dx, dw = q.gated_gemm_backward(s["dy"], pre, s["w"], s["x"], activation=c["act"])
        return {"out": out, "dpre": dpre, "dx": dx, "dw": dw}
    if c["kind"] == "lora":
        to = s["base"] if c["out"] == "f32" else None  # a float32 base is added to in place, as the plain form does
        if not c["train"]:
            return q.lora_gemm(s["x"], s["a"], s["b"], s["offsets"], s["ids"], scale=s["scale"], base=s["base"], out=to,
                               out_dtype=DTYPES[c["out"]])
        out, z = q.lora_gemm(s["x"], s["a"], s["b"], s["offsets"], s["ids"], scale=s["scale"], base=s["base"], out=to,
                             out_dtype=DTYPES[c["out"]], return_z=True)
        dx, da, db = q.lora_gemm_backward(s["dy"], s["x"], z, s["a"], s["b"], s["offsets"], s["ids"], scale=s["scale"],
                                          base=s["dx"])
        return {"out": out, "dx": dx, "da": da, "db": db}
    if not c["train"]:
        y, res = q.block_norm(s["res"], s["w"], block=s["block"], block_weight=s["post"], gate=s["gate"],
                              residual_scale=c["scale"], eps=EPS)
        return {"y": y, "res": res}
    g = q.block_norm_backward(s["dy"], s["dres"], s["res"], s["w"], block=s["block"], block_weight=s["post"],
                              gate=s["gate"], residual_scale=c["scale"], eps=EPS)
    out = {"dres": g.residual, "dw": g.weight, "dblock": g.block}
    if c["post"]:
        out["dpost"] = g.block_weight
    if c["gates"]:
        out["dgate"] = g.gate
    return out


def run(state):
    return _calls(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------- the work, and the definition in 64 bits


def work(case):
    c = case
    if c["kind"] == "gated":
        m, f, k = c["m"], c["f"], c["k"]
        size = 2 * f * k * BYTES[c["weight"]] + 2 * m * k + m * f * BYTES[c["out"]] + (4 * m * f if c["addend"] else 0)
        flops = 4 * m * f * k
        if c["train"]:  # gradient in, dpre, dx and dw out
            return {"bytes": size + 2 * m * f + 4 * m * f + 2 * m * k + 4 * f * k, "flops": 3 * flops}
        return {"bytes": size, "flops": flops}
    if c["kind"] == "lora":
        t, r, k, n = c["t"], c["r"], c["k"], c["n"]
        counts, ids = _counts(c), _ids(c)
        live, used = sum(m for m, z in zip(counts, ids) if z >= 0), len({z for z in ids if z >= 0})
        size = 2 * live * k + 2 * used * r * (k + n) + t * n * BYTES[c["out"]] * (2 if c["base"] else 1) + 4 * c["adapters"]
        flops = 2 * live * r * (k + n)
        if c["train"]:
            return {"bytes": size + 2 * live * n + 2 * 2 * t * k + 4 * c["adapters"] * r * (k + n), "flops": 3 * flops}
        return {"bytes": size, "flops": flops}
    t, h, res, io, par = c["t"], c["h"], BYTES[c["res"]], BYTES[c["io"]], BYTES[c["par"]]
    rows = 1 + (1 if c["post"] else 0) + c["gates"]
    if c["train"]:
        return {"bytes": t * h * (3 * res + 3 * io) + 2 * rows * h * par, "flops": t * h * (30 if c["post"] else 16)}
    return {"bytes": t * h * (2 * res + 2 * io) + rows * h * par, "flops": t * h * (12 if c["post"] else 8)}


def _act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, 0.0), torch.where(v > 0, 1.0, 0.0).double()
    if act == "silu":
        sig = torch.sigmoid(v)
        return v * sig, sig + v * sig * torch.sigmoid(-v)
    rate = math.sqrt(2.0 / math.pi)
    th = torch.tanh(rate * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * rate * (1 + 3 * 0.044715 * v * v)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] == "gated":
        f, x = c["f"], s["x"].double()
        gate = s["alpha"] * torch.mm(x, s["w"][:f].double().t())
        up = s["alpha"] * torch.mm(x, s["w"][f:].double().t())
        if s["addend"] is not None:
            gate, up = gate + s["addend"][:, :f].double(), up + s["addend"][:, f:].double()
        val, slope = _act64(gate, c["act"])
        if not c["train"]:
            return val * up
        dy = s["dy"].double()
        dg, du = dy * up * slope, dy * val
        return {"out": val * up, "dpre": torch.cat([dg, du], 1),
                "dx": torch.mm(dg, s["w"][:f].double()) + torch.mm(du, s["w"][f:].double()),
                "dw": torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)], 0)}
    if c["kind"] == "lora":
        t, k, n = c["t"], c["k"], c["n"]
        out = torch.zeros((t, n), dtype=torch.float64, device=DEV) if s["base"] is None else s["base"].double()
        da, db = torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
        dx = s["dx"].double() if c["train"] else None
        edges, ids, scale = s["offsets"].tolist(), s["ids"].tolist(), s["scale"].double().tolist()
        for z, l in enumerate(ids):
            cut = slice(edges[z], edges[z + 1])
            if l < 0 or edges[z] == edges[z + 1]:
                continue
            x, a, b = s["x"][cut].double(), s["a"][l].double(), s["b"][l].double()
            low = torch.mm(x, a.t())
            out[cut] += scale[l] * torch.mm(low, b.t())
            if c["train"]:
                dy = s["dy"][cut].double()
                dlow = scale[l] * torch.mm(dy, b)
                dx[cut] += torch.mm(dlow, a)
                da[l] += torch.mm(dlow.t(), x)
                db[l] += scale[l] * torch.mm(dy.t(), low)
        return {"out": out, "dx": dx, "da": da, "db": db} if c["train"] else out
    per = c["t"] // c["gates"] if c["gates"] else 1
    gate = s["gate"].double()[torch.arange(c["t"], device=DEV) // per] if c["gates"] else torch.ones((), device=DEV).double()
    r, o, w = s["res"].double(), s["block"].double(), s["w"].double()

    def unit_of(x):  # x over its root mean square, and that root
        root = torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / c["h"] + EPS)
        return x / root, root

    if not c["train"]:
        res = c["scale"] * r + gate * (unit_of(o)[0] * s["post"].double() if c["post"] else o)
        return {"y": unit_of(res.to(DTYPES[c["res"]]).double())[0] * w, "res": res}
    dy = s["dy"].double()
    unit, root = unit_of(r)
    along = torch.linalg.vecdot(dy * w, unit).unsqueeze(1) / c["h"]
    d = s["dres"].double() + (dy * w - along * unit) / root
    out = {"dres": c["scale"] * d, "dw": torch.linalg.vecdot(dy, unit, dim=0)}
    if c["post"]:
        unit_o, root_o = unit_of(o)
        grad = d * gate
        out["dpost"] = torch.linalg.vecdot(grad, unit_o, dim=0)
        grad = grad * s["post"].double()
        out["dblock"] = (grad - torch.linalg.vecdot(grad, unit_o).unsqueeze(1) / c["h"] * unit_o) / root_o
        o = unit_o * s["post"].double()
    else:
        out["dblock"] = d * gate
    if c["gates"]:
        out["dgate"] = torch.stack([part.sum(0) for part in (d * o).split(per)]) if c["gates"] <= 512 else \
            (d * o).unflatten(0, (c["gates"], per)).sum(1)
    return out
