"""Cases that measure the operators around the modulated norm: the norm of queries and keys with the position
rotation, the embedding lookup and its gradient, and the global gradient norm with clipping.

``run`` computes each in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
``own`` is true, through the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CLIP_EPS = 1e-6


def listed():
    return [
        # one new token of eight streams, far along: the latency of a serving step
        {"name": "rope_fwd_decode", "op": "rope_fwd", "dtype": "bf16", "B": 8, "S": 1, "Hq": 24, "Hk": 24, "Dh": 128,
         "Dr": 128, "interleaved": True, "fused": True, "pads": False, "far": True, "P": 32768},
        # the image latents of the headline workload: 24 heads of 128, views of a fused projection's output
        {"name": "rope_fwd_latents", "op": "rope_fwd", "dtype": "bf16", "B": 2, "S": 4096, "Hq": 24, "Hk": 24,
         "Dh": 128, "Dr": 128, "interleaved": True, "fused": True, "pads": False, "far": False, "P": 4096},
        # a padded batch of text: shared key heads, half rotation over a part of an odd head size, fp32
        {"name": "rope_fwd_text_f32", "op": "rope_fwd", "dtype": "f32", "B": 3, "S": 1531, "Hq": 20, "Hk": 4, "Dh": 96,
         "Dr": 64, "interleaved": False, "fused": False, "pads": True, "far": False, "P": 1600},
        # the training step of the headline workload, from attention's gradients
        {"name": "rope_bwd_latents", "op": "rope_bwd", "dtype": "bf16", "B": 2, "S": 4096, "Hq": 24, "Hk": 24,
         "Dh": 128, "Dr": 128, "interleaved": True, "fused": True, "pads": False, "far": False, "P": 4096},
        # a small padded training batch in fp32 with heads of 72 channels
        {"name": "rope_bwd_text_f32", "op": "rope_bwd", "dtype": "f32", "B": 5, "S": 333, "Hq": 16, "Hk": 8, "Dh": 72,
         "Dr": 72, "interleaved": False, "fused": False, "pads": True, "far": False, "P": 400},
        # class labels of a batch of samples (the last row: no class)
        {"name": "embed_fwd_labels", "op": "embed_fwd", "dtype": "bf16", "n": 257, "V": 1001, "D": 3072,
         "ids": "labels", "scale": 1.0},
        # the tokens of a text batch, scaled by sqrt(D)
        {"name": "embed_fwd_text", "op": "embed_fwd", "dtype": "f32", "n": 16383, "V": 50021, "D": 2048,
         "ids": "text", "scale": math.sqrt(2048.0)},
        # label gradients of 4096 samples, a tenth of them without a class
        {"name": "embed_bwd_labels", "op": "embed_bwd", "dtype": "bf16", "grad": "f32", "n": 4096, "V": 1001,
         "D": 3072, "ids": "labels", "scale": 1.0},
        # the table gradient of a text batch: a few tokens very often, most of the table never
        {"name": "embed_bwd_text", "op": "embed_bwd", "dtype": "bf16", "grad": "bf16", "n": 32768, "V": 50021,
         "D": 1024, "ids": "text", "scale": 32.0},
        # the gradients of one small layer: the latency of the norm alone
        {"name": "norm_layer", "op": "norm", "tensors": 6, "big": 512 * 1024, "ragged": False, "mixed": False,
         "factor": 0.0},
        # sixty tensors of odd sizes and both types, written into flat buckets
        {"name": "clip_ragged", "op": "clip", "tensors": 60, "big": 1500000, "ragged": True, "mixed": True,
         "factor": 0.5},
        # the fp32 weight and bias gradients of sixteen modulations
        {"name": "clip_modulations", "op": "clip", "tensors": 32, "big": 6144 * 3072, "ragged": False, "mixed": False,
         "factor": 0.3},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "embed_fwd", "embed_bwd", "norm", "clip"])
    if op in ("rope_fwd", "rope_bwd"):
        Dh = 8 * rng.randint(4, 32)
        Hk = _log(rng, 1, 24)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        rows = _log(rng, 1, max(1, 2 * 4096 * 48 * 128 // ((Hq + Hk) * Dh * 2)))
        B = min(rows, _log(rng, 1, 64))
        S = max(1, rows // B)
        return {"op": op, "dtype": rng.choice(["bf16", "f32"]), "B": B, "S": S, "Hq": Hq, "Hk": Hk, "Dh": Dh,
                "Dr": 8 * rng.randint(0, Dh // 8), "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5,
                "pads": rng.random() < 0.5, "far": rng.random() < 0.3, "P": S + rng.randint(0, 4096)}
    if op in ("embed_fwd", "embed_bwd"):
        D = 8 * _log(rng, 8, 1024)
        n = _log(rng, 1, max(1, 32768 * 1024 // D))
        V = _log(rng, 2, max(2, 50021 * 1024 // D))
        case = {"op": op, "dtype": rng.choice(["bf16", "f32"]), "n": n, "V": V, "D": D,
                "ids": rng.choice(["labels", "text"]), "scale": rng.choice([1.0, 0.5, math.sqrt(D)])}
        if op == "embed_bwd":
            case["grad"] = "f32" if case["dtype"] == "f32" else rng.choice(["f32", "bf16"])
        return case
    tensors = _log(rng, 1, 64)
    return {"op": op, "tensors": tensors, "big": _log(rng, 3, 16 * 6144 * 3072 // max(tensors, 16)),
            "ragged": rng.random() < 0.6, "mixed": rng.random() < 0.5,
            "factor": 0.0 if op == "norm" else rng.choice([0.1, 0.5, 0.9, 2.0])}


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------

def _sizes(case):
    """Elements and types of the tensors of a gradient list: weights and their biases, or ragged ones."""
    n, big = case["tensors"], case["big"]
    if case["ragged"]:
        sizes = [max(1, int(big * ((i * 37) % 101 + 1) / 101) | 1) for i in range(n)]
    else:
        sizes = [big if i % 2 == 0 else max(1, int(2 * math.sqrt(big / 2))) for i in range(n)]
    types = ["bf16" if case["mixed"] and i % 3 != 0 else "f32" for i in range(n)]
    return sizes, types


def _views(flat, sizes):
    ends = torch.tensor(sizes).cumsum(0).tolist()
    return [flat[e - s:e] for s, e in zip(sizes, ends)]


def _prepare_rope(case, gen, dev):
    t = DTYPES[case["dtype"]]
    B, S, Hq, Hk, Dh, Dr, P = (case[k] for k in ("B", "S", "Hq", "Hk", "Dh", "Dr", "P"))

    def rows(H):
        return torch.randn((B, S, H, Dh), generator=gen, device=dev)

    scale = torch.exp(0.5 * torch.randn((B, S, 1, 1), generator=gen, device=dev))  # rows of unlike size
    if case["fused"]:  # views of the projection's output [B, S, (Hq + 2 Hk) Dh]
        qkv = (rows(Hq + 2 * Hk) * scale).to(t)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        q, k = (rows(Hq) * scale).to(t), (rows(Hk) * scale).to(t)
    wq = (1 + 0.1 * torch.randn(Dh, generator=gen, device=dev)).to(t)
    wk = (1 + 0.1 * torch.randn(Dh, generator=gen, device=dev)).to(t)
    if case["far"]:  # each stream at a place of its own
        first = torch.randint(0, P - S + 1, (B, 1), generator=gen, device=dev)
        pos = first + torch.arange(S, device=dev)
    else:
        pos = torch.arange(S, device=dev).expand(B, S)
    if case["pads"]:  # rows behind a sequence's end have no position
        lens = torch.randint(0, S + 1, (B, 1), generator=gen, device=dev)
        lens[0] = S
        pos = torch.where(torch.arange(S, device=dev) < lens, pos, -1)
    pos = pos.to(torch.int32).contiguous()
    inv = 10000.0 ** (-torch.arange(Dr // 2, device=dev, dtype=torch.float64) / max(1, Dr // 2))
    angle = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * inv
    state = {"q": q, "k": k, "wq": wq, "wk": wk, "cos": angle.cos().float(), "sin": angle.sin().float(), "pos": pos,
             "case": case}
    if case["op"] == "rope_bwd":
        state["gq"] = (0.1 * rows(Hq)).to(t)
        state["gk"] = (0.1 * rows(Hk)).to(t)
    return state


def _prepare_embed(case, gen, dev):
    t = DTYPES[case["dtype"]]
    n, V, D = case["n"], case["V"], case["D"]
    if case["ids"] == "labels":  # even over the classes, a tenth with the last one (no class)
        ids = torch.randint(0, V, (n,), generator=gen, device=dev)
        ids = torch.where(torch.rand(n, generator=gen, device=dev) < 0.1, V - 1, ids)
    else:  # text: a token's frequency falls with its rank, and some places are padding
        u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1.0)) - 1).long().clamp_(0, V - 1)
        ids = torch.where(torch.rand(n, generator=gen, device=dev) < 0.02, -1, ids)
    state = {"ids": ids, "case": case}
    if case["op"] == "embed_fwd":
        state["table"] = (0.02 * torch.randn((V, D), generator=gen, device=dev)).to(t)
    else:
        state["g"] = (0.1 * torch.randn((n, D), generator=gen, device=dev)).to(t)
    return state


def _prepare_grads(case, gen, dev):
    sizes, types = _sizes(case)
    total = sum(sizes)
    spread = [10.0 ** (-(i % 5)) for i in range(len(sizes))]  # layers' gradients differ in size
    grads = [(s * torch.randn(n, generator=gen, device=dev)).to(DTYPES[t]) for n, t, s in zip(sizes, types, spread)]
    norm = math.sqrt(sum(n * s * s for n, s in zip(sizes, spread)))
    state = {"grads": grads, "case": case, "max_norm": case["factor"] * norm, "total": total}
    if case["op"] == "clip":
        state["flat"] = {t: torch.empty(sum(n for n, u in zip(sizes, types) if u == t), dtype=DTYPES[t], device=dev)
                         for t in ("f32", "bf16") if t in types}
        views = {t: iter(_views(f, [n for n, u in zip(sizes, types) if u == t])) for t, f in state["flat"].items()}
        state["outs"] = [next(views[t]) for t in types]
    return state


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    if case["op"].startswith("rope"):
        return _prepare_rope(case, gen, dev)
    if case["op"].startswith("embed"):
        return _prepare_embed(case, gen, dev)
    return _prepare_grads(case, gen, dev)


# ------------------------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------------------------

def _turn(n, c, s, interleaved, back):
    """The rotation of the first 2 * c.shape[-1] channels of n (its transpose if back)."""
    half = c.shape[-1]
    s = -s if back else s
    if interleaved:
        a, b = n[..., 0:2 * half:2], n[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = n[..., :half], n[..., half:2 * half]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, n[..., 2 * half:]), -1)


def _angles(st):
    pos = st["pos"].long()
    at = pos.clamp(min=0)
    return st["cos"][at][:, :, None], st["sin"][at][:, :, None], (pos >= 0)[:, :, None, None]


def _plain_rope_fwd(st):
    c, s, real = _angles(st)

    def one(x, w):
        xf = x.float()
        n = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * w.float()
        return torch.where(real, _turn(n, c, s, st["case"]["interleaved"], False), 0.0).to(x.dtype)

    return {"q": one(st["q"], st["wq"]), "k": one(st["k"], st["wk"])}


def _plain_rope_bwd(st):
    c, s, real = _angles(st)

    def one(dy, x, w):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        g = torch.where(real, _turn(dy.float(), c, s, st["case"]["interleaved"], True), 0.0)
        dw = (g * (xf * r)).sum((0, 1, 2))
        h = g * w.float()
        dx = r * (h - xf * (r * r * (h * xf).mean(-1, keepdim=True)))
        return torch.where(real, dx, 0.0).to(x.dtype), dw

    dq, dwq = one(st["gq"], st["q"], st["wq"])
    dk, dwk = one(st["gk"], st["k"], st["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_embed_fwd(st):
    ids, table = st["ids"], st["table"]
    rows = table[ids.clamp(min=0)].float() * st["case"]["scale"]
    return {"out": torch.where((ids >= 0)[:, None], rows, 0.0).to(table.dtype)}


def _plain_embed_bwd(st):
    case, ids = st["case"], st["ids"]
    acc = torch.zeros((case["V"] + 1, case["D"]), device=ids.device)
    acc.index_add_(0, torch.where(ids >= 0, ids, case["V"]), st["g"].float())
    return {"d_table": (acc[:-1] * case["scale"]).to(DTYPES[case["grad"]])}


def _plain_norm(grads):
    squares = [g.double().square().sum() for g in grads]  # long sums: 64 bits
    return torch.stack(squares).sum().sqrt()


def _plain_clip(st):
    norm = _plain_norm(st["grads"])
    coef = (st["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    out = {"norm": norm.float()}
    for t in st["flat"]:
        flat = torch.cat([g for g in st["grads"] if g.dtype == DTYPES[t]])
        out[t] = (flat.float() * coef).to(DTYPES[t])
    return out


# ------------------------------------------------------------------------------------------------------------------
# the package's entry points
# ------------------------------------------------------------------------------------------------------------------

def _own(st):
    from invariant_dit_adaln_gb300 import binding
    case = st["case"]
    op = case["op"]
    f32 = case.get("dtype") == "f32"
    if op == "rope_fwd":
        call = binding.adaln_f32_qk_norm_rope_fwd if f32 else binding.adaln_qk_norm_rope_fwd
        q, k = call(st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"], pos=st["pos"], eps=EPS,
                    interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "rope_bwd":
        call = binding.adaln_f32_qk_norm_rope_bwd if f32 else binding.adaln_qk_norm_rope_bwd
        dq, dk, dwq, dwk = call(st["gq"], st["gk"], st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"],
                                pos=st["pos"], eps=EPS, interleaved=case["interleaved"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "embed_fwd":
        call = binding.adaln_f32_embed_fwd if f32 else binding.adaln_embed_fwd
        return {"out": call(st["ids"], st["table"], scale=case["scale"])}
    if op == "embed_bwd":
        shape = (case["V"], case["D"])
        if f32:
            return {"d_table": binding.adaln_f32_embed_bwd(st["g"], st["ids"], case["V"], scale=case["scale"])}
        grad = torch.empty(shape, dtype=DTYPES[case["grad"]], device=st["g"].device)
        name = "d_table_acc" if case["grad"] == "f32" else "d_table"
        binding.adaln_embed_bwd(st["g"], st["ids"], case["V"], scale=case["scale"], **{name: grad})
        return {"d_table": grad}
    if op == "norm":
        return {"norm": binding.adaln_grad_norm(st["grads"])[0]}
    _, stats = binding.adaln_grad_clip(st["grads"], st["max_norm"], outs=st["outs"])
    return {"norm": stats[0], **st["flat"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope_fwd":
        return _plain_rope_fwd(state)
    if op == "rope_bwd":
        return _plain_rope_bwd(state)
    if op == "embed_fwd":
        return _plain_embed_fwd(state)
    if op == "embed_bwd":
        return _plain_embed_bwd(state)
    if op == "norm":
        return {"norm": _plain_norm(state["grads"]).float()}
    return _plain_clip(state)


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op.startswith("rope"):
        rows = case["B"] * case["S"]
        elems = rows * (case["Hq"] + case["Hk"]) * case["Dh"]
        table = min(rows, case["P"]) * case["Dr"] * 4 + rows * 4
        weights = 2 * case["Dh"] * size
        if op == "rope_fwd":
            return {"bytes": 2 * elems * size + table + weights, "flops": 8 * elems}
        return {"bytes": 3 * elems * size + table + weights + 2 * case["Dh"] * 4, "flops": 18 * elems}
    if op.startswith("embed"):
        n, V, D = case["n"], case["V"], case["D"]
        if case["ids"] == "labels":  # the rows that n draws touch, on average
            touched = V * (1 - (1 - 0.9 / V) ** n)
        else:
            chance = [(math.log(b + 1) - math.log(a + 1)) / math.log(V + 1)
                      for a, b in _bins(V)]
            touched = sum((b - a) * (1 - (1 - p / (b - a)) ** (0.98 * n)) for (a, b), p in zip(_bins(V), chance))
        if op == "embed_fwd":
            return {"bytes": (touched + n) * D * size + 8 * n, "flops": n * D}
        return {"bytes": n * D * size + V * D * (2 if case["grad"] == "bf16" else 4) + 8 * n, "flops": 2 * n * D}
    sizes, types = _sizes(case)
    total = sum(n * (2 if t == "bf16" else 4) for n, t in zip(sizes, types))
    if op == "norm":
        return {"bytes": total + 4, "flops": 2 * sum(sizes)}
    return {"bytes": 2 * total + 4, "flops": 3 * sum(sizes)}


def _bins(V):
    """Token ranks in about fifty ranges of like logarithmic width: [a, b)."""
    edges = sorted({min(V, int(math.exp(i * math.log(V + 1.0) / 50)) - 1) for i in range(51)} | {0, V})
    return list(zip(edges[:-1], edges[1:]))


def _exact_rope(case, st):
    Dr, inter = case["Dr"], case["interleaved"]
    B, S, Dh = case["B"], case["S"], case["Dh"]
    j = torch.arange(Dr // 2, device="cuda")
    first, second = (2 * j, 2 * j + 1) if inter else (j, j + Dr // 2)
    real = (st["pos"] >= 0).double()[:, :, None]
    at = st["pos"].long().clamp(min=0)
    z = torch.complex(st["cos"].double()[at], st["sin"].double()[at])[:, :, None]

    def forward(x, w):
        n = x / (x.pow(2).sum(-1, keepdim=True) / Dh + EPS).sqrt() * w
        y = n.clone()
        if Dr:
            turned = torch.complex(n[..., first], n[..., second]) * z
            y[..., first] = turned.real
            y[..., second] = turned.imag
        return y * real[..., None]

    out = {}
    for name in ("q", "k"):
        x, w = st[name].double(), st["w" + name].double()
        if case["op"] == "rope_fwd":
            out[name] = forward(x, w)
        else:
            with torch.enable_grad():
                x.requires_grad_(True)
                w.requires_grad_(True)
                out["d" + name], out["dw" + name] = torch.autograd.grad(forward(x, w), (x, w), st["g" + name].double())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("rope"):
        return _exact_rope(case, st)
    if op == "embed_fwd":
        table = torch.cat((st["table"].double(), torch.zeros((1, case["D"]), dtype=torch.float64, device="cuda")))
        return {"out": torch.nn.functional.embedding(st["ids"] % (case["V"] + 1), table) * case["scale"]}
    if op == "embed_bwd":
        # running sums over the occurrences in token order, and their differences at the tokens' ends
        order = st["ids"].argsort(stable=True)
        ids = st["ids"][order]
        sums = torch.cat((torch.zeros((1, case["D"]), dtype=torch.float64, device="cuda"),
                          st["g"].double()[order].cumsum(0)))
        v = torch.arange(case["V"], device="cuda")
        return {"d_table": (sums[torch.searchsorted(ids, v, right=True)] - sums[torch.searchsorted(ids, v)])
                * case["scale"]}
    flat = {t: torch.cat([g.double() for g in st["grads"] if g.dtype == d] or [torch.empty(0, device="cuda").double()])
            for t, d in DTYPES.items()}
    norm = math.sqrt(sum(float(torch.dot(f, f)) for f in flat.values()))
    if op == "norm":
        return {"norm": torch.tensor(norm, dtype=torch.float64)}
    coef = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
    return {"norm": torch.tensor(norm, dtype=torch.float64), **{t: flat[t] * coef for t in st["flat"]}}
