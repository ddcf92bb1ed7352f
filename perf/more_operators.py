"""Cases that measure the operators of fine-tuning: the modulated norm with its input kept in 8 bits for the backward
pass, and low-rank adapters, one for each sample, beside a shared projection.

``run`` computes each in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
``own`` is true, through the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
GROUP = 32


def listed():
    return [
        # a training step of the headline workload's final norm, its input kept in 8 bits between the two passes
        {"name": "ckpt8_step_latents", "op": "ckpt8_step", "dtype": "bf16", "B": 2, "S": 4096, "D": 3072},
        # the same in fp32 on a small text batch of odd lengths, with channels that are no multiple of a group
        {"name": "ckpt8_step_text_f32", "op": "ckpt8_step", "dtype": "f32", "B": 3, "S": 513, "D": 1160},
        # the backward of a short prompt: latency
        {"name": "ckpt8_bwd_prompt", "op": "ckpt8_bwd", "dtype": "bf16", "B": 4, "S": 77, "D": 768},
        # the norm's output taken again, as the input of the next projection's weight gradient
        {"name": "ckpt8_again_latents", "op": "ckpt8_again", "dtype": "bf16", "B": 2, "S": 4096, "D": 3072},
        # an activation of another layer put away and taken back
        {"name": "ckpt8_keep_ragged", "op": "ckpt8_keep", "dtype": "bf16", "B": 5, "S": 1531, "D": 2056},
        # the modulation of 64 requests, each with one of 24 fine-tunes or none: latency of a serving step
        {"name": "lora_fwd_requests", "op": "lora_fwd", "dtype": "bf16", "B": 64, "S": 1, "K": 3072, "N": 6144, "R": 16,
         "NA": 24, "ragged": False},
        # fused query, key and value projection of eight requests of unlike lengths
        {"name": "lora_fwd_tokens", "op": "lora_fwd", "dtype": "bf16", "B": 8, "S": 1024, "K": 3072, "N": 9216, "R": 32,
         "NA": 5, "ragged": True},
        # one prompt in fp32
        {"name": "lora_fwd_prompt_f32", "op": "lora_fwd", "dtype": "f32", "B": 1, "S": 77, "K": 768, "N": 1544, "R": 8,
         "NA": 2, "ragged": False},
        # fine-tuning one adapter of a square projection at the headline workload
        {"name": "lora_step_latents", "op": "lora_step", "dtype": "bf16", "B": 2, "S": 4096, "K": 3072, "N": 3072,
         "R": 16, "NA": 1, "ragged": False},
        # a small text batch in fp32, three adapters
        {"name": "lora_step_text_f32", "op": "lora_step", "dtype": "f32", "B": 5, "S": 333, "K": 1160, "N": 1536,
         "R": 8, "NA": 3, "ragged": True},
        # adapters of the modulation itself: a conditioning row a sample
        {"name": "lora_step_samples", "op": "lora_step", "dtype": "bf16", "B": 257, "S": 1, "K": 3072, "N": 6144,
         "R": 16, "NA": 4, "ragged": False},
        # large rank, odd lengths, two adapters
        {"name": "lora_step_rank128", "op": "lora_step", "dtype": "bf16", "B": 3, "S": 1531, "K": 2048, "N": 2560,
         "R": 128, "NA": 2, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ckpt8_step", "ckpt8_bwd", "ckpt8_again", "ckpt8_keep", "lora_fwd", "lora_fwd", "lora_step",
                     "lora_step"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("ckpt8"):
        D = 8 * _log(rng, 8, 1024 if dtype == "bf16" else 512)
        rows = _log(rng, 1, 2 * 4096 * 3072 // D // (1 if dtype == "bf16" else 2))
        B = min(rows, _log(rng, 1, 64))
        return {"op": op, "dtype": dtype, "B": B, "S": max(1, min(65536, rows // B)), "D": D}
    K, N, R = 8 * _log(rng, 8, 768), 8 * _log(rng, 8, 1152), 8 * _log(rng, 1, 16)
    rows = _log(rng, 1, max(1, 2 * 4096 * 6144 // (K + N) * 16 // max(16, R) // (1 if dtype == "bf16" else 4)))
    B = min(rows, _log(rng, 1, 256))
    return {"op": op, "dtype": dtype, "B": B, "S": max(1, min(65536, rows // B)), "K": K, "N": N, "R": R,
            "NA": _log(rng, 1, 24), "ragged": rng.random() < 0.5}


def _lens(case):
    """Rows of each sample: all, or falling from S to 1 and 0."""
    B, S = case["B"], case["S"]
    if not case["ragged"]:
        return [S] * B
    lens = [max(0, S - i * S // B - i % 2) for i in range(B)]
    return lens if B < 4 else lens[:-2] + [1, 0]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = DTYPES[case["dtype"]]
    B, S = case["B"], case["S"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"].startswith("ckpt8"):
        D = case["D"]
        # rows and channels of unlike size, and a mean
        x = normal(B, S, D) * torch.exp(0.5 * normal(B, S, 1)) * torch.exp(0.7 * normal(D)) + 0.3 * normal(D)
        state = {"case": case, "x": x.to(t)}
        if case["op"] == "ckpt8_keep":
            return state
        state["emb"] = (0.3 * normal(B, 2 * D)).to(t)
        if case["op"] != "ckpt8_again":
            state["dy"] = normal(B, S, D).to(t)
        if case["op"] != "ckpt8_step":  # what the forward left
            xf = state.pop("x").float()
            state["mean"] = xf.mean(-1)
            state["rstd"] = torch.rsqrt(xf.var(-1, correction=0) + EPS)
            state["ckpt"] = _record(xf)
        return state
    K, N, R, NA = (case[k] for k in ("K", "N", "R", "NA"))
    state = {"case": case, "x": normal(B, S, K).to(t), "y": normal(B, S, N).to(t),
             "A": (normal(NA, R, K) / math.sqrt(K)).to(t), "U": (normal(NA, R, N) / math.sqrt(R)).to(t),
             "scale": 0.5 + torch.rand(NA, generator=gen, device=dev)}
    ids = torch.randint(0, NA, (B,), generator=gen, device=dev, dtype=torch.int32)
    if B > 1:
        ids[B // 2] = -1  # a request without an adapter
    state["ids"] = ids
    state["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    state["out"] = torch.zeros((B, S, N), dtype=t, device=dev)
    if case["op"] == "lora_step":
        state["d_out"] = normal(B, S, N).to(t)
        state["d_base"] = normal(B, S, K).to(t)
        state["dx"] = torch.zeros((B, S, K), dtype=t, device=dev)
    return state


def _groups(x):
    """x in groups of 32 channels, the last one filled with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _codes(x):
    """(codes, exponents): the least exponent k >= -126 that brings a group below 127.5 steps of 2^k."""
    g = _groups(x)
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True))
    k = (e - 7 + (m >= 127.5 / 128).to(e.dtype)).clamp(min=-126)
    return torch.ldexp(g, -k).round(), k


def _kept(x):
    """The values that the 8 bits stand for."""
    q, k = _codes(x)
    return torch.ldexp(q, k).flatten(-2)[..., :x.shape[-1]]


def _record(x):
    """Codes and scale bytes of each row, each part filled up to 16 bytes."""
    q, k = _codes(x)
    q = q.to(torch.int8).flatten(-2)[..., :x.shape[-1]]
    s = (k.squeeze(-1) + 127).to(torch.uint8)
    return torch.cat((torch.nn.functional.pad(q, (0, -q.shape[-1] % 16)).view(torch.uint8),
                      torch.nn.functional.pad(s, (0, -s.shape[-1] % 16))), -1).contiguous()


def _of_record(ckpt, D):
    """The values of records."""
    first = (D + 15) // 16 * 16
    n = (D + GROUP - 1) // GROUP
    k = ckpt[..., first:first + n].to(torch.int32) - 127
    return torch.ldexp(_groups(ckpt[..., :D].view(torch.int8).float()), k[..., None]).flatten(-2)[..., :D]


def _modulation(emb, t):
    """(1 + scale), a tensor of the activations' type, and shift."""
    scale, shift = emb.float()[:, None].chunk(2, -1)
    return (1 + scale).to(t).float(), shift


def _plain_norm_bwd(dy, x8, emb, mean, rstd, t):
    onep, _ = _modulation(emb, t)
    g = dy.float()
    r = rstd[..., None]
    xhat = (x8 - mean[..., None]) * r
    gh, p = g * onep, g * xhat
    dx = r * (gh - gh.mean(-1, keepdim=True) - xhat * (p * onep).mean(-1, keepdim=True))
    return dx.to(t), torch.cat((p.sum(1), g.sum(1)), -1)


def _plain_ckpt8(st):
    case = st["case"]
    t, op = DTYPES[case["dtype"]], case["op"]
    if op == "ckpt8_keep":
        return {"x": _kept(st["x"].float()).to(t)}
    if op == "ckpt8_step":
        x = st["x"].float()
        mean = x.mean(-1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
        onep, shift = _modulation(st["emb"], t)
        out = (c * rstd * onep + shift).to(t)
        dx, d_emb = _plain_norm_bwd(st["dy"], _kept(x), st["emb"], mean[..., 0], rstd[..., 0], t)
        return {"out": out, "mean": mean[..., 0], "rstd": rstd[..., 0], "dx": dx, "d_emb": d_emb}
    x8 = _of_record(st["ckpt"], case["D"])
    if op == "ckpt8_again":
        onep, shift = _modulation(st["emb"], t)
        return {"out": ((x8 - st["mean"][..., None]) * st["rstd"][..., None] * onep + shift).to(t)}
    dx, d_emb = _plain_norm_bwd(st["dy"], x8, st["emb"], st["mean"], st["rstd"], t)
    return {"dx": dx, "d_emb": d_emb}


def _plain_lora(st):
    case = st["case"]
    t = DTYPES[case["dtype"]]
    B, S, NA = case["B"], case["S"], case["NA"]
    at = st["ids"].long().clamp(min=0)
    rows = torch.ones((B, S, 1), dtype=torch.bool, device="cuda")
    if st["lens"] is not None:
        rows = (torch.arange(S, device="cuda") < st["lens"][:, None])[..., None]
    factor = torch.where(st["ids"] >= 0, st["scale"][at], 0.0)[:, None, None]
    A, U = st["A"].float()[at], st["U"].float()[at]
    x = st["x"].float()
    h = torch.where(rows, factor * (x @ A.transpose(1, 2)), 0.0)
    out = torch.where(rows, st["y"].float() + h @ U, 0.0).to(t)
    if case["op"] == "lora_fwd":
        return {"out": out}
    d = st["d_out"].float()
    e = torch.where(rows, factor * (d @ U.transpose(1, 2)), 0.0)
    dx = torch.where(rows, st["d_base"].float() + e @ A, 0.0).to(t)
    dA = torch.zeros((NA, case["R"], case["K"]), device="cuda").index_add_(0, at, e.transpose(1, 2) @ x)
    dU = torch.zeros((NA, case["R"], case["N"]), device="cuda").index_add_(0, at, h.transpose(1, 2) @ d)
    return {"out": out, "dx": dx, "dA": dA, "dU": dU}


def _own(st):
    from invariant_dit_adaln_gb300 import binding as b
    case = st["case"]
    op, f32 = case["op"], case["dtype"] == "f32"
    if op.startswith("ckpt8"):
        if op == "ckpt8_keep":
            ckpt = (b.adaln_f32_ckpt8_pack if f32 else b.adaln_ckpt8_pack)(st["x"])
            return {"x": (b.adaln_f32_ckpt8_unpack if f32 else b.adaln_ckpt8_unpack)(ckpt, case["D"])}
        if op == "ckpt8_again":
            again = b.adaln_f32_out_again_ckpt8 if f32 else b.adaln_out_again_ckpt8
            return {"out": again(st["ckpt"], st["emb"], st["mean"], st["rstd"])}
        bwd = b.adaln_f32_out_bwd_ckpt8 if f32 else b.adaln_out_bwd_ckpt8
        if op == "ckpt8_bwd":
            dx, d_emb = bwd(st["dy"], st["ckpt"], st["emb"], st["mean"], st["rstd"])
            return {"dx": dx, "d_emb": d_emb}
        fwd = b.adaln_f32_out_fwd_ckpt8 if f32 else b.adaln_out_fwd_ckpt8
        out, mean, rstd, ckpt = fwd(st["x"], st["emb"], eps=EPS)
        dx, d_emb = bwd(st["dy"], ckpt, st["emb"], mean, rstd)
        return {"out": out, "mean": mean, "rstd": rstd, "dx": dx, "d_emb": d_emb}
    adapters = (st["A"], st["U"], st["scale"], st["ids"])
    fwd = b.adaln_f32_lora_fwd if f32 else b.adaln_lora_fwd
    out, kept = fwd(st["x"], *adapters, y=st["y"], lens=st["lens"], out=st["out"])
    if op == "lora_fwd":
        return {"out": out}
    bwd = b.adaln_f32_lora_bwd if f32 else b.adaln_lora_bwd
    dx, dA, dU = bwd(st["d_out"], st["x"], kept, *adapters, lens=st["lens"], dx_base=st["d_base"], dx=st["dx"])
    return {"out": out, "dx": dx, "dA": dA, "dU": dU}


def run(state):
    if own:
        return _own(state)
    return (_plain_ckpt8 if state["case"]["op"].startswith("ckpt8") else _plain_lora)(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, S, op = case["B"], case["S"], case["op"]
    if op.startswith("ckpt8"):
        D = case["D"]
        record = (D + 15) // 16 * 16 + ((D + GROUP - 1) // GROUP + 15) // 16 * 16
        kept = B * S * record + 8 * B * S + 2 * B * D * e  # records, statistics, modulation
        each = B * S * D * e
        d_emb = 8 * B * D
        return {"ckpt8_keep": {"bytes": 2 * each + 2 * B * S * record, "flops": 4 * B * S * D},
                "ckpt8_again": {"bytes": kept + each, "flops": 6 * B * S * D},
                "ckpt8_bwd": {"bytes": kept + 2 * each + d_emb, "flops": 20 * B * S * D},
                "ckpt8_step": {"bytes": 2 * kept + 4 * each + d_emb, "flops": 32 * B * S * D}}[op]
    K, N, R, NA = (case[k] for k in ("K", "N", "R", "NA"))
    rows, adapters = sum(_lens(case)), min(NA, B) * R * (K + N)
    n = {"bytes": e * (rows * (K + 2 * N) + adapters), "flops": 2 * rows * R * (K + N)}
    if op == "lora_step":
        n["bytes"] += e * (rows * (3 * K + N) + adapters) + 4 * NA * R * (K + N)
        n["flops"] += 4 * rows * R * (K + N)
    return n


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_kept(x):
    """Each group's multiple of 2^k, k the least integer >= -126 with max|x| / 127.5 < 2^k."""
    D = x.shape[-1]
    n = -(-D // GROUP)
    full = torch.zeros((*x.shape[:-1], n * GROUP), dtype=torch.float64, device=x.device)
    full[..., :D] = x
    g = full.view(*x.shape[:-1], n, GROUP)
    top = g.abs().max(-1, keepdim=True).values
    k = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300) / 127.5)) + 1, -126.0).clamp(min=-126)
    step = torch.exp2(k)
    return (torch.round(g / step) * step).view(full.shape)[..., :D]


def _exact_ckpt8(case, st):
    op, t, D = case["op"], DTYPES[case["dtype"]], case["D"]
    if op == "ckpt8_keep":
        return {"x": _exact_kept(st["x"].double())}
    emb = st["emb"].double()
    onep = (1 + emb[:, :D]).to(t).double()[:, None]  # rounded once to the activations' type
    shift = emb[:, None, D:]
    got = {}
    if op == "ckpt8_step":
        x = st["x"].double()
        mean = x.mean(-1)
        rstd = 1 / torch.sqrt((x - mean[..., None]).square().mean(-1) + EPS)
        x8 = _exact_kept(x)
        got = {"out": (x - mean[..., None]) * rstd[..., None] * onep + shift, "mean": mean, "rstd": rstd}
    else:
        mean, rstd = st["mean"].double(), st["rstd"].double()
        at = -(-D // 16) * 16
        steps = torch.exp2(st["ckpt"][..., at:at + -(-D // GROUP)].double() - 127)
        code = st["ckpt"][..., :D].double()
        code = torch.where(code > 127, code - 256, code)
        x8 = code * steps.repeat_interleave(GROUP, -1)[..., :D]
    xhat = (x8 - mean[..., None]) * rstd[..., None]
    if op == "ckpt8_again":
        return {"out": xhat * onep + shift}
    g = st["dy"].double()
    gh = g * onep
    got["dx"] = rstd[..., None] * (gh - gh.sum(-1, keepdim=True) / D - xhat * (gh * xhat).sum(-1, keepdim=True) / D)
    got["d_emb"] = torch.cat(((g * xhat).sum(1), g.sum(1)), 1)
    return got


def _exact_lora(case, st):
    B, S, NA, R = (case[k] for k in ("B", "S", "NA", "R"))
    live = torch.arange(S, device="cuda")[None, :] < torch.tensor(_lens(case), device="cuda")[:, None]
    # which adapter a sample has, as a matrix of its scales
    pick = (st["ids"][:, None] == torch.arange(NA, device="cuda")).double()
    s = pick * st["scale"].double()
    A, U = st["A"].double().view(NA, -1), st["U"].double().view(NA, -1)
    As, Us = (pick @ A).view(B, R, -1), (pick @ U).view(B, R, -1)
    each = s.sum(1)[:, None, None] * live[..., None]
    x = st["x"].double()
    h = torch.einsum("bsk,brk->bsr", x, As) * each
    out = (st["y"].double() + torch.einsum("bsr,brn->bsn", h, Us)) * live[..., None]
    if case["op"] == "lora_fwd":
        return {"out": out}
    d = st["d_out"].double()
    e = torch.einsum("bsn,brn->bsr", d, Us) * each
    dx = (st["d_base"].double() + torch.einsum("bsr,brk->bsk", e, As)) * live[..., None]
    dA = pick.T @ torch.einsum("bsr,bsk->brk", e, x).reshape(B, -1)
    dU = pick.T @ torch.einsum("bsr,bsn->brn", h, d).reshape(B, -1)
    return {"out": out, "dx": dx, "dA": dA.view(NA, R, -1), "dU": dU.view(NA, R, -1)}


def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_ckpt8 if case["op"].startswith("ckpt8") else _exact_lora)(case, st)
