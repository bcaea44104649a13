"""Measured cases of the paged key-value cache: writing it (bf16 as it is, or quantised to e4m3), reading it back, and
the attention of single new tokens over it.

A case names one operator and its sizes. `prepare` makes what a server holds before the call (the fused QKV rows, the
cache pages, page tables, slots and workspaces), `run` makes one call, `exact` gives the same outputs in 64 bits.

The cache is K and V pages [n_pages][Hkv][page][D] in bf16 or e4m3; an e4m3 cache has a scale pair (K, V) for each
token and head in [n_pages][Hkv][page][2] fp32. The scale is the smallest power of two 2^e, e >= -64, under which the
vector's largest magnitude is at most 448.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rows(op, name, T, kv, page, Hq=28, Hkv=4, D=128, pad=0, spare=0):
    return {"name": name, "op": op, "T": T, "kv": kv, "page": page, "Hq": Hq, "Hkv": Hkv, "D": D, "pad": pad,
            "spare": spare}


def _decode(name, R, lo, hi, kv, page, Hq=28, Hkv=4, D=128, idle=0):
    return {"name": name, "op": "decode", "R": R, "lo": lo, "hi": hi, "kv": kv, "page": page, "Hq": Hq, "Hkv": Hkv,
            "D": D, "idle": idle}


def listed():
    return [
        # one decoding step of 64 sequences: a new token each, quantised, three padded rows
        _rows("write", "write_step_64_e4m3", 64, "e4m3", 16, pad=3, spare=512),
        # a prompt of the BAGEL-shaped layer goes into the cache as it is
        _rows("write", "write_prompt_4096_bf16", 4096, "bf16", 16, spare=16),
        # a large CFG pack (12 sequences) is quantised as it is written
        _rows("write", "write_pack_36864_e4m3", 36864, "e4m3", 64, spare=64),
        # the tail of a cached prompt comes back for a chunk of prefill, odd length
        _rows("read", "read_prompt_777_e4m3", 777, "e4m3", 16, spare=64),
        # small heads, pages that are no power of two
        _rows("read", "read_heads64_16385_bf16", 16385, "bf16", 48, Hq=8, Hkv=8, D=64, spare=16),
        # every prompt of the CFG pack for the denoising steps' joint attention
        _rows("read", "read_pack_36864_e4m3", 36864, "e4m3", 64, spare=64),
        # a single short chat: latency
        _decode("decode_1x500_bf16", 1, 500, 500, "bf16", 16),
        # the CFG pack's prompts, one token each
        _decode("decode_12x2500_bf16", 12, 1500, 2500, "bf16", 16),
        # small heads, short ragged sequences, some slots of the batch idle
        _decode("decode_33x1500_heads64_bf16", 33, 1, 1500, "bf16", 48, Hq=4, Hkv=2, D=64, idle=5),
        # one very long context
        _decode("decode_1x131072_e4m3", 1, 131072, 131072, "e4m3", 64),
        # a serving batch of long ragged contexts
        _decode("decode_64x8192_bf16", 64, 1000, 8192, "bf16", 16),
        # a large serving batch over a quantised cache
        _decode("decode_256x4096_e4m3", 256, 200, 4096, "e4m3", 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode"))
    kv, page, D = rng.choice(("bf16", "e4m3")), rng.choice((16, 32, 48, 64, 128)), rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8, 12, 16))
    if op != "decode":
        T = min(_log(rng, 1, 36864), 36864 * 4608 // ((G + 2) * Hkv * D))
        c = _rows(op, "", T, kv, page, G * Hkv, Hkv, D, pad=rng.choice((0, 0, T // 8)), spare=rng.randint(1, 64))
    else:
        R = _log(rng, 1, 256)
        most = min(131072, (1 << 27) // (R * Hkv * D))  # keys a row: at most the largest listed case's elements
        hi = _log(rng, 1, most)
        lo = rng.randint(1, hi)
        c = _decode("", R, lo, hi, kv, page, G * Hkv, Hkv, D, idle=rng.choice((0, 0, R // 5)))
    del c["name"]
    return c


def _lens(c):
    """The sequences' lengths: the same for every seed, so that the work of a case is known."""
    r = random.Random("lens %d %d %d" % (c["R"], c["lo"], c["hi"]))
    lens = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["R"] - 1)]
    for i in range(c["idle"]):  # the batch's last slots are empty
        lens[len(lens) - 1 - i] = 0
    return lens


def work(case):
    c = case
    size = 1 if c["kv"] == "e4m3" else 2
    per_key = c["Hkv"] * 2 * (c["D"] * size + (4 if c["kv"] == "e4m3" else 0))  # K and V of a token in the cache
    if c["op"] == "decode":
        lens = _lens(c)
        table = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": sum(lens) * per_key + 2 * c["R"] * c["Hq"] * c["D"] * 2 + 4 * (table + c["R"]),
                "flops": 4.0 * sum(lens) * c["Hq"] * c["D"]}
    n = c["T"] - c["pad"]
    return {"bytes": n * (per_key + c["Hkv"] * 2 * c["D"] * 2) + 4 * c["T"], "flops": 0}


# ---------------------------------------------------------------------------
# what a server holds before the call
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _cache(c, n_pages, gen):
    """K and V pages full of earlier tokens: values of unit size, with tokens louder or quieter than others."""
    shape = (n_pages, c["Hkv"], c["page"], c["D"])
    made = []
    for _ in range(2):
        x = _normal(gen, *shape)
        x *= torch.exp(0.5 * _normal(gen, *shape[:-1], 1))
        made.append(x.to(torch.bfloat16))
        del x
    if c["kv"] == "bf16":
        return made[0], made[1], None
    scales = torch.empty(shape[:-1] + (2,), device=DEV)
    codes = []
    for i in range(2):
        q, scales[..., i] = _quantise(made[i].float())
        codes.append(q)
    return codes[0], codes[1], scales


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    N = (c["Hq"] + 2 * c["Hkv"]) * c["D"]
    s = {"c": c, "scale": 1.0 / math.sqrt(c["D"])}
    if c["op"] == "decode":
        lens = _lens(c)
        pages = [-(-n // c["page"]) for n in lens]
        n_pages = max(1, sum(pages))
        order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        width = max(1, max(pages))
        # row r's pages are the next ones of a shuffled pool, the rest of its table is unused (-1)
        start = torch.tensor([0] + pages, device=DEV).cumsum(0)[:-1]
        col = torch.arange(width, device=DEV)
        at = (start[:, None] + col[None, :]).clamp(max=n_pages - 1)
        used = col[None, :] < torch.tensor(pages, device=DEV)[:, None]
        s["table"] = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["k"], s["v"], s["scales"] = _cache(c, n_pages, gen)
        s["qkv"] = _normal(gen, c["R"], N).to(torch.bfloat16)
        s["out"] = torch.empty((c["R"], c["Hq"] * c["D"]), dtype=torch.bfloat16, device=DEV)
        rows = c["R"]
    else:
        n_pages = -(-c["T"] // c["page"]) + c["spare"]
        # whole pages in shuffled order, as an allocator hands them out
        order = torch.randperm(n_pages, generator=gen, device=DEV)
        i = torch.arange(c["T"], device=DEV)
        s["slots"] = (order[i // c["page"]] * c["page"] + i % c["page"]).to(torch.int32)
        s["slots"][c["T"] - c["pad"]:] = -1
        s["k"], s["v"], s["scales"] = _cache(c, n_pages, gen)
        s["qkv"] = _normal(gen, c["T"], N).to(torch.bfloat16)
        rows = c["T"]
    s["ws"] = torch.zeros(_workspace(c, rows, s), dtype=torch.uint8, device=DEV)
    return s


def _workspace(c, rows, s):
    """Bytes of workspace: the calls' error word, and for decoding each key range's partial result."""
    if c["op"] != "decode":
        return 64
    return 64 + rows * c["Hq"] * (c["D"] + 2) * 4 * 160


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _quantise(x):
    """fp32 vectors [..., D] to (e4m3 codes, power-of-two scales [...])."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-64)
    scale = torch.where(torch.isfinite(a), torch.ldexp(torch.ones_like(a), e), torch.full_like(a, float("nan")))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _bytes(t):
    """The tensor for indexing: an e4m3 tensor as its bytes."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _outputs_of_write(s):
    return {"k": s["k"], "v": s["v"]} if s["scales"] is None else {"k": s["k"], "v": s["v"], "scales": s["scales"]}


def _plain_write(s):
    c = s["c"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    page, off = slots // c["page"], slots % c["page"]
    kv = s["qkv"][keep][:, c["Hq"] * c["D"]:].reshape(-1, 2, c["Hkv"], c["D"])
    if c["kv"] == "bf16":
        s["k"][page, :, off] = kv[:, 0]
        s["v"][page, :, off] = kv[:, 1]
    else:
        q, scale = _quantise(kv.float())
        q = q.view(torch.uint8)
        s["k"].view(torch.uint8)[page, :, off] = q[:, 0]
        s["v"].view(torch.uint8)[page, :, off] = q[:, 1]
        s["scales"][page, :, off] = scale.permute(0, 2, 1)
    return _outputs_of_write(s)


def _plain_read(s):
    c = s["c"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    page, off = slots // c["page"], slots % c["page"]
    kv = torch.stack([_bytes(s["k"])[page, :, off], _bytes(s["v"])[page, :, off]], 1)
    if c["kv"] == "e4m3":
        scale = s["scales"][page, :, off].permute(0, 2, 1)
        kv = (kv.view(torch.float8_e4m3fn).float() * scale[..., None]).to(torch.bfloat16)
    s["qkv"][keep, c["Hq"] * c["D"]:] = kv.reshape(kv.shape[0], -1)
    return s["qkv"]


def _gathered(s, t, which):
    """The cache's pages of every row as fp32 [R][Hkv][keys][D], and their fp32 scales applied."""
    c = s["c"]
    table = s["table"].long().clamp(min=0)
    x = _bytes(t)[table]  # [R][pages][Hkv][page][D]
    x = x.view(torch.float8_e4m3fn).float() if c["kv"] == "e4m3" else x.float()
    if c["kv"] == "e4m3":
        x *= s["scales"][..., which][table][..., None]
    return x.transpose(1, 2).reshape(c["R"], c["Hkv"], -1, c["D"])


def _plain_decode(s):
    c = s["c"]
    R, Hq, Hkv, D = c["R"], c["Hq"], c["Hkv"], c["D"]
    q = s["qkv"][:, : Hq * D].float().reshape(R, Hkv, Hq // Hkv, D)
    k = _gathered(s, s["k"], 0)
    seen = torch.arange(k.shape[2], device=DEV)[None, :] < s["lens"][:, None]
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    x = torch.where(seen[:, None, None, :], x, torch.full_like(x, float("-inf")))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    v = _gathered(s, s["v"], 1)
    v = torch.where(seen[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(R, Hq * D).to(torch.bfloat16)


def run(state):
    s = state
    c = s["c"]
    if own:
        import mixture_transformers_token_gb300 as mot

        if c["op"] == "write":
            mot.mot_kv_cache_write(s["qkv"], s["slots"], s["k"], s["v"], c["Hq"], s["ws"], scales=s["scales"])
            return _outputs_of_write(s)
        if c["op"] == "read":
            return mot.mot_kv_cache_read(s["k"], s["v"], s["slots"], s["qkv"], c["Hq"], s["ws"], scales=s["scales"])
        return mot.mot_paged_decode_attention(s["qkv"], s["table"], s["lens"], s["k"], s["v"], c["Hq"], s["ws"],
                                              scales=s["scales"], scale=s["scale"], out=s["out"])
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode}[c["op"]](s)


# ---------------------------------------------------------------------------
# the same outputs from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(x):
    """float64 vectors [..., D] to (the e4m3 values, the scales), from the format's definition: a sign, 4 exponent
    bits (2^-6 to 2^8), 3 fraction bits, steps of 2^-9 below 2^-6, ties to even."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.clamp(a, min=2.0 ** -200) / 448.0))
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)  # log2 next to a border
    e = torch.where(a <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-64.0)
    scale = torch.exp2(e)
    y = x / scale[..., None]
    b = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6)))
    b = torch.where(torch.exp2(b + 1) <= y.abs(), b + 1, b)
    step = torch.exp2(b - 3)
    return torch.round(y / step) * step, scale


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["op"] != "decode":
        rows = torch.nonzero(s["slots"] >= 0).reshape(-1)
        slots = s["slots"][rows].long()
        at = ((slots // page)[:, None] * Hkv + torch.arange(Hkv, device=DEV)[None, :]) * page + (slots % page)[:, None]
    if c["op"] == "write":
        kv = s["qkv"][rows][:, Hq * D:].double().reshape(-1, 2, Hkv, D)
        k, v = (s[n].to(torch.float32).double().reshape(-1, D).clone() for n in ("k", "v"))
        if c["kv"] == "bf16":
            k[at], v[at] = kv[:, 0], kv[:, 1]
            return {"k": k.reshape(s["k"].shape), "v": v.reshape(s["v"].shape)}
        code, scale = _exact_e4m3(kv)
        k[at], v[at] = code[:, 0], code[:, 1]
        scales = s["scales"].double().reshape(-1, 2).clone()
        scales[at] = scale.permute(0, 2, 1)
        return {"k": k.reshape(s["k"].shape), "v": v.reshape(s["v"].shape), "scales": scales.reshape(s["scales"].shape)}
    if c["op"] == "read":
        out = s["qkv"].double()
        both = []
        for i, n in enumerate(("k", "v")):
            x = s[n].to(torch.float32).double().reshape(-1, D)[at]
            if c["kv"] == "e4m3":
                x = x * s["scales"].double().reshape(-1, 2)[at][..., i, None]
            both.append(x.reshape(len(rows), Hkv * D))
        out[rows, Hq * D:] = torch.cat(both, 1)
        return out
    out = torch.zeros((c["R"], Hq * D), dtype=torch.float64, device=DEV)
    for r, n in enumerate(_lens(c)):
        if n == 0:
            continue
        pages = s["table"][r, : -(-n // page)].long()
        kv = []
        for i, name in enumerate(("k", "v")):
            x = _bytes(s[name])[pages].view(s[name].dtype).to(torch.float32).double()
            if c["kv"] == "e4m3":
                x = x * s["scales"][pages][..., i].double()[..., None]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n])
        q = s["qkv"][r, : Hq * D].double().reshape(Hkv, Hq // Hkv, D)
        w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, kv[0]) / math.sqrt(D), -1)
        out[r] = torch.einsum("hgn,hnd->hgd", w, kv[1]).reshape(-1)
    return out
