"""Measured cases of what a training step of the routed layer needs beyond its projections and norms: the backward pass
of joint attention, the backward pass of the QK norm and RoPE, and the AdamW step of many tensors.

A case names one operator and its sizes. `prepare` makes what a training program holds before the call (the forward's
tensors and incoming gradients, or weights, gradients and optimizer states), `run` makes one call, `exact` gives the
same outputs in 64 bits.

attn   dqkv [T][(Hq + 2 Hkv) D] from dout, qkv, out [T][Hq D] (bf16) and lse [Hq][T] (the natural log of each softmax
       sum). A sequence is (q_start, k_start, nq, nk, n_causal): its queries are the last nq of nk key positions, rows
       below n_causal are causal, the others see every key. Columns that are no sequence's query or key are kept.
rope   per head x of D values (pre-norm projection): u = x rstd w, out_i = u_i c - u_{i+D/2} s, out_{i+D/2} =
       u_{i+D/2} c + u_i s; dx and the gradient of w from the gradient of out. Value heads pass through.
adamw  m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, p -= lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd p)
       on fp32 weights p with a bf16 copy. 8-bit states: m and sqrt(v) as e4m3 in blocks of 256 whose scale is the
       block's largest magnitude over 448, rounded up or down by 16 random bits an element (Philox4x32-7 of the
       element's index, the tensor's index, the step and a seed); a positive v never gets the code of zero, and blocks
       below 2^-100 become zero.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 256  # elements of an 8-bit state that share a scale
EPS = 1e-6   # of the norm
THETA = 1e6
SEED = 0x5EED0123456789
HYPER = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "step": 7, "grad_scale": 0.5}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attn(name, n, lo, hi, und, Hq=28, Hkv=4, D=128, prefix=0, share=False, pad=0):
    return {"name": name, "op": "attn", "n": n, "lo": lo, "hi": hi, "und": und, "Hq": Hq, "Hkv": Hkv, "D": D,
            "prefix": prefix, "share": share, "pad": pad}


def _rope(name, T, table, gen, Hq=28, Hkv=4, D=128):
    return {"name": name, "op": "rope", "T": T, "table": table, "gen": gen, "Hq": Hq, "Hkv": Hkv, "D": D}


def _adamw(name, sizes, state, grad, copies=1, p16=True):
    return {"name": name, "op": "adamw", "sizes": sizes, "copies": copies, "state": state, "grad": grad, "p16": p16}


def listed():
    qkv, o, mlp = 4608 * 3584, 3584 * 3584, 18944 * 3584
    return [
        # the tiny layer's only sequence: latency
        _attn("attn_tiny_64", 1, 64, 64, 100, 4, 2, 64),
        # one packed sample of the BAGEL-shaped layer: prompt rows, then latents
        _attn("attn_layer_4096", 1, 4096, 4096, 70),
        # text samples of any length packed together, small heads, rows behind the last sample
        _attn("attn_ragged_37x700_heads64", 37, 1, 700, 100, 8, 8, 64, pad=13),
        # a group of eight images' latents over the keys of one shared prompt of odd length
        _attn("attn_shared_prompt_777", 8, 1024, 1024, 0, prefix=777, share=True),
        # a large pack: twelve samples of prompt and latents
        _attn("attn_pack_12x3000", 12, 2900, 3000, 66),
        # the tiny layer: latency
        _rope("rope_tiny_64", 64, "bf16", 50, 4, 2, 64),
        # the BAGEL-shaped layer, a quarter of its rows latents
        _rope("rope_layer_4096", 4096, "bf16", 25),
        # a large pack of odd length under the fp32 rotation
        _rope("rope_pack_36001_fp32", 36001, "fp32", 33),
        # norm weights of 28 layers: many small tensors
        _adamw("adamw_norms_112", "3584,3584,128,128", "fp32", "fp32", copies=28),
        # the attention weights of one layer, fp32 states
        _adamw("adamw_attention_fp32", "%d,%d,3584,128,128" % (qkv, o), "fp32", "fp32"),
        # one weight set of a whole layer, 8-bit states and bf16 gradients
        _adamw("adamw_layer_e4m3", "%d,%d,%d,%d,%d,3584,3584,128,128" % (qkv, o, mlp, mlp, mlp), "e4m3", "bf16"),
        # one weight set of a whole layer, fp32 states
        _adamw("adamw_layer_fp32", "%d,%d,%d,%d,%d,3584,3584,128,128" % (qkv, o, mlp, mlp, mlp), "fp32", "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "rope", "adamw"))
    D, Hkv = rng.choice((64, 128)), rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 12))
    if op == "attn":
        while True:
            n = rng.choice((1, 1, 2, 3, 8, 24, 64))
            hi = _log(rng, 1, 8192)
            lo = rng.choice((hi, rng.randint(1, hi), 1))
            prefix = rng.choice((0, 0, _log(rng, 1, 8192)))
            # scores of the plain form and rows of the pack: at most the largest listed case's
            if (n + 1) * Hq * D * max(hi, prefix) * (hi + prefix) <= 12 * 28 * 128 * 3000 * 3000 and n * (hi + prefix) <= 65536:
                break
        share = prefix > 0 and rng.choice((False, True))
        c = _attn("", n, lo, hi, rng.choice((0, 30, 66, 100)), Hq, Hkv, D, prefix, share, rng.choice((0, 1, 77)))
    elif op == "rope":
        c = _rope("", min(_log(rng, 1, 36864), 36001 * 4608 // ((Hq + 2 * Hkv) * D)), rng.choice(("bf16", "fp32")),
                  rng.choice((0, 25, 50, 100)), Hq, Hkv, D)
    else:
        sizes = [_log(rng, 1, 1 << 24) for _ in range(rng.choice((1, 2, 5, 9)))]
        most = max(1, (1 << 27) // sum(sizes))
        c = _adamw("", ",".join(str(n) for n in sizes), rng.choice(("fp32", "e4m3")), rng.choice(("fp32", "bf16")),
                   min(most, rng.choice((1, 1, 3, 20))), rng.choice((True, True, False)))
    del c["name"]
    return c


def _pack(c):
    """The sequences' descriptors and the number of rows: the same for every seed, so that the work is known."""
    r = random.Random("pack %d %d %d" % (c["n"], c["lo"], c["hi"]))
    lens = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["n"] - 1)]
    seqs, at = [], 0
    if c["share"]:  # the prompt, then groups of rows that see the prompt's keys alone
        seqs.append((0, 0, c["prefix"], c["prefix"], c["prefix"]))
        at = c["prefix"]
    for nq in lens:
        if c["share"]:
            seqs.append((at, 0, nq, c["prefix"], 0))
            at += nq
        else:  # cached rows before the first query are keys alone
            seqs.append((at + c["prefix"], at, nq, c["prefix"] + nq, nq * c["und"] // 100))
            at += c["prefix"] + nq
    return seqs, at + c["pad"]


def _sizes(c):
    return [int(n) for n in c["sizes"].split(",")] * c["copies"]


def work(case):
    c = case
    if c["op"] == "attn":
        seqs, T = _pack(c)
        pairs = sum(nc * (nk - nq) + nc * (nc + 1) // 2 + (nq - nc) * nk for _, _, nq, nk, nc in seqs)
        rows, N = T - c["pad"], (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": rows * (2 * N * 2 + 2 * c["Hq"] * c["D"] * 2 + 4 * c["Hq"]), "flops": 10.0 * pairs * c["Hq"] * c["D"]}
    if c["op"] == "rope":  # d_out and its result; of the pre-norm rows only the normed heads
        qk, half = (c["Hq"] + c["Hkv"]) * c["D"], (2 if c["table"] == "bf16" else 4) * c["D"]
        return {"bytes": c["T"] * (2 * (qk + c["Hkv"] * c["D"]) * 2 + qk * 2 + 4 + half), "flops": 0}
    n = sum(_sizes(c))
    state = 16 if c["state"] == "fp32" else 4 + 16 / BLOCK
    return {"bytes": n * (8 + (2 if c["p16"] else 0) + (4 if c["grad"] == "fp32" else 2) + state), "flops": 0}


# ---------------------------------------------------------------------------
# what a training program holds before the call
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _gathered_rows(s):
    """Row indexes [n_seq][rows] of every sequence's queries and keys (clamped past its end), and which are its own."""
    q0, k0, nq, nk, nc = (s["seqs"][:, i].long()[:, None] for i in range(5))
    i = torch.arange(s["most_q"], device=DEV)[None, :]
    j = torch.arange(s["most_k"], device=DEV)[None, :]
    T = s["qkv"].shape[0]
    # the keys that query i sees: all, or for a causal row those up to its own position
    last = torch.where(i < nc, nk - nq + i, nk - 1)
    return (q0 + i).clamp(max=T - 1), i < nq, (k0 + j).clamp(max=T - 1), j < nk, last


def _heads(x, rows, first, Hkv, G, D):
    """Columns of the rows as fp32 [n_seq][Hkv][G][rows][D], heads from column head `first` on."""
    y = x[:, first * D:(first + Hkv * G) * D][rows].float()
    return y.reshape(*rows.shape, Hkv, G, D).permute(0, 2, 3, 1, 4)


def _scores(s):
    c = s["c"]
    G = c["Hq"] // c["Hkv"]
    qi, has_q, ki, has_k, last = _gathered_rows(s)
    q = _heads(s["qkv"], qi, 0, c["Hkv"], G, c["D"])
    k = _heads(s["qkv"], ki, c["Hq"], c["Hkv"], 1, c["D"])
    v = _heads(s["qkv"], ki, c["Hq"] + c["Hkv"], c["Hkv"], 1, c["D"])
    seen = (torch.arange(s["most_k"], device=DEV)[None, None, :] <= last[:, :, None]) & has_q[:, :, None] & has_k[:, None, :]
    return qi, has_q, ki, has_k, q, k, v, seen[:, None, None]


def _prepare_attn(c, gen):
    seqs, T = _pack(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    N = (Hq + 2 * Hkv) * D
    s = {"c": c, "scale": 1.0 / math.sqrt(D), "seqs": torch.tensor(seqs, dtype=torch.int32, device=DEV),
         "most_q": max(x[2] for x in seqs), "most_k": max(x[3] for x in seqs)}
    s["qkv"] = _normal(gen, T, N).to(torch.bfloat16)
    s["dout"] = _normal(gen, T, Hq * D).to(torch.bfloat16)
    s["dqkv"] = _normal(gen, T, N).to(torch.bfloat16)
    # the forward's outputs, a sequence and KV head at a time
    s["out"] = torch.zeros((T, Hq * D), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((Hq, T), device=DEV)
    G = Hq // Hkv
    for q0, k0, nq, nk, nc in seqs:
        j, i = torch.arange(nk, device=DEV), torch.arange(nq, device=DEV)
        hidden = (i < nc)[:, None] & (j[None, :] > nk - nq + i[:, None])
        for g in range(Hkv):
            cut = lambda h, n, a, m: s["qkv"][a:a + m, h * D:(h + n) * D].float().reshape(m, n, D).transpose(0, 1)  # noqa: E731
            x = torch.matmul(cut(g * G, G, q0, nq), cut(Hq + g, 1, k0, nk).transpose(1, 2)) * s["scale"]
            x.masked_fill_(hidden, float("-inf"))
            lse = torch.logsumexp(x, -1)
            o = torch.matmul(torch.exp(x - lse[..., None]), cut(Hq + Hkv + g, 1, k0, nk))
            s["lse"][g * G:(g + 1) * G, q0:q0 + nq] = lse
            s["out"][q0:q0 + nq, g * G * D:(g + 1) * G * D] = o.transpose(0, 1).reshape(nq, G * D).to(torch.bfloat16)
    if own:
        import mixture_transformers_token_gb300 as mot

        n = mot.mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, len(seqs))
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s


def _prepare_rope(c, gen):
    T, D = c["T"], c["D"]
    N = (c["Hq"] + 2 * c["Hkv"]) * D
    s = {"c": c}
    s["x"] = _normal(gen, T, N).to(torch.bfloat16)
    s["d_out"] = _normal(gen, T, N).to(torch.bfloat16)
    s["w"] = [(1 + 0.1 * _normal(gen, 2, D)).to(torch.bfloat16) for _ in range(2)]  # q's and k's, und and gen
    s["mod"] = (torch.rand(T, generator=gen, device=DEV) * 100 < c["gen"]).to(torch.uint8)
    s["pos"] = torch.arange(T, device=DEV, dtype=torch.int32)
    inv = THETA ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    angle = torch.arange(T, device=DEV, dtype=torch.float64)[:, None] * inv[None, :]
    s["cs"] = torch.stack([angle.cos(), angle.sin()], -1).to(torch.bfloat16 if c["table"] == "bf16" else torch.float32)
    s["dx"] = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    s["dw"] = torch.zeros((2, 2, D), device=DEV)
    if own:  # the layer's plan, which the forward made, and room for partial weight gradients
        import mixture_transformers_token_gb300 as mot

        s["ws"] = mot.mot_route_plan(s["mod"])
        n = mot.mot_qk_norm_rope_backward_workspace_bytes(T, D)
        s["scratch"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s


def _prepare_adamw(c, gen):
    sizes = _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    first = [sum(blocks[:i]) for i in range(len(blocks))]
    NB = sum(blocks)
    s = {"c": c, "sizes": sizes, "first": first}
    # every tensor starts at a block's border of one long array; what lies between tensors is zero
    n_of = torch.tensor(sizes, device=DEV)
    s["tensor"] = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), torch.tensor(blocks, device=DEV), output_size=NB)
    s["inner"] = torch.arange(NB, device=DEV) - torch.tensor(first, device=DEV)[s["tensor"]]  # block within its tensor
    has = torch.arange(BLOCK, device=DEV)[None, :] < (n_of[s["tensor"]] - s["inner"] * BLOCK)[:, None]
    decays = [0.0 if n <= 8192 else 0.1 for n in sizes]  # norm weights do not decay
    s["decays"] = decays
    s["decay"] = torch.tensor(decays, device=DEV)[s["tensor"]]

    def values(scale):  # unit rows of a weight, some louder than others
        x = _normal(gen, NB, BLOCK)
        x *= scale * torch.exp(0.5 * _normal(gen, NB, 1))
        return x.masked_fill_(~has, 0.0)

    s["p"] = values(0.02)
    s["p16"] = s["p"].to(torch.bfloat16) if c["p16"] else None
    s["g"] = values(2e-3).to(torch.bfloat16 if c["grad"] == "bf16" else torch.float32)
    m, r = values(5e-4), values(1e-3).abs_()
    del has
    if c["state"] == "fp32":
        s["m"], s["v"], s["scales"] = m, r.square_(), None
    else:
        s["scales"] = torch.empty((NB, 2), device=DEV)
        half = torch.full((NB, BLOCK), 1 << 19, dtype=torch.int32, device=DEV)
        s["m"], s["scales"][:, 0] = _quantise(m, half)
        s["v"], s["scales"][:, 1] = _quantise(r, half)
    s["hyper"] = torch.tensor(_hyper_words(), dtype=torch.int32, device=DEV).view(torch.float32)
    if own:  # the error word and the list of tensors, which a program makes once
        import mixture_transformers_token_gb300 as mot

        cut = lambda name, i: None if s[name] is None else s[name].view(-1)[first[i] * BLOCK:first[i] * BLOCK + sizes[i]]  # noqa: E731
        each = range(len(sizes))
        s["ws"] = torch.zeros(64, dtype=torch.uint8, device=DEV)
        s["plan"] = mot.AdamWTensors(
            [cut("p", i) for i in each], [cut("g", i) for i in each], [cut("m", i) for i in each], [cut("v", i) for i in each],
            p16=[cut("p16", i) for i in each] if c["p16"] else None,
            scales=[s["scales"][first[i]:first[i] + blocks[i]] for i in each] if c["state"] == "e4m3" else None,
            weight_decay=decays)
    return s


def _hyper_words():
    """The step's numbers in fp32, each rounded once from 64 bits, and the step itself, as 16 words."""
    h = HYPER
    values = [h["lr"], h["beta1"], 1 - h["beta1"], h["beta2"], 1 - h["beta2"], h["lr"] / (1 - h["beta1"] ** h["step"]),
              1 / math.sqrt(1 - h["beta2"] ** h["step"]), h["eps"], h["grad_scale"]]
    words = torch.tensor(values, dtype=torch.float64).float().view(torch.int32).tolist()
    return words + [h["step"]] + [0] * 6


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return {"attn": _prepare_attn, "rope": _prepare_rope, "adamw": _prepare_adamw}[c["op"]](c, gen)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_attn(s):
    c = s["c"]
    Hq, Hkv, D, T = c["Hq"], c["Hkv"], c["D"], s["qkv"].shape[0]
    G, n = Hq // Hkv, s["seqs"].shape[0]
    qi, has_q, ki, has_k, q, k, v, seen = _scores(s)
    do = _heads(s["dout"], qi, 0, Hkv, G, D)
    delta = (do * _heads(s["out"], qi, 0, Hkv, G, D)).sum(-1, keepdim=True)
    lse = s["lse"][:, qi].permute(1, 0, 2).reshape(n, Hkv, G, -1, 1)
    p = torch.matmul(q, k.transpose(-1, -2))
    p.mul_(s["scale"]).sub_(lse).exp_().masked_fill_(~seen, 0.0)
    flat = lambda x: x.reshape(n, Hkv, -1, x.shape[-1])  # noqa: E731  the heads of a group, one after another
    dv = torch.matmul(flat(p).transpose(-1, -2), flat(do))
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds.sub_(delta).mul_(p).mul_(s["scale"])
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(flat(ds).transpose(-1, -2), flat(q))
    # queries belong to one sequence, keys may belong to several
    rows = torch.where(has_q, qi, T).reshape(-1)
    dq_all = torch.zeros((T + 1, Hq * D), device=DEV).index_copy_(0, rows, dq.permute(0, 3, 1, 2, 4).reshape(-1, Hq * D))
    is_q = torch.zeros(T + 1, dtype=torch.bool, device=DEV).index_fill_(0, rows, True)[:T, None]
    rows = torch.where(has_k, ki, T).reshape(-1)
    dkv = torch.stack([dk, dv], 1).permute(0, 3, 1, 2, 4).reshape(-1, 2 * Hkv * D)
    dkv_all = torch.zeros((T + 1, 2 * Hkv * D), device=DEV).index_add_(0, rows, dkv)
    is_k = torch.zeros(T + 1, dtype=torch.bool, device=DEV).index_fill_(0, rows, True)[:T, None]
    new = torch.cat([dq_all[:T], dkv_all[:T]], 1).to(torch.bfloat16)
    written = torch.cat([is_q.expand(-1, Hq * D), is_k.expand(-1, 2 * Hkv * D)], 1)
    return torch.where(written, new, s["dqkv"])


def _plain_rope(s):
    c = s["c"]
    T, D, Hq, Hkv = c["T"], c["D"], c["Hq"], c["Hkv"]
    nqk, half = Hq + Hkv, D // 2
    x = s["x"][:, :nqk * D].float().reshape(T, nqk, D)
    d = s["d_out"][:, :nqk * D].float().reshape(T, nqk, D)
    cs = s["cs"][s["pos"].long()].float()
    co, si = cs[:, None, :, 0], cs[:, None, :, 1]
    du = torch.cat([d[..., :half] * co + d[..., half:] * si, d[..., half:] * co - d[..., :half] * si], -1)
    kind = s["mod"].long()
    w = torch.cat([s["w"][0].float()[kind][:, None].expand(-1, Hq, -1), s["w"][1].float()[kind][:, None].expand(-1, Hkv, -1)], 1)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * rstd
    g = du * w
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    per = du * xh
    per = torch.stack([per[:, :Hq].sum(1), per[:, Hq:].sum(1)], 0)  # [q, k][T][D]
    gen = kind.to(torch.float32)[None, :, None]
    dw = torch.stack([(per * (1 - gen)).sum(1), (per * gen).sum(1)], 1)
    return {"dx": torch.cat([dx.reshape(T, nqk * D).to(torch.bfloat16), s["d_out"][:, nqk * D:]], 1), "dw": dw}


def _philox(block_lo, block_hi, tensor, step, seed):
    """Philox4x32-7 of the counter (block_lo, block_hi, tensor, step): four 32-bit words as int64 arrays."""
    low = 0xFFFFFFFF
    x = [block_lo, block_hi, tensor, torch.full_like(block_lo, step)]
    k0, k1 = seed & low, seed >> 32 & low

    def half(a, by):  # high and low words of a * by, exact in 64 bits whose sign wraps
        y = a * by
        return (y >> 32) & low, y & low

    for _ in range(7):
        h0, l0 = half(x[0], 0xD2511F53)
        h1, l1 = half(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return x


def _random_words(s):
    """One 32-bit word for each element of the states, [blocks][256]."""
    at = (s["inner"] * (BLOCK // 4))[:, None] + torch.arange(BLOCK // 4, device=DEV)[None, :]
    tensor = s["tensor"][:, None].expand_as(at)
    return torch.stack(_philox(at & 0xFFFFFFFF, at >> 32, tensor, HYPER["step"], SEED), -1).reshape(-1, BLOCK)


def _quantise(x, up):
    """fp32 blocks to (e4m3, scales): up in [0, 2^20) is added below the last kept bit before the rest is cut off."""
    a = x.abs().amax(-1)
    fine, zero = torch.isfinite(a), torch.zeros_like(a)
    some = a >= 2.0 ** -100
    scale = torch.where(fine, torch.where(some, a / 448.0, zero), torch.full_like(a, float("nan")))
    y = x * torch.where(fine & some, 448.0 / a, zero)[:, None]
    y = torch.where(fine[:, None], y, torch.zeros_like(y))
    z = y.abs().clamp(max=448.0)
    lift = torch.where(z < 2.0 ** -6, torch.full_like(z, 2.0 ** -6), torch.zeros_like(z))  # subnormals keep 2^-9 steps
    z = ((z + lift).view(torch.int32) + up & ~0xFFFFF).view(torch.float32) - lift
    return torch.copysign(z, y).to(torch.float8_e4m3fn), scale


def _plain_adamw(s):
    c, h = s["c"], s["hyper"]
    lr, b1, c1, b2, c2, lb1, rb2, eps, gs = (h[i] for i in range(9))
    g = s["g"].float() * gs
    if c["state"] == "fp32":
        m, v = s["m"], s["v"]
    else:
        m = s["m"].float() * s["scales"][:, :1]
        v = (s["v"].float() * s["scales"][:, 1:]).square()
    m = m * b1 + g * c1
    v = v * b2 + g * g * c2
    r = v.sqrt()
    u = m * lb1 / (r * rb2 + eps)
    s["p"].sub_(u + s["p"] * (lr * s["decay"])[:, None])
    if c["p16"]:
        s["p16"].copy_(s["p"])
    if c["state"] == "fp32":
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        word = _random_words(s)
        code, scale = _quantise(m, ((word & 0xFFFF) << 4).int())
        s["m"].view(torch.uint8).copy_(code.view(torch.uint8))
        s["scales"][:, 0] = scale
        code, scale = _quantise(r, ((word >> 16) << 4).int())
        code = code.view(torch.uint8)
        code = torch.where((code == 0) & (v > 0) & (scale > 0)[:, None], torch.ones_like(code), code)
        s["v"].view(torch.uint8).copy_(code)
        s["scales"][:, 1] = scale
    return _outputs_of_adamw(s)


def _outputs_of_adamw(s):
    return {name: s[name] for name in ("p", "p16", "m", "v", "scales") if s[name] is not None}


def run(state):
    s = state
    c = s["c"]
    if own:
        import mixture_transformers_token_gb300 as mot

        if c["op"] == "attn":
            return mot.mot_joint_attention_backward(s["dout"], s["qkv"], s["out"], s["lse"], s["seqs"], c["Hq"], c["Hkv"],
                                                    c["D"], s["ws"], scale=s["scale"], dqkv=s["dqkv"])
        if c["op"] == "rope":
            dx, dw = mot.mot_qk_norm_rope_backward(s["d_out"], s["x"], s["w"][0], s["w"][1], s["pos"], s["cs"], c["Hq"],
                                                   c["Hkv"], c["D"], EPS, s["ws"], dx=s["dx"], dw=s["dw"],
                                                   scratch=s["scratch"])
            return {"dx": dx, "dw": dw}
        mot.mot_adamw_step(s["plan"], s["hyper"], s["ws"], seed=SEED)
        return _outputs_of_adamw(s)
    return {"attn": _plain_attn, "rope": _plain_rope, "adamw": _plain_adamw}[c["op"]](s)


# ---------------------------------------------------------------------------
# the same outputs from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_attn(s):
    """The gradient by differentiating the forward definition, a sequence and KV head at a time."""
    c = s["c"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    sums = torch.zeros(s["qkv"].shape, dtype=torch.float64, device=DEV)
    written = torch.zeros(s["qkv"].shape, dtype=torch.bool, device=DEV)
    for q0, k0, nq, nk, nc in s["seqs"].tolist():
        see = torch.ones((nq, nk), dtype=torch.bool, device=DEV)
        see[:nc] = torch.tril(see[:nc], diagonal=nk - nq)
        for g in range(Hkv):
            at = {"q": (slice(q0, q0 + nq), slice(g * G * D, (g + 1) * G * D)),
                  "k": (slice(k0, k0 + nk), slice((Hq + g) * D, (Hq + g + 1) * D)),
                  "v": (slice(k0, k0 + nk), slice((Hq + Hkv + g) * D, (Hq + Hkv + g + 1) * D))}
            leaf = {n: s["qkv"][i].double().requires_grad_() for n, i in at.items()}
            x = torch.einsum("qgd,kd->gqk", leaf["q"].reshape(nq, G, D), leaf["k"]) / math.sqrt(D)
            w = torch.softmax(x.masked_fill(~see, float("-inf")), -1)
            o = torch.einsum("gqk,kd->qgd", w, leaf["v"]).reshape(nq, G * D)
            o.backward(s["dout"][at["q"]].double())
            for n, i in at.items():
                sums[i] += leaf[n].grad
                written[i] = True
            del leaf, x, w, o
    return torch.where(written, sums, s["dqkv"].double())


def _exact_rope(s):
    """The gradient by differentiating the forward definition, a slice of rows at a time."""
    c = s["c"]
    T, D, Hq, Hkv = c["T"], c["D"], c["Hq"], c["Hkv"]
    w = torch.stack([x.double() for x in s["w"]]).requires_grad_()  # [q, k][und, gen][D]
    head = torch.tensor([0] * Hq + [1] * Hkv, device=DEV)
    dx = s["d_out"].double()
    for a in range(0, T, 4096):
        b = min(T, a + 4096)
        x = s["x"][a:b, :(Hq + Hkv) * D].double().reshape(b - a, Hq + Hkv, D).requires_grad_()
        mine = w[head[None, :], s["mod"][a:b].long()[:, None]]
        u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * mine
        z = torch.view_as_complex(torch.stack([u[..., : D // 2], u[..., D // 2:]], -1).contiguous())
        z = z * torch.view_as_complex(s["cs"][s["pos"][a:b].long()].double())[:, None]
        d = dx[a:b, :(Hq + Hkv) * D].reshape(b - a, Hq + Hkv, D)
        (z.real * d[..., : D // 2] + z.imag * d[..., D // 2:]).sum().backward()
        dx[a:b, :(Hq + Hkv) * D] = x.grad.reshape(b - a, -1)
    return {"dx": dx, "dw": w.grad}


def _exact_e4m3(x, up):
    """float64 blocks and up in [0, 1) to (the e4m3 values, the scales): steps of 2^-9 below 2^-6, else of the value's
    own binade; the steps that fit, one more where what is left and up make a whole one."""
    a = x.abs().amax(-1)
    a = torch.where(a < 2.0 ** -100, torch.zeros_like(a), a)
    y = x * torch.where(a > 0, 448.0 / a, a)[:, None]
    b = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6)))
    b = torch.where(torch.exp2(b + 1) <= y.abs(), b + 1, b)
    b = torch.where(torch.exp2(b) > torch.clamp(y.abs(), min=2.0 ** -6), b - 1, b)
    step = torch.exp2(b - 3)
    return torch.clamp(torch.sign(y) * torch.floor(y.abs() / step + up) * step, -448.0, 448.0), a / 448.0


def _exact_adamw(s):
    c, h = s["c"], HYPER
    g = s["g"].double() * h["grad_scale"]
    m, v = s["m"].float().double(), s["v"].float().double()
    if c["state"] != "fp32":
        m, v = m * s["scales"][:, :1].double(), (v * s["scales"][:, 1:].double()) ** 2
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    del g
    p = s["p"].double()
    hat = m / (1 - h["beta1"] ** h["step"]) / (torch.sqrt(v / (1 - h["beta2"] ** h["step"])) + h["eps"])
    p = p - h["lr"] * (hat + s["decay"].double()[:, None] * p)
    del hat
    out = {"p": p}
    if c["p16"]:
        out["p16"] = p
    if c["state"] == "fp32":
        return {**out, "m": m, "v": v}
    word = _random_words(s)
    scales = torch.empty(s["scales"].shape, dtype=torch.float64, device=DEV)
    out["m"], scales[:, 0] = _exact_e4m3(m, (word & 0xFFFF).double() / 65536)
    code, scales[:, 1] = _exact_e4m3(v.sqrt(), (word >> 16).double() / 65536)
    out["v"] = torch.where((code == 0) & (v > 0) & (scales[:, 1:] > 0), torch.full_like(code, 2.0 ** -9), code)
    out["scales"] = scales
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "adamw": _exact_adamw}[s["c"]["op"]](s)
