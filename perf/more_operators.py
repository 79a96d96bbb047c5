"""Cases of the 4-bit key/value cache and the attention that reads it, with their plain forms.

``own`` false: ``run`` computes an operator from elementary torch operations in
float32 (whatever the inputs' type), rounded once at the end.  ``own`` true:
``run`` makes the library's calls.  The operators:

* ``store``   new tokens' keys and values [B,Hkv,Nn,d] into a paged cache that
  holds them in 4 bits, and back as the values they stand for (what a prefill
  attends to, so that it sees what decoding will see).
* ``read``    the cached tokens of a batch as dense keys and values [B,Hkv,N,d],
  zeros past a sequence's length.
* ``attend``  attention of each sequence's last Nq tokens, q [B,Hq,Nq,d], over
  the cache: query t sees its sequence's keys up to its own, query head h uses
  key/value head h / (Hq / Hkv); with the log of the sum of exponentials.

A group of 16 neighbouring entries of a token's key (or value) of one head has
one scale: s = amax / 6 rounded to e4m3 (4 exponent and 3 mantissa bits, at
most 448); an entry x is held as the nearest e2m1 code to x / s, that is one of
+-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code.  All of that applies to
x / k_scale (x / v_scale); a code stands for code * s * k_scale.  The cache is
uint8 [pages, Hkv, page, 9 d / 8]; of a page and head every 16 tokens are 18 d
bytes: key codes [d/16][16 tokens][8], key scales [16 tokens][d/16], value codes
[d][8] (of a channel's 16 tokens), value scales [d/16][16 tokens]; of two codes
in a byte the first is in the low half.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decoding step of a serving batch writes one token a sequence: latency
        {"name": "store_step", "op": "store", "dtype": "bf16", "B": 64, "Hkv": 8, "Nn": 1, "lo": 500, "hi": 8200, "page": 64, "d": 128},
        # a batch of prompts of unequal lengths is prefilled
        {"name": "store_prompts", "op": "store", "dtype": "bf16", "B": 8, "Hkv": 8, "Nn": 8192, "lo": 900, "hi": 8192, "page": 64, "d": 128},
        # float32 evaluation of a small model, a chunk after a past, odd sizes
        {"name": "store_f32", "op": "store", "dtype": "f32", "B": 6, "Hkv": 5, "Nn": 1333, "lo": 1333, "hi": 3001, "page": 48, "d": 80},
        # two short conversations of a small model move to another engine
        {"name": "read_small", "op": "read", "dtype": "bf16", "B": 2, "Hkv": 4, "lo": 130, "hi": 777, "page": 16, "d": 64},
        # long contexts read back for a dense pass over them
        {"name": "read_long", "op": "read", "dtype": "bf16", "B": 8, "Hkv": 8, "lo": 3000, "hi": 16384, "page": 64, "d": 128},
        # one user's next token; latency
        {"name": "attend_one", "op": "attend", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 1, "lo": 1000, "hi": 1000, "page": 64, "d": 128},
        # a serving batch of ragged conversations
        {"name": "attend_serving", "op": "attend", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "lo": 500, "hi": 8200, "page": 64, "d": 128},
        # eight query heads a key head, three drafted tokens beside the last one, small pages
        {"name": "attend_drafts", "op": "attend", "dtype": "bf16", "B": 32, "Hq": 64, "Hkv": 8, "Nq": 4, "lo": 1000, "hi": 16384, "page": 16, "d": 128},
        # long documents, the largest cache
        {"name": "attend_long", "op": "attend", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "lo": 4096, "hi": 32768, "page": 128, "d": 128},
        # a small model with a key head for every query head, odd lengths, one sequence empty
        {"name": "attend_heads", "op": "attend", "dtype": "bf16", "B": 17, "Hq": 16, "Hkv": 16, "Nq": 1, "lo": 0, "hi": 4001, "page": 32, "d": 64},
        # one chunk of a long prompt against what is cached of it
        {"name": "attend_chunk", "op": "attend", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 512, "lo": 8704, "hi": 8704, "page": 64, "d": 128},
        # float32 evaluation, odd sizes
        {"name": "attend_f32", "op": "attend", "dtype": "f32", "B": 6, "Hq": 32, "Hkv": 8, "Nq": 3, "lo": 0, "hi": 3001, "page": 16, "d": 96},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["store", "read", "attend", "attend", "attend"])
    f32 = rng.random() < 0.25
    c = {"op": op, "dtype": "f32" if f32 else "bf16", "Hkv": rng.choice([1, 2, 3, 4, 8, 16]), "page": rng.choice([16, 32, 48, 64, 128])}
    if op == "attend":
        hi = _log(rng, 20, 3000 if f32 else 32768)
        c |= {"B": _log(rng, 1, 8 if f32 else 64), "Hq": c["Hkv"] * rng.choice([1, 2, 4, 5, 8]), "Nq": rng.choice([1, 1, 1, 2, 3, 4, 7, 61]),
              "lo": hi // rng.choice([1, 2, 16]), "hi": hi, "d": rng.choice([64, 96, 128])}
        return c
    hi = _log(rng, 20, 3000 if f32 else 16384)
    c |= {"B": _log(rng, 1, 8 if f32 else 64), "lo": hi // rng.choice([1, 2, 16]), "hi": hi, "d": 16 * rng.randint(2, 8) if f32 else rng.choice([64, 80, 96, 128])}
    if op == "store":
        # either a few new tokens after what was there, or whole prompts of unequal lengths
        c["Nn"] = hi if rng.random() < 0.5 else rng.randint(1, max(1, min(c["lo"], 9)))
    return c


def draw(rng):
    largest = {}  # of each operator and type
    for c in listed():
        w = work(c)
        k = (c["op"], c["dtype"])
        largest[k] = {n: max(w[n], largest.get(k, w)[n]) for n in w}
    largest["read", "f32"] = {"bytes": 5.0e7, "flops": 5.0e7}
    while True:
        c = _drawn(rng)
        w, most = work(c), largest[c["op"], c["dtype"]]
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _lens(case):
    """The lengths of the batch's sequences: spread between the case's bounds, out of order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    step = 3 if B % 5 == 0 else 5
    return [hi if B == 1 else lo + (hi - lo) * ((step * i + 2) % B) // (B - 1) for i in range(B)]


def _new(case):
    """How many tokens of each sequence a ``store`` writes: whole prompts where Nn is their longest, else the last Nn."""
    return [min(n, case["Nn"]) for n in _lens(case)]


def _pairs(n_q, n_k):
    """Query-key pairs of n_q new tokens over n_k keys, each token seeing the keys up to its own."""
    first = n_k - n_q + 1
    if first >= 0:
        return n_q * first + n_q * (n_q - 1) // 2
    return n_k * (n_k + 1) // 2


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, Hkv, d, lens = case["B"], case["Hkv"], case["d"], _lens(case)
    tables = 4 * (B + sum(-(-n // case["page"]) for n in lens))
    if case["op"] == "store":
        n = Hkv * sum(_new(case))  # inputs read, the cache written and read, values written, to the batch's width
        return {"bytes": n * (2 * e * d + 2 * (9 * d // 8)) + B * Hkv * case["Nn"] * 2 * e * d + tables, "flops": 8 * n * d}
    if case["op"] == "read":
        return {"bytes": Hkv * (sum(lens) * (9 * d // 8) + B * max(lens) * 2 * e * d) + tables, "flops": 4 * Hkv * sum(lens) * d}
    Hq, Nq = case["Hq"], case["Nq"]
    rows = B * Hq * Nq
    return {"bytes": rows * (2 * e * d + 4) + Hkv * sum(lens) * (9 * d // 8) + tables,
            "flops": 4 * d * Hq * sum(_pairs(Nq, n) for n in lens)}


# ---------------------------------------------------------------- the cache's format, in elementary operations

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x, scale):
    """Codes (uint8 0..15) and scales (e4m3, as bytes [..., d/16]) of x [..., d]."""
    g = (x.float() / scale).unflatten(-1, (-1, 16))
    s = (g.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = g.abs() / s.float()[..., None]
    code = torch.zeros_like(t, dtype=torch.uint8)
    for i, (a, b) in enumerate(zip(LEVELS, LEVELS[1:])):  # past the middle of two neighbours; on it, to the even code
        code += (t > (a + b) / 2) if i % 2 == 0 else (t >= (a + b) / 2)
    code += (g < 0) * (code > 0) * 8
    return code.flatten(-2), s.view(torch.uint8)


def _bytes(codes):
    """Two codes a byte, along the last dimension."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _codes(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def _levels(codes):
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    return torch.index_select(table, 0, codes.flatten().int()).view(codes.shape)


def _pack(k, v, k_scale, v_scale):
    """Cache bytes [..., n/16, 18 d] of k and v [..., n, d], n a multiple of 16."""
    d = k.shape[-1]
    kc, ks = _quantise(k.unflatten(-2, (-1, 16)), k_scale)  # [..., blocks, 16, d], [..., blocks, 16, d/16]
    vc, vs = _quantise(v.unflatten(-2, (-1, 16)), v_scale)
    kc = _bytes(kc.unflatten(-1, (d // 16, 16))).transpose(-3, -2)  # [..., d/16, 16 tokens, 8]
    return torch.cat([kc.flatten(-3), ks.flatten(-2), _bytes(vc.transpose(-1, -2)).flatten(-2), vs.transpose(-1, -2).flatten(-2)], -1)


def _unpack(blocks, d, k_scale, v_scale):
    """float32 k and v [..., n, d] of cache bytes [..., n/16, 18 d]."""
    kc, ks, vc, vs = blocks.split([8 * d, d, 8 * d, d], -1)
    ks = ks.unflatten(-1, (16, d // 16)).contiguous().view(torch.float8_e4m3fn).float()  # [..., 16, d/16]
    vs = vs.unflatten(-1, (d // 16, 16)).contiguous().view(torch.float8_e4m3fn).float()  # [..., d/16, 16]
    k = _levels(_codes(kc.unflatten(-1, (d // 16, 16, 8)))).transpose(-3, -2) * ks[..., None]  # [..., 16, d/16, 16]
    v = _levels(_codes(vc.unflatten(-1, (d // 16, 16, 8)))) * vs[..., None, :]  # [..., d/16, 16 channels, 16 tokens]
    k = (k * k_scale).flatten(-2)
    v = (v * v_scale).flatten(-3, -2).transpose(-1, -2)
    return k.flatten(-3, -2), v.flatten(-3, -2)


def _dense(s, seqs, n):
    """float32 keys and values [len(seqs), Hkv, n, d] of some sequences, zeros past their lengths."""
    case = s["case"]
    d, Hkv = case["d"], case["Hkv"]
    pages = s["table"][seqs, : -(-n // case["page"])].long()
    blocks = s["cache"][pages].transpose(1, 2).reshape(len(seqs), Hkv, -1, 18 * d)[:, :, : -(-n // 16)]
    k, v = _unpack(blocks, d, s["k_scale"], s["v_scale"])
    held = (torch.arange(n, device=k.device) < s["lens"][seqs, None])[:, None, :, None]
    return torch.where(held, k[:, :, :n], 0.0), torch.where(held, v[:, :, :n], 0.0)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]
    B, Hkv, page, d = (case[n] for n in ("B", "Hkv", "page", "d"))
    lens = _lens(case)
    held = [-(-n // page) for n in lens]
    pages, wide = sum(held) + 3, max(1, max(held))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def keys(*shape):  # a few channels are larger than the others, as they are in keys
        return normal(*shape) * torch.exp(0.7 * normal(shape[-1]))

    cache = torch.empty((pages, Hkv, page, 9 * d // 8), dtype=torch.uint8, device="cuda")
    k_scale, v_scale = 0.0625, 0.03125
    if case["op"] == "store" and case["Nn"] >= max(lens):
        cache.zero_()
    else:
        some = max(1, (1 << 27) // (Hkv * page * d))
        for p in range(0, pages, some):
            n = min(some, pages - p)
            cache[p : p + n] = _pack(keys(n, Hkv, page, d), normal(n, Hkv, page, d), k_scale, v_scale).view(n, Hkv, page, 9 * d // 8)
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    mine = torch.tensor([[p < n for p in range(wide)] for n in held], device="cuda")
    table = torch.zeros((B, wide), dtype=torch.int32, device="cuda")
    table[mine] = order[: pages - 3]
    s = {"case": case, "cache": cache, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "n": max(1, max(lens)), "k_scale": k_scale, "v_scale": v_scale}
    if case["op"] == "store":
        Nn = case["Nn"]
        s |= {"k": keys(B, Hkv, Nn, d).to(t), "v": normal(B, Hkv, Nn, d).to(t),
              "new": torch.tensor(_new(case), dtype=torch.int32, device="cuda"), "first": s["lens"] - Nn,
              "k_out": torch.empty((B, Hkv, Nn, d), device="cuda", dtype=t), "v_out": torch.empty((B, Hkv, Nn, d), device="cuda", dtype=t)}
    elif case["op"] == "read":
        s |= {"k_out": torch.empty((B, Hkv, s["n"], d), device="cuda", dtype=t), "v_out": torch.empty((B, Hkv, s["n"], d), device="cuda", dtype=t)}
    else:
        shape = (B, case["Hq"], case["Nq"], d)
        s |= {"q": normal(*shape).to(t), "scale": 1.0 / math.sqrt(d), "o": torch.empty(shape, device="cuda", dtype=t), "lse": torch.empty(shape[:3], device="cuda")}
    return s


# ---------------------------------------------------------------- the operators

def _store(s):
    Nn, t = s["case"]["Nn"], s["k"].dtype
    written = (torch.arange(Nn, device="cuda")[None, :] >= Nn - s["new"][:, None])[:, None, :, None]
    out = []
    for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        codes, scales = _quantise(x, scale)
        value = (_levels(codes).unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None] * scale).flatten(-2)
        out.append(torch.where(written, value, 0.0).to(t))
    return tuple(out)


def _read(s):
    k, v, t = s["k_out"], s["v_out"], s["k_out"].dtype
    some = max(1, (1 << 28) // (k.shape[1] * k.shape[2] * k.shape[3]))
    for b in range(0, len(k), some):
        x, y = _dense(s, torch.arange(b, min(b + some, len(k)), device="cuda"), s["n"])
        k[b : b + some], v[b : b + some] = x.to(t), y.to(t)
    return k, v


def _attend(s):
    q = s["q"].float()
    B, Hq, Nq, d = q.shape
    Hkv, n = s["case"]["Hkv"], s["n"]
    G = Hq // Hkv
    t = torch.arange(Nq, device=q.device).repeat(G)
    some = max(1, (1 << 28) // (Hkv * n * d))
    for b in range(0, B, some):
        seqs = torch.arange(b, min(b + some, B), device=q.device)
        k, v = _dense(s, seqs, n)
        x = torch.matmul(q[seqs].view(-1, Hkv, G * Nq, d), k.transpose(2, 3)) * s["scale"]
        sees = torch.arange(n, device=q.device) < (s["lens"][seqs, None] - (Nq - 1 - t))[..., None]
        x = torch.where(sees[:, None], x, -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
        s["o"][seqs] = o.view(-1, Hq, Nq, d).to(s["o"].dtype)
        s["lse"][seqs] = (m + torch.log(l)).view(-1, Hq, Nq)
    return s["o"], s["lse"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from exact_tiled_attention_02_gb300 import binding as fa
        scales = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "store":
            fa.fa_cache_fp4_write(s["k"], s["v"], s["cache"], s["lens"], block_table=s["table"], n_new=s["new"], **scales)
            return fa.fa_cache_fp4_read(s["cache"], s["lens"], s["case"]["Nn"], block_table=s["table"], first=s["first"], k=s["k_out"], v=s["v_out"], **scales)
        if op == "read":
            return fa.fa_cache_fp4_read(s["cache"], s["lens"], s["n"], block_table=s["table"], k=s["k_out"], v=s["v_out"], **scales)
        return fa.fa_fwd_cache_fp4(s["q"], s["cache"], s["lens"], scale=s["scale"], block_table=s["table"], o=s["o"], lse=s["lse"], **scales)
    return _store(s) if op == "store" else _read(s) if op == "read" else _attend(s)


# ---------------------------------------------------------------- the definition in 64 bits

def _nearest(x, values):
    """The nearest of ascending float64 ``values`` to each x, ties to the even index."""
    i = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    below, above = values[i - 1], values[i]
    up = (x - below > above - x) | ((x - below == above - x) & (i % 2 == 0))
    return torch.where(up, above, below)


def _e4m3():
    """The non-negative values of e4m3, ascending."""
    return torch.tensor([m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1], dtype=torch.float64, device="cuda")


def _exact_store(x, scale):
    g = x.double().unflatten(-1, (-1, 16)) / scale
    s = _nearest(g.abs().amax(-1, keepdim=True) / 6, _e4m3())
    m = _nearest(torch.where(s > 0, g.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g)), torch.tensor(LEVELS, dtype=torch.float64, device="cuda"))
    return (torch.copysign(m, g) * s * scale).flatten(-2)


def _exact_sequence(s, b):
    """float64 keys and values [Hkv, n, d] of sequence b."""
    case = s["case"]
    d, n, page = case["d"], _lens(case)[b], case["page"]
    e4m3 = _e4m3()
    e4m3 = torch.cat([e4m3, e4m3[-1:] * math.nan, -e4m3, e4m3[-1:] * math.nan])
    e2m1 = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    e2m1 = torch.cat([e2m1, -e2m1])
    raw = s["cache"][s["table"][b, : -(-n // page)].long()].permute(1, 0, 2, 3).reshape(case["Hkv"], -1, 18 * d)
    token = torch.arange(n, device="cuda")[:, None]
    c = torch.arange(d, device="cuda")[None, :]
    j, blk = token % 16, raw[:, (token // 16)[:, 0]].int()  # each token's block

    def entry(at, nibble, scale_at, scale):  # byte positions within the block [n, d]
        byte = torch.gather(blk, 2, at.expand(n, d)[None].expand(case["Hkv"], -1, -1))
        sc = torch.gather(blk, 2, scale_at.expand(n, d)[None].expand(case["Hkv"], -1, -1))
        return e2m1[((byte >> (4 * nibble)) & 15).long()] * e4m3[sc.long()] * scale

    k = entry((c // 16) * 128 + j * 8 + (c % 16) // 2, (c % 2).int(), 8 * d + j * (d // 16) + c // 16, s["k_scale"])
    v = entry(9 * d + c * 8 + j // 2, (j % 2).int(), 17 * d + (c // 16) * 16 + j, s["v_scale"])
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "store":
        Nn, out = case["Nn"], []
        for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            y = _exact_store(x, scale)
            for b, n in enumerate(_new(case)):
                y[b, :, : Nn - n] = 0
            out.append(y)
        return tuple(out)
    if case["op"] == "read":
        if work(case)["bytes"] > 1.5e9:
            return None
        k, v = (torch.zeros((B, Hkv, s["n"], d), dtype=torch.float64, device="cuda") for _ in range(2))
        for b, n in enumerate(_lens(case)):
            if n:
                k[b, :, :n], v[b, :, :n] = _exact_sequence(s, b)
        return k, v
    Hq, Nq = case["Hq"], case["Nq"]
    o = torch.zeros((B, Hq, Nq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        if not n:
            continue
        k, v = _exact_sequence(s, b)
        sees = torch.arange(n, device="cuda")[None, :] <= n - Nq + torch.arange(Nq, device="cuda")[:, None]
        for h in range(Hkv):
            G = Hq // Hkv
            x = (s["q"][b, h * G : (h + 1) * G].double() @ k[h].T * s["scale"]).masked_fill(~sees, -math.inf)
            total = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(torch.isinf(total), torch.zeros_like(total), total)[..., None])
            o[b, h * G : (h + 1) * G], lse[b, h * G : (h + 1) * G] = w @ v[h], total
    return o, lse
