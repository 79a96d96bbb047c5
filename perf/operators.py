"""Cases of the latent-attention and shared-prefix operators, with their plain forms.

``own`` false: ``run`` computes an operator from elementary torch operations in
float32 (whatever the inputs' type), rounded once at the end.  ``own`` true:
``run`` makes the library call.  The operators:

* ``prefix``   attention of a decoding batch whose sequences share one long
  prefix: q [B,Hq,Nq,d]; prefix keys and values [Hkv,Np,d]; each sequence's own
  keys and values [B,Hkv,Ns,d], of which ``lens[b]`` are valid.
* ``absorbed`` latent attention in its absorbed form: q [B,H,Nq,dc+dr] against
  a paged cache of latent vectors [pages,page,dc+dr]; values are the first dc
  entries of the same vectors.
* ``fwd``, ``train``  latent attention in its expanded form, causal: q
  [B,H,Nq,dn+dr], per-head keys [B,H,Nk,dn], rotary keys shared by the heads
  [B,Nk,dr], values [B,H,Nk,dv]; ``train`` is one forward and backward.

In all of them query t of a sequence's Nq new tokens sees its keys up to its
own, the last query being the last key's.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a short chat behind a system prompt, small model: one token for four users; latency
        {"name": "prefix_small", "op": "prefix", "dtype": "bf16", "B": 4, "Hq": 16, "Hkv": 4, "Nq": 1, "Np": 1000, "Ns": 128, "d": 64},
        # a serving batch behind a long document or few-shot prompt
        {"name": "prefix_serving", "op": "prefix", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "Np": 16384, "Ns": 1024, "d": 128},
        # many samples of one long prompt, four drafted tokens each
        {"name": "prefix_large", "op": "prefix", "dtype": "bf16", "B": 128, "Hq": 32, "Hkv": 8, "Nq": 4, "Np": 32768, "Ns": 2048, "d": 128},
        # float32 evaluation, a head of its own for every query head, odd sizes
        {"name": "prefix_f32", "op": "prefix", "dtype": "f32", "B": 7, "Hq": 8, "Hkv": 8, "Nq": 3, "Np": 2999, "Ns": 333, "d": 80},
        # one user's next token; latency
        {"name": "absorbed_one", "op": "absorbed", "dtype": "bf16", "B": 1, "H": 16, "Nq": 1, "lo": 777, "hi": 777, "page": 64, "dc": 512, "dr": 64},
        # a serving batch of ragged conversations, heads split over eight devices
        {"name": "absorbed_serving", "op": "absorbed", "dtype": "bf16", "B": 64, "H": 16, "Nq": 1, "lo": 500, "hi": 8200, "page": 64, "dc": 512, "dr": 64},
        # every head on one device, two tokens a step (one drafted), long contexts, small pages
        {"name": "absorbed_large", "op": "absorbed", "dtype": "bf16", "B": 64, "H": 128, "Nq": 2, "lo": 1000, "hi": 16384, "page": 16, "dc": 512, "dr": 64},
        # float32 evaluation, small latents, odd sizes
        {"name": "absorbed_f32", "op": "absorbed", "dtype": "f32", "B": 5, "H": 12, "Nq": 1, "lo": 0, "hi": 2047, "page": 24, "dc": 192, "dr": 40},
        # prefill of a prompt
        {"name": "fwd_prefill", "op": "fwd", "dtype": "bf16", "B": 1, "H": 16, "Nq": 8192, "Nk": 8192, "dn": 128, "dr": 64, "dv": 128},
        # one chunk of a prompt against what was prefilled before it, odd lengths
        {"name": "fwd_chunk", "op": "fwd", "dtype": "bf16", "B": 3, "H": 16, "Nq": 500, "Nk": 2777, "dn": 128, "dr": 64, "dv": 128},
        # a training step's attention
        {"name": "train_bf16", "op": "train", "dtype": "bf16", "B": 2, "H": 16, "Nq": 4096, "Nk": 4096, "dn": 128, "dr": 64, "dv": 128},
        # a small model in float32, odd sizes
        {"name": "train_f32", "op": "train", "dtype": "f32", "B": 2, "H": 3, "Nq": 333, "Nk": 333, "dn": 48, "dr": 20, "dv": 40},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["prefix", "prefix", "absorbed", "absorbed", "fwd", "train"])
    f32 = rng.random() < 0.25
    c = {"op": op, "dtype": "f32" if f32 else "bf16"}
    if op == "prefix":
        hkv = rng.choice([1, 2, 4, 8])
        c |= {"B": _log(rng, 1, 16 if f32 else 128), "Hq": hkv * rng.choice([1, 2, 4, 5, 8]), "Hkv": hkv, "Nq": rng.choice([1, 1, 1, 2, 3, 4]),
              "Np": _log(rng, 64, 4000 if f32 else 32768), "Ns": _log(rng, 8, 500 if f32 else 2048), "d": rng.randint(16, 128) if f32 else rng.choice([64, 96, 128])}
    elif op == "absorbed":
        hi = _log(rng, 50, 2500 if f32 else 16384)
        c |= {"B": _log(rng, 1, 8 if f32 else 64), "H": rng.choice([8, 12, 16]) if f32 else rng.choice([16, 20, 32, 64, 128]), "Nq": rng.choice([1, 1, 2, 3]),
              "lo": hi // rng.choice([1, 2, 16]), "hi": hi, "page": rng.choice([16, 32, 48, 64, 128]),
              "dc": rng.randint(32, 256) if f32 else rng.choice([256, 512, 512]), "dr": rng.randint(8, 64) if f32 else 64}
    else:
        nk = _log(rng, 33, (600 if op == "train" else 1500) if f32 else (4096 if op == "train" else 8192))
        nq = nk if op == "train" or rng.random() < 0.5 else max(1, int(nk * rng.uniform(0.05, 1)))
        c |= {"B": rng.choice([1, 2, 3]), "H": rng.choice([2, 3, 8] if f32 else [2, 5, 16]), "Nq": nq, "Nk": nk,
              "dn": rng.randint(16, 64) if f32 else 128, "dr": rng.randint(8, 32) if f32 else 64, "dv": rng.randint(16, 64) if f32 else 128}
    return c


def draw(rng):
    most = {"bf16": 3.0e11, "f32": 4.0e9}  # flops: under those of the largest listed cases
    while True:
        c = _drawn(rng)
        if work(c)["flops"] <= most[c["dtype"]]:
            return c


def _lens(case):
    """The valid lengths of the batch's sequences: spread between the case's bounds, out of order."""
    B = case["B"]
    lo, hi = (case["Ns"] // 2, case["Ns"]) if case["op"] == "prefix" else (case["lo"], case["hi"])
    return [hi if B == 1 else lo + (hi - lo) * ((5 * i + 2) % B) // (B - 1) if B % 5 else lo + (hi - lo) * ((3 * i + 2) % B) // (B - 1) for i in range(B)]


def _pairs(n_q, n_k):
    """Query-key pairs of n_q new tokens over n_k keys, each token seeing the keys up to its own."""
    first = n_k - n_q + 1
    if first >= 0:
        return n_q * first + n_q * (n_q - 1) // 2
    return n_k * (n_k + 1) // 2


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "prefix":
        B, Hq, Hkv, Nq, Np, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "Np", "d"))
        lens = _lens(case)
        rows = B * Hq * Nq
        return {"bytes": e * d * (2 * rows + 2 * Hkv * (Np + sum(lens))) + 4 * rows + 4 * B,
                "flops": 4 * d * Hq * (B * Nq * Np + sum(_pairs(Nq, n) for n in lens))}
    if case["op"] == "absorbed":
        B, H, Nq, dc, dr = (case[k] for k in ("B", "H", "Nq", "dc", "dr"))
        lens = _lens(case)
        rows = B * H * Nq
        return {"bytes": e * (rows * (2 * dc + dr) + sum(lens) * (dc + dr)) + 4 * rows + 4 * B + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 2 * (2 * dc + dr) * H * sum(_pairs(Nq, n) for n in lens)}
    B, H, Nq, Nk, dn, dr, dv = (case[k] for k in ("B", "H", "Nq", "Nk", "dn", "dr", "dv"))
    q, k, v, o = B * H * Nq * (dn + dr), B * H * Nk * dn + B * Nk * dr, B * H * Nk * dv, B * H * Nq * dv
    pairs = B * H * _pairs(Nq, Nk)
    if case["op"] == "fwd":
        return {"bytes": e * (q + k + v + o) + 4 * B * H * Nq, "flops": 2 * pairs * (dn + dr + dv)}
    return {"bytes": e * (2 * (q + k + v) + 2 * o) + 4 * B * H * Nq, "flops": 2 * pairs * ((dn + dr + dv) + 3 * (dn + dr) + 2 * dv)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    s = {"case": case}
    if case["op"] == "prefix":
        B, Hq, Hkv, Nq, Np, Ns, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "Np", "Ns", "d"))
        s |= {"q": normal(B, Hq, Nq, d), "kp": normal(Hkv, Np, d), "vp": normal(Hkv, Np, d), "k": normal(B, Hkv, Ns, d), "v": normal(B, Hkv, Ns, d)}
        s |= {"lens": torch.tensor(_lens(case), dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(d)}
        s |= {"o": torch.empty_like(s["q"]), "lse": torch.empty((B, Hq, Nq), device="cuda")}
    elif case["op"] == "absorbed":
        B, H, Nq, page, dc, dr = (case[k] for k in ("B", "H", "Nq", "page", "dc", "dr"))
        lens = _lens(case)
        wide = max(1, -(-max(lens) // page))
        pages = sum(-(-n // page) for n in lens) + 3
        order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        held = torch.tensor([[p < -(-n // page) for p in range(wide)] for n in lens], device="cuda")
        table = torch.zeros((B, wide), dtype=torch.int32, device="cuda")
        table[held] = order[: pages - 3]
        s |= {"q": normal(B, H, Nq, dc + dr), "cache": normal(pages, page, dc + dr), "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
        s |= {"scale": 1.0 / math.sqrt(192.0), "o": torch.empty((B, H, Nq, dc), device="cuda", dtype=t), "lse": torch.empty((B, H, Nq), device="cuda")}
    else:
        B, H, Nq, Nk, dn, dr, dv = (case[k] for k in ("B", "H", "Nq", "Nk", "dn", "dr", "dv"))
        s |= {"q": normal(B, H, Nq, dn + dr), "kn": normal(B, H, Nk, dn), "kr": normal(B, Nk, dr), "v": normal(B, H, Nk, dv)}
        s |= {"scale": 1.0 / math.sqrt(dn + dr), "do": normal(B, H, Nq, dv) if case["op"] == "train" else None}
    return s


def _softmax(s):
    """exp(s - max), its row sums and the log of the sums of exp(s); a row of -inf gives zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    n = p.sum(-1, keepdim=True)
    return p, torch.where(n == 0, torch.ones_like(n), n), (m + torch.log(n))[..., 0]


def _prefix(s):
    q, kp, vp, k, v = (s[n].float() for n in ("q", "kp", "vp", "k", "v"))
    B, Hq, Nq, d = q.shape
    Hkv, Np = kp.shape[:2]
    Ns, G = k.shape[2], Hq // Hkv
    rows = q.view(B, Hkv, G * Nq, d)
    far = torch.matmul(rows.transpose(0, 1).reshape(Hkv, B * G * Nq, d), kp.transpose(1, 2)).view(Hkv, B, G * Nq, Np).transpose(0, 1)
    near = torch.matmul(rows, k.transpose(2, 3))
    t = torch.arange(Nq, device=q.device).repeat(G)
    sees = torch.arange(Ns, device=q.device)[None, None, :] < (s["lens"][:, None] - (Nq - 1 - t)[None, :])[:, :, None]
    near = torch.where(sees[:, None], near, torch.full_like(near, -math.inf))
    p, n, lse = _softmax(torch.cat([far, near], -1) * s["scale"])
    o = torch.matmul(p[..., :Np].transpose(0, 1).reshape(Hkv, B * G * Nq, Np), vp).view(Hkv, B, G * Nq, d).transpose(0, 1) + torch.matmul(p[..., Np:], v)
    return (o / n).reshape(B, Hq, Nq, d).to(s["q"].dtype), lse.reshape(B, Hq, Nq)


def _absorbed(s):
    q, dc = s["q"].float(), s["case"]["dc"]
    B, H, Nq, dk = q.shape
    c = s["cache"][s["table"].long()].float().view(B, -1, dk)
    x = torch.matmul(q.view(B, H * Nq, dk), c.transpose(1, 2)) * s["scale"]
    t = torch.arange(Nq, device=q.device).repeat(H)
    sees = torch.arange(c.shape[1], device=q.device)[None, None, :] < (s["lens"][:, None] - (Nq - 1 - t)[None, :])[:, :, None]
    p, n, lse = _softmax(torch.where(sees, x, torch.full_like(x, -math.inf)))
    return (torch.matmul(p, c[..., :dc]) / n).view(B, H, Nq, dc).to(s["q"].dtype), lse.view(B, H, Nq)


def _expanded(s, train):
    q, kn, kr, v = (s[n].float() for n in ("q", "kn", "kr", "v"))
    B, H, Nq, _ = q.shape
    Nk, dn = kn.shape[2:]
    t = s["q"].dtype
    x = (torch.matmul(q[..., :dn], kn.transpose(2, 3)) + torch.matmul(q[..., dn:], kr[:, None].transpose(2, 3))) * s["scale"]
    sees = torch.arange(Nk, device=q.device)[None, :] <= torch.arange(Nq, device=q.device)[:, None] + (Nk - Nq)
    p, n, lse = _softmax(torch.where(sees, x, torch.full_like(x, -math.inf)))
    p = p / n
    o = torch.matmul(p, v)
    if not train:
        return o.to(t), lse
    do = s["do"].float()
    ds = p * (torch.matmul(do, v.transpose(2, 3)) - (do * o).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.cat([torch.matmul(ds, kn), torch.matmul(ds, kr[:, None])], -1)
    dkn = torch.matmul(ds.transpose(2, 3), q[..., :dn])
    dkr = torch.matmul(ds.transpose(2, 3), q[..., dn:]).sum(1)
    dv = torch.matmul(p.transpose(2, 3), do)
    return o.to(t), lse, dq.to(t), dkn.to(t), dkr.to(t), dv.to(t)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from exact_tiled_attention_02_gb300 import binding as fa
        if op == "prefix":
            return fa.fa_fwd_shared_prefix(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], scale=s["scale"], o=s["o"], lse=s["lse"])
        if op == "absorbed":
            return fa.fa_fwd_latent_absorbed(s["q"], s["cache"], s["lens"], block_table=s["table"], dc=s["case"]["dc"], scale=s["scale"], o=s["o"], lse=s["lse"])
        o, lse = fa.fa_fwd_latent(s["q"], s["kn"], s["kr"], s["v"], scale=s["scale"], causal=True)
        if op == "fwd":
            return o, lse
        return (o, lse) + fa.fa_bwd_latent(s["q"], s["kn"], s["kr"], s["v"], o, lse, s["do"], scale=s["scale"], causal=True)
    if op == "prefix":
        return _prefix(s)
    if op == "absorbed":
        return _absorbed(s)
    return _expanded(s, op == "train")


def _exact_rows(q, keys, values, scale, sees):
    """softmax(q keys^T scale) values over the keys that a row sees, and the log of the sum of exponentials; all float64."""
    x = (q @ keys.transpose(-1, -2)) * scale
    x = x.masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return w @ values, lse


def exact(case, seed):
    s = prepare(case, seed)
    dev = s["q"].device
    if case["op"] in ("prefix", "absorbed"):
        q = s["q"].double()
        outs, sums = [], []
        for b, n in enumerate(_lens(case)):  # one sequence at a time, over its own keys only
            Nq = q.shape[2]
            if case["op"] == "prefix":
                G, Np = case["Hq"] // case["Hkv"], case["Np"]
                keys = torch.cat([s["kp"], s["k"][b, :, :n]], 1).double().repeat_interleave(G, 0)
                values = torch.cat([s["vp"], s["v"][b, :, :n]], 1).double().repeat_interleave(G, 0)
            else:
                Np = 0
                pages = s["table"][b, : -(-n // case["page"])].long()
                keys = s["cache"][pages].reshape(-1, q.shape[-1])[:n].double()[None]
                values = keys[..., : case["dc"]]
            place = torch.arange(Np + n, device=dev)[None, :]
            sees = (place < Np) | (place - Np <= n - Nq + torch.arange(Nq, device=dev)[:, None])
            if Np + n == 0:
                o, lse = torch.zeros((q.shape[1], Nq, values.shape[-1]), dtype=torch.float64, device=dev), torch.full((q.shape[1], Nq), -math.inf, dtype=torch.float64, device=dev)
            else:
                o, lse = _exact_rows(q[b], keys, values, s["scale"], sees)
            outs.append(o)
            sums.append(lse)
        return torch.stack(outs), torch.stack(sums)
    train = case["op"] == "train"
    leaf = [s[n].double().requires_grad_(train) for n in ("q", "kn", "kr", "v")]
    q, kn, kr, v = leaf
    keys = torch.cat([kn, kr[:, None].expand(-1, kn.shape[1], -1, -1)], -1)
    Nq, Nk = q.shape[2], kn.shape[2]
    sees = torch.ones((Nq, Nk), dtype=torch.bool, device=dev).tril(Nk - Nq)
    if not train:
        return _exact_rows(q, keys, v, s["scale"], sees)
    o, lse = _exact_rows(q, keys, v, s["scale"], sees)
    grads = torch.autograd.grad(o, leaf, s["do"].double())
    return (o.detach(), lse.detach()) + tuple(grads)
