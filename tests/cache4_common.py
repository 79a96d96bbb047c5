"""Inputs and error bounds of the 4-bit cache's GPU tests."""

import numpy as np

import oracle
from tests import seq_bounds as sb


def random_cache(rng, pages, Hkv, page, d):
    """Blocks of random codes and scales (between 1/8 and 4, some zero), as bytes."""
    blocks = rng.integers(0, 256, (pages, Hkv, page // 16, 18 * d)).astype(np.uint8)
    scales = rng.integers(0x20, 0x48, (pages, Hkv, page // 16, 2, d)).astype(np.uint8)
    scales[rng.random(scales.shape) < 0.02] = 0
    blocks[..., 8 * d:9 * d], blocks[..., 17 * d:] = scales[..., 0, :], scales[..., 1, :]
    return blocks.reshape(pages, Hkv, page, 9 * d // 8)


def place(rng, B, max_pages, lens, page, spare=2):
    """A block table over shuffled pages (entries past a length are out of range), and the number of pages."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = list(rng.permutation(pages))
    table = np.full((B, max_pages), -7, dtype=np.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    return table, pages


def poison(cache, table, lens, page, d):
    """Bytes at positions that no length covers: NaN scales and every code."""
    cache = cache.reshape(*cache.shape[:2], page // 16, 18 * d)
    held = {int(table[b, i]) for b, n in enumerate(lens) for i in range(-(-n // page))}
    for p in range(cache.shape[0]):
        if p not in held:
            cache[p] = 0xFF
    for b, n in enumerate(lens):
        if n % page == 0:
            continue
        pg, first = cache[table[b, n // page]], n % page
        for blk in range(first // 16, page // 16):
            for h in range(cache.shape[1]):
                kc, ks, vc, vs = (x.copy() for x in oracle.cache4_unpack(pg[h, blk], d))
                t = max(first - 16 * blk, 0)
                kc[t:], vc[t:], ks[t:], vs[t:] = 15, 15, 0x7F, 0xFF
                pg[h, blk] = oracle.cache4_pack(kc, ks, vc, vs)


def dense(cache, table, b, n, d, page, k_scale, v_scale):
    """float64 keys and values [Hkv, n, d] of a sequence."""
    Hkv = cache.shape[1]
    blocks = cache.reshape(cache.shape[0], Hkv, page // 16, 18 * d)
    out = np.zeros((2, Hkv, -(-n // 16) * 16, d))
    for i in range(-(-n // 16)):
        pg = b if table is None else int(table[b, i * 16 // page])
        if not 0 <= pg < cache.shape[0]:
            continue
        for h in range(Hkv):
            kc, ks, vc, vs = oracle.cache4_unpack(blocks[pg, h, i % (page // 16)], d)
            out[0, h, 16 * i:16 * i + 16] = oracle.cache4_values(kc, ks, k_scale)
            out[1, h, 16 * i:16 * i + 16] = oracle.cache4_values(vc, vs, v_scale)
    return out[0, :, :n], out[1, :, :n]


def forward(q, k, v, scale, dtype):
    """(O, lse, tolerance of O, tolerance of lse) of a sequence's new tokens q [Hq, Nq, d] over k, v [Hkv, n, d].

    K, V = code * scale * tensor's scale; code * scale is exact in fp16 and
    fp32, so what is rounded is q (fp16 terms relative to its row's largest
    entry: 2^-39 of that at most, less than the sums' steps), the fp32 sums
    (seq_bounds), P, and the output's own type.  P is taken 2^7 times as large,
    as one fp16 number in bf16 calls, half a step 2^-11 relative, and as two in
    float32 ones, 2^-22, and in both no finer than fp16's least half step, 2^-25
    of 2^7 P: for each of n keys 2^-32, relative to a sum of P of at least its
    largest, 1.  The tensors' scales cost two fp32 roundings more, within the
    sums' margin.
    """
    G = q.shape[0] // k.shape[0]
    k, v = k.repeat(G, 0), v.repeat(G, 0)
    sees = oracle.new_token_mask(q.shape[1], k.shape[1])
    p, lse = oracle.masked_probabilities(q, k, scale, sees)
    o = np.matmul(p, v)
    _, e = sb._score_errors(q, k, scale, sees)
    av = np.matmul(p, np.abs(v))
    n = sees.sum(-1)[:, None]
    least = n * 2.0 ** -32 * (np.abs(v).max(1, keepdims=True) if v.shape[1] else 0.0)
    tol = (e + 2.0 ** -22 + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22)) * av + least + sb.HALF[dtype] * np.abs(o) + 1e-30
    return o, lse, tol, e[..., 0] + 2.0 ** -22 + 2.0 ** -24 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
