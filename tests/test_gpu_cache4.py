"""The 4-bit key/value cache on the GPU: what is written bit for bit, what is
read back number for number, attention element by element against the float64
definition."""

import numpy as np
import pytest

import oracle
from tests import cache4_common as cc
from tests import seq_bounds as sb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_02_gb300 import binding
    return binding


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def tokens(rng, dtype, *shape):
    """Keys or values with small, large, zero, saturating and tied groups."""
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)))
    g = x.reshape(*shape[:-1], shape[-1] // 16, 16)
    kind = rng.integers(0, 12, g.shape[:-1])
    g[kind == 0] = 0
    g[kind == 1] *= 1e-4
    g[kind == 2] *= 1e4
    g[kind == 3] = rng.integers(-24, 25, g.shape)[kind == 3] / 4  # on the borders between codes where amax is 6
    return torch.from_numpy(x).float().to(TYPES[dtype])


WRITES = [
    # dtype, B, Hkv, Nn, page, d, lens, n_new, scales
    ("bf16", 1, 1, 1, 16, 16, [1], None, (1.0, 1.0)),
    ("bf16", 3, 2, 1, 16, 128, [1, 16, 17], None, (0.25, 2.0)),
    ("bf16", 3, 2, 2, 32, 64, [2, 17, 33], None, (1.0, 1.0)),          # across a block and a page
    ("bf16", 2, 3, 40, 48, 96, [40, 131], None, (0.3, 0.7)),            # scales that are no powers of two
    ("bf16", 4, 2, 33, 16, 80, [33, 5, 0, 20], [33, 5, 0, 20], (1.0, 0.125)),  # prompts of unequal lengths
    ("bf16", 3, 1, 7, 64, 256, [70, 71, 64], [7, 0, 3], (1.0, 1.0)),
    ("f32", 2, 5, 19, 32, 48, [19, 64], None, (0.0625, 1e-3)),
    ("f32", 2, 1, 1, 128, 208, [128, 129], None, (1.0, 1.0)),
    ("f32", 2, 2, 9, 16, 128, [4, 30], None, (1.0, 1.0)),               # rows before position 0
]


@pytest.mark.parametrize("dtype,B,Hkv,Nn,page,d,lens,n_new,scales", WRITES)
def test_write_and_read(fa, dtype, B, Hkv, Nn, page, d, lens, n_new, scales):
    rng = np.random.default_rng(B * 1000 + d)
    max_pages = max(1, -(-max(lens) // page)) + 1
    table, pages = cc.place(rng, B, max_pages, lens, page)
    before = cc.random_cache(rng, pages, Hkv, page, d)
    k, v = tokens(rng, dtype, B, Hkv, Nn, d), tokens(rng, dtype, B, Hkv, Nn, d)
    for b in range(B):  # padding may hold anything
        k[b, :, :Nn - (Nn if n_new is None else n_new[b])] = float("nan")
    cache = torch.from_numpy(before).cuda()
    fa.fa_cache_fp4_write(k.cuda(), v.cuda(), cache, i32(lens), block_table=i32(table), k_scale=scales[0],
                          v_scale=scales[1], n_new=None if n_new is None else i32(n_new))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    want = before.reshape(pages, Hkv, page // 16, 18 * d).copy()
    # the division by the tensor's scale is float32's
    y = [(x.float() / torch.tensor(s, dtype=torch.float32)).double().numpy() for x, s in zip((k, v), scales)]
    for b in range(B):
        n = Nn if n_new is None else n_new[b]
        for t in range(max(Nn - n, Nn - lens[b]), Nn):
            pos = lens[b] - Nn + t
            blk = want[table[b, pos // page], :, pos % page // 16]
            for h in range(Hkv):
                parts = [x.copy() for x in oracle.cache4_unpack(blk[h], d)]
                for i in range(2):
                    parts[2 * i][pos % 16], parts[2 * i + 1][pos % 16] = oracle.cache4_quantise(y[i][b, h, t], 1.0)
                blk[h] = oracle.cache4_pack(*parts)
    got = cache.cpu().numpy().reshape(want.shape)
    written = want != before.reshape(want.shape)

    def plain(x):  # minus zero is zero, and a group of NaN is one whatever its codes
        out = []
        for blk in x.reshape(-1, 18 * d):
            kc, ks, vc, vs = oracle.cache4_unpack(blk, d)
            out.append([np.where(kc == 8, 0, kc), ks, np.where(vc == 8, 0, vc), vs])
        return [np.stack(a) for a in zip(*out)]

    for a, b in zip(plain(got), plain(want)):
        assert (a == b).all()
    assert (got[~written & (got != want)] & 0x77 == want[~written & (got != want)] & 0x77).all()

    # what was written, and around it: positions first .. first + N - 1
    N = Nn + 21
    first = [n - Nn - 10 for n in lens]
    for out in ("f32", "bf16"):
        rk, rv = fa.fa_cache_fp4_read(cache, i32(lens), N, TYPES[out], block_table=i32(table), first=i32(first),
                                      k_scale=scales[0], v_scale=scales[1])
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        for b in range(B):
            # code * scale exactly, times the tensor's scale in float32, then the output's type
            ks, vs = cc.dense(cache.cpu().numpy(), table, b, lens[b], d, page, 1.0, 1.0)
            for r, x, s in ((rk, ks, scales[0]), (rv, vs, scales[1])):
                ref = torch.zeros((Hkv, N, d))
                for t in range(N):
                    if 0 <= first[b] + t < lens[b]:
                        ref[:, t] = torch.from_numpy(x[:, first[b] + t]).float() * torch.tensor(s, dtype=torch.float32)
                assert torch.equal(torch.nan_to_num(r[b].cpu().float(), nan=-7e7), torch.nan_to_num(ref.to(TYPES[out]).float(), nan=-7e7))


def test_write_special_numbers(fa):
    k = torch.zeros(1, 1, 5, 32)
    k[0, 0, 0, 3], k[0, 0, 1, 5], k[0, 0, 2, 20], k[0, 0, 3, 1], k[0, 0, 4, 16] = float("nan"), float("-inf"), 1e30, 1e-30, 6.0
    for t in (torch.float32, torch.bfloat16):
        cache = torch.zeros(1, 1, 16, 36, dtype=torch.uint8, device="cuda")
        x = k.to(t).cuda()
        fa.fa_cache_fp4_write(x, x, cache, i32([5]))
        for r in fa.fa_cache_fp4_read(cache, i32([5]), 5, torch.float32):
            r = r[0, 0].cpu()
            assert torch.isnan(r[0, :16]).all() and (r[0, 16:] == 0).all()
            assert r[1, 5] == -2688 and r[2, 20] == 2688 and r[4, 16] == 6
            r[0, :16] = r[1, 5] = r[2, 20] = r[4, 16] = 0
            assert (r == 0).all()


def test_tables_and_lengths_out_of_range(fa):
    """Nothing out of range is read or written, and it is reported."""
    rng = np.random.default_rng(5)
    B, Hkv, page, d = 4, 2, 16, 64
    table = i32([[0, 9], [1, -1], [2, 3], [4, 5]])  # 9 and -1: no such page
    lens = i32([20, 32, 33, -2])                     # 33 of 32; -2
    before = torch.from_numpy(cc.random_cache(rng, 6, Hkv, page, d)).cuda()
    cache = before.clone()
    k = tokens(rng, "f32", B, Hkv, 20, d).cuda()
    fa.fa_cache_fp4_write(k, k, cache, lens, block_table=table)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
    assert torch.equal(cache[2:], before[2:]) and not torch.equal(cache[:2], before[:2])
    k, v = fa.fa_cache_fp4_read(before, lens, 40, torch.float32, block_table=table)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
    assert (k[:2, :, 16:] == 0).all() and (k[2, :, 32:] == 0).all() and (k[3] == 0).all()
    for b, n in ((0, 16), (1, 16), (2, 32)):
        kd, vd = cc.dense(before.cpu().numpy(), table.cpu().numpy(), b, n, d, page, 1.0, 1.0)
        assert (sb.f64(k[b, :, :n]) == kd).all() and (sb.f64(v[b, :, :n]) == vd).all()
    fa.fa_cache_fp4_write(k[:, :, :3].contiguous(), k[:, :, :3].contiguous(), cache, i32([3] * 4), block_table=table, n_new=i32([4, -1, 3, 0]))
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
    for dtype in ("bf16", "f32"):
        q = torch.from_numpy(rng.standard_normal((B, 4, 2, d))).to(TYPES[dtype])
        o, lse = fa.fa_fwd_cache_fp4(q.cuda(), before, lens, block_table=table)
        assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
        for b, n in enumerate((20, 32, 32, 0)):  # a missing page reads as zeros
            kd, vd = cc.dense(before.cpu().numpy(), table.cpu().numpy(), b, n, d, page, 1.0, 1.0)
            ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), kd, vd, d ** -0.5, dtype)
            sb.check("o", sb.f64(o[b]), ref, tol)
            sb.check("lse", sb.f64(lse[b]), lr, tol_l)


ATTENDS = [
    # dtype, B, Hq, Hkv, Nq, page, d, lens, q multiplier
    ("bf16", 1, 1, 1, 1, 16, 64, [1], 1),                           # the smallest call
    ("bf16", 2, 2, 1, 1, 16, 128, [0, 2], 1),                       # an empty sequence
    ("bf16", 7, 8, 2, 1, 64, 128, [1, 63, 64, 127, 128, 129, 256], 1),  # lengths around a tile
    ("bf16", 5, 10, 2, 3, 48, 96, [2, 1, 130, 300, 3], 1),          # rows that see nothing; pages across tiles
    ("bf16", 3, 16, 2, 4, 16, 64, [1000, 17, 515], 4),              # 32 rows; large scores
    ("bf16", 2, 20, 4, 7, 32, 128, [700, 333], 1),                  # 35 rows
    ("bf16", 2, 8, 1, 13, 128, 96, [1, 640], 2),                    # 104 rows in groups
    ("bf16", 1, 4, 1, 100, 64, 128, [1500], 1),                     # 400 rows
    ("bf16", 1, 8, 8, 1, 64, 128, [30001], 2),                      # one long sequence
    ("bf16", 40, 4, 1, 1, 16, 64, [7 * i % 331 for i in range(40)], 1),  # many pieces a CTA
    ("bf16", 33, 8, 8, 2, 32, 96, [(19 * i + 3) % 401 for i in range(33)], 1),
    ("bf16", 150, 8, 1, 4, 16, 128, [(37 * i + 5) % 700 for i in range(150)], 1),   # 32 rows, several sequences a CTA
    ("bf16", 150, 4, 1, 12, 16, 64, [(41 * i + 9) % 700 for i in range(150)], 1),   # 48 rows
    ("f32", 150, 8, 1, 4, 32, 96, [(43 * i + 2) % 600 for i in range(150)], 1),
    ("f32", 150, 4, 1, 1, 32, 128, [(43 * i + 2) % 600 for i in range(150)], 1),
    ("bf16", 3, 6, 2, 2, 16, 80, [5, 90, 200], 1),                  # widths without a tensor-core form
    ("bf16", 2, 4, 2, 1, 32, 256, [65, 400], 1),
    ("bf16", 2, 3, 3, 5, 16, 16, [4, 100], 1),
    ("f32", 1, 1, 1, 1, 16, 16, [1], 1),
    ("f32", 4, 6, 2, 3, 16, 80, [0, 2, 64, 201], 1),
    ("f32", 2, 12, 4, 5, 48, 128, [129, 1000], 3),
    ("f32", 3, 4, 2, 1, 32, 256, [1, 65, 513], 1),
    ("f32", 9, 8, 8, 1, 64, 96, [0, 1, 63, 64, 65, 127, 128, 129, 700], 1),
    ("f32", 1, 4, 1, 30, 64, 64, [3000], 1),
]


@pytest.mark.parametrize("dtype,B,Hq,Hkv,Nq,page,d,lens,mult", ATTENDS)
def test_attention(fa, dtype, B, Hq, Hkv, Nq, page, d, lens, mult):
    rng = np.random.default_rng(Hq * 100 + d)
    max_pages = max(1, -(-max(lens) // page)) + 1
    table, pages = cc.place(rng, B, max_pages, lens, page)
    cache = cc.random_cache(rng, pages, Hkv, page, d)
    cc.poison(cache, table, lens, page, d)
    ks, vs, scale = 0.3, 1.7, 1.1 / d
    q = torch.from_numpy(rng.standard_normal((B, Hq, Nq, d)) * mult).to(TYPES[dtype])
    args = (q.cuda(), torch.from_numpy(cache).cuda(), i32(lens))
    kw = dict(scale=scale, block_table=i32(table), k_scale=ks, v_scale=vs)
    o, lse = fa.fa_fwd_cache_fp4(*args, **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for b in range(B):
        k, v = cc.dense(cache, table, b, lens[b], d, page, float(np.float32(ks)), float(np.float32(vs)))
        ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), k, v, float(np.float32(scale)), dtype)
        sb.check(f"lse {b}", sb.f64(lse[b]), lr, tol_l)
        sb.check(f"o {b}", sb.f64(o[b]), ref, tol)
    again, none = fa.fa_fwd_cache_fp4(*args, want_lse=False, **kw)
    assert none is None and torch.equal(again, o)  # bit for bit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_any_magnitude(fa, dtype):
    """Query rows of one group whose entries differ by many powers of two, within a row too."""
    rng = np.random.default_rng(11)
    d, n = 128, 300
    cache = cc.random_cache(rng, 5, 1, 64, d)
    q = rng.standard_normal((1, 8, 1, d))
    q *= 2.0 ** np.array([0, -60, -30, -10, 0, 3, -90, 0]).reshape(1, 8, 1, 1)
    q[0, 4] *= 2.0 ** -rng.integers(0, 40, (1, d))
    q[0, 7] = 0
    q = torch.from_numpy(q).to(TYPES[dtype])
    table = np.arange(5, dtype=np.int32)[None]
    o, lse = fa.fa_fwd_cache_fp4(q.cuda(), torch.from_numpy(cache).cuda(), i32([n]), block_table=i32(table))
    k, v = cc.dense(cache, table, 0, n, d, 64, 1.0, 1.0)
    ref, lr, tol, tol_l = cc.forward(sb.f64(q[0]), k, v, d ** -0.5, dtype)
    sb.check("lse", sb.f64(lse[0]), lr, tol_l)
    sb.check("o", sb.f64(o[0]), ref, tol)


def test_without_a_table(fa):
    rng = np.random.default_rng(3)
    B, Hkv, page, d, lens = 3, 2, 320, 64, [320, 0, 77]
    cache = cc.random_cache(rng, B + 1, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((B, 4, 1, d))).bfloat16()
    o, lse = fa.fa_fwd_cache_fp4(q.cuda(), torch.from_numpy(cache).cuda(), i32(lens))
    for b in range(B):
        k, v = cc.dense(cache, None, b, lens[b], d, page, 1.0, 1.0)
        ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), k, v, d ** -0.5, "bf16")
        sb.check("o", sb.f64(o[b]), ref, tol)
        sb.check("lse", sb.f64(lse[b]), lr, tol_l)


@pytest.mark.parametrize("dtype,d,Nq", [("bf16", 128, 1), ("bf16", 64, 20), ("f32", 96, 2), ("bf16", 80, 1)])
def test_a_batch_without_any_token(fa, dtype, d, Nq):
    q = torch.randn(3, 4, Nq, d).to(TYPES[dtype]).cuda()
    cache = torch.full((2, 2, 16, 9 * d // 8), 0xFF, dtype=torch.uint8, device="cuda")
    kw = dict(block_table=i32([[-1, 7]] * 3))
    o, lse = fa.fa_fwd_cache_fp4(q, cache, i32([0, 0, 0]), **kw)
    k, v = fa.fa_cache_fp4_read(cache, i32([0, 0, 0]), 5, **kw)
    fa.fa_cache_fp4_write(q[:, :2].contiguous(), q[:, :2].contiguous(), cache, i32([0, 0, 0]), n_new=i32([0, 0, 0]), **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    assert (o == 0).all() and (lse == -float("inf")).all() and (k == 0).all() and (v == 0).all() and (cache == 0xFF).all()


@pytest.mark.parametrize("Hq,Hkv,Nq,d", [(8, 8, 1, 128), (16, 4, 1, 64), (40, 8, 1, 96), (24, 3, 1, 128), (64, 4, 1, 128),
                                         (48, 16, 1, 64), (10, 2, 4, 128), (6, 1, 9, 96), (4, 1, 33, 64), (2, 1, 97, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_row_count(fa, dtype, Hq, Hkv, Nq, d):
    """1 to 194 rows a key head: every width of the products, and groups of rows."""
    rng = np.random.default_rng(Hq + Nq)
    lens, page = [Nq + 3, 0, 517, 128, 2], 32
    table, pages = cc.place(rng, 5, 20, lens, page)
    cache = cc.random_cache(rng, pages, Hkv, page, d)
    cc.poison(cache, table, lens, page, d)
    q = torch.from_numpy(rng.standard_normal((5, Hq, Nq, d))).to(TYPES[dtype])
    o, lse = fa.fa_fwd_cache_fp4(q.cuda(), torch.from_numpy(cache).cuda(), i32(lens), scale=0.02, block_table=i32(table))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for b, n in enumerate(lens):
        k, v = cc.dense(cache, table, b, n, d, page, 1.0, 1.0)
        ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), k, v, float(np.float32(0.02)), dtype)
        sb.check(f"lse {b}", sb.f64(lse[b]), lr, tol_l)
        sb.check(f"o {b}", sb.f64(o[b]), ref, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_rise_and_fall(fa, dtype):
    """Keys that grow along a sequence (references rise tile after tile, O is
    rescaled), fall, or jump by thousands; scores of 2^40 and of 2^-40."""
    d, n, page = 128, 1000, 16
    rng = np.random.default_rng(6)
    blocks = cc.random_cache(rng, 63, 1, page, d).reshape(63, 1, 1, 18 * d)
    table = np.arange(63, dtype=np.int32)[None]
    for grow in (lambda i: i // 2, lambda i: 62 - i, lambda i: 60 * (i % 2), lambda i: 55 if i == 40 else 5):
        for i in range(63):
            blocks[i, ..., 8 * d:9 * d] = 0x10 + grow(i)
        cache = blocks.reshape(63, 1, page, 144)
        for scale in (0.01, 0.5, 2.0 ** 20, 2.0 ** -60):
            q = torch.from_numpy(rng.standard_normal((1, 4, 2, d))).to(TYPES[dtype])
            o, lse = fa.fa_fwd_cache_fp4(q.cuda(), torch.from_numpy(cache).cuda(), i32([n]), scale=scale, block_table=i32(table))
            k, v = cc.dense(cache, table, 0, n, d, page, 1.0, 1.0)
            ref, lr, tol, tol_l = cc.forward(sb.f64(q[0]), k, v, scale, dtype)
            sb.check("lse", sb.f64(lse[0]), lr, tol_l)
            if scale < 2:  # past that the bound on a score's error allows any softmax
                sb.check("o", sb.f64(o[0]), ref, tol)
            assert torch.isfinite(o).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 80)])
def test_a_token_that_is_no_number(fa, dtype, d):
    """A NaN among a sequence's keys or values is not lost, and stays with its sequence and head."""
    rng = np.random.default_rng(8)
    k, v = tokens(rng, dtype, 3, 2, 200, d), tokens(rng, dtype, 3, 2, 200, d)
    k[0, 1, 150, 7], v[2, 0, 3, 20] = float("nan"), float("nan")
    cache = torch.zeros((3, 2, 208, 9 * d // 8), dtype=torch.uint8, device="cuda")
    lens = i32([200, 200, 200])
    fa.fa_cache_fp4_write(k.cuda(), v.cuda(), cache, lens)
    q = torch.from_numpy(rng.standard_normal((3, 8, 1, d))).to(TYPES[dtype]).cuda()
    o, lse = fa.fa_fwd_cache_fp4(q, cache, lens)
    o, lse = torch.isnan(o[:, :, 0]).cpu(), torch.isnan(lse[:, :, 0]).cpu()
    want_o, want_l = torch.zeros(3, 8, d, dtype=torch.bool), torch.zeros(3, 8, dtype=torch.bool)
    want_o[0, 4:] = want_l[0, 4:] = True
    want_o[2, :4, 16:32] = True
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [100, -100])
def test_queries_far_from_one(fa, dtype, power):
    """Queries of 2^100 and 2^-100 with a scale that brings the scores back."""
    rng = np.random.default_rng(12)
    d, n, page = 96, 250, 32
    cache = cc.random_cache(rng, 8, 2, page, d)
    table = np.arange(8, dtype=np.int32)[None]
    q = torch.from_numpy(rng.standard_normal((1, 6, 3, d)) * 2.0 ** power).to(TYPES[dtype])
    scale = 0.1 * 2.0 ** -power
    o, lse = fa.fa_fwd_cache_fp4(q.cuda(), torch.from_numpy(cache).cuda(), i32([n]), scale=scale, block_table=i32(table))
    k, v = cc.dense(cache, table, 0, n, d, page, 1.0, 1.0)
    ref, lr, tol, tol_l = cc.forward(sb.f64(q[0]), k, v, float(np.float32(scale)), dtype)
    sb.check("lse", sb.f64(lse[0]), lr, tol_l)
    sb.check("o", sb.f64(o[0]), ref, tol)
