"""The 4-bit cache's calls at their borders: capacities near 2^31 tokens,
pages that sequences share, numbers on the borders of the format, bytes around
what a call writes."""

import numpy as np
import pytest

import oracle
from tests import cache4_common as cc

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


def quantised(x, scale):
    """What float64 ``x`` is held as, its division by the tensor's scale float32's."""
    y = (torch.from_numpy(x).float() / torch.tensor(scale, dtype=torch.float32)).double().numpy()
    return oracle.cache4_quantise(y, 1.0)


def test_more_rows_than_positions_are_left(fa):
    """A sequence of 2^31 - 2^20 tokens (its table repeats one page) and 2^21
    rows, of which one is new: of the blocks that so many rows could touch, those
    past the end would begin beyond 2^31."""
    page, max_pages, Nn, d = 1 << 20, 2047, 1 << 21, 16
    rng = np.random.default_rng(0)
    cache = torch.full((1, 1, page, 9 * d // 8), 0x11, dtype=torch.uint8, device="cuda")
    k = torch.full((1, 1, Nn, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    new = [torch.from_numpy(rng.standard_normal(d)).bfloat16() for _ in range(2)]
    k[0, 0, -1], v[0, 0, -1] = new[0].cuda(), new[1].cuda()
    fa.fa_cache_fp4_write(k, v, cache, i32([page * max_pages]), block_table=i32([[0] * max_pages]), n_new=i32([1]))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    got = cache.view(-1, 18 * d)
    assert (got[:-1] == 0x11).all()
    parts = [x.copy() for x in oracle.cache4_unpack(np.full(18 * d, 0x11), d)]
    for i, x in enumerate(new):
        parts[2 * i][15], parts[2 * i + 1][15] = oracle.cache4_quantise(x.double().numpy(), 1.0)
    have = oracle.cache4_unpack(got[-1].cpu().numpy(), d)
    for a, b in zip(have, parts):
        assert (np.where(a == 8, 0, a) == np.where(b == 8, 0, b)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_without_new_tokens_leaves_its_page_alone(fa, dtype):
    """One sequence of 200 writes to a page that all of them hold; the others'
    lengths end in the block that it writes to.  Nothing it wrote is lost, and a
    table without pages is not looked at where there is nothing to write."""
    B, Hkv, page, d = 200, 4, 64, 128
    rng = np.random.default_rng(1)
    lens, n_new = [25] * B, [0] * B
    lens[100], n_new[100] = 30, 6
    table = np.zeros((B, 2), dtype=np.int32)
    table[7] = table[150] = -1
    for seed in range(30):
        k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, 6, d))).to(TYPES[dtype]).cuda() for _ in range(2))
        alone = torch.full((3, Hkv, page, 9 * d // 8), 0x11, dtype=torch.uint8, device="cuda")
        cache = alone.clone()
        one = slice(100, 101)
        fa.fa_cache_fp4_write(k[one], v[one], alone, i32(lens[one]), block_table=i32(table[one]))
        fa.fa_cache_fp4_write(k, v, cache, i32(lens), block_table=i32(table), n_new=i32(n_new))
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        assert torch.equal(cache, alone) and not (cache[0] == 0x11).all()


@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("power", [-124, -60, 110])
def test_values_scale_of_any_magnitude(fa, d, power):
    """O is proportional to v_scale, far from 1 too: a power of two moves it as a
    whole.  What may differ: O is a float32 number of its own (2^-24), a piece of a
    sequence is one before pieces are merged (2^-24 again, and the merge's sums are
    of numbers scaled alike), and below 2^-126 each of at most 64 pieces and the
    result is rounded to 2^-149."""
    rng = np.random.default_rng(2)
    B, Hq, Hkv, page, lens = 3, 8, 2, 32, [1000, 5, 129]
    table, pages = cc.place(rng, B, 32, lens, page)
    cache = torch.from_numpy(cc.random_cache(rng, pages, Hkv, page, d)).cuda()
    q = torch.from_numpy(rng.standard_normal((B, Hq, 1, d))).float().cuda()
    kw = dict(block_table=i32(table), k_scale=0.25)
    one, lse = fa.fa_fwd_cache_fp4(q, cache, i32(lens), v_scale=1.0, **kw)
    far, lse2 = fa.fa_fwd_cache_fp4(q, cache, i32(lens), v_scale=2.0 ** power, **kw)
    assert fa.fa_last_device_status() == fa.FA_OK and torch.equal(lse, lse2)
    want = one.double() * 2.0 ** power
    assert ((far.double() - want).abs() <= 2.0 ** -21 * want.abs() + 65 * 2.0 ** -150).all()
    assert (want != 0).any()


def steps_around(x, dtype, n):
    """Each of positive ``x`` (exact in ``dtype``), and n numbers of that type to either side."""
    ints = torch.int32 if dtype == torch.float32 else torch.int16
    bits = x.to(dtype).view(ints)
    return torch.stack([(bits + i).view(dtype) for i in range(-n, n + 1)], -1)


def groups_on_borders(dtype, scale):
    """[groups, 16]: a largest entry at or a few steps from every border between two
    e4m3 scales (or the e4m3 numbers themselves), times 6 and the tensor's scale;
    the others at or near the borders between codes under either scale."""
    e4m3 = torch.from_numpy(oracle.cache4.E4M3)
    middle = (e4m3[1:] + e4m3[:-1]) / 2
    amax = torch.cat([6 * middle, 6 * e4m3[1:]])  # at most 7 significant bits
    s = torch.cat([torch.stack([e4m3[:-1], e4m3[1:]], -1), torch.stack([e4m3[1:], e4m3[1:]], -1)])
    codes = torch.from_numpy((oracle.cache4.E2M1[1:] + oracle.cache4.E2M1[:-1]) / 2)
    top = steps_around(amax * scale, dtype, 4).double()                                      # [A, 9]
    near = torch.where(s > 0, s, s[:, 1:])[..., None] * codes                                # [A, 2, 7]
    near = steps_around((near * scale).float().to(dtype), dtype, 2).double().flatten(1)      # [A, 70]
    near = torch.nn.functional.pad(near, (0, 5)).view(-1, 5, 15)                             # in fives of 15
    g = torch.cat([top[:, :, None, None].expand(-1, -1, 5, 1), near[:, None].expand(-1, 9, -1, -1)], -1)
    return torch.minimum(g, g[..., :1]).reshape(-1, 16)  # (none larger than the first)


def test_groups_on_borders_are_there():
    """Of the float32 groups with a power-of-two scale: scales at every tie and one step to either side."""
    x = groups_on_borders(torch.float32, 0.125)
    amax = x[:, 0] / 0.125
    mids = torch.from_numpy((oracle.cache4.E4M3[1:] + oracle.cache4.E4M3[:-1]) / 2) * 6
    below, above = (torch.nextafter(mids.float(), torch.tensor(t)).double() for t in (0.0, float("inf")))
    for want in (mids, below, above):
        assert torch.isin(want, amax).all()
    assert (x.abs().amax(-1) == x[:, 0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.125, 1.0, 0.06, 1.7])
def test_borders_of_scales_and_codes(fa, dtype, scale):
    """Every border of e4m3 and of e2m1, on it and a few steps of the type beside
    it: scales and codes are the definition's, bit for bit."""
    x = groups_on_borders(TYPES[dtype], scale)
    n = -(-x.shape[0] // 16) * 16
    x = torch.nn.functional.pad(x, (0, 0, 0, n - x.shape[0])).to(TYPES[dtype])
    k, v = x[None, None], -x.flip(-1)[None, None].contiguous()
    cache = torch.zeros((1, 1, n, 18), dtype=torch.uint8, device="cuda")
    fa.fa_cache_fp4_write(k.cuda(), v.cuda(), cache, i32([n]), k_scale=scale, v_scale=scale)
    torch.cuda.synchronize()
    got = cache.cpu().numpy().reshape(-1, 18 * 16)
    parts = [np.concatenate(a) for a in zip(*(oracle.cache4_unpack(blk, 16) for blk in got))]
    for i, t in enumerate((k, v)):
        codes, s = quantised(t[0, 0].double().numpy(), scale)
        assert (parts[2 * i + 1] == s).all()
        assert (np.where(parts[2 * i] == 8, 0, parts[2 * i]) == codes).all()  # minus zero is zero


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_write_stays_within_its_tokens(fa, dtype):
    """The cache inside a larger buffer, its pages' unused ones, inputs and the
    bytes of every other token: all as they were.  New tokens across borders of
    blocks and pages."""
    B, Hkv, Nn, page, d = 5, 3, 40, 32, 80
    rng = np.random.default_rng(3)
    lens, n_new = [70, 33, 40, 129, 16], [40, 3, 0, 17, 1]
    table, pages = cc.place(rng, B, 6, lens, page)
    before = cc.random_cache(rng, pages, Hkv, page, d)
    buf = torch.full((before.size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    cache = buf[4096:4096 + before.size].view(before.shape)
    cache.copy_(torch.from_numpy(before))
    k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, Nn, d))).to(TYPES[dtype]).cuda() for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    fa.fa_cache_fp4_write(k, v, cache, i32(lens), block_table=i32(table), n_new=i32(n_new), k_scale=0.5, v_scale=0.3)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    assert (buf[:4096] == 0xA5).all() and (buf[-4096:] == 0xA5).all()
    assert torch.equal(k, k0) and torch.equal(v, v0)
    new = np.zeros((pages, page), dtype=bool)
    for b in range(B):
        for pos in range(lens[b] - n_new[b], lens[b]):
            new[table[b, pos // page], pos % page] = True
    shape = (pages, Hkv, page // 16, 18 * d)
    was, now = before.reshape(shape), cache.cpu().numpy().reshape(shape)
    changed = 0
    for p, h, i in np.ndindex(shape[:3]):
        keep = ~new[p, 16 * i:16 * i + 16]
        for a, c in zip(oracle.cache4_unpack(was[p, h, i], d), oracle.cache4_unpack(now[p, h, i], d)):
            assert (a[keep] == c[keep]).all()
            changed += int((a[~keep] != c[~keep]).sum())
    assert changed > 0.8 * 61 * Hkv * 2 * d  # (61 new tokens; a random code is the same one time in 16)
