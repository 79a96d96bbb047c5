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
