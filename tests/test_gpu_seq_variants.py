"""Widths, row counts and part counts of the serving calls that no other
table of cases reaches, element by element against the float64 definition."""

import pytest

from tests import seq_bounds as sb
from tests.test_gpu_latent import absorbed, expect_absorbed
from tests.test_gpu_shared_prefix import expect, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_02_gb300 import binding
    return binding


def _absorbed(fa, dtype, B, H, Nq, page, dc, dr, lens, seed):
    q, cache, tab, rows = absorbed(dtype, B, H, Nq, page, dc, dr, lens, seed=seed)
    o_ref, lse_ref, tol_o, tol_l = expect_absorbed(dtype, q, rows, dc, 192 ** -0.5)
    o, lse = fa.fa_fwd_latent_absorbed(q.cuda(), cache.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), dc,
                                       192 ** -0.5, block_table=tab.cuda())
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


def _prefix(fa, dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens, seed):
    host = make(dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens, seed=seed)
    o_ref, lse_ref, tol_o, tol_l = expect(dtype, *host, lens, d ** -0.5)
    o, lse = fa.fa_fwd_shared_prefix(*[t.cuda() for t in host], torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


@pytest.mark.parametrize("H,Nq,page,lens", [
    (20, 1, 16, [0, 15, 64, 65, 333]),     # 32 columns
    (10, 3, 48, [2, 3, 47, 200]),          # 30 rows, the first before its sequence
    (64, 2, 48, [1, 129, 700]),            # 64 columns, two groups of rows
    (50, 1, 64, [64, 5000]),               # 50 rows, many pieces
    (5, 3, 32, [1, 31, 33]),               # 15 rows
])
def test_absorbed_256_wide(fa, H, Nq, page, lens):
    _absorbed(fa, "bf16", len(lens), H, Nq, page, 256, 64, lens, seed=H + Nq)


@pytest.mark.parametrize("Hq,Hkv,Nq,d,Np,lens", [
    (16, 2, 3, 128, 130, [3, 64, 129, 0, 2]),   # 24 rows a sequence and key head
    (16, 2, 4, 128, 0, [65, 1]),                # 32 rows, no prefix
    (25, 5, 5, 96, 200, [4, 70, 128]),          # 25 rows
    (8, 1, 4, 96, 0, [130, 3]),                 # 32 rows, no prefix
    (17, 1, 1, 128, 700, [66, 1, 0]),           # 17 rows
])
def test_prefix_with_17_to_32_rows_a_key_head(fa, Hq, Hkv, Nq, d, Np, lens):
    _prefix(fa, "bf16", len(lens), Hq, Hkv, Nq, Np, max(lens) + 5, d, lens, seed=Hq + d)


def test_float32_merge_of_more_than_32_parts(fa):
    _prefix(fa, "f32", 1, 1, 1, 1, 2500, 0, 33, [0], seed=1)           # 40 parts
    _prefix(fa, "f32", 1, 2, 1, 2, 4096, 4096, 64, [4000], seed=2)     # 64 and 64
    _prefix(fa, "f32", 1, 2, 1, 2, 4096, 4096, 64, [1], seed=3)        # most parts without a key
    _absorbed(fa, "f32", 1, 3, 1, 24, 192, 40, [3000], seed=4)         # 47 parts
    _absorbed(fa, "f32", 2, 16, 2, 16, 300, 20, [5000, 33], seed=5)    # 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absorbed_sequences_may_share_pages(fa, dtype):
    """The same pages in two sequences' tables, and one page twice in a sequence's."""
    q, cache, tab, rows = absorbed(dtype, 3, 16, 1, 32, 512, 64, [160, 96, 64], seed=11)
    tab[1, :2] = tab[0, :2]   # sequence 1 begins like sequence 0
    tab[2, 1] = tab[2, 0]
    rows[1][:64] = rows[0][:64]
    rows[2][32:] = rows[2][:32]
    lens = [160, 96, 64]
    o_ref, lse_ref, tol_o, tol_l = expect_absorbed(dtype, q, rows, 512, 0.07)
    o, lse = fa.fa_fwd_latent_absorbed(q.cuda(), cache.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 512,
                                       0.07, block_table=tab.cuda())
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


@pytest.mark.parametrize("dtype,Hq,Hkv,Nq,Np,d,lens", [
    ("bf16", 8, 2, 200, 0, 64, [200, 130]),    # a prompt: every token new, the second row of rows before its sequence
    ("bf16", 4, 4, 150, 70, 128, [150, 400]),  # a chunk behind a prefix, one with a past of its own
    ("f32", 6, 2, 70, 0, 40, [70, 20]),
])
def test_prompt_through_the_prefix_call(fa, dtype, Hq, Hkv, Nq, Np, d, lens):
    """Nq new tokens with as many own keys: causal attention of a prompt with shared key heads."""
    _prefix(fa, dtype, len(lens), Hq, Hkv, Nq, Np, max(lens), d, lens, seed=Nq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_lse(fa, dtype):
    """No lse wanted: the same O, bit for bit, whichever kernel writes it."""
    host = make(dtype, 3, 8, 2, 1, 300, 90, 64, [90, 0, 7], seed=1)
    args = [t.cuda() for t in host] + [torch.tensor([90, 0, 7], dtype=torch.int32, device="cuda")]
    o, lse = fa.fa_fwd_shared_prefix(*args)
    bare, none = fa.fa_fwd_shared_prefix(*args, want_lse=False)
    assert none is None and lse is not None and torch.equal(o, bare)
    q, cache, tab, _ = absorbed(dtype, 3, 16, 1, 16, 512, 64, [300, 0, 20], seed=2)  # merged, empty and whole pieces
    args = (q.cuda(), cache.cuda(), torch.tensor([300, 0, 20], dtype=torch.int32, device="cuda"), 512, 0.07)
    o, _ = fa.fa_fwd_latent_absorbed(*args, block_table=tab.cuda())
    bare, none = fa.fa_fwd_latent_absorbed(*args, block_table=tab.cuda(), want_lse=False)
    assert none is None and torch.equal(o, bare)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(3)
    q, kn, kr, v = (torch.randn(s, generator=g).to(t).cuda() for s in ((2, 3, 150, 192), (2, 3, 150, 128), (2, 150, 64), (2, 3, 150, 128)))
    o, _ = fa.fa_fwd_latent(q, kn, kr, v)
    bare, none = fa.fa_fwd_latent(q, kn, kr, v, want_lse=False)
    assert none is None and torch.equal(o, bare)
