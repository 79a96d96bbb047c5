"""Host-side refusals of the 4-bit cache's entry points: every invalid request
is rejected before any CUDA call (the pointers are fake)."""

import ctypes

import pytest

P = 1 << 20  # a fake, aligned pointer value; never dereferenced
VP = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def b():
    from exact_tiled_attention_02_gb300 import binding
    return binding


def write(b, k=P, v=P, c=P, t=P, lens=P, new=P, B=2, Hkv=4, Nn=3, n_pages=100, page=64, max_pages=10, d=128, ks=1.0,
          vs=1.0, dt=1):
    return b.lib.fa_cache_fp4_write(VP(k), VP(v), VP(c), VP(t), VP(lens), VP(new), B, Hkv, Nn, n_pages, page,
                                    max_pages, d, ks, vs, dt, VP(0))


def read(b, k=P, v=P, c=P, t=P, lens=P, new=P, B=2, Hkv=4, Nn=3, n_pages=100, page=64, max_pages=10, d=128, ks=1.0,
         vs=1.0, dt=1):
    return b.lib.fa_cache_fp4_read(VP(c), VP(t), VP(lens), VP(new), VP(k), VP(v), B, Hkv, Nn, n_pages, page, max_pages,
                                   d, ks, vs, dt, VP(0))


def attend(b, q=P, c=P, t=P, lens=P, o=P, lse=P, B=2, Hq=8, Hkv=4, Nq=1, n_pages=100, page=64, max_pages=10, d=128,
           scale=0.1, ks=1.0, vs=1.0, dt=1, ws=P, wsb=BIG):
    return b.lib.fa_fwd_cache_fp4(VP(q), VP(c), VP(t), VP(lens), VP(o), VP(lse), B, Hq, Hkv, Nq, n_pages, page,
                                  max_pages, d, scale, ks, vs, dt, VP(ws), wsb, VP(0))


CACHE = [
    (dict(c=0), 1), (dict(lens=0), 1), (dict(c=P + 8), 1), (dict(t=P + 2), 1), (dict(lens=P + 1), 1),
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(n_pages=0), 1), (dict(page=0), 1), (dict(max_pages=0), 1), (dict(d=0), 1),
    (dict(d=-16), 1), (dict(page=1 << 20, max_pages=1 << 20), 1), (dict(n_pages=1 << 30, page=1 << 16), 1),
    (dict(t=0), 1), (dict(t=0, max_pages=1, n_pages=1), 1),  # without a table: one page a sequence
    (dict(ks=0.0), 1), (dict(vs=-1.0), 1), (dict(ks=float("nan")), 1), (dict(vs=float("inf")), 1), (dict(dt=2), 1),
    (dict(page=24), 2), (dict(d=120), 2), (dict(d=272), 2), (dict(d=8), 2),
]
TOKENS = CACHE + [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=P + 8), 1), (dict(v=P + 2), 1), (dict(new=P + 2), 1), (dict(Nn=0), 1),
    (dict(Nn=-5), 1), (dict(Nn=1 << 30, Hkv=64), 1), (dict(B=1 << 20, Hkv=1 << 14, Nn=1, max_pages=1, n_pages=1), 1),
]


@pytest.mark.parametrize("kw,code", TOKENS)
def test_write_rejects_on_host(b, kw, code):
    assert write(b, **kw) == code


@pytest.mark.parametrize("kw,code", TOKENS)
def test_read_rejects_on_host(b, kw, code):
    assert read(b, **kw) == code


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(q=0), 1), (dict(o=0), 1), (dict(ws=0), 1), (dict(q=P + 8), 1), (dict(o=P + 4), 1), (dict(lse=P + 2), 1),
    (dict(ws=P + 128), 1), (dict(wsb=16), 1), (dict(Hq=0), 1), (dict(Hq=9), 1), (dict(Nq=0), 1),
    (dict(B=1 << 20, Hq=1 << 10), 1), (dict(Nq=1 << 26), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=1e30, ks=1e30), 1), (dict(B=1 << 20, max_pages=1 << 10), 1),
])
def test_attention_rejects_on_host(b, kw, code):
    assert attend(b, **kw) == code


def test_sizes(b):
    assert b.fa_cache_fp4_bytes(100, 8, 64, 128) == 100 * 8 * 64 * 144
    assert b.fa_cache_fp4_bytes(1, 1, 16, 16) == 18 * 16
    assert b.fa_cache_fp4_bytes(1, 1, 24, 128) == 0 and b.fa_cache_fp4_bytes(0, 1, 16, 128) == 0
    assert b.fa_cache_fp4_bytes(1 << 20, 1 << 20, 16, 128) == 0
    need = b.fa_fwd_cache_fp4_workspace_bytes
    assert need(2, 8, 4, 1, 64, 10, 128) > 0
    assert need(2, 9, 4, 1, 64, 10, 128) == 0 and need(2, 8, 4, 0, 64, 10, 128) == 0
    assert need(1 << 20, 8, 4, 1, 64, 1 << 10, 128) == 0 and need(2, 8, 4, 1, 1 << 20, 1 << 20, 128) == 0
    assert need(2, 8, 4, 1, 64, 10, 512) == 0


def test_binding_checks_tensors(b):
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 4, 3, 64)
    with pytest.raises(ValueError):
        b.fa_cache_fp4_write(k, k, torch.zeros(9, 4, 16, 72, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.fa_fwd_cache_fp4(k, torch.zeros(9, 4, 16, 72, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.fa_cache_fp4_read(torch.zeros(9, 4, 16, 72, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32), 5)
    with pytest.raises(ValueError):
        b.fa_cache_fp4_read(torch.zeros(9, 16, 72, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32), 5)
