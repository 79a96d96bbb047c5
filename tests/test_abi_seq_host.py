"""Host-side refusals of the shared-prefix and latent entry points: every
invalid request is rejected before any CUDA call (the pointers are fake)."""

import ctypes

import pytest

P = 1 << 20  # a fake, aligned pointer value; never dereferenced
VP = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def b():
    from exact_tiled_attention_02_gb300 import binding
    return binding


def prefix(b, q=P, kp=P, vp=P, k=P, v=P, lens=P, o=P, lse=P, B=2, Hq=8, Hkv=2, Nq=1, Np=100, Ns=50, d=64, scale=0.1,
           dt=1, ws=P, wsb=BIG):
    return b.lib.fa_fwd_shared_prefix(VP(q), VP(kp), VP(vp), VP(k), VP(v), VP(lens), VP(o), VP(lse), B, Hq, Hkv, Nq,
                                      Np, Ns, d, scale, dt, VP(ws), wsb, VP(0))


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(lens=0), 1),
    (dict(o=0), 1), (dict(ws=0), 1), (dict(q=P + 8), 1), (dict(vp=P + 2), 1), (dict(lens=P + 2), 1),
    (dict(lse=P + 1), 1), (dict(ws=P + 16), 1), (dict(wsb=100), 1),
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=9), 1), (dict(Hkv=3), 1), (dict(Nq=0), 1),
    (dict(Np=-1), 1), (dict(Ns=-1), 1), (dict(d=0), 1), (dict(B=1 << 30, Hq=64), 1), (dict(Np=(1 << 30) + 1, d=128, Hkv=8), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(dt=5), 1),
    (dict(d=80), 2), (dict(d=256), 2), (dict(dt=0, d=129), 2),
])
def test_shared_prefix_rejects_on_host(b, kw, code):
    assert prefix(b, **kw) == code


def absorbed(b, q=P, c=P, t=P, lens=P, o=P, lse=P, B=2, H=16, Nq=1, n_pages=100, page=64, max_pages=10, dc=512, dr=64,
             scale=0.1, dt=1, ws=P, wsb=BIG):
    return b.lib.fa_fwd_latent_absorbed(VP(q), VP(c), VP(t), VP(lens), VP(o), VP(lse), B, H, Nq, n_pages, page,
                                        max_pages, dc, dr, scale, dt, VP(ws), wsb, VP(0))


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(c=0), 1), (dict(lens=0), 1), (dict(o=0), 1), (dict(ws=0), 1), (dict(c=P + 8), 1),
    (dict(t=P + 2), 1), (dict(lens=P + 1), 1), (dict(lse=P + 2), 1), (dict(ws=P + 128), 1), (dict(wsb=64), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Nq=0), 1), (dict(n_pages=0), 1), (dict(page=0), 1), (dict(max_pages=0), 1),
    (dict(page=1 << 20, max_pages=1 << 20), 1), (dict(dc=0), 1), (dict(dr=0), 1), (dict(H=1 << 30, B=64), 1),
    (dict(t=0), 1), (dict(t=0, max_pages=1, n_pages=1), 1),  # without a table: one page a sequence
    (dict(scale=-1.0), 1), (dict(dt=2), 1),
    (dict(dc=128), 2), (dict(dr=32), 2), (dict(page=24), 2), (dict(dt=0, dc=513), 2), (dict(dt=0, dr=129), 2),
])
def test_absorbed_rejects_on_host(b, kw, code):
    assert absorbed(b, **kw) == code


def latent(b, q=P, kn=P, kr=P, v=P, o=P, lse=P, B=2, H=4, Nq=10, Nk=10, dn=128, dr=64, dv=128, scale=0.1, causal=1,
           dt=1):
    return b.lib.fa_fwd_latent(VP(q), VP(kn), VP(kr), VP(v), VP(o), VP(lse), B, H, Nq, Nk, dn, dr, dv, scale, causal,
                               dt, VP(0))


def latent_bwd(b, q=P, kn=P, kr=P, v=P, o=P, lse=P, do=P, dq=P, dkn=P, dkr=P, dvo=P, B=2, H=4, Nq=10, Nk=10, dn=128,
               dr=64, dv=128, scale=0.1, causal=1, dt=1, ws=P, wsb=BIG):
    return b.lib.fa_bwd_latent(VP(q), VP(kn), VP(kr), VP(v), VP(o), VP(lse), VP(do), VP(dq), VP(dkn), VP(dkr), VP(dvo),
                               B, H, Nq, Nk, dn, dr, dv, scale, causal, dt, VP(ws), wsb, VP(0))


COMMON = [
    (dict(q=0), 1), (dict(kn=0), 1), (dict(kr=0), 1), (dict(v=0), 1), (dict(o=0), 1), (dict(q=P + 4), 1),
    (dict(kr=P + 8), 1), (dict(lse=P + 2), 1), (dict(B=0), 1), (dict(H=0), 1), (dict(Nq=0), 1), (dict(Nk=0), 1),
    (dict(dn=0), 1), (dict(dr=0), 1), (dict(dv=0), 1), (dict(B=1 << 20, H=1 << 20), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(causal=2), 1), (dict(dt=9), 1),
    (dict(dn=64), 2), (dict(dr=32), 2), (dict(dv=64), 2), (dict(dt=0, dn=200, dr=57), 2), (dict(dt=0, dv=129), 2),
]


@pytest.mark.parametrize("kw,code", COMMON)
def test_latent_rejects_on_host(b, kw, code):
    assert latent(b, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(lse=0), 1), (dict(do=0), 1), (dict(dq=0), 1), (dict(dkn=0), 1), (dict(dkr=0), 1), (dict(dvo=0), 1),
    (dict(dkr=P + 8), 1), (dict(ws=0), 1), (dict(ws=P + 8), 1), (dict(wsb=64), 1),
])
def test_latent_bwd_rejects_on_host(b, kw, code):
    assert latent_bwd(b, **kw) == code


def test_workspace_sizes(b):
    assert b.fa_fwd_shared_prefix_workspace_bytes(0, 8, 2, 1, 10, 10, 64) == 0
    assert b.fa_fwd_shared_prefix_workspace_bytes(2, 9, 2, 1, 10, 10, 64) == 0
    assert b.fa_fwd_latent_absorbed_workspace_bytes(1, 0, 1, 64, 4, 512) == 0
    assert b.fa_bwd_latent_workspace_bytes(1, 1, 0, 1, 128, 64, 128) == 0
    for n in (b.fa_fwd_shared_prefix_workspace_bytes(2, 8, 2, 1, 1000, 10, 64),
              b.fa_fwd_latent_absorbed_workspace_bytes(3, 16, 1, 64, 40, 512),
              b.fa_bwd_latent_workspace_bytes(1, 2, 100, 100, 128, 64, 128)):
        assert n > 0 and n % 256 == 0
    # two padded row arrays, then the rotary gradient of each head
    assert b.fa_bwd_latent_workspace_bytes(1, 2, 100, 70, 128, 64, 128) == 2 * (2 * 128 * 4) + 2 * 70 * 64 * 4


def test_absorbed_refuses_too_many_rows_before_it_plans(b):
    """B H Nq of 2^28 and more, among them products past 32 bits: the query
    answers 0, as the call refuses; one row fewer than 2^28 is planned."""
    for B, H, Nq in ((1, 65536, 65536), (1, 65536, 32768), (1 << 20, 1 << 9, 1), (1, 1 << 28, 1), (4, 1 << 26, 1)):
        assert b.lib.fa_fwd_latent_absorbed_workspace_bytes(B, H, Nq, 64, 4, 192) == 0, (B, H, Nq)
        assert absorbed(b, B=B, H=H, Nq=Nq) == 1, (B, H, Nq)
    assert 0 < b.lib.fa_fwd_latent_absorbed_workspace_bytes(1, (1 << 28) - 1, 1, 64, 4, 192) < 1 << 44
    # a table past 2^40 entries, a latent past 4096: the call's other refusals
    assert b.lib.fa_fwd_latent_absorbed_workspace_bytes(1, 1, 1, 64, 4, 4097) == 0


def test_prefix_length_ends_at_the_rooms_of_the_other_lengths(b):
    """Np above 2^31 - 256, where counts of 64- or 128-key tiles pass 32 bits:
    the query answers 0 and the call refuses, whatever workspace it is given."""
    size = b.lib.fa_fwd_shared_prefix_workspace_bytes
    for Np in ((1 << 31) - 255, (1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1):
        for ws in (BIG, (1 << 64) - 1):
            assert prefix(b, B=1, Hq=1, Hkv=1, Np=Np, Ns=1, wsb=ws) == 1, Np
        assert size(1, 1, 1, 1, Np, 1, 64) == 0, Np
    assert 0 < size(1, 1, 1, 1, (1 << 31) - 256, 1, 64) < 1 << 30


def test_room_of_a_batch_is_limited_in_whole_tiles(b):
    """The documented limit: 7,040,929 tiles of 64 tokens, each sequence's room rounded up."""
    most = 7040929
    prefix_bytes, absorbed_bytes = b.lib.fa_fwd_shared_prefix_workspace_bytes, b.lib.fa_fwd_latent_absorbed_workspace_bytes
    for n, Ns in ((most, 1), (most, 64), (1, most * 64), (most // 2, 65)):
        assert prefix_bytes(n, 1, 1, 1, 0, Ns, 64) > 0, (n, Ns)
    for n, Ns in ((most + 1, 1), (most, 65), (1, most * 64 + 1), (most // 2 + 1, 65)):
        assert prefix_bytes(n, 1, 1, 1, 0, Ns, 64) == 0, (n, Ns)
        for dt in (0, 1):
            assert prefix(b, B=n, Hq=1, Hkv=1, Np=0, Ns=Ns, dt=dt) == 1, (n, Ns)
    for n, page, pages in ((most, 1, 1), (most, 16, 4), (1, 64, most), (most // 2, 5, 13)):
        assert absorbed_bytes(n, 1, 1, page, pages, 512) > 0, (n, page, pages)
    for n, page, pages in ((most + 1, 1, 1), (most, 5, 13), (1, 64, most + 1)):
        assert absorbed_bytes(n, 1, 1, page, pages, 512) == 0, (n, page, pages)
        for dt in (0, 1):
            assert absorbed(b, B=n, H=1, page=page, max_pages=pages, n_pages=1, dt=dt) == 1, (n, page, pages)


def test_expanded_lengths_are_limited(b):
    size = b.lib.fa_bwd_latent_workspace_bytes
    for Nq, Nk in ((1 << 30, 1), (1, 1 << 30)):
        assert latent(b, B=1, H=1, Nq=Nq, Nk=Nk, dn=1, dr=1, dv=1, dt=0) == 1
        assert latent_bwd(b, B=1, H=1, Nq=Nq, Nk=Nk, dn=1, dr=1, dv=1, dt=0) == 1
        assert size(1, 1, Nq, Nk, 1, 1, 1) == 0
        assert size(1, 1, max(1, Nq - 1), max(1, Nk - 1), 1, 1, 1) > 0


def test_latent_backward_limits_its_padded_rows(b):
    """B H Nq, Nq rounded up to 128, below 2^33: where the first launch would be refused, the query and the call refuse."""
    size = b.lib.fa_bwd_latent_workspace_bytes
    assert size(1 << 13, (1 << 13) - 1, 128, 1, 1, 1, 1) > 0
    for B, H, Nq in ((1 << 13, 1 << 13, 1), (1 << 13, (1 << 13) - 1, 129), (1 << 10, 1 << 20, 1)):
        assert size(B, H, Nq, 1, 1, 1, 1) == 0, (B, H, Nq)
        for dt in (0, 1):
            assert latent_bwd(b, B=B, H=H, Nq=Nq, Nk=1, dn=1, dr=1, dv=1, dt=dt, wsb=(1 << 64) - 1) == 1, (B, H, Nq)
