"""Offsets beyond 32 bits in the latent and shared-prefix operators: the last
sequences of tensors with more than 2^31 elements, against the definition."""

import numpy as np
import pytest

import oracle
from tests import seq_bounds as sb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB free on the device")
    from exact_tiled_attention_02_gb300 import binding
    return binding


def test_absorbed_at_the_end_of_a_long_cache(fa):
    pages, page = 60000, 64  # 60000 * 64 * 576 = 2.2e9 entries
    cache = torch.empty((pages, page, 576), device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[0, pages - 1, pages - 3], [pages - 2, 1, pages - 4]], dtype=torch.int32, device="cuda")
    for p in table.flatten().tolist():
        cache[p] = torch.randn((page, 576), device="cuda")
    q = torch.randn((2, 16, 1, 576), device="cuda").bfloat16()
    lens = [150, 129]
    o, lse = fa.fa_fwd_latent_absorbed(q, cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), 512, 0.07,
                                       block_table=table)
    assert fa.fa_last_device_status() == fa.FA_OK
    for b, n in enumerate(lens):
        x = sb.f64(cache[table[b].long()].reshape(-1, 576)[:n])[None]
        ref, lr, tol_o, tol_l = sb.forward(sb.f64(q[b]), x, x[..., :512], 0.07, oracle.new_token_mask(1, n), "bf16")
        sb.check("o", sb.f64(o[b]), ref, tol_o)
        sb.check("lse", sb.f64(lse[b]), lr, tol_l)


def test_shared_prefix_with_long_padded_sequences(fa):
    B, Hq, Hkv, Np, Ns, d = 17, 4, 1, 130, 1 << 20, 128  # own keys: 2.3e9 entries
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, kp, vp = n(B, Hq, 1, d), n(Hkv, Np, d), n(Hkv, Np, d)
    k, v = (torch.empty((B, Hkv, Ns, d), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = [3] * 15 + [65, 100]
    for b, m in enumerate(lens):
        k[b, :, :m], v[b, :, :m] = n(Hkv, m, d), n(Hkv, m, d)
        k[b, :, m:m + 64], v[b, :, m:m + 64] = float("nan"), float("nan")
    o, lse = fa.fa_fwd_shared_prefix(q, kp, vp, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert fa.fa_last_device_status() == fa.FA_OK
    for b in (0, 15, 16):
        m = lens[b]
        keys = np.concatenate([sb.f64(kp), sb.f64(k[b, :, :m])], 1).repeat(Hq, 0)
        vals = np.concatenate([sb.f64(vp), sb.f64(v[b, :, :m])], 1).repeat(Hq, 0)
        ref, lr, tol_o, tol_l = sb.forward(sb.f64(q[b]), keys, vals, d ** -0.5, True, "bf16")
        sb.check("o", sb.f64(o[b]), ref, tol_o)
        sb.check("lse", sb.f64(lse[b]), lr, tol_l)


def test_expanded_forward_and_backward_past_32_bits(fa):
    B, H, N = 33000, 4, 128  # v: 2.2e9 entries
    g = torch.Generator(device="cuda").manual_seed(1)
    t = dict(device="cuda", dtype=torch.bfloat16)
    q, kn, kr = torch.empty((B, H, N, 192), **t), torch.empty((B, H, N, 128), **t), torch.empty((B, N, 64), **t)
    v, do = torch.empty((B, H, N, 128), **t), torch.empty((B, H, N, 128), **t)
    for x in (q, kn, kr, v, do):
        x.normal_(generator=g)
    o, lse = fa.fa_fwd_latent(q, kn, kr, v)
    grads = fa.fa_bwd_latent(q, kn, kr, v, o, lse, do)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    vis = oracle.new_token_mask(N, N)
    for b in (0, B - 1):
        keys = np.concatenate([sb.f64(kn[b]), np.broadcast_to(sb.f64(kr[b])[None], (H, N, 64))], -1)
        args = (sb.f64(q[b]), keys, sb.f64(v[b]))
        ref, lr, tol_o, tol_l = sb.forward(*args, 192 ** -0.5, vis, "bf16")
        sb.check("o", sb.f64(o[b]), ref, tol_o)
        sb.check("lse", sb.f64(lse[b]), lr, tol_l)
        (dq, dk, dv), (tq, tk, tv) = sb.backward(*args, sb.f64(do[b]), 192 ** -0.5, vis, "bf16")
        u = sb.HALF["bf16"]
        for name, got, want, tol in (("dq", grads[0][b], dq, tq), ("dk_nope", grads[1][b], dk[..., :128], tk[..., :128]),
                                     ("dk_rope", grads[2][b], dk[..., 128:].sum(0), tk[..., 128:].sum(0)),
                                     ("dv", grads[3][b], dv, tv)):
            sb.check(name, sb.f64(got), want, tol + u * (np.abs(want) + tol) + 1e-30)
