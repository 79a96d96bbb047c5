"""Persistent kernels of the latent and shared-prefix operators where a CTA
takes several items of unequal length, whole batches and heads element by
element against the float64 definition."""

import numpy as np
import pytest

import oracle
from tests import seq_bounds as sb
from tests.test_gpu_latent import expanded, keys_of
from tests.test_gpu_shared_prefix import expect, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_02_gb300 import binding
    return binding


def _check_step(fa, B, H, Nq, Nk, causal, seed):
    host = expanded("bf16", B, H, Nq, Nk, 128, 64, 128, seed=seed)
    q, kn, kr, v, do = (t.cuda() for t in host)
    vis = oracle.new_token_mask(Nq, Nk) if causal else np.ones((Nq, Nk), bool)
    scale = 192 ** -0.5
    o, lse = fa.fa_fwd_latent(q, kn, kr, v, causal=causal)
    grads = fa.fa_bwd_latent(q, kn, kr, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    u = sb.HALF["bf16"]
    for b in range(B):  # one sequence at a time: the definition's arrays stay small
        args = (sb.f64(host[0][b]), keys_of(host[1][b:b + 1], host[2][b:b + 1])[0], sb.f64(host[3][b]))
        o_ref, lse_ref, tol_o, tol_l = sb.forward(*args, scale, vis, "bf16")
        sb.check(f"o[{b}]", sb.f64(o[b]), o_ref, tol_o)
        sb.check(f"lse[{b}]", sb.f64(lse[b]), lse_ref, tol_l)
        (dq, dk, dv), (tq, tk, tv) = sb.backward(*args, sb.f64(host[4][b]), scale, vis, "bf16")
        for name, got, want, tol in (("dq", grads[0], dq, tq), ("dk_nope", grads[1], dk[..., :128], tk[..., :128]),
                                     ("dk_rope", grads[2], dk[..., 128:].sum(0),
                                      tk[..., 128:].sum(0) + H * 2.0 ** -24 * np.abs(dk[..., 128:]).sum(0)),
                                     ("dv", grads[3], dv, tv)):
            sb.check(f"{name}[{b}]", sb.f64(got[b]), want, tol + u * (np.abs(want) + tol) + 1e-30)


STEPS = [
    # B, H, Nq, Nk, causal
    (2, 31, 520, 520, True),   # 3 pairs of query tiles of 2 to 5 key tiles; 5 key tiles of 1 to 9 steps
    (2, 40, 700, 130, True),   # rows that see nothing: items without a step between others
    (2, 40, 300, 777, True),   # a chunk against a longer past, a second query tile of 44 rows
    (3, 52, 129, 200, False),  # no mask: a second query tile of one row
    (1, 160, 140, 1, True),    # one key
]


@pytest.mark.parametrize("B,H,Nq,Nk,causal", STEPS)
def test_expanded_step_over_several_items_a_cta(fa, B, H, Nq, Nk, causal):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * H * -(-Nq // 256) > sms and B * H * -(-Nk // 128) > sms  # items of the forward and of the keys form
    _check_step(fa, B, H, Nq, Nk, causal, seed=Nq + 3 * Nk)


PREFIX = [
    # B, Hq, Hkv, Nq, Np, Ns, d, a length's step: at 152 SMs
    (157, 32, 8, 8, 300, 40, 64, 17),   # 160 pieces on 80 CTAs, the last query tile one sequence
    (96, 32, 8, 3, 2000, 512, 96, 37),  # 120 pieces, the prefix in three, on 64 CTAs
    (40, 64, 4, 16, 1100, 0, 64, 1),    # no keys after the prefix
]


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Np,Ns,d,step", PREFIX)
def test_prefix_over_several_items_a_cta(fa, B, Hq, Hkv, Nq, Np, Ns, d, step):
    lens = [step * i % (Ns + 1) for i in range(B)]
    host = make("bf16", B, Hq, Hkv, Nq, Np, Ns, d, lens, seed=B + Np)
    o, lse = fa.fa_fwd_shared_prefix(*[t.cuda() for t in host], torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    q, kp, vp, k, v = host
    for b in range(B):
        o_ref, lse_ref, tol_o, tol_l = expect("bf16", q[b:b + 1], kp, vp, k[b:b + 1], v[b:b + 1], lens[b:b + 1], d ** -0.5)
        sb.check(f"o[{b}]", sb.f64(o[b:b + 1]), o_ref, tol_o)
        sb.check(f"lse[{b}]", sb.f64(lse[b:b + 1]), lse_ref, tol_l)


def test_expanded_chunk_padded_on_the_right(fa):
    """Chunks of unequal length after pasts of one length, padded on the right
    (finite values, dO = 0): results and gradients of the real tokens are those
    of the call without padding, bit for bit for the forward and dq."""
    past, Nq, real = 90, 200, 133
    Nk = past + Nq
    q, kn, kr, v, do = (t.cuda() for t in expanded("bf16", 2, 3, Nq, Nk, 128, 64, 128, seed=21))
    do[:, :, real:] = 0
    o, lse = fa.fa_fwd_latent(q, kn, kr, v)
    grads = fa.fa_bwd_latent(q, kn, kr, v, o, lse, do)
    n = past + real
    cut = [t.contiguous() for t in (q[:, :, :real], kn[:, :, :n], kr[:, :n], v[:, :, :n])]
    o2, lse2 = fa.fa_fwd_latent(*cut)
    want = fa.fa_bwd_latent(*cut, o2, lse2, do[:, :, :real].contiguous())
    assert torch.equal(o[:, :, :real], o2) and torch.equal(lse[:, :, :real], lse2)
    assert torch.equal(grads[0][:, :, :real], want[0])
    # dk and dv: the padded rows add products with zeros, so that only the sign of a zero could differ
    for got, ref in ((grads[1][:, :, :n], want[1]), (grads[2][:, :n], want[2]), (grads[3][:, :, :n], want[3])):
        assert (got == ref).all()
    for g in (grads[1][:, :, n:], grads[2][:, n:], grads[3][:, :, n:]):
        assert (g == 0).all()
