"""The language-model operators as they are used: together, on streams, and
against the framework's other attention calls."""

import numpy as np
import pytest

from tests import seq_bounds as sb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_02_gb300 import binding
    return binding


def _normal(*shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32).to(dtype).cuda()


def test_prefill_then_decode_of_a_latent_model(fa):
    """Prefill in the expanded form, decode in the absorbed one: with the
    up-projections folded into q and applied to O, both are the same
    attention.  float32: the projections here are float64 products rounded to
    float32 once, so the two differ by those roundings (2^-24 relative of sums
    of dc products, a few entries deep) and the kernels' sums."""
    B, H, N, dc, dn, dr, dv, page = 2, 4, 150, 64, 48, 16, 40, 16
    c = _normal(B, N, dc, seed=1)
    kr = _normal(B, N, dr, seed=2)
    q = _normal(B, H, N, dn + dr, seed=3)
    wk, wv = _normal(H, dn, dc, seed=4) / 8, _normal(H, dv, dc, seed=5) / 8
    kn = torch.einsum("bnc,hdc->bhnd", c.double(), wk.double()).float().contiguous()
    v = torch.einsum("bnc,hdc->bhnd", c.double(), wv.double()).float().contiguous()
    scale = (dn + dr) ** -0.5
    o, lse = fa.fa_fwd_latent(q, kn, kr, v, scale=scale)
    # the last three tokens again, as new tokens over a paged cache
    T = 3
    pages = -(-N // page)
    order = torch.randperm(B * pages + 2, generator=torch.Generator().manual_seed(6))[:B * pages].view(B, pages)
    cache = torch.full((B * pages + 2, page, dc + dr), float("nan"), device="cuda")
    rows = torch.cat([c, kr], -1)
    for b in range(B):
        for p in range(pages):
            part = rows[b, p * page:(p + 1) * page]
            cache[order[b, p], :len(part)] = part
    qa = torch.cat([torch.einsum("bhtd,hdc->bhtc", q[:, :, -T:, :dn].double(), wk.double()).float(), q[:, :, -T:, dn:]], -1)
    lat, lse2 = fa.fa_fwd_latent_absorbed(qa.contiguous(), cache, torch.full((B,), N, dtype=torch.int32, device="cuda"), dc,
                                          scale, block_table=order.int().cuda())
    o2 = torch.einsum("bhtc,hdc->bhtd", lat.double(), wv.double())
    # each side: scores off by (dc + dn + dr + 8) 2^-22 of their absolute sums (under 40 here), P and so O by twice that
    # relative to sum P |v| (under 4), the kernels' sums over 150 keys within the same
    tol = 2 * 2 * (dc + dn + dr + 8) * 2.0 ** -22 * 40 * 4
    assert float((o2 - o[:, :, -T:].double()).abs().max()) <= tol
    assert float((lse2 - lse[:, :, -T:]).abs().max()) <= tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_prefix_is_the_last_row_of_full_attention(fa, dtype):
    """One new token after a prefix and some of its own: the last query row of
    fa_fwd over the whole sequence."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    H, Np, d, lens = 3, 200, 64, [1, 56, 30]
    kp, vp = _normal(H, Np, d, seed=1, dtype=t), _normal(H, Np, d, seed=2, dtype=t)
    k, v = _normal(3, H, 56, d, seed=3, dtype=t), _normal(3, H, 56, d, seed=4, dtype=t)
    q = _normal(3, H, 1, d, seed=5, dtype=t)
    o, lse = fa.fa_fwd_shared_prefix(q, kp, vp, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lens):
        ks, vs = torch.cat([kp, k[b, :, :n]], 1)[None].contiguous(), torch.cat([vp, v[b, :, :n]], 1)[None].contiguous()
        qs = torch.zeros_like(ks)
        qs[0, :, -1] = q[b, :, 0]
        of, lf = fa.fa_fwd(qs, ks, vs)
        ref, lr, tol_o, tol_l = sb.forward(sb.f64(q[b]), sb.f64(ks[0]), sb.f64(vs[0]), d ** -0.5, True, dtype)
        sb.check("o", sb.f64(o[b]), ref, tol_o)
        sb.check("fa_fwd", sb.f64(of[0, :, -1:]), ref, tol_o)
        assert (np.abs(sb.f64(lse[b]) - sb.f64(lf[0, :, -1:])) <= 2 * tol_l).all()


def test_two_steps_on_two_streams(fa):
    """Each stream its own buffers and workspace (allocated by the calls): results as alone, bit for bit."""
    t = torch.bfloat16
    sets = []
    for i in range(2):
        q, kn, kr = (_normal(*s, seed=10 * i + j, dtype=t) for j, s in enumerate(((2, 4, 333, 192), (2, 4, 333, 128), (2, 333, 64))))
        v, do = _normal(2, 4, 333, 128, seed=10 * i + 5, dtype=t), _normal(2, 4, 333, 128, seed=10 * i + 6, dtype=t)
        sets.append((q, kn, kr, v, do))

    def step(x, stream=None):
        q, kn, kr, v, do = x
        o, lse = fa.fa_fwd_latent(q, kn, kr, v, stream=stream)
        return (o, lse) + fa.fa_bwd_latent(q, kn, kr, v, o, lse, do, stream=stream)

    alone = [step(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            both[i].append(step(sets[i], s))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for i in range(2):
        for got in both[i]:
            for a, b in zip(got, alone[i]):
                assert torch.equal(a, b)


def test_decode_loop_over_a_growing_cache(fa):
    """Token after token, as a server does: every step's result is the
    definition's over the cache so far."""
    B, H, page, dc, dr = 3, 16, 16, 512, 64
    lens = torch.tensor([14, 0, 63], dtype=torch.int32, device="cuda")
    cache = torch.randn((20, page, dc + dr), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:18].view(3, 6).int().cuda()
    import oracle
    for step in range(4):
        lens += 1
        q = _normal(B, H, 1, dc + dr, seed=step, dtype=torch.bfloat16)
        o, lse = fa.fa_fwd_latent_absorbed(q, cache, lens, dc, 0.07, block_table=table)
        for b in range(B):
            n = int(lens[b])
            x = sb.f64(cache[table[b].long()].reshape(-1, dc + dr)[:n])[None]
            ref, lr, tol_o, tol_l = sb.forward(sb.f64(q[b]), x, x[..., :dc], 0.07, oracle.new_token_mask(1, n), "bf16")
            sb.check("o", sb.f64(o[b]), ref, tol_o)
            sb.check("lse", sb.f64(lse[b]), lr, tol_l)


def test_given_stream_orders_after_its_work(fa):
    """The calls run on the stream given, behind what is queued there."""
    s = torch.cuda.Stream()
    q, cache = _normal(2, 16, 1, 576, seed=1, dtype=torch.bfloat16), _normal(8, 64, 576, seed=2, dtype=torch.bfloat16)
    lens = torch.tensor([200, 100], dtype=torch.int32, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    ref = fa.fa_fwd_latent_absorbed(q, cache, lens, 512, 0.07, block_table=table)
    late = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):
            x = x @ x
        late.copy_(q)
    got = fa.fa_fwd_latent_absorbed(late, cache, lens, 512, 0.07, block_table=table, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_two_captured_graphs_with_workspaces_of_their_own(fa):
    t = torch.bfloat16
    kp, vp = _normal(2, 300, 64, seed=1, dtype=t), _normal(2, 300, 64, seed=2, dtype=t)
    graphs, outs, refs = [], [], []
    for i in range(2):
        q, k, v = (_normal(*s, seed=20 * i + j, dtype=t) for j, s in enumerate(((5, 8, 1, 64), (5, 2, 90, 64), (5, 2, 90, 64))))
        lens = torch.tensor([90, 0, 1, 64, 65], dtype=torch.int32, device="cuda")
        refs.append(fa.fa_fwd_shared_prefix(q, kp, vp, k, v, lens))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # the workspace comes from the graph's own pool
            outs.append(fa.fa_fwd_shared_prefix(q, kp, vp, k, v, lens))
        graphs.append((g, q, k, v, lens))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g[0].replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])
