"""Latent attention on the GPU: the expanded form's forward and backward and
the absorbed form over a paged cache, element by element against the float64
definition within the bounds of tests/seq_bounds.py."""

import numpy as np
import pytest

import oracle
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


# ------------------------------------------------------------ expanded form
def expanded(dtype, B, H, Nq, Nk, dn, dr, dv, seed=0, mult=1.0):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g).mul_(mult).to(TYPES[dtype])

    return n(B, H, Nq, dn + dr), n(B, H, Nk, dn), n(B, Nk, dr), n(B, H, Nk, dv), n(B, H, Nq, dv)


def keys_of(kn, kr):
    kn, kr = sb.f64(kn), sb.f64(kr)
    return np.concatenate([kn, np.broadcast_to(kr[:, None], kn.shape[:3] + kr.shape[-1:])], -1)


EXPANDED = [
    # dtype, B, H, Nq, Nk, dn, dr, dv, causal
    ("bf16", 1, 1, 1, 1, 128, 64, 128, True),
    ("bf16", 1, 2, 1, 200, 128, 64, 128, True),     # one new token
    ("bf16", 2, 3, 130, 130, 128, 64, 128, True),
    ("bf16", 1, 2, 300, 300, 128, 64, 128, False),
    ("bf16", 1, 2, 127, 385, 128, 64, 128, True),   # a chunk against a longer past
    ("bf16", 2, 1, 257, 64, 128, 64, 128, True),    # the first 193 rows see nothing
    ("bf16", 1, 1, 140, 129, 128, 64, 128, True),
    ("bf16", 1, 1, 65, 700, 128, 64, 128, False),
    ("bf16", 1, 5, 600, 600, 128, 64, 128, True),
    ("f32", 1, 1, 1, 1, 1, 1, 1, True),
    ("f32", 2, 3, 70, 70, 48, 20, 40, True),
    ("f32", 1, 2, 40, 133, 65, 7, 128, True),
    ("f32", 1, 2, 90, 30, 128, 64, 64, True),
    ("f32", 2, 2, 33, 65, 192, 64, 33, False),
    # heads enough that a CTA takes 32 or 64 rows, at every register width of the backward
    ("f32", 8, 10, 65, 65, 20, 7, 40, True),
    ("f32", 8, 10, 65, 65, 48, 20, 40, True),
    ("f32", 8, 10, 65, 100, 64, 64, 128, False),
    ("f32", 8, 10, 70, 65, 96, 64, 128, True),
    ("f32", 8, 10, 65, 65, 96, 64, 60, True),
    ("f32", 8, 10, 65, 65, 192, 64, 60, True),
    ("f32", 8, 10, 65, 65, 192, 64, 128, True),
]


@pytest.mark.parametrize("dtype,B,H,Nq,Nk,dn,dr,dv,causal", EXPANDED)
def test_expanded_forward_and_backward(fa, dtype, B, H, Nq, Nk, dn, dr, dv, causal):
    host = expanded(dtype, B, H, Nq, Nk, dn, dr, dv, seed=Nq + Nk)
    q, kn, kr, v, do = (t.cuda() for t in host)
    vis = oracle.new_token_mask(Nq, Nk) if causal else np.ones((Nq, Nk), bool)
    scale = (dn + dr) ** -0.5
    args = (sb.f64(host[0]), keys_of(host[1], host[2]), sb.f64(host[3]))
    o_ref, lse_ref, tol_o, tol_l = sb.forward(*args, scale, vis, dtype)
    o, lse = fa.fa_fwd_latent(q, kn, kr, v, causal=causal)
    grads = fa.fa_bwd_latent(q, kn, kr, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)
    (dq, dk, dv_), (tq, tk, tv) = sb.backward(*args, sb.f64(host[4]), scale, vis, dtype)
    u = sb.HALF[dtype]
    for name, got, want, tol in (("dq", grads[0], dq, tq), ("dk_nope", grads[1], dk[..., :dn], tk[..., :dn]),
                                 ("dk_rope", grads[2], dk[..., dn:].sum(1),
                                  tk[..., dn:].sum(1) + H * 2.0 ** -24 * np.abs(dk[..., dn:]).sum(1)),
                                 ("dv", grads[3], dv_, tv)):
        sb.check(name, sb.f64(got), want, tol + u * (np.abs(want) + tol) + 1e-30)


def test_expanded_gradient_against_differences(fa):
    """float32: the change of sum(O dO) along a direction, by central differences of the forward."""
    host = expanded("f32", 1, 2, 20, 24, 16, 8, 12, seed=4)
    q, kn, kr, v, do = (t.cuda() for t in host)
    o, lse = fa.fa_fwd_latent(q, kn, kr, v)
    grads = fa.fa_bwd_latent(q, kn, kr, v, o, lse, do)
    h = 2.0 ** -7
    for i, (x, g) in enumerate(zip((q, kn, kr, v), grads)):
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).cuda()
        d /= d.norm()
        ins = [q, kn, kr, v]
        f = []
        for sgn in (1.0, -1.0):
            ins[i] = x + sgn * h * d
            f.append(float((fa.fa_fwd_latent(*ins)[0].double() * do.double()).sum()))
        num, ana = (f[0] - f[1]) / (2 * h), float((g.double() * d.double()).sum())
        # truncation h^2 / 6 times a third derivative along a unit vector (a few |do||v|, about 22 * 3.5), rounding
        # 480 terms of 2^-22 over 2 h
        tol = h * h / 6 * 400 + 480 * 2.0 ** -22 / (2 * h)
        assert abs(num - ana) <= tol, (i, num, ana, tol)


def test_expanded_large_logits(fa):
    host = expanded("bf16", 1, 2, 300, 300, 128, 64, 128, seed=6, mult=4.0)
    vis = oracle.new_token_mask(300, 300)
    o_ref, lse_ref, tol_o, tol_l = sb.forward(sb.f64(host[0]), keys_of(host[1], host[2]), sb.f64(host[3]), 192 ** -0.5,
                                              vis, "bf16")
    o, lse = fa.fa_fwd_latent(*(t.cuda() for t in host[:4]))
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


def test_expanded_repeats_bit_for_bit(fa):
    q, kn, kr, v, do = (t.cuda() for t in expanded("bf16", 2, 3, 400, 400, 128, 64, 128, seed=7))
    need = fa.fa_bwd_latent_workspace_bytes(2, 3, 400, 400, 128, 64, 128)
    outs = []
    for fill in (0, 255):
        o, lse = fa.fa_fwd_latent(q, kn, kr, v)
        ws = torch.full((need,), fill, device="cuda", dtype=torch.uint8)
        outs.append((o, lse) + fa.fa_bwd_latent(q, kn, kr, v, o, lse, do, workspace=ws))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_expanded_step_replays_in_a_graph(fa):
    bufs = [t.cuda() for t in expanded("bf16", 1, 2, 260, 260, 128, 64, 128, seed=9)]
    q, kn, kr, v, do = bufs
    o, lse = torch.empty((1, 2, 260, 128), device="cuda", dtype=q.dtype), torch.empty((1, 2, 260), device="cuda")
    grads = [torch.empty_like(t) for t in (q, kn, kr, v)]
    ws = torch.empty(fa.fa_bwd_latent_workspace_bytes(1, 2, 260, 260, 128, 64, 128), device="cuda", dtype=torch.uint8)

    def step():
        fa.fa_fwd_latent(q, kn, kr, v, o=o, lse=lse)
        fa.fa_bwd_latent(q, kn, kr, v, o, lse, do, dq=grads[0], dk_nope=grads[1], dk_rope=grads[2], dv=grads[3],
                         workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for dst, src in zip(bufs, expanded("bf16", 1, 2, 260, 260, 128, 64, 128, seed=10)):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    ref_o, ref_l = fa.fa_fwd_latent(q, kn, kr, v)
    ref = fa.fa_bwd_latent(q, kn, kr, v, ref_o, ref_l, do)
    assert torch.equal(o, ref_o) and torch.equal(lse, ref_l)
    for a, b in zip(grads, ref):
        assert torch.equal(a, b)


def test_expanded_right_padding_changes_nothing(fa):
    """causal: the rows of a short sequence do not depend on the (finite) padding behind them."""
    q, kn, kr, v, do = (t.cuda() for t in expanded("bf16", 2, 2, 200, 200, 128, 64, 128, seed=12))
    o, lse = fa.fa_fwd_latent(q, kn, kr, v)
    cut = [t[:, :, :150].contiguous() for t in (q, kn, v)]
    o2, lse2 = fa.fa_fwd_latent(cut[0], cut[1], kr[:, :150].contiguous(), cut[2])
    assert torch.equal(o[:, :, :150], o2) and torch.equal(lse[:, :, :150], lse2)


# ------------------------------------------------------------ absorbed form
def absorbed(dtype, B, H, Nq, page, dc, dr, lens, seed=0, mult=1.0, spare=2, table=True):
    """Host tensors: q, cache, table (or None), and each sequence's rows gathered in order."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    q = torch.randn((B, H, Nq, dc + dr), generator=g).mul_(mult).to(t)
    if table:
        wide = max(1, max(-(-n // page) for n in lens))
        held = [-(-n // page) for n in lens]
        pages = sum(held) + spare
        order = torch.randperm(pages, generator=g).tolist()
        tab = torch.full((B, wide), -7, dtype=torch.int32)  # entries past a sequence's length are not read
        at = 0
        for b, n in enumerate(held):
            tab[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
    else:
        tab, pages = None, B
    cache = torch.full((pages, page, dc + dr), float("nan")).to(t)  # what no length covers is NaN
    rows = []
    for b, n in enumerate(lens):
        x = torch.randn((n, dc + dr), generator=g).mul_(mult).to(t)
        for p in range(-(-n // page)):
            part = x[p * page:(p + 1) * page]
            cache[int(tab[b, p]) if table else b, :len(part)] = part
        rows.append(x)
    return q, cache, tab, rows


def expect_absorbed(dtype, q, rows, dc, scale):
    out = []
    for b, x in enumerate(rows):
        x = sb.f64(x)[None]
        vis = oracle.new_token_mask(q.shape[2], x.shape[1])
        out.append(sb.forward(sb.f64(q[b]), x, x[..., :dc], scale, vis, dtype))
    return tuple(np.stack(x) for x in zip(*out))


ABSORBED = [
    # dtype, B, H, Nq, page, dc, dr, lens, with a table
    ("bf16", 1, 1, 1, 16, 512, 64, [1], True),
    ("bf16", 3, 16, 1, 64, 512, 64, [0, 64, 777], True),           # an empty sequence
    ("bf16", 4, 16, 1, 16, 512, 64, [15, 16, 17, 200], True),      # pages that end inside a tile
    ("bf16", 3, 16, 2, 48, 512, 64, [1, 47, 333], True),           # a row before its sequence
    ("bf16", 2, 128, 1, 64, 512, 64, [300, 65], True),             # two groups of 64 rows
    ("bf16", 2, 20, 3, 32, 512, 64, [129, 2], True),               # 60 rows
    ("bf16", 2, 33, 2, 16, 512, 64, [100, 63], True),              # 66 rows: a second group of two
    ("bf16", 3, 16, 1, 100, 512, 64, [100, 1, 63], False),         # no table: a padded cache
    ("bf16", 9, 8, 1, 64, 256, 64, [5, 0, 64, 65, 128, 1000, 1, 0, 2], True),
    ("bf16", 1, 16, 1, 64, 512, 64, [9000], True),                 # one long sequence over every SM
    ("f32", 1, 1, 1, 3, 1, 1, [1], True),
    ("f32", 4, 12, 1, 24, 192, 40, [0, 1, 25, 300], True),
    ("f32", 2, 5, 4, 7, 512, 128, [3, 100], True),
    ("f32", 2, 30, 3, 64, 65, 9, [64, 10], False),
]


@pytest.mark.parametrize("dtype,B,H,Nq,page,dc,dr,lens,table", ABSORBED)
def test_absorbed_against_definition(fa, dtype, B, H, Nq, page, dc, dr, lens, table):
    q, cache, tab, rows = absorbed(dtype, B, H, Nq, page, dc, dr, lens, seed=B + H, table=table)
    scale = 192 ** -0.5
    o_ref, lse_ref, tol_o, tol_l = expect_absorbed(dtype, q, rows, dc, scale)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_latent_absorbed(q.cuda(), cache.cuda(), ln, dc, scale,
                                       block_table=None if tab is None else tab.cuda())
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absorbed_large_logits(fa, dtype):
    q, cache, tab, rows = absorbed(dtype, 2, 16, 1, 32, 512, 64, [500, 70], seed=2, mult=3.0)
    o_ref, lse_ref, tol_o, tol_l = expect_absorbed(dtype, q, rows, 512, 0.1)
    o, lse = fa.fa_fwd_latent_absorbed(q.cuda(), cache.cuda(), torch.tensor([500, 70], dtype=torch.int32).cuda(), 512,
                                       0.1, block_table=tab.cuda())
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absorbed_pages_and_lengths_out_of_range_are_reported(fa, dtype):
    """A page outside the cache counts as a page of zeros, a length past the capacity as the capacity."""
    q, cache, tab, rows = absorbed(dtype, 2, 16, 1, 32, 512, 64, [128, 64], seed=3)
    zero = [r.clone() for r in rows]
    zero[0][32:64] = 0
    zero[1][:32] = 0
    o_ref, lse_ref, tol_o, tol_l = expect_absorbed(dtype, q, zero, 512, 0.07)
    tab[0, 1], tab[1, 0] = 10 ** 6, -1
    tab[1, 2:] = tab[1, 1]
    ln = torch.tensor([10 ** 9, 64], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_latent_absorbed(q.cuda(), cache.cuda(), ln, 512, 0.07, block_table=tab.cuda())
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


def test_absorbed_repeats_bit_for_bit_and_leaves_guards(fa):
    q, cache, tab, _ = absorbed("bf16", 3, 16, 1, 16, 512, 64, [900, 0, 65], seed=4)
    q, cache, tab = q.cuda(), cache.cuda(), tab.cuda()
    ln = torch.tensor([900, 0, 65], dtype=torch.int32, device="cuda")
    need = fa.fa_fwd_latent_absorbed_workspace_bytes(3, 16, 1, 16, tab.shape[1], 512)
    n = 3 * 16 * 512
    outs = []
    for fill in (0, 255):
        guard = torch.full((n + 2048,), 7.0, device="cuda", dtype=q.dtype)
        ws = torch.full((need,), fill, device="cuda", dtype=torch.uint8)
        o = guard[1024:1024 + n].view(3, 16, 1, 512)
        _, lse = fa.fa_fwd_latent_absorbed(q, cache, ln, 512, 0.07, block_table=tab, o=o, workspace=ws)
        torch.cuda.synchronize()
        assert (guard[:1024] == 7).all() and (guard[-1024:] == 7).all()
        outs.append((o.clone(), lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_absorbed_replays_in_a_graph_with_new_lengths_and_pages(fa):
    q, cache, tab, _ = absorbed("bf16", 3, 16, 1, 16, 512, 64, [300, 300, 300], seed=5)
    q, cache, tab = q.cuda(), torch.nan_to_num(cache).cuda(), tab.cuda()
    ln = torch.tensor([300, 20, 7], dtype=torch.int32, device="cuda")
    o, lse = torch.empty((3, 16, 1, 512), device="cuda", dtype=q.dtype), torch.empty((3, 16, 1), device="cuda")
    ws = torch.empty(fa.fa_fwd_latent_absorbed_workspace_bytes(3, 16, 1, 16, tab.shape[1], 512), device="cuda",
                     dtype=torch.uint8)
    call = lambda: fa.fa_fwd_latent_absorbed(q, cache, ln, 512, 0.07, block_table=tab, o=o, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1, 0, 299], [300, 300, 300]):
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        tab.copy_(tab.flip(0).contiguous())
        graph.replay()
        torch.cuda.synchronize()
        ref = fa.fa_fwd_latent_absorbed(q, cache, ln, 512, 0.07, block_table=tab)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# ---------------------------------------------------------------- refusals
def test_refusals(fa):
    q, kn, kr, v, do = (t.cuda() for t in expanded("bf16", 2, 2, 8, 8, 128, 64, 128))
    for bad in ((q, kn, kr[:1], v), (q, kn[:, :1], kr, v), (q, kn, kr, v[:, :, :4]), (q.float(), kn, kr, v),
                (q[0], kn, kr, v), (q, kn, kr.cpu(), v), (q, q, kr, v), (q.transpose(1, 2), kn, kr, v)):
        with pytest.raises(ValueError):
            fa.fa_fwd_latent(*bad)
    o, lse = fa.fa_fwd_latent(q, kn, kr, v)
    with pytest.raises(ValueError):
        fa.fa_bwd_latent(q, kn, kr, v, o, lse.half(), do)
    with pytest.raises(ValueError):
        fa.fa_bwd_latent(q, kn, kr, v, o, lse, do[:1])
    with pytest.raises(fa.FaError):
        fa.fa_fwd_latent(q, kn, kr, v, scale=-1.0)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_latent(q[..., :160].contiguous(), kn, kr[..., :32].contiguous(), v)
    with pytest.raises(TypeError):
        fa.fa_fwd_latent(q.half(), kn.half(), kr.half(), v.half())
    aq, cache, tab, _ = absorbed("bf16", 2, 4, 1, 16, 512, 64, [16, 16])
    aq, cache, tab = aq.cuda(), cache.cuda(), tab.cuda()
    ln = torch.tensor([16, 16], dtype=torch.int32, device="cuda")
    for kw in (dict(block_table=tab.long()), dict(block_table=tab[:1]), dict(block_table=tab.cpu())):
        with pytest.raises(ValueError):
            fa.fa_fwd_latent_absorbed(aq, cache, ln, 512, 0.1, **kw)
    with pytest.raises(ValueError):
        fa.fa_fwd_latent_absorbed(aq, cache, ln, 576, 0.1, block_table=tab)
    with pytest.raises(ValueError):
        fa.fa_fwd_latent_absorbed(aq, cache[:, :, :500].contiguous(), ln, 512, 0.1, block_table=tab)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_latent_absorbed(aq, cache[:1], ln, 512, 0.1)  # fewer pages than sequences
    with pytest.raises(fa.FaError):
        fa.fa_fwd_latent_absorbed(aq, cache, ln, 500, 0.1, block_table=tab)
