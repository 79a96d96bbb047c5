"""Shared-prefix attention on the GPU, element by element against the float64
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


def make(dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens, seed=0, mult=1.0, poison=True):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]

    def n(*shape):
        return torch.randn(shape, generator=g).mul_(mult).to(t)

    q, kp, vp, k, v = n(B, Hq, Nq, d), n(Hkv, Np, d), n(Hkv, Np, d), n(B, Hkv, Ns, d), n(B, Hkv, Ns, d)
    if poison:  # positions past a sequence's length may hold anything
        for b, m in enumerate(lens):
            k[b, :, m:] = float("nan")
            v[b, :, m:] = float("inf")
    return q, kp, vp, k, v


def expect(dtype, q, kp, vp, k, v, lens, scale):
    """(O, lse, tolerances) for the whole batch."""
    B, Hq, Nq, d = q.shape
    G = Hq // kp.shape[0]
    out = []
    for b, m in enumerate(lens):
        keys = np.concatenate([sb.f64(kp), sb.f64(k[b, :, :m])], 1).repeat(G, 0)
        vals = np.concatenate([sb.f64(vp), sb.f64(v[b, :, :m])], 1).repeat(G, 0)
        Np = kp.shape[1]
        vis = np.concatenate([np.ones((Nq, Np), bool), oracle.new_token_mask(Nq, m)], 1)
        out.append(sb.forward(sb.f64(q[b]), keys, vals, scale, vis, dtype))
    return tuple(np.stack(x) for x in zip(*out))


CASES = [
    # dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens
    ("bf16", 1, 1, 1, 1, 1, 1, 64, [1]),                    # the smallest call
    ("bf16", 1, 1, 1, 1, 1, 0, 64, [0]),                    # nothing after the prefix
    ("bf16", 2, 4, 2, 1, 0, 9, 64, [9, 0]),                 # no prefix; the second row sees nothing
    ("bf16", 5, 8, 2, 1, 127, 70, 64, [1, 63, 64, 65, 70]),  # lengths around a tile
    ("bf16", 3, 10, 2, 3, 129, 130, 96, [2, 130, 3]),       # five query heads a key head; rows before a short sequence
    ("bf16", 2, 16, 2, 9, 300, 65, 128, [5, 65]),           # 72 rows a group
    ("bf16", 40, 16, 2, 1, 1000, 33, 128, [i % 34 for i in range(40)]),  # 320 rows share the prefix
    ("bf16", 33, 8, 8, 2, 513, 20, 64, [i % 21 for i in range(33)]),
    ("bf16", 2, 8, 1, 40, 200, 50, 128, [50, 41]),          # 320 rows of one sequence
    ("bf16", 3, 8, 1, 6, 100, 130, 64, [130, 70, 0]),       # 48 rows a sequence
    ("bf16", 3, 10, 2, 7, 0, 130, 96, [64, 129, 1]),        # 35 rows, no prefix
    ("bf16", 24, 16, 2, 8, 130, 700, 128, [700 - 29 * i for i in range(24)]),  # 64 rows, many pieces
    ("bf16", 24, 16, 2, 4, 130, 700, 64, [700 - 29 * i for i in range(24)]),   # 32 rows
    ("f32", 1, 8, 8, 40, 100, 130, 64, [130]),              # rows enough for wider tiles
    ("bf16", 1, 2, 1, 1, 5000, 3000, 128, [2999]),          # many splits of both parts
    ("f32", 1, 1, 1, 1, 1, 0, 1, [0]),
    ("f32", 3, 6, 2, 1, 65, 40, 80, [0, 1, 40]),
    ("f32", 2, 4, 4, 5, 100, 30, 37, [3, 30]),
    ("f32", 9, 8, 2, 2, 700, 129, 128, [129, 0, 1, 2, 64, 65, 128, 127, 3]),
]


@pytest.mark.parametrize("dtype,B,Hq,Hkv,Nq,Np,Ns,d,lens", CASES)
def test_against_definition(fa, dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens):
    host = make(dtype, B, Hq, Hkv, Nq, Np, Ns, d, lens, seed=B + Np)
    o_ref, lse_ref, tol_o, tol_l = expect(dtype, *host, lens, d ** -0.5)
    dev = [t.cuda() for t in host]
    o, lse = fa.fa_fwd_shared_prefix(*dev, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits(fa, dtype):
    """Scores of some hundreds: the running maximum rises across tiles and parts."""
    lens = [65, 130, 1]
    host = make(dtype, 3, 4, 2, 2, 400, 130, 64, lens, seed=3, mult=6.0)
    o_ref, lse_ref, tol_o, tol_l = expect(dtype, *host, lens, 0.125)
    o, lse = fa.fa_fwd_shared_prefix(*[t.cuda() for t in host], torch.tensor(lens, dtype=torch.int32, device="cuda"))
    sb.check("o", sb.f64(o), o_ref, tol_o)
    sb.check("lse", sb.f64(lse), lse_ref, tol_l)


def test_repeats_bit_for_bit_and_leaves_guards(fa):
    """Two calls agree bit for bit; nothing is written around the outputs; a poisoned workspace changes nothing."""
    lens = [70, 3, 0, 33]
    q, kp, vp, k, v = (t.cuda() for t in make("bf16", 4, 8, 2, 1, 700, 70, 64, lens, seed=8))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = fa.fa_fwd_shared_prefix_workspace_bytes(4, 8, 2, 1, 700, 70, 64)
    outs = []
    for fill in (0, 255):
        guard = torch.full((q.numel() + 2048,), 7.0, device="cuda", dtype=q.dtype)
        lguard = torch.full((4 * 8 + 512,), 7.0, device="cuda")
        ws = torch.full((need,), fill, device="cuda", dtype=torch.uint8)
        o, lse = guard[1024:1024 + q.numel()].view(q.shape), lguard[256:256 + 32].view(4, 8, 1)
        fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln, o=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert (guard[:1024] == 7).all() and (guard[-1024:] == 7).all()
        assert (lguard[:256] == 7).all() and (lguard[-256:] == 7).all()
        outs.append((o.clone(), lse.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_out_of_range_are_reported(fa, dtype):
    """A length past the capacity counts as the capacity, one below 0 as 0, and the status says so."""
    lens = [40, 0]
    host = make(dtype, 2, 2, 1, 1, 50, 40, 64, lens, seed=5)
    dev = [t.cuda() for t in host]
    good = fa.fa_fwd_shared_prefix(*dev, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert fa.fa_last_device_status() == fa.FA_OK
    bad = fa.fa_fwd_shared_prefix(*dev, torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda"))
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID
    assert fa.fa_last_device_status() == fa.FA_OK  # cleared by reading
    assert torch.equal(good[0], bad[0]) and torch.equal(good[1], bad[1])


def test_replays_in_a_graph_with_new_lengths(fa):
    lens = [33, 64, 7]
    q, kp, vp, k, v = (t.cuda() for t in make("bf16", 3, 8, 2, 2, 300, 64, 128, [64] * 3, seed=11))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((3, 8, 2), device="cuda")
    ws = torch.empty(fa.fa_fwd_shared_prefix_workspace_bytes(3, 8, 2, 2, 300, 64, 128), device="cuda", dtype=torch.uint8)
    call = lambda: fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln, o=o, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1, 0, 64], [64, 64, 64]):
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        ref = fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_on_a_busy_stream_of_its_own(fa):
    lens = [20, 30]
    dev = [t.cuda() for t in make("bf16", 2, 4, 2, 1, 200, 30, 64, lens, seed=13)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = fa.fa_fwd_shared_prefix(*dev, ln)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
    got = [fa.fa_fwd_shared_prefix(*dev, ln, stream=s) for _ in range(3)]
    s.synchronize()
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_refusals(fa):
    q, kp, vp, k, v = (t.cuda() for t in make("bf16", 2, 4, 2, 1, 20, 8, 64, [8, 8], seed=1))
    ln = torch.tensor([8, 8], dtype=torch.int32, device="cuda")
    for bad in ((q.float(), kp, vp, k, v, ln), (q, kp[:1], vp, k, v, ln), (q, kp, vp[:, :10], k, v, ln),
                (q, kp, vp, k[:1], v, ln), (q, kp, vp, k, v[:, :, :4], ln), (q, kp, vp, k, v, ln.long()),
                (q, kp, vp, k, v, ln[:1]), (q, kp, vp, k, v, ln.cpu()), (q, kp.cpu(), vp, k, v, ln),
                (q[0], kp, vp, k, v, ln), (q.transpose(0, 1), kp, vp, k, v, ln)):
        with pytest.raises(ValueError):
            fa.fa_fwd_shared_prefix(*bad)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln, scale=0.0)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln, workspace=torch.empty(256, device="cuda", dtype=torch.uint8))
    with pytest.raises(ValueError):
        fa.fa_fwd_shared_prefix(q, kp, vp, k, v, ln, o=torch.empty(1, device="cuda"))
    with pytest.raises(TypeError):
        fa.fa_fwd_shared_prefix(*(t.half() for t in (q, kp, vp, k, v)), ln)
