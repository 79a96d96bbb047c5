"""The 4-bit cache's calls as they are used: a decode loop that writes and
attends, against the framework's other attention calls, on streams, in graphs,
past 32-bit offsets, with bytes that nothing may change."""

import numpy as np
import pytest

import oracle
from tests import cache4_common as cc
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def normal(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 80), ("f32", 64)])
def test_prefill_and_decode_loop(fa, dtype, d):
    """Ragged prompts written at once, then token after token, as a server does:
    every step is the definition's over what the cache then stands for, and what
    it stands for is the tokens within their quantisation."""
    t, B, Hq, Hkv, page, ks, vs = TYPES[dtype], 3, 8, 2, 16, 0.25, 0.5
    lens0 = [37, 0, 16]
    cache = torch.zeros((14, Hkv, page, 9 * d // 8), dtype=torch.uint8, device="cuda")
    table = i32(np.random.default_rng(0).permutation(14)[:12].reshape(3, 4))
    kw = dict(block_table=table, k_scale=ks, v_scale=vs)
    N = max(lens0)
    k0, v0 = normal(B, Hkv, N, d, seed=1, dtype=t), normal(B, Hkv, N, d, seed=2, dtype=t)
    fa.fa_cache_fp4_write(k0, v0, cache, i32(lens0), n_new=i32(lens0), **kw)
    said = [[x[b, :, N - n:].float().cpu() for b, n in enumerate(lens0)] for x in (k0, v0)]
    lens = i32(lens0)
    for step, Nq in enumerate((1, 1, 3, 1)):
        lens += Nq
        q, k, v = normal(B, Hq, Nq, d, seed=10 + step, dtype=t), normal(B, Hkv, Nq, d, seed=20 + step, dtype=t), normal(B, Hkv, Nq, d, seed=30 + step, dtype=t)
        fa.fa_cache_fp4_write(k, v, cache, lens, **kw)
        o, lse = fa.fa_fwd_cache_fp4(q, cache, lens, **kw)
        rk, rv = fa.fa_cache_fp4_read(cache, lens, int(lens.max()), torch.float32, **kw)
        for b in range(B):
            n = int(lens[b])
            for x, new in zip(said, (k, v)):
                x[b] = torch.cat([x[b], new[b].float().cpu()], 1)
            for x, r, s in ((said[0][b], rk, ks), (said[1][b], rv, vs)):
                got = r[b, :, :n].cpu()
                g = x.reshape(*x.shape[:-1], -1, 16)
                # half the widest gap (6 - 4) of amax / 6, which is rounded by 1/16 and to no finer than 2^-9
                tol = (g.abs().amax(-1, keepdim=True) / 6 * (1 + 1 / 16) + s * 2.0 ** -9).expand_as(g).reshape(x.shape)
                assert ((got - x).abs() <= tol).all()
            kd, vd = cc.dense(cache.cpu().numpy(), table.cpu().numpy(), b, n, d, page, ks, vs)
            ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), kd, vd, d ** -0.5, dtype)
            sb.check("o", sb.f64(o[b]), ref, tol)
            sb.check("lse", sb.f64(lse[b]), lr, tol_l)
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.parametrize("dtype,Nq", [("bf16", 1), ("bf16", 5), ("f32", 2)])
def test_is_dense_attention_over_what_is_read_back(fa, dtype, Nq):
    """The shared-prefix call with no prefix, over the keys and values read back.
    The tensors' scales are powers of two, so bf16 holds what is read back exactly
    (6 significant bits)."""
    t, B, Hq, Hkv, page, d, lens = TYPES[dtype], 4, 12, 4, 32, 128, [300, 1, 64, 129]
    rng = np.random.default_rng(4)
    table, pages = cc.place(rng, B, 10, lens, page)
    cache = torch.from_numpy(cc.random_cache(rng, pages, Hkv, page, d)).cuda()
    kw = dict(block_table=i32(table), k_scale=0.25, v_scale=0.5)
    q = torch.from_numpy(rng.standard_normal((B, Hq, Nq, d))).to(t).cuda()
    o, lse = fa.fa_fwd_cache_fp4(q, cache, i32(lens), **kw)
    k, v = fa.fa_cache_fp4_read(cache, i32(lens), 300, t, **kw)
    none = torch.empty((Hkv, 0, d), dtype=t, device="cuda")
    o2, lse2 = fa.fa_fwd_shared_prefix(q, none, none, k, v, i32(lens))
    for b, n in enumerate(lens):
        kd, vd = sb.f64(k[b, :, :n]), sb.f64(v[b, :, :n])
        _, _, tol, tol_l = cc.forward(sb.f64(q[b]), kd, vd, d ** -0.5, dtype)
        G = Hq // Hkv
        ref, lr, tol2, tol_l2 = sb.forward(sb.f64(q[b]), kd.repeat(G, 0), vd.repeat(G, 0), d ** -0.5, oracle.new_token_mask(Nq, n), dtype)
        sb.check("o", sb.f64(o[b]), ref, tol)
        assert (np.abs(sb.f64(o[b]) - sb.f64(o2[b])) <= tol + tol2).all()
        fin = np.isfinite(lr)
        assert (np.abs(sb.f64(lse[b]) - sb.f64(lse2[b]))[fin] <= (tol_l + tol_l2)[fin]).all()


def _case(seed, dtype=torch.bfloat16, d=128, Nq=1, B=5, Hq=16, Hkv=4, page=32):
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, 500, B)]
    table, pages = cc.place(rng, B, 16, lens, page)
    return dict(cache=torch.from_numpy(cc.random_cache(rng, pages, Hkv, page, d)).cuda(), table=i32(table), lens=i32(lens),
                q=normal(B, Hq, Nq, d, seed=seed, dtype=dtype), k=normal(B, Hkv, Nq, d, seed=seed + 1, dtype=dtype),
                v=normal(B, Hkv, Nq, d, seed=seed + 2, dtype=dtype))


def _step(fa, s, stream=None):
    fa.fa_cache_fp4_write(s["k"], s["v"], s["cache"], s["lens"], block_table=s["table"], stream=stream)
    o, lse = fa.fa_fwd_cache_fp4(s["q"], s["cache"], s["lens"], block_table=s["table"], stream=stream)
    return (o, lse) + fa.fa_cache_fp4_read(s["cache"], s["lens"], 40, torch.bfloat16, block_table=s["table"], stream=stream)


def test_two_steps_on_two_streams(fa):
    """Each stream its own cache and workspace (allocated by the call): results as alone, bit for bit."""
    sets = [_case(1), _case(9, Nq=3, d=64)]
    alone = [_step(fa, s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            both[i].append(_step(fa, sets[i], st))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for i in range(2):
        for got in both[i]:
            for a, b in zip(got, alone[i]):
                assert torch.equal(a, b)


def test_given_stream_orders_after_its_work(fa):
    s = _case(3)
    ref = _step(fa, s)
    late = torch.zeros_like(s["q"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        x = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):
            x = x @ x
        late.copy_(s["q"])
    got = _step(fa, {**s, "q": late}, st)
    st.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,Nq", [("bf16", 1), ("bf16", 9), ("f32", 2)])
def test_a_captured_step_follows_its_lengths(fa, dtype, Nq):
    """One graph of write and attention, replayed while the lengths grow in device memory."""
    s = _case(20, dtype=TYPES[dtype], Nq=Nq)
    s["lens"].copy_(i32([Nq, 31, 120, 15, 200]))
    s["table"] = i32(np.arange(80).reshape(5, 16))
    s["cache"] = torch.zeros((80,) + tuple(s["cache"].shape[1:]), dtype=torch.uint8, device="cuda")
    ws = torch.empty(fa.fa_fwd_cache_fp4_workspace_bytes(5, 16, 4, Nq, 32, 16, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:3], device="cuda")

    def step():
        fa.fa_cache_fp4_write(s["k"], s["v"], s["cache"], s["lens"], block_table=s["table"])
        fa.fa_fwd_cache_fp4(s["q"], s["cache"], s["lens"], block_table=s["table"], o=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for name, seed in (("q", 50), ("k", 60), ("v", 70)):
            s[name].copy_(normal(*s[name].shape, seed=seed + i, dtype=TYPES[dtype]))
        s["lens"] += i32([Nq, 1, 100, 0, 33])
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        ref = fa.fa_fwd_cache_fp4(s["q"], s["cache"], s["lens"], block_table=s["table"])
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        assert fa.fa_last_device_status() == fa.FA_OK


def test_two_captured_graphs_with_workspaces_of_their_own(fa):
    sets, graphs, outs, refs = [_case(30), _case(40, Nq=2)], [], [], []
    for s in sets:
        refs.append(_step(fa, s))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # the workspace comes from the graph's own pool
            outs.append(_step(fa, s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        for a, b in zip(o, r):
            assert torch.equal(a, b)


def test_nothing_beyond_outputs_is_written(fa):
    """Outputs inside larger buffers: the bytes around them stay; of the cache, those of other tokens."""
    s = _case(50, Nq=2, d=96, Hq=20)
    B, Hq, Nq, d = s["q"].shape

    def inside(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)

    ob, o = inside((B, Hq, Nq, d), torch.bfloat16)
    lb, lse = inside((B, Hq, Nq), torch.float32)
    kb, k = inside((B, 4, 45, d), torch.bfloat16)
    vb, v = inside((B, 4, 45, d), torch.bfloat16)
    need = fa.fa_fwd_cache_fp4_workspace_bytes(B, Hq, 4, Nq, 32, 16, d)
    ws = torch.full((need + 256,), 9, dtype=torch.uint8, device="cuda")
    before = s["cache"].clone()
    fa.fa_fwd_cache_fp4(s["q"], s["cache"], s["lens"], block_table=s["table"], o=o, lse=lse, workspace=ws[:need])
    fa.fa_cache_fp4_read(s["cache"], s["lens"], 45, block_table=s["table"], first=s["lens"] - 40, k=k, v=v)
    torch.cuda.synchronize()
    assert torch.equal(before, s["cache"])
    for buf in (ob, lb, kb, vb):
        assert (buf[:256] == 7).all() and (buf[-256:] == 7).all()
    assert (ws[need:] == 9).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 80)])
def test_past_32_bit_offsets(fa, dtype, d):
    """A cache past 4 GB, its first and last pages in use; write, read and attention."""
    Hkv, page = 8, 64
    pages = (1 << 32) // (Hkv * page * 9 * d // 8) + 40
    cache = torch.zeros((pages, Hkv, page, 9 * d // 8), dtype=torch.uint8, device="cuda")
    order = [pages - 1, 0, pages - 2, pages // 2, pages - 30, 3]
    table, lens = i32([order[:3], order[3:]]), [150, 129]
    n = max(lens)
    k, v = normal(2, Hkv, n, d, seed=1, dtype=TYPES[dtype]), normal(2, Hkv, n, d, seed=2, dtype=TYPES[dtype])
    q = normal(2, 16, 1, d, seed=3, dtype=TYPES[dtype])
    fa.fa_cache_fp4_write(k, v, cache, i32(lens), block_table=table, n_new=i32(lens), k_scale=0.5, v_scale=0.5)
    rk, rv = fa.fa_cache_fp4_read(cache, i32(lens), n, torch.float32, block_table=table, k_scale=0.5, v_scale=0.5)
    o, lse = fa.fa_fwd_cache_fp4(q, cache, i32(lens), block_table=table, k_scale=0.5, v_scale=0.5)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for b, m in enumerate(lens):
        want = []
        for x, r in ((k, rk), (v, rv)):
            codes, s = oracle.cache4_quantise(sb.f64(x[b, :, n - m:]) / 0.5, 1.0)
            want.append(oracle.cache4_values(codes, s, 0.5))
            assert (sb.f64(r[b, :, :m]) == want[-1]).all()
        ref, lr, tol, tol_l = cc.forward(sb.f64(q[b]), *want, d ** -0.5, dtype)
        sb.check("o", sb.f64(o[b]), ref, tol)
        sb.check("lse", sb.f64(lse[b]), lr, tol_l)
    assert int((cache[4:pages // 2] != 0).sum()) == 0  # other pages untouched


def test_rows_past_32_bit_offsets(fa):
    """Dense keys and values of more than 2^31 entries, read and written."""
    B, Hkv, N, d, page = 3, 8, 700_000, 128, 64
    per = -(-N // page)
    cache = torch.randint(0, 256, (per, Hkv, page, 144), dtype=torch.uint8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    blocks = cache.view(per, Hkv, page // 16, 18 * d)
    blocks[..., 8 * d:9 * d] &= 0x3F
    blocks[..., 17 * d:] &= 0x3F
    table = torch.arange(per, dtype=torch.int32, device="cuda").repeat(B, 1)  # one sequence, read three times
    lens = i32([N, N - 5, N])
    k, v = fa.fa_cache_fp4_read(cache, lens, N, torch.bfloat16, block_table=table)
    for x in (k, v):
        assert torch.equal(x[0, :, :N - 5], x[1, :, :N - 5]) and torch.equal(x[0], x[2]) and (x[1, :, N - 5:] == 0).all()
    kd, vd = cc.dense(cache[per - 2:].cpu().numpy(), np.array([[0, 1]]), 0, N - (per - 2) * page, d, page, 1.0, 1.0)
    assert (sb.f64(k[2, :, (per - 2) * page:]) == kd).all() and (sb.f64(v[2, :, (per - 2) * page:]) == vd).all()
    # what was read quantises to itself: 6 significant bits, and a group's largest entry is at most 6 s
    # with every group's largest code made 6
    again = torch.zeros((3 * per, Hkv, page, 144), dtype=torch.uint8, device="cuda")
    own = torch.arange(3 * per, dtype=torch.int32, device="cuda").view(3, per)
    k[..., ::16], v[..., ::16] = 12.0, -12.0
    k.clamp_(-12, 12), v.clamp_(-12, 12)
    fa.fa_cache_fp4_write(k, v, again, i32([N] * 3), block_table=own)
    rows = slice(N - 100, N)
    rk, rv = fa.fa_cache_fp4_read(again, i32([N] * 3), 100, torch.bfloat16, block_table=own, first=i32([N - 100] * 3))
    for x, r in ((k, rk), (v, rv)):
        codes, s = oracle.cache4_quantise(sb.f64(x[2, :, rows]), 1.0)
        assert (sb.f64(r[2]) == oracle.cache4_values(codes, s, 1.0)).all()
    assert fa.fa_last_device_status() == fa.FA_OK


def test_package_names(fa):
    import exact_tiled_attention_02_gb300 as pkg
    for name in ("fa_cache_fp4_write", "fa_cache_fp4_read", "fa_fwd_cache_fp4", "fa_cache_fp4_bytes"):
        assert getattr(pkg, name) is getattr(fa, name)
