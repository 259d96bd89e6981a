"""MXFP4 pools, attention with accumulated key weights, and eviction by weight on the GPU, against
the definitions in 64 bits (oracle/mxfp4.py, oracle/eviction.py).

Tolerances.  Codes, scale bytes, kept positions and moved bytes are exact.
* Scores: an fp32 sum of D products is off by at most (D + 2) 2^-24 sum|q_d k_d|; with |q|, |k| of
  N(0, 1) inputs, D = 128 and scale D^-1/2, scale sum|q k| log2(e) stays below 24, so a score (log2
  domain) is off by less than 2e-4, and so is a log-sum-exp; 2^x turns that into 3e-4 relative
  (2 x 2e-4 ln 2), with 2^x itself and the sums below 1e-5: weights within 4e-4 relative.
* MXFP4 attention rounds each probability to f16 (2^-12 relative; scales are applied in fp32) and
  uses the codes as they are: |out - ref| <= (2^-12 + 4e-4) max|v|.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import e4m3_decode  # noqa: E402
from oracle import eviction, mxfp4  # noqa: E402

BS = 16
KSC, VSC = 0.0125, 0.015625


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_286_gb300 import build
    build.build()


def bits_f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """Pools of one kind with random contents (stale slots hold NaN patterns) and their values."""

    def __init__(self, ctx, qlens, hq, hkv, d, kind, seed=0, spare=3, spread=0, cols=1, bound=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.qlens = np.array(ctx, np.int32), np.array(qlens, np.int32)
        self.hq, self.hkv, self.d, self.kind = hq, hkv, d, kind
        self.bound = max(bound, int(self.ctx.max()))                # max_context_len of the calls
        S = len(ctx)
        nblk = -(-self.ctx // BS)
        nb = int(nblk.sum()) + spare
        ids = rng.permutation(nb)
        self.tables = np.full((S, max(1, int(nblk.max())) + cols), -1, np.int32)
        at = 0
        for s in range(S):
            self.tables[s, :nblk[s]] = ids[at:at + nblk[s]]
            at += nblk[s]
        self.free = ids[at:]
        self.scale = d ** -0.5

        def pool(sc):
            x = torch.randn((nb, hkv, BS, d), generator=g)
            if spread:  # scale blocks of very different size
                e = torch.randint(-spread, spread + 1, (nb, hkv, BS, d // 32, 1), generator=g)
                x = (x.reshape(nb, hkv, BS, -1, 32) * torch.exp2(e.float())).reshape(x.shape)
            x = x.bfloat16()
            stale = torch.ones(nb, BS, dtype=torch.bool)
            for s in range(S):
                for j in range(int(nblk[s])):
                    stale[self.tables[s, j], :max(0, min(BS, int(self.ctx[s]) - BS * j))] = False
            stale = stale[:, None, :].expand(nb, hkv, BS)
            if kind == "bf16":
                raw = x.clone()
                raw[stale] = float("nan")
                return raw.cuda(), bits_f64(x)
            if kind == "e4m3":
                q = (x.float() / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                vals = e4m3_decode(q.numpy()) * float(np.float32(sc))
                q[stale] = 0x7F
                return q.cuda(), vals
            codes, byte = mxfp4.encode(bits_f64(x))
            vals = mxfp4.decode(codes, byte)
            byte[stale.numpy()] = 255
            codes[stale.numpy()] = 13
            return torch.from_numpy(mxfp4.pack_tiles(codes, byte)).cuda(), vals

        self.k, self.kv = pool(KSC)
        self.v, self.vv = pool(VSC)
        T = int(self.qlens.sum())
        self.q = torch.randn((T, hq, d), generator=g).bfloat16()
        self.qsl = np.concatenate([[0], np.cumsum(self.qlens)]).astype(np.int32)
        self.scales = dict(k_scale=KSC, v_scale=VSC) if kind == "e4m3" else {}

    def dev(self):
        return [torch.from_numpy(x).cuda() for x in (self.tables, self.ctx, self.qsl)]

    def context(self, s):
        L = int(self.ctx[s])
        ids = self.tables[s, :-(-L // BS)]
        f = lambda p: p[ids].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[:L]  # noqa: E731
        return f(self.kv), f(self.vv)

    def reference(self):
        q = bits_f64(self.q)
        outs, ws = [], []
        for s in range(len(self.ctx)):
            L, n = int(self.ctx[s]), int(self.qlens[s])
            if n == 0:
                ws.append(None)
                continue
            K, V = self.context(s)
            o, w = eviction.attend_with_weights(q[self.qsl[s]:self.qsl[s] + n], K, V, L - n, self.scale)
            outs.append(o)
            ws.append(w)
        return np.concatenate(outs), ws

    def workspace(self, pa, weights=False):
        f = pa.attention_key_weights_workspace_size if weights else pa.attention_workspace_size
        return pa.new_workspace(f(len(self.ctx), self.q.shape[0], self.hq, self.hkv, self.d,
                                  self.bound, int(self.qlens.max())))

    def hints(self):
        return dict(scale=self.scale, max_context_len=self.bound,
                    max_query_len=int(self.qlens.max()), **self.scales)


# ---------------------------------------------------------------------------------------------
# MXFP4 append and read
# ---------------------------------------------------------------------------------------------
def mx_inputs(d, T, hkv, seed):
    """Blocks of every scale, with zeros, ties, subnormals, infinities and NaN among them."""
    rng = np.random.default_rng(seed)
    bits = rng.integers(0, 1 << 16, (T, hkv, d), dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).clone()
    n = T // 2
    e = torch.from_numpy(rng.integers(-130, 127, (n, hkv, d // 32, 1))).float()
    y = torch.from_numpy(rng.standard_normal((n, hkv, d // 32, 32)).astype(np.float32))
    x[:n] = (y.double() * torch.exp2(e.double())).float().reshape(n, hkv, d).bfloat16()
    # exact multiples of a quarter of the scale: every value between codes, ties included
    grid = torch.from_numpy(rng.integers(-31, 32, (n // 2, hkv, d)).astype(np.float32)) / 4
    x[:n // 2] = grid.bfloat16()
    x[0] = 0.0
    x[1, 0, :32] = -0.0
    x[2, 0, 5] = float("inf")
    x[3, 0, 7] = float("nan")
    return x


@pytest.mark.parametrize("d,hkv,T", [(128, 8, 301), (64, 3, 97), (128, 1, 33), (64, 1, 1024)])
def test_mxfp4_append_and_read(d, hkv, T):
    import paged_kv_cache_286_gb300 as pa
    k, v = mx_inputs(d, T, hkv, 1), mx_inputs(d, T, hkv, 2)
    nb = T // BS + 3
    rng = np.random.default_rng(3)
    slots = rng.permutation(nb * BS)[:T].astype(np.int64)
    slots[4] = -1
    kc, vc = pa.new_mxfp4_cache(nb, hkv, d), pa.new_mxfp4_cache(nb, hkv, d)
    kc.fill_(0xAB), vc.fill_(0xAB)
    ws = pa.new_workspace(256)
    ts = torch.from_numpy(slots).cuda()
    pa.cache_append(k.cuda(), v.cuda(), ts, kc, vc, ws)
    outs = {t: pa.cache_read(ts, kc, vc, ws, out_dtype=t) for t in (torch.bfloat16, torch.float32)}
    assert pa.check_error(ws) == 0
    for x, pool, i in ((k, kc, 0), (v, vc, 1)):
        codes, byte = mxfp4.encode(bits_f64(x))
        start = mxfp4.unpack_tiles(np.full((nb, hkv, 17 * d // 2), 0xAB, np.uint8))
        for t in range(T):
            if slots[t] >= 0:
                start[0][slots[t] // BS, :, slots[t] % BS] = codes[t]
                start[1][slots[t] // BS, :, slots[t] % BS] = byte[t]
        assert np.array_equal(pool.cpu().numpy(), mxfp4.pack_tiles(*start))
        want = mxfp4.decode(codes, byte)
        want[np.broadcast_to((byte == 0)[..., None], byte.shape + (32,)).reshape(want.shape)] *= 0  # 2^-127
        want[4] = 0.0
        for t in outs:
            got = outs[t][i].float().cpu().numpy()
            w32 = want.astype(np.float32)
            assert outs[t][i].dtype == t
            assert np.array_equal(got, w32, equal_nan=True)


def test_read_of_bf16_and_e4m3_pools_and_bad_slots():
    import paged_kv_cache_286_gb300 as pa
    for kind in ("bf16", "e4m3"):
        c = Case([40, 17], [1, 1], 4, 2, 128, kind, seed=4)
        slots = np.array([int(c.tables[0, 1]) * BS + 3, -5, int(c.tables[1, 0]) * BS, 10 ** 9], np.int64)
        ws = pa.new_workspace(256)
        k, v = pa.cache_read(torch.from_numpy(slots).cuda(), c.k, c.v, ws, out_dtype=torch.float32, **c.scales)
        assert pa.check_error(ws, raise_on_error=False) == 0x2
        for got, vals in ((k, c.kv), (v, c.vv)):
            got = got.cpu().numpy()
            assert not got[1].any() and not got[3].any()
            for i in (0, 2):
                want = vals[slots[i] // BS, :, slots[i] % BS]
                assert np.abs(got[i] - want).max() <= 2.0 ** -24 * np.abs(want).max()


@pytest.mark.parametrize("d", [64, 128])
def test_copy_blocks_of_an_mxfp4_pool(d):
    import ctypes
    import paged_kv_cache_286_gb300 as pa
    g = torch.Generator().manual_seed(6)
    k = torch.randint(0, 256, (9, 3, 17 * d // 2), generator=g, dtype=torch.uint8).cuda()
    v = k.flip(0).contiguous()
    want = [x.clone() for x in (k, v)]
    for x in want:
        x[7], x[0] = x[2], x[5]
    pairs = torch.tensor([[2, 7], [5, 0]], dtype=torch.int32, device="cuda")
    ws = pa.new_workspace(256)
    desc = pa.cache_desc(k)
    pa._lib.check(pa.library().pa_copy_blocks(pa._ptr(k), pa._ptr(v), ctypes.byref(desc), pa._ptr(pairs), 2,
                                              pa._ptr(ws), None))
    assert pa.check_error(ws) == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


# ---------------------------------------------------------------------------------------------
# attention over MXFP4 pools
# ---------------------------------------------------------------------------------------------
EDGE = [1, 15, 16, 17, 32, 33, 100, 511, 513, 2000]


def check_mx(c, out):
    ref, _ = c.reference()
    got = bits_f64(out)
    assert np.isfinite(got).all()
    # per scale block of the output: a block's own values bound its error
    for s in range(len(c.ctx)):
        if c.qlens[s] == 0:
            continue
        _, V = c.context(s)
        top = np.abs(V).reshape(V.shape[0], c.hkv, c.d // 32, 32).max((0, 3))       # [hkv, blocks]
        top = np.repeat(np.repeat(top, 32, -1), c.hq // c.hkv, 0)
        rows = slice(c.qsl[s], c.qsl[s + 1])
        tol = (2.0 ** -12 + 4e-4) * top
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ref[rows])
        assert (np.abs(got[rows] - ref[rows]) <= tol).all(), s


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 2, 128), (12, 3, 64), (16, 1, 128), (5, 1, 64), (32, 4, 64)])
@pytest.mark.parametrize("spread", [0, 12])
def test_mxfp4_decode(hq, hkv, d, spread):
    import paged_kv_cache_286_gb300 as pa
    c = Case(EDGE, [1] * len(EDGE), hq, hkv, d, "mxfp4", seed=hq + d, spread=spread)
    if spread:  # scores stay in range: q small where keys are large
        c.q = (c.q.float() * 2.0 ** -12).bfloat16()
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    ws[256:] = 0xFF
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws) == 0
    check_mx(c, out)


@pytest.mark.parametrize("qlens,ctx", [
    ([2, 3, 7, 16], [40, 3, 200, 16]), ([37, 1, 64], [37, 900, 300]), ([0, 5, 0, 1], [10, 70, 33, 1]),
    ([130, 1, 5], [700, 2100, 5]),
])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (8, 2, 128), (16, 1, 128), (9, 3, 128)])
def test_mxfp4_runs(qlens, ctx, hq, hkv, d):
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, "mxfp4", seed=sum(ctx) + d)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    for dt in (torch.float32, torch.bfloat16):
        out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, out_dtype=dt, **c.hints())
        assert pa.check_error(ws) == 0
        check_mx(c, out)


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("share", [1.0, 0.5, 0.0])
def test_mxfp4_chunks_with_room_to_stage_all_some_and_none(d, hq, hkv, share):
    """Long runs go to the prefill tiles through a bf16 copy in what the workspace has past the
    attention's own part, and to the split-KV kernel where it has no room for them."""
    import paged_kv_cache_286_gb300 as pa
    qlens, ctx = [60, 1, 200, 3, 45, 7], [500, 900, 200, 77, 1300, 700]
    c = Case(ctx, qlens, hq, hkv, d, "mxfp4", seed=31 + d)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    group = hq // hkv
    blocks = min(len(qlens), sum(qlens) // (32 // group + 1)) * -(-1300 // BS)
    ws = ws[:ws.numel() - int((1 - share) * blocks) * hkv * BS * d * 4]
    ws[256:] = 0xFF
    before = np.random.default_rng(1).random((6, hkv, 1300)).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, out_dtype=dt, **c.hints())
        assert pa.check_error(ws) == 0
        check_mx(c, out)
    W = torch.from_numpy(before).cuda()
    ws = c.workspace(pa, True)
    ws = ws[:ws.numel() - int((1 - share) * blocks) * hkv * BS * d * 4]
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0
    check_weights(c, before, W.cpu().numpy(), list(range(6)), 1.0)
    good = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    t[2, 3] = 10 ** 6                                    # a bad block: its sequence's rows are lost
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x1
    assert torch.equal(out[:61], good[:61]) and torch.equal(out[261:], good[261:])


@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 64), (8, 2, 64), (16, 8, 128), (24, 6, 128)])
@pytest.mark.parametrize("qlens", [1, 2])
@pytest.mark.parametrize("spread", [0, 12])
def test_mxfp4_small_groups(hq, hkv, d, qlens, spread):
    """Groups of two and four, of which two kv heads share a tile of rows where a step may have
    enough items: many sequences under a wide bound."""
    import paged_kv_cache_286_gb300 as pa
    lens = [max(x, qlens) for x in EDGE] + [33, 100, 5, 17, 64] * 50
    c = Case(lens, [1 + (i % qlens) for i in range(len(lens))], hq, hkv, d, "mxfp4", seed=hq + hkv + d, spread=spread,
             bound=8192)
    if spread:
        c.q = (c.q.float() * 2.0 ** -12).bfloat16()
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    ws[256:] = 0xFF
    for dt in (torch.float32, torch.bfloat16):
        out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, out_dtype=dt, **c.hints())
        assert pa.check_error(ws) == 0
        check_mx(c, out)
    before = np.zeros((len(lens), hkv, 8192), np.float32)
    W = torch.from_numpy(before).cuda()
    wsw = c.workspace(pa, True)
    out2 = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, wsw, out_dtype=dt, **c.hints())
    assert pa.check_error(wsw) == 0
    assert torch.equal(out, out2)
    check_weights(c, before, W.cpu().numpy(), list(range(len(lens))), 1.0)


@pytest.mark.parametrize("kind", ["mxfp4", "e4m3"])
def test_many_sequences_of_two_heads_per_item(kind):
    """More sequences than the plan orders at a time, in its order of length: some without query
    tokens, some of one key, and one that breaks the bound on contexts and is left out."""
    import paged_kv_cache_286_gb300 as pa
    rng = np.random.default_rng(41)
    lens = rng.integers(1, 200, 1100)
    lens[::7] = 1
    lens[[5, 1030]] = [1500, 1400]
    qlens = (rng.random(1100) < 0.9).astype(np.int32)
    qlens[[5, 9, 1030]] = 1
    c = Case(lens, qlens, 8, 2, 128, kind, seed=42)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    ws[256:] = 0xFF
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws) == 0
    check_mx(c, out)
    ctx[9] = 1501
    row = int(c.qsl[9])
    again = torch.full_like(out, 7.0)
    pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, out=again, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x4
    out[row] = 7.0
    assert torch.equal(again, out)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 8, 64)])
def test_mxfp4_partitions_cut_to_even_rounds(hq, hkv, d):
    """Contexts of up to 3,000 keys under a bound for which the partitions are longer than 128 blocks."""
    import paged_kv_cache_286_gb300 as pa
    lens = [3000, 1, 2353, 2352, 640, 17, 2999, 100, 16, 15, 2000, 33, 1040, 48, 2, 2368]
    c = Case(lens, [1] * 16, hq, hkv, d, "mxfp4", seed=d, bound=32768)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    ws[256:] = 0xFF
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws) == 0
    check_mx(c, out)


@pytest.mark.parametrize("d", [64, 128])
def test_mxfp4_without_a_workspace(d):
    """The built-in scratch: a step with a chunk, which is not staged there."""
    import ctypes
    import paged_kv_cache_286_gb300 as pa
    qlens, ctx = [40, 1, 2], [300, 900, 50]
    c = Case(ctx, qlens, 8, 2, d, "mxfp4", seed=17)
    t, ctx, qsl = c.dev()
    L, q = pa.library(), c.q.cuda()
    word = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    out = torch.empty(43, 8, d, device="cuda")
    desc = pa.cache_desc(c.k)
    for _ in range(2):
        pa._lib.check(L.pa_attention_noalloc(
            pa._ptr(q), 43, pa._ptr(c.k), pa._ptr(c.v), ctypes.byref(desc), pa._ptr(t), t.size(1), pa._ptr(ctx),
            pa._ptr(qsl), 3, c.bound, 40, 8, 2, d, c.scale, pa._ptr(out), 2, pa._ptr(word), None))
        torch.cuda.synchronize()
        assert word.item() == 0
        check_mx(c, out)


def test_mxfp4_steps_in_graphs_on_two_streams():
    """Two captured steps (append, attention with a staged chunk, key weights, eviction) with
    workspaces of their own, replayed at once, give what the same calls give one after the other."""
    import paged_kv_cache_286_gb300 as pa
    cases = [Case([500, 900, 77], [60, 1, 3], 8, 2, 128, "mxfp4", seed=s) for s in (1, 2)]

    def state(c):
        t, ctx, qsl = c.dev()
        slots = torch.from_numpy(np.concatenate([c.tables[s][:1] * BS + np.arange(3) for s in range(3)]).astype(np.int64)).cuda()
        W = torch.zeros(3, 2, 900, device="cuda")
        keep = torch.tensor([200, 333, 77], dtype=torch.int32, device="cuda")
        kv = [torch.randn(9, 2, 128, generator=torch.Generator().manual_seed(c.hq + i)).bfloat16().cuda() for i in range(2)]
        ws = c.workspace(pa, True)
        ws[256:] = 0xFF
        return dict(c=c, t=t, ctx=ctx, qsl=qsl, slots=slots, W=W, keep=keep, kv=kv, ws=ws, k=c.k.clone(), v=c.v.clone(),
                    q=c.q.cuda(), out=torch.empty(64, 8, 128, device="cuda"),
                    kept=torch.empty(3, 2, 400, dtype=torch.int32, device="cuda"),
                    lens=torch.empty(3, dtype=torch.int32, device="cuda"))

    def run(s):
        c = s["c"]
        pa.cache_append(*s["kv"], s["slots"], s["k"], s["v"], s["ws"])
        pa.attention_key_weights(s["q"], s["k"], s["v"], s["t"], s["ctx"], s["qsl"], s["W"], s["ws"], out=s["out"],
                                 **c.hints())
        pa.evict_keys(s["k"], s["v"], s["t"], s["ctx"], s["keep"], s["W"], s["ws"], max_context_len=900,
                      max_keep_len=400, recent=10, kept=s["kept"], new_lens=s["lens"])

    want = [state(c) for c in cases]
    for s in want:
        for _ in range(2):
            run(s)
    torch.cuda.synchronize()
    got = [state(c) for c in cases]
    streams, graphs = [torch.cuda.Stream() for _ in cases], []
    for s, st in zip(got, streams):
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            run(s)
        graphs.append(graph)
    for _ in range(2):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert pa.check_error(b["ws"]) == 0
        for x in ("out", "W", "kept", "lens", "k", "v"):
            assert torch.equal(a[x], b[x]), x


@pytest.mark.parametrize("head", [0, 1])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("at", [0, 37])
def test_mxfp4_nan_block_stays_in_its_head(head, which, at):
    import paged_kv_cache_286_gb300 as pa
    c = Case([50, 300], [1, 1], 16, 4, 128, "mxfp4", seed=9, bound=1 << 20)  # (two heads an item)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    good = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    blk, off = int(c.tables[0, at // BS]), at % BS
    pool = c.k if which == "k" else c.v
    pool[blk, head, off * 64:(off + 1) * 64] = 0
    pool[blk, head, 1024 + off * 4 + 3] = 255                       # dims 96 .. 127
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    mine = torch.arange(16, device="cuda") // 4 == head
    assert torch.equal(out[1], good[1]) and torch.equal(out[0, ~mine], good[0, ~mine])
    nan = out[0, mine].isnan()
    assert nan.all() if which == "k" else (nan[:, 96:].all() and not nan[:, :96].any())


def test_mxfp4_nan_block_reaches_only_the_rows_that_see_it():
    import paged_kv_cache_286_gb300 as pa
    for which in ("k", "v"):
        c = Case([50], [4], 2, 1, 128, "mxfp4", seed=9)
        blk, off = int(c.tables[0, 48 // BS]), 48 % BS              # position 48: queries 2 and 3 see it
        pool = c.k if which == "k" else c.v
        pool[blk, 0, off * 64:(off + 1) * 64] = 0
        pool[blk, 0, 1024 + off * 4] = 255                          # dims 0 .. 31
        t, ctx, qsl = c.dev()
        ws = c.workspace(pa)
        out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints()).isnan().cpu()
        assert not out[:2].any()
        assert out[2:].all() if which == "k" else (out[2:, :, :32].all() and not out[2:, :, 32:].any())


def test_mxfp4_bad_block_ids_and_lengths():
    import paged_kv_cache_286_gb300 as pa
    c = Case([100, 64, 33], [1, 1, 1], 4, 2, 128, "mxfp4", seed=10)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    good = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    t[0, 1] = 10 ** 6
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x1
    assert torch.equal(out[1:], good[1:]) and torch.isfinite(out).all()
    t2, ctx2, _ = c.dev()
    ctx2[1] = 101                                                    # more than the host's bound
    pa.attention(c.q.cuda(), c.k, c.v, t2, ctx2, qsl, ws, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x4


# ---------------------------------------------------------------------------------------------
# accumulated key weights
# ---------------------------------------------------------------------------------------------
def check_weights(c, before, after, rows, decay):
    _, ws = c.reference()
    want = before.astype(np.float64)
    for s, w in enumerate(ws):
        if w is not None and rows[s] >= 0:
            L = int(c.ctx[s])
            want[rows[s], :, :L] = decay * want[rows[s], :, :L] + w
    touched = np.zeros(before.shape, bool)
    for s, w in enumerate(ws):
        if w is not None and rows[s] >= 0:
            touched[rows[s], :, :int(c.ctx[s])] = True
    assert np.array_equal(after[~touched], before[~touched])        # bit for bit
    assert (np.abs(after - want) <= 4e-4 * np.abs(want) + 1e-12)[touched].all()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("mxfp4", 128), ("mxfp4", 64)])
@pytest.mark.parametrize("qlens,ctx,hq,hkv", [
    ([1] * 10, EDGE, 8, 2), ([1] * 10, EDGE, 3, 3), ([1] * 10, EDGE, 16, 1),
    ([2, 3, 7, 16], [40, 3, 200, 16], 8, 2), ([37, 1, 64, 0], [37, 900, 300, 12], 8, 2),
    ([130, 1, 5], [700, 2100, 5], 4, 4), ([33, 200], [2000, 200], 16, 2),
])
def test_key_weights(kind, d, qlens, ctx, hq, hkv):
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, kind, seed=sum(ctx) + hq + d)
    t, ctx, qsl = c.dev()
    S = len(qlens)
    ws = c.workspace(pa, True)
    ws[256:] = 0xFF
    rng = np.random.default_rng(1)
    rows = rng.permutation(S + 2)[:S].astype(np.int32)
    before = rng.random((S + 2, hkv, int(c.ctx.max()) + 3)).astype(np.float32)
    W = torch.from_numpy(before).cuda()
    plain = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, c.workspace(pa), **c.hints())
    out = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, weight_rows=torch.from_numpy(rows).cuda(),
                                   decay=0.75, **c.hints())
    assert pa.check_error(ws) == 0
    assert torch.equal(out, plain)
    check_weights(c, before, W.cpu().numpy(), rows, 0.75)
    W2 = torch.from_numpy(before).cuda()                              # the same bits again
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W2, ws, weight_rows=torch.from_numpy(rows).cuda(),
                             decay=0.75, **c.hints())
    assert torch.equal(W, W2)


def test_key_weights_of_a_step_whose_scores_are_not_kept():
    """A bound on the context so large that the scores would take more than 1 GiB: K is read again."""
    import paged_kv_cache_286_gb300 as pa
    c = Case([300, 70, 1000], [1, 2, 1], 8, 2, 128, "bf16", seed=5)
    t, ctx, qsl = c.dev()
    far = 12_000_000
    sizes = [pa.attention_key_weights_workspace_size(3, 4, 8, 2, 128, m, 2) for m in (far - 8_000_000, far)]
    assert sizes[1] < sizes[0] + (1 << 29)
    W = torch.zeros(3, 2, far, device="cuda")
    ws = pa.new_workspace(sizes[1])
    hints = dict(c.hints(), max_context_len=far)
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, **hints)
    assert pa.check_error(ws) == 0
    W = W[..., :1003].contiguous()
    check_weights(c, np.zeros(W.shape, np.float32), W.cpu().numpy(), [0, 1, 2], 1.0)


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 16), (64, 16, 16), (128, 64, 16), (128, 40, 20), (64, 128, 16)])
def test_key_weights_of_chunks_on_the_tensor_cores(d, hq, hkv):
    """Enough key chunks for a CTA each: long runs beside short ones, a chunk without a prefix, runs
    that end inside a tile, keys that end inside a block, and a block outside the pool."""
    import paged_kv_cache_286_gb300 as pa
    qlens, ctx = [200, 1, 33, 70, 0, 129], [1300, 500, 33, 900, 44, 641]
    c = Case(ctx, qlens, hq, hkv, d, "bf16", seed=d + hq)
    t, ctx, qsl = c.dev()
    before = np.random.default_rng(2).random((6, hkv, 1301)).astype(np.float32)
    W = torch.from_numpy(before).cuda()
    ws = c.workspace(pa, True)
    ws[256:] = 0xFF
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, decay=0.5, **c.hints())
    assert pa.check_error(ws) == 0
    check_weights(c, before, W.cpu().numpy(), list(range(6)), 0.5)
    W2 = torch.from_numpy(before).cuda()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W2, ws, decay=0.5, **c.hints())
    assert torch.equal(W, W2)
    t[3, 20] = -7
    W2 = torch.from_numpy(before).cuda()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W2, ws, decay=0.5, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x1
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(W[keep], W2[keep])
    assert torch.equal(W2[3, :, 320:336].cpu(), torch.from_numpy(before[3, :, 320:336] * np.float32(0.5)))


@pytest.mark.parametrize("kind,d,hq,hkv", [("e4m3", 128, 16, 16), ("e4m3", 128, 64, 16), ("mxfp4", 128, 40, 20),
                                           ("mxfp4", 64, 32, 16), ("mxfp4", 128, 128, 16)])
def test_key_weights_of_chunks_over_small_pools_on_the_tensor_cores(kind, d, hq, hkv):
    """As above; the keys are converted on their way in."""
    import paged_kv_cache_286_gb300 as pa
    qlens, ctx = [200, 1, 33, 70, 0, 129, 300], [1300, 500, 33, 900, 44, 641, 2000]
    c = Case(ctx, qlens, hq, hkv, d, kind, seed=d + hq)
    t, ctx, qsl = c.dev()
    before = np.random.default_rng(2).random((7, hkv, 2003)).astype(np.float32)
    W = torch.from_numpy(before).cuda()
    ws = c.workspace(pa, True)
    ws[256:] = 0xFF
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, decay=0.5, **c.hints())
    assert pa.check_error(ws) == 0
    check_weights(c, before, W.cpu().numpy(), list(range(7)), 0.5)
    W2 = torch.from_numpy(before).cuda()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W2, ws, decay=0.5, **c.hints())
    assert torch.equal(W, W2)
    t[3, 20] = 10 ** 6
    W2 = torch.from_numpy(before).cuda()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W2, ws, decay=0.5, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x1
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(W[keep], W2[keep])
    assert torch.equal(W2[3, :, 320:336].cpu(), torch.from_numpy(before[3, :, 320:336] * np.float32(0.5)))


def test_key_weights_wait_that_expires_reports_a_timeout():
    import paged_kv_cache_286_gb300 as pa
    c = Case([1300, 500], [200, 1], 16, 16, 64, "bf16", seed=3)
    t, ctx, qsl = c.dev()
    L = pa.library()
    ws = c.workspace(pa, True)
    want = torch.zeros(2, 16, 1300, device="cuda")
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, want, ws, **c.hints())
    W = torch.zeros_like(want)
    try:
        L.pa_set_wait_limit_ns(20_000_000)
        L.pa_test_skip_one_copy(1)
        pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, **c.hints())
        assert pa.check_error(ws, raise_on_error=False) & 0x8
    finally:
        L.pa_test_skip_one_copy(0)
        L.pa_set_wait_limit_ns(0)
    W.zero_()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0 and torch.equal(W, want)


def test_key_weights_rows_left_out():
    import paged_kv_cache_286_gb300 as pa
    c = Case([40, 70, 33], [1, 2, 1], 4, 2, 64, "bf16", seed=2)
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa, True)
    W = torch.rand(3, 2, 70, device="cuda")
    before = W.cpu().numpy().copy()
    rows = torch.tensor([2, -1, 7], dtype=torch.int32, device="cuda")
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, weight_rows=rows, **c.hints())
    assert pa.check_error(ws, raise_on_error=False) == 0x10
    check_weights(c, before, W.cpu().numpy(), [2, -1, -1], 1.0)


def test_key_weights_step_in_a_graph_on_a_side_stream():
    import paged_kv_cache_286_gb300 as pa
    c = Case([300, 70, 1000], [1, 1, 1], 8, 2, 128, "bf16", seed=3)
    t, ctx, qsl = c.dev()
    q = c.q.cuda()
    want = torch.zeros(3, 2, 1000, device="cuda")
    ws = c.workspace(pa, True)
    for _ in range(3):
        ref = pa.attention_key_weights(q, c.k, c.v, t, ctx, qsl, want, ws, decay=0.5, **c.hints())
    W = torch.zeros_like(want)
    out = torch.empty_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            pa.attention_key_weights(q, c.k, c.v, t, ctx, qsl, W, ws, decay=0.5, out=out, **c.hints())
        for _ in range(3):
            g.replay()
    side.synchronize()
    assert torch.equal(W, want) and torch.equal(out, ref)


# ---------------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------------
def tile_rows(pool, kind, d):
    """Raw rows [NB, H, 16, bytes] of a pool (MXFP4: codes and scale bytes side by side)."""
    if kind != "mxfp4":
        x = pool.view(torch.uint8) if pool.dtype != torch.uint8 else pool
        return x.cpu().numpy().copy()
    x = pool.cpu().numpy()
    nb, h, _ = x.shape
    return np.concatenate([x[..., :8 * d].reshape(nb, h, 16, d // 2), x[..., 8 * d:].reshape(nb, h, 16, d // 32)], -1)


def evict_reference(c, W, ctx, keep, recent, max_keep, dst_tables, rows, dst_rows):
    k, v = (tile_rows(p, c.kind, c.d) for p in (c.k, c.v))
    k2, v2, W2 = k.copy(), v.copy(), W.copy()
    kept_all = np.full((len(ctx), c.hkv, max_keep), -1, np.int32)
    for s, L in enumerate(ctx):
        for h in range(c.hkv):
            kept = eviction.choose(W[rows[s], h], int(L), int(keep[s]), recent)
            n = len(kept)
            kept_all[s, h, :n] = kept
            W2[dst_rows[s], h, :n] = W[rows[s], h, kept]
            W2[dst_rows[s], h, n:L] = 0
            i = np.arange(n)
            src = c.tables[s, kept // BS], h, kept % BS
            dst = dst_tables[s, i // BS], h, i % BS
            k2[dst], v2[dst] = k[src], v[src]
    return kept_all, np.minimum(keep, ctx), k2, v2, W2


WEIGHTS = {
    "random": lambda rng, shape: rng.random(shape),
    "ties": lambda rng, shape: rng.integers(0, 3, shape),
    "equal": lambda rng, shape: np.full(shape, 0.25),
    "odd": lambda rng, shape: rng.choice([0.0, -0.0, -1.5, np.inf, -np.inf, np.nan, 1e-40, 3.0, 3.0000002], shape),
    "close": lambda rng, shape: 1.0 + rng.integers(0, 40, shape) * 2.0 ** -23,
}


@pytest.mark.parametrize("weights", sorted(WEIGHTS))
@pytest.mark.parametrize("kind,d,hkv", [("bf16", 128, 2), ("bf16", 64, 1), ("e4m3", 128, 3), ("mxfp4", 128, 2),
                                        ("mxfp4", 64, 2)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(weights, kind, d, hkv, in_place):
    import paged_kv_cache_286_gb300 as pa
    ctx = [1, 2, 16, 17, 100, 333, 2049, 5000, 40]
    keep = np.array([1, 1, 7, 17, 33, 200, 2048, 1777, 0], np.int32)
    for recent in (0, 1, 100, 10 ** 6):
        c = Case(ctx, [1] * len(ctx), hkv, hkv, d, kind, seed=7, spare=sum(-(-x // BS) for x in ctx))
        S = len(ctx)
        rng = np.random.default_rng(8)
        W = WEIGHTS[weights](rng, (2 * S, hkv, 5003)).astype(np.float32)
        rows = rng.permutation(2 * S).astype(np.int32)
        rows, dst_rows = rows[:S], (rows[:S] if in_place else rows[S:])
        dst = c.tables.copy()
        if not in_place:                                             # some own blocks, some fresh ones
            fresh = iter(c.free)
            for s in range(S):
                for j in range(-(-int(keep[s]) // BS)):
                    if (s + j) % 3 or s == 5:
                        dst[s, j] = next(fresh)
        kept_w, lens_w, k_w, v_w, W_w = evict_reference(c, W, c.ctx, keep, recent, 2048, dst, rows, dst_rows)
        Wt = torch.from_numpy(W).cuda()
        ws = pa.new_workspace(pa.evict_workspace_size(S, hkv, 5000, 2048))
        cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        kept, lens = pa.evict_keys(c.k, c.v, cu(c.tables), cu(c.ctx), cu(keep), Wt, ws, max_context_len=5000,
                                   max_keep_len=2048, recent=recent, dst_tables=None if in_place else cu(dst),
                                   weight_rows=cu(rows), dst_weight_rows=None if in_place else cu(dst_rows))
        assert pa.check_error(ws) == 0
        assert np.array_equal(kept.cpu().numpy(), kept_w)
        assert np.array_equal(lens.cpu().numpy(), lens_w)
        assert np.array_equal(Wt.cpu().numpy(), W_w, equal_nan=True)
        assert np.array_equal(tile_rows(c.k, kind, d), k_w) and np.array_equal(tile_rows(c.v, kind, d), v_w)


@pytest.mark.parametrize("weights", ["random", "ties", "odd", "equal"])
@pytest.mark.parametrize("ctx,keep,hkv", [
    ([70000, 65537], [30011, 65536], 1),          # more than a CTA's shared memory holds
    ([9000, 4097, 1, 40, 8191, 16], [1, 4096, 1, 0, 8190, 16], 2),
    ([5000, 300, 4999], [2500, 299, 4999], 1),
    ([450000, 17], [200000, 3], 1),
])
def test_evict_long_rows_and_default_rows(ctx, keep, hkv, weights):
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, [1] * len(ctx), hkv, hkv, 64, "bf16", seed=12)
    rng = np.random.default_rng(5)
    top = max(ctx)
    W0 = WEIGHTS[weights](rng, (len(ctx), hkv, top + 1)).astype(np.float32)
    if weights == "random":
        W0 = W0 ** 8
    keep = np.array(keep, np.int32)
    rows = list(range(len(ctx)))
    ws = pa.new_workspace(pa.evict_workspace_size(len(ctx), hkv, top, int(keep.max())))
    t, lens, _ = c.dev()
    for recent in (0, 555):
        args = evict_reference(c, W0, c.ctx, keep, recent, int(keep.max()), c.tables, rows, rows)
        k, v, Wt = c.k.clone(), c.v.clone(), torch.from_numpy(W0).cuda()
        kept, new = pa.evict_keys(k, v, t, lens, torch.from_numpy(keep).cuda(), Wt, ws, max_context_len=top,
                                  max_keep_len=int(keep.max()), recent=recent)
        assert pa.check_error(ws) == 0
        assert np.array_equal(kept.cpu().numpy(), args[0]) and np.array_equal(new.cpu().numpy(), args[1])
        assert np.array_equal(Wt.cpu().numpy(), args[4], equal_nan=True)
        assert np.array_equal(tile_rows(k, "bf16", 64), args[2])
        assert np.array_equal(tile_rows(v, "bf16", 64), args[3])


@pytest.mark.parametrize("weights", sorted(WEIGHTS))
@pytest.mark.parametrize("bound", [300, 5000, 20000])
def test_evict_of_many_rows(weights, bound):
    """More rows than fill the GPU, under bounds that choose each width of the selection."""
    import paged_kv_cache_286_gb300 as pa
    rng = np.random.default_rng(31)
    ctx = rng.integers(1, 301, 160)
    keep = np.maximum(1, (ctx * rng.random(160)).astype(np.int32)).astype(np.int32)
    c = Case(ctx, [1] * 160, 2, 2, 64, "bf16", seed=15)
    W0 = WEIGHTS[weights](rng, (160, 2, bound)).astype(np.float32)
    rows = list(range(160))
    want = evict_reference(c, W0, c.ctx, keep, 7, 300, c.tables, rows, rows)
    Wt, (t, lens, _) = torch.from_numpy(W0).cuda(), c.dev()
    t = torch.nn.functional.pad(t, (0, -(-bound // BS) - t.size(1)), value=-1) if bound > 300 else t
    ws = pa.new_workspace(256)
    kept, new = pa.evict_keys(c.k, c.v, t, lens, torch.from_numpy(keep).cuda(), Wt, ws, max_context_len=bound,
                              max_keep_len=300, recent=7)
    assert pa.check_error(ws) == 0
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(new.cpu().numpy(), want[1])
    assert np.array_equal(Wt.cpu().numpy(), want[4], equal_nan=True)
    assert np.array_equal(tile_rows(c.k, "bf16", 64), want[2]) and np.array_equal(tile_rows(c.v, "bf16", 64), want[3])


def test_evict_of_empty_sequences_and_to_nothing():
    import paged_kv_cache_286_gb300 as pa
    c = Case([40, 16, 50], [1] * 3, 2, 2, 64, "bf16", seed=14)
    t, _, _ = c.dev()
    ctx = torch.tensor([40, 0, 50], dtype=torch.int32, device="cuda")
    keep = torch.tensor([0, 9, 0], dtype=torch.int32, device="cuda")
    W = torch.rand(3, 2, 64, device="cuda")
    w0, k0 = W.cpu().numpy().copy(), tile_rows(c.k, "bf16", 64)
    ws = pa.new_workspace(256)
    for most in (8, 0):
        kept, lens = pa.evict_keys(c.k, c.v, t, ctx, keep, W, ws, max_context_len=64, max_keep_len=most, recent=4)
        assert pa.check_error(ws) == 0
        assert lens.tolist() == [0, 0, 0] and kept.shape == (3, 2, most) and (kept == -1).all()
        got = W.cpu().numpy()
        assert (got[0, :, :40] == 0).all() and (got[2, :, :50] == 0).all()
        assert np.array_equal(got[0, :, 40:], w0[0, :, 40:]) and np.array_equal(got[1], w0[1])
        assert np.array_equal(tile_rows(c.k, "bf16", 64), k0)


def test_evict_leaves_bad_sequences_as_they_are():
    import paged_kv_cache_286_gb300 as pa
    c = Case([40, 50, 60, 70, 80, 90], [1] * 6, 2, 2, 64, "bf16", seed=13)
    t, _, _ = c.dev()
    ctx = torch.tensor([40, -3, 60, 70, 80, 1000], dtype=torch.int32, device="cuda")
    keep = torch.tensor([20, 5, -1, 33, 20, 20], dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 1, 2, 3, -1, 5], dtype=torch.int32, device="cuda")
    W = torch.rand(6, 2, 100, device="cuda")
    k0, w0 = tile_rows(c.k, "bf16", 64), W.cpu().numpy().copy()
    ws = pa.new_workspace(256)
    kept, lens = pa.evict_keys(c.k, c.v, t, ctx, keep, W, ws, max_context_len=100, max_keep_len=32, recent=4,
                               weight_rows=rows)
    assert pa.check_error(ws, raise_on_error=False) == 0x4
    assert lens.tolist() == [20, -3, 60, 70, 80, 1000]
    assert (kept[1:] == -1).all() and (kept[0, :, :20] >= 0).all()
    changed = np.zeros(k0.shape[0], bool)
    changed[c.tables[0, :2]] = True
    assert np.array_equal(tile_rows(c.k, "bf16", 64)[~changed], k0[~changed])
    assert np.array_equal(W.cpu().numpy()[1:], w0[1:])
    # a block outside the pool: its keys do not move
    t[0, 0] = -1
    pa.evict_keys(c.k, c.v, t[:1], ctx[:1], keep[:1], W, ws, max_context_len=100, max_keep_len=32, recent=4)
    assert pa.check_error(ws, raise_on_error=False) == 0x1
    rows[0] = 6
    pa.evict_keys(c.k, c.v, t[:1], ctx[:1], keep[:1], W, ws, max_context_len=100, max_keep_len=32, recent=4,
                  weight_rows=rows[:1])
    assert pa.check_error(ws, raise_on_error=False) == 0x10


def test_far_blocks():
    """Pools larger than 4 GiB: the keys in their last blocks."""
    import paged_kv_cache_286_gb300 as pa
    nb, hkv, d, L = 140000, 8, 128, 100
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros((nb, hkv, BS, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[-7:], v[-7:] = (torch.randn((7, hkv, BS, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, hkv, d), generator=g, device="cuda").bfloat16()
    far = torch.arange(nb - 7, nb, dtype=torch.int32, device="cuda")[None]
    near = far - (nb - 7)
    res = []
    for kk, vv, t in ((k, v, far), (k[-7:].clone(), v[-7:].clone(), near)):
        ctx = torch.tensor([L], dtype=torch.int32, device="cuda")
        qsl = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        W = torch.zeros(1, hkv, L, device="cuda")
        ws = pa.new_workspace(pa.attention_key_weights_workspace_size(1, 1, hkv, hkv, d, L, 1))
        out = pa.attention_key_weights(q, kk, vv, t, ctx, qsl, W, ws, scale=d ** -0.5, max_context_len=L, max_query_len=1)
        kept, _ = pa.evict_keys(kk, vv, t, ctx, torch.tensor([37], dtype=torch.int32, device="cuda"), W, ws,
                                max_context_len=L, max_keep_len=37, recent=5)
        assert pa.check_error(ws) == 0
        res.append((out, W, kept, kk[-7:], vv[-7:]))
    for a, b in zip(*res):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_serving_loop_with_a_key_budget(kind):
    """A prompt, decode steps that accumulate weights, eviction when a sequence passes its budget
    (planned by the block manager: a block shared with a fork is copied out of, not written), and more
    steps over what is left; every step against a dense model of each head's keys in 64 bits."""
    import paged_kv_cache_286_gb300 as pa
    from paged_kv_cache_286_gb300.block_manager import BlockManager
    hq, hkv, d, nb, width, budget, recent = 4, 2, 128, 40, 12, 60, 9
    bm = BlockManager(nb)
    g = torch.Generator().manual_seed(21)
    if kind == "mxfp4":
        kc, vc = pa.new_mxfp4_cache(nb, hkv, d), pa.new_mxfp4_cache(nb, hkv, d)
        stored = lambda x: mxfp4.decode(*mxfp4.encode(bits_f64(x)))  # noqa: E731
        tol_w, tol_o = 1e-3, 2.0 ** -12 + 4e-4
    else:
        kc = torch.zeros((nb, hkv, BS, d), dtype=torch.bfloat16, device="cuda")
        vc, stored = torch.zeros_like(kc), bits_f64
        tol_w, tol_o = 1e-3, 4e-4
    keys = {s: [[] for _ in range(hkv)] for s in (0, 1)}   # per head: lists of (k, v)
    weight = {s: [[] for _ in range(hkv)] for s in (0, 1)}
    W = torch.zeros(2, hkv, width * BS, device="cuda")
    ws = pa.new_workspace(pa.attention_key_weights_workspace_size(2, 80, hq, hkv, d, width * BS, 80))

    def step(news):
        """news: {seq: new tokens}"""
        seqs = sorted(news)
        ks, vs, slots = [], [], []
        for s in seqs:
            sl, pairs = bm.append(s, news[s])
            assert not pairs
            k, v = (torch.randn(news[s], hkv, d, generator=g).bfloat16() for _ in range(2))
            ks.append(k), vs.append(v), slots.append(sl)
            for h in range(hkv):
                keys[s][h] += list(zip(stored(k)[:, h], stored(v)[:, h]))
                weight[s][h] += [0.0] * news[s]
        T = sum(news.values())
        pa.cache_append(torch.cat(ks).cuda(), torch.cat(vs).cuda(), torch.from_numpy(np.concatenate(slots)).cuda(), kc, vc, ws)
        q = torch.randn(T, hq, d, generator=g).bfloat16()
        ctx = np.array([bm.num_tokens(s) for s in seqs], np.int32)
        qsl = np.concatenate([[0], np.cumsum([news[s] for s in seqs])]).astype(np.int32)
        cu = lambda x: torch.from_numpy(np.asarray(x)).cuda()  # noqa: E731
        out = pa.attention_key_weights(q.cuda(), kc, vc, cu(bm.tables(seqs, width)), cu(ctx), cu(qsl), W, ws, scale=d ** -0.5,
                                       max_context_len=width * BS, max_query_len=80,
                                       weight_rows=cu(np.array(seqs, np.int32)))
        assert pa.check_error(ws) == 0
        got, Wn = bits_f64(out), W.cpu().numpy()
        for i, s in enumerate(seqs):
            K, V = (np.stack([np.stack([kv[j] for kv in keys[s][h]]) for h in range(hkv)], 1) for j in (0, 1))
            assert len(K) == ctx[i]
            o, w = eviction.attend_with_weights(bits_f64(q)[qsl[i]:qsl[i + 1]], K, V, len(K) - news[s], d ** -0.5)
            assert np.abs(got[qsl[i]:qsl[i + 1]] - o).max() <= tol_o * np.abs(V).max()
            for h in range(hkv):
                weight[s][h] = list(np.array(weight[s][h]) + w[h])
                assert np.abs(Wn[s, h, :len(K)] - weight[s][h]).max() <= tol_w * max(weight[s][h])
                weight[s][h] = [float(x) for x in Wn[s, h, :len(K)]]  # what the choice goes by
        return ctx

    def evict(s):
        cu = lambda x: torch.from_numpy(np.asarray(x)).cuda()  # noqa: E731
        L = bm.num_tokens(s)
        table = bm.tables([s], width)
        dst = bm.evict(s, min(budget, L), width)[None]
        kept, lens = pa.evict_keys(kc, vc, cu(table), cu(np.array([L], np.int32)), cu(np.array([budget], np.int32)), W, ws,
                                   max_context_len=width * BS, max_keep_len=budget, recent=recent, dst_tables=cu(dst),
                                   weight_rows=cu(np.array([s], np.int32)))
        assert pa.check_error(ws) == 0 and lens.item() == bm.num_tokens(s)
        for h in range(hkv):
            want = eviction.choose(np.array(weight[s][h], np.float32), L, budget, recent)
            assert np.array_equal(kept[0, h].cpu().numpy()[:len(want)], want)
            keys[s][h] = [keys[s][h][j] for j in want]
            weight[s][h] = [weight[s][h][j] for j in want]

    step({0: 80})
    bm.fork(0, 1)                                   # shares all five blocks
    keys[1] = [list(x) for x in keys[0]]
    weight[1] = [list(x) for x in weight[0]]
    W[1] = W[0]
    before = set(bm.block_table(0).tolist())
    evict(0)                                        # its shared blocks are left to sequence 1
    assert not before & set(bm.block_table(0).tolist())
    for i in range(40):
        step({0: 1, 1: 1} if i % 3 else {0: 2, 1: 3})
        for s in (0, 1):
            if bm.num_tokens(s) > budget + 20:
                evict(s)
    step({1: 30})
