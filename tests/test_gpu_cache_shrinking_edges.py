"""Edges of the operators that shrink the cache, on the GPU, against the definitions in 64 bits: the
smallest scales of MXFP4 pools, sequences evicted in one call, keys that hold infinities, queries of any
size, waits that run out, and key weights that start from nothing.

Tolerances are those of test_gpu_cache_shrinking.py (a score off by less than 2e-4 in the log2 domain,
so a weight or a log-sum-exp's power by 4e-4; MXFP4 attention rounds a probability to f16, 2^-12);
codes, bytes, positions and moves are exact."""

import numpy as np
import pytest
import torch

from test_gpu_cache_shrinking import (BS, Case, bits_f64, check_weights, evict_reference, mx_inputs,
                                      tile_rows)

pytestmark = pytest.mark.gpu

from oracle import mxfp4  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_286_gb300 import build
    build.build()


# ---------------------------------------------------------------------------------------------
# the smallest scales: byte 0 is 2^-127, whose codes reach 1.5 * 2^-125
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d,hkv,T", [(128, 8, 301), (64, 3, 97), (128, 1, 33), (64, 1, 1024)])
def test_mxfp4_append_and_read_of_every_scale(d, hkv, T):
    import paged_kv_cache_286_gb300 as pa
    k, v = mx_inputs(d, T, hkv, 1), mx_inputs(d, T, hkv, 2)
    # whole blocks of the two smallest scales: every multiple of 2^-128, and of 2^-129, up to 31
    tiny = np.arange(T * hkv * d).reshape(T, hkv, d) % 32 * 2.0 ** -128
    k[T - 9:] = torch.from_numpy(tiny[T - 9:]).bfloat16()
    v[T - 9:] = -k[T - 9:] / 2
    nb = T // BS + 3
    slots = np.random.default_rng(3).permutation(nb * BS)[:T].astype(np.int64)
    slots[4] = -1
    kc, vc = pa.new_mxfp4_cache(nb, hkv, d), pa.new_mxfp4_cache(nb, hkv, d)
    ws = pa.new_workspace(256)
    ts = torch.from_numpy(slots).cuda()
    pa.cache_append(k.cuda(), v.cuda(), ts, kc, vc, ws)
    outs = {t: pa.cache_read(ts, kc, vc, ws, out_dtype=t) for t in (torch.bfloat16, torch.float32)}
    assert pa.check_error(ws) == 0
    for i, x in enumerate((k, v)):
        codes, byte = mxfp4.encode(bits_f64(x))
        want = mxfp4.decode(codes, byte)
        assert want[T - 9:].any() and (byte[T - 9:] == 1 - i).all()
        want[4] = 0.0
        for t in outs:
            assert outs[t][i].dtype == t
            assert np.array_equal(outs[t][i].float().cpu().numpy(), want.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("d", [64, 128])
def test_mxfp4_read_of_any_bytes(d):
    """Every scale byte beside every code; 6 * 2^127 is past fp32's and bf16's range."""
    import paged_kv_cache_286_gb300 as pa
    pool = np.random.default_rng(d).integers(0, 256, (2, 20, 3, 17 * d // 2), dtype=np.uint8)
    want = mxfp4.decode(*mxfp4.unpack_tiles(pool[0])), mxfp4.decode(*mxfp4.unpack_tiles(pool[1]))
    slots = torch.arange(20 * BS, device="cuda")
    ws = pa.new_workspace(256)
    for t in (torch.bfloat16, torch.float32):
        got = pa.cache_read(slots, *(torch.from_numpy(p).cuda() for p in pool), ws, out_dtype=t)
        assert pa.check_error(ws) == 0
        for g, w in zip(got, want):
            with np.errstate(over="ignore"):
                w = w.transpose(0, 2, 1, 3).reshape(-1, 3, d).astype(np.float32)
            assert np.array_equal(g.float().cpu().numpy(), w, equal_nan=True)


def smallest(c, which):
    """The case with its keys or values in blocks of scale bytes 0 and 1."""
    vals = c.kv if which == "k" else c.vv
    codes, byte = mxfp4.encode(np.where(np.isfinite(vals), vals, 0.0) * 2.0 ** -126)
    assert byte.max() <= 1 and (byte == 0).mean() > 0.5
    pool, vals = torch.from_numpy(mxfp4.pack_tiles(codes, byte)).cuda(), mxfp4.decode(codes, byte)
    if which == "k":
        c.k, c.kv = pool, vals
        c.q = (c.q.float() * 2.0 ** 112).bfloat16()                  # scores of the usual size
        c.scale *= 2.0 ** 14
    else:
        c.v, c.vv = pool, vals


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 4, 4), (128, 2, 2), (64, 16, 1)])
@pytest.mark.parametrize("qlens", [(1, 1, 1, 1), (1, 3, 2, 1), (40, 1, 60, 2)])
def test_mxfp4_attention_over_the_smallest_scales(which, d, hq, hkv, qlens):
    """Decode tokens, short runs and staged chunks, their weights too."""
    import paged_kv_cache_286_gb300 as pa
    c = Case([700, 33, 90, 16], qlens, hq, hkv, d, "mxfp4", seed=d + hq)
    smallest(c, which)
    t, ctx, qsl = c.dev()
    before = np.zeros((4, hkv, 700), np.float32)
    W = torch.from_numpy(before).cuda()
    ws, ref = c.workspace(pa, True), c.reference()[0]
    ws[256:] = 0xFF
    out = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, ctx, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0
    got = bits_f64(out)
    top = np.abs(c.vv).max()
    # 2^-149: outputs of the smallest values are subnormal
    assert np.abs(got - ref).max() <= (2.0 ** -12 + 4e-4) * top + 8 * 2.0 ** -149
    assert np.abs(ref).max() > 0.1 * top
    check_weights(c, before, W.cpu().numpy(), list(range(4)), 1.0)


# ---------------------------------------------------------------------------------------------
# several sequences evicted in one call
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("mxfp4", 64)])
def test_forks_and_neighbours_evicted_in_one_call(kind, d):
    """A parent, its two forks and a sequence of its own, planned by one evict_batch call: what each
    keeps is what it would keep alone, and a fork that stays out of the call keeps its keys."""
    import paged_kv_cache_286_gb300 as pa
    from paged_kv_cache_286_gb300.block_manager import BlockManager
    hkv, L, keep, recent = 3, 1500, [600, 333, 1499, 40], 17
    bm = BlockManager(340)
    bm.append(0, L)
    for s in (1, 2, 4):
        bm.fork(0, s)
    bm.append(3, 700)
    seqs = [0, 1, 2, 3]
    lens = [bm.num_tokens(s) for s in seqs]
    width = -(-L // BS)
    c = Case([L], [1], hkv, hkv, d, kind, seed=5, spare=340 - width)
    c.tables = bm.tables(seqs + [4], width)
    k0, v0 = (tile_rows(p, kind, d) for p in (c.k, c.v))
    W0 = np.random.default_rng(6).random((4, hkv, L)).astype(np.float32)
    dst = bm.evict_batch(seqs, keep, width)
    want = evict_reference(c, W0, np.array(lens), np.array(keep), recent, 1499, dst, seqs, seqs)
    cu = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(x, t)).cuda()  # noqa: E731
    W = torch.from_numpy(W0).cuda()
    ws = pa.new_workspace(pa.evict_workspace_size(4, hkv, L, 1499))
    kept, new = pa.evict_keys(c.k, c.v, cu(c.tables[:4]), cu(lens), cu(keep), W, ws, max_context_len=L,
                              max_keep_len=1499, recent=recent, dst_tables=cu(dst))
    assert pa.check_error(ws) == 0
    assert np.array_equal(kept.cpu().numpy(), want[0]) and new.tolist() == keep
    assert np.array_equal(W.cpu().numpy(), want[4])
    k1, v1 = (tile_rows(p, kind, d) for p in (c.k, c.v))
    assert np.array_equal(k1, want[2]) and np.array_equal(v1, want[3])
    still = c.tables[4]
    assert bm.block_table(4).tolist() == still.tolist()
    assert np.array_equal(k1[still], k0[still]) and np.array_equal(v1[still], v0[still])


# ---------------------------------------------------------------------------------------------
# keys that hold infinities
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d,hq,hkv,ctx,qlens", [
    (128, 1, 1, [300, 40], [37, 1]), (64, 6, 2, [300, 40], [45, 2]), (128, 3, 3, [513, 70], [33, 5]),  # mma.sync
    (128, 16, 16, [1300, 900], [201, 70]), (64, 16, 16, [1300, 900], [201, 1]),                     # tcgen05
])
def test_key_weights_of_keys_with_infinities(d, hq, hkv, ctx, qlens):
    """A key whose scores are all minus infinity receives nothing: decay * W, whatever the rows of the
    last tile that no query fills."""
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, "bf16", seed=d + hq)
    c.q[..., 3] = -c.q[..., 3].abs() - 0.5
    at = [0, 5, ctx[0] - qlens[0]]                                   # seen by every query of the first run
    for j in at:
        c.k[int(c.tables[0, j // BS]), :, j % BS, 3] = float("inf")
        c.kv[int(c.tables[0, j // BS]), :, j % BS, 3] = np.inf
    t, cl, qsl = c.dev()
    before = np.random.default_rng(2).random((2, hkv, max(ctx))).astype(np.float32)
    W = torch.from_numpy(before).cuda()
    ws = c.workspace(pa, True)
    ws[256:] = 0xFF
    out = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, decay=0.5, **c.hints())
    assert pa.check_error(ws) == 0
    assert torch.isfinite(out).all()
    check_weights(c, before, W.cpu().numpy(), [0, 1], 0.5)
    assert np.array_equal(W[0][:, at].cpu().numpy(), before[0][:, at] / 2)


# ---------------------------------------------------------------------------------------------
# queries of any size over MXFP4 keys
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv,qlens", [(4, 4, (1, 1, 1)), (8, 2, (1, 3, 2)), (16, 1, (2, 1, 1))])
@pytest.mark.parametrize("size", [120, -120])
def test_mxfp4_queries_of_any_size(hq, hkv, qlens, size):
    """q of 2^120 and 2^-120, the scale in proportion: scores, and so outputs, of the usual size."""
    import paged_kv_cache_286_gb300 as pa
    c = Case([300, 33, 90], qlens, hq, hkv, 128, "mxfp4", seed=hq)
    c.q = (c.q.float() * 2.0 ** size).bfloat16()
    c.scale *= 2.0 ** -size
    t, ctx, qsl = c.dev()
    ws = c.workspace(pa)
    ref = c.reference()[0]
    out = pa.attention(c.q.cuda(), c.k, c.v, t, ctx, qsl, ws, **c.hints())
    assert pa.check_error(ws) == 0
    assert np.abs(bits_f64(out) - ref).max() <= (2.0 ** -12 + 4e-4) * np.abs(c.vv).max()


# ---------------------------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d,hq,hkv,ctx,qlens", [
    (128, 8, 2, [500, 70], [1, 1]), (64, 4, 4, [500, 70], [1, 2]),           # decode tokens
    (128, 8, 2, [500, 700], [1, 60]), (64, 16, 16, [1300, 500], [200, 1]),   # both passes over K
])
def test_weights_stay_as_they_are_when_the_attention_times_out(d, hq, hkv, ctx, qlens):
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, "bf16", seed=3)
    t, cl, qsl = c.dev()
    L, ws = pa.library(), c.workspace(pa, True)
    ws[256:] = 0xFF
    before = torch.rand(2, hkv, max(ctx), device="cuda")
    want, W = before.clone(), before.clone()
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, want, ws, **c.hints())
    assert pa.check_error(ws) == 0
    try:
        L.pa_set_wait_limit_ns(20_000_000)
        L.pa_test_skip_one_copy(1)
        pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
        L.pa_test_skip_one_copy(0)
        # a step behind it, before anyone has looked
        pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
        assert pa.check_error(ws, raise_on_error=False) & 0x8
    finally:
        L.pa_test_skip_one_copy(0)
        L.pa_set_wait_limit_ns(0)
    assert torch.equal(W, before)
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0 and torch.equal(W, want)


@pytest.mark.parametrize("d,hq,hkv,ctx,qlens", [(128, 16, 16, [1300, 500], [200, 1]), (64, 16, 16, [1300, 900], [200, 77])])
def test_a_wait_of_the_weights_themselves_that_runs_out(d, hq, hkv, ctx, qlens):
    """The attention is done, the rows of the weights are lost, and the next call is whole again."""
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, "bf16", seed=3)
    t, cl, qsl = c.dev()
    L, ws = pa.library(), c.workspace(pa, True)
    ws[256:] = 0xFF
    W = torch.rand(3, hkv, max(ctx), device="cuda")
    before = W.clone()
    out = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
    want = W.clone()
    assert pa.check_error(ws) == 0
    W.copy_(before)
    try:
        L.pa_set_wait_limit_ns(20_000_000)
        L.pa_test_skip_one_copy(2)
        again = pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
        assert pa.check_error(ws, raise_on_error=False) == 0x8
    finally:
        L.pa_test_skip_one_copy(0)
        L.pa_set_wait_limit_ns(0)
    assert torch.equal(again, out) and torch.equal(W[2], before[2])
    W.copy_(before)
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0 and torch.equal(W, want)


# ---------------------------------------------------------------------------------------------
# key weights that start from nothing
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("mxfp4", 128), ("mxfp4", 64)])
@pytest.mark.parametrize("qlens,ctx,hq,hkv", [
    ([1] * 6, [1, 17, 100, 513, 2000, 5000], 8, 2), ([1] * 4, [33, 1000, 16, 4097], 3, 3), ([5, 1, 2], [700, 2100, 5], 3, 1),
    ([1500], [1500], 1, 1), ([1500], [1900], 3, 1), ([1500, 1], [1700, 300], 4, 1),
])
def test_key_weights_from_zeros(kind, d, qlens, ctx, hq, hkv):
    """Nothing but what the step adds is there for the bound to be a part of; and runs of 1,500 tokens."""
    import paged_kv_cache_286_gb300 as pa
    c = Case(ctx, qlens, hq, hkv, d, kind, seed=sum(ctx) + hq + d)
    t, cl, qsl = c.dev()
    before = np.zeros((len(ctx), hkv, max(ctx)), np.float32)
    W = torch.from_numpy(before).cuda()
    ws = c.workspace(pa, True)
    ws[256:] = 0xFF
    pa.attention_key_weights(c.q.cuda(), c.k, c.v, t, cl, qsl, W, ws, **c.hints())
    assert pa.check_error(ws) == 0
    check_weights(c, before, W.cpu().numpy(), list(range(len(ctx))), 1.0)
