"""Host side of the cache-shrinking calls: refusals, the block manager's evict, and the 64-bit
definitions against worked values."""

import ctypes
import os
import sys

import numpy as np
import pytest

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "tests"))
from oracle import eviction, mxfp4  # noqa: E402

pa_build = pytest.importorskip("paged_kv_cache_286_gb300.build")
FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    from paged_kv_cache_286_gb300 import _lib
    return _lib.load()


def _desc(**kw):
    from paged_kv_cache_286_gb300 import _lib
    d = dict(num_blocks=32, block_size=16, num_kv_heads=4, head_dim=64, cache_dtype=3, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return _lib.CacheDesc(**d)


def at(x):
    return ctypes.c_void_p(x)


# ---- MXFP4 definitions ------------------------------------------------------------------------
def test_e2m1_values_and_rounding():
    assert mxfp4.VALUES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert mxfp4.VALUES[8:].tolist() == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    x = np.zeros(32)
    x[:14] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.75, 0.26, 7.9, -6.5, 0.2, -0.1]
    codes, byte = mxfp4.encode(x[None])
    assert byte.tolist() == [[127]]           # 7.9: floor(log2) - 2 = 0
    got = mxfp4.decode(codes, byte)[0, :14]
    assert got.tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -1, 0.5, 6, -6, 0, -0.0]


def test_scales_of_extreme_blocks():
    x = np.zeros((5, 32))
    x[1, 3] = 2.0 ** -126                      # below the smallest scale's reach
    x[2, 0] = 2.0 ** 127
    x[3, 1] = np.inf
    x[4, 9] = np.nan
    codes, byte = mxfp4.encode(x)
    assert byte[:, 0].tolist() == [0, 0, 252, 253, 255]
    assert mxfp4.decode(codes, byte)[1, 3] == 2.0 ** -126
    assert mxfp4.decode(codes, byte)[2, 0] == 2.0 ** 127
    assert np.isnan(mxfp4.decode(codes, byte)[4]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_tiles_round_trip_and_word_order(d):
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (3, 2, 16, d), dtype=np.uint8)
    byte = rng.integers(0, 256, (3, 2, 16, d // 32), dtype=np.uint8)
    pool = mxfp4.pack_tiles(codes, byte)
    assert pool.shape == (3, 2, 17 * d // 2)
    c2, b2 = mxfp4.unpack_tiles(pool)
    assert np.array_equal(c2, codes) and np.array_equal(b2, byte)
    # word 1 of row 5 (bytes 2 and 3): dims 32 .. 35
    row = pool[1, 1, 5 * d // 2:]
    assert row[2] == codes[1, 1, 5, 32] | codes[1, 1, 5, 33] << 4
    assert row[3] == codes[1, 1, 5, 34] | codes[1, 1, 5, 35] << 4


def test_choose():
    w = np.array([5, 1, 5, np.nan, 0, -0.0, 9, 2.0])
    assert eviction.choose(w, 8, 4, 1).tolist() == [0, 2, 6, 7]
    assert eviction.choose(w, 8, 3, 0).tolist() == [0, 2, 6]
    assert eviction.choose(w, 6, 5, 0).tolist() == [0, 1, 2, 4, 5]      # NaN goes first
    assert eviction.choose(w, 6, 4, 0).tolist() == [0, 1, 2, 4]         # 0 and -0 tie: the lower stays
    assert eviction.choose(w, 8, 3, 99).tolist() == [5, 6, 7]
    assert eviction.choose(w, 3, 9, 1).tolist() == [0, 1, 2]
    assert eviction.choose(w, 8, 0, 2).tolist() == []


def test_weights_sum_to_the_rows():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    _, w = eviction.attend_with_weights(q, K, V, 6, 0.3)
    assert np.allclose(w.sum(1), 6.0)                                    # 3 queries x 2 heads
    assert (w[:, 7] < w[:, :9].sum(1)).all() and (w[:, 8] > 0).all()
    _, w1 = eviction.attend_with_weights(q[:1], K[:7], V[:7], 6, 0.3)
    assert (w1[:, :7] < w[:, :7]).all()


# ---- refusals -----------------------------------------------------------------------------------
@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=32), 2), (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(block_size=32), 2),
    (dict(num_kv_heads=0), 1), (dict(num_blocks=1 << 25), 1), (dict(cache_dtype=2), 2), (dict(cache_dtype=4), 2),
])
def test_mxfp4_descriptors(lib, kw, status):
    d = _desc(**kw)
    assert lib.pa_cache_append(FAKE, FAKE, FAKE, 4, FAKE, FAKE, ctypes.byref(d), FAKE, None) == status
    assert lib.pa_cache_read(FAKE, 4, FAKE, FAKE, ctypes.byref(d), FAKE, FAKE, 2, FAKE, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(slots=None), 1), (dict(kc=None), 1), (dict(k=None), 1), (dict(v=at(0x100008)), 1),
    (dict(odt=1), 2), (dict(odt=3), 2), (dict(ws=None), 1), (dict(slots=at(0x100004)), 1), (dict(T=0), 0),
])
def test_cache_read_refusals(lib, kw, status):
    a = dict(slots=FAKE, T=4, kc=FAKE, vc=FAKE, k=FAKE, v=FAKE, odt=0, ws=FAKE)
    a.update(kw)
    d = _desc()
    assert lib.pa_cache_read(a["slots"], a["T"], a["kc"], a["vc"], ctypes.byref(d), a["k"], a["v"], a["odt"], a["ws"],
                             None) == status


def _weights(lib, **kw):
    d = kw.pop("desc", _desc(cache_dtype=0))
    a = dict(q=FAKE, T=4, k=FAKE, v=FAKE, tables=FAKE, maxb=5, ctx=FAKE, qsl=FAKE, S=4, maxctx=80, maxq=1, hq=4, hkv=4,
             dim=64, scale=0.125, out=FAKE, odt=2, W=FAKE, rows=None, nrows=4, maxkeys=80, decay=1.0, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    return lib.pa_attention_key_weights(
        a["q"], a["T"], a["k"], a["v"], ctypes.byref(d), a["tables"], a["maxb"], a["ctx"], a["qsl"], a["S"], a["maxctx"],
        a["maxq"], a["hq"], a["hkv"], a["dim"], a["scale"], a["out"], a["odt"], a["W"], a["rows"], a["nrows"],
        a["maxkeys"], a["decay"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=6), 1), (dict(hq=128), 2), (dict(odt=1), 2), (dict(scale=float("inf")), 1), (dict(W=None), 1),
    (dict(W=at(0x100002)), 1), (dict(rows=at(0x100002)), 1), (dict(nrows=3), 1), (dict(nrows=-1), 1),
    (dict(maxkeys=79), 1), (dict(maxkeys=-1), 1), (dict(decay=-0.5), 1), (dict(decay=float("nan")), 1),
    (dict(decay=float("inf")), 1), (dict(ws=None), 1), (dict(wsb=300), 1), (dict(ws=at(0x100010)), 1), (dict(S=-1), 1),
    (dict(desc=_desc(num_kv_heads=2)), 1),
])
def test_key_weights_refusals(lib, kw, status):
    assert _weights(lib, **kw) == status
    assert lib.pa_last_error_string().decode()


def test_key_weights_with_nothing_to_do(lib):
    assert _weights(lib, S=0) == 0 and _weights(lib, T=0) == 0


def test_key_weights_workspace_holds_the_attention_s(lib):
    a = lib.pa_attention_workspace_size(16, 16, 32, 8, 128, 16, 32768, 1)
    b = lib.pa_attention_key_weights_workspace_size(16, 16, 32, 8, 128, 16, 32768, 1)
    assert b >= a + 16 * 32 * 4
    # the attention's size alone is refused
    assert _weights(lib, wsb=lib.pa_attention_workspace_size(4, 4, 4, 4, 64, 16, 80, 1)) == 1


def _evict(lib, **kw):
    d = kw.pop("desc", _desc(cache_dtype=0))
    a = dict(k=FAKE, v=FAKE, tables=FAKE, dst=None, maxb=5, ctx=at(0x200000), keep=at(0x210000), S=4, maxctx=80,
             maxkeep=40, recent=4, W=FAKE, rows=None, drows=None, nrows=4, maxkeys=80, kept=FAKE, lens=at(0x220000),
             ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.pa_evict_keys(
        a["k"], a["v"], ctypes.byref(d), a["tables"], a["dst"], a["maxb"], a["ctx"], a["keep"], a["S"], a["maxctx"],
        a["maxkeep"], a["recent"], a["W"], a["rows"], a["drows"], a["nrows"], a["maxkeys"], a["kept"], a["lens"],
        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(maxkeep=-1), 1), (dict(recent=-1), 1), (dict(maxctx=0), 1), (dict(W=None), 1),
    (dict(nrows=3), 1), (dict(maxkeys=79), 1), (dict(k=None), 1), (dict(tables=None), 1), (dict(ctx=None), 1),
    (dict(keep=None), 1), (dict(lens=None), 1), (dict(kept=None), 1), (dict(maxb=0), 1), (dict(k=at(0x100008)), 1),
    (dict(dst=at(0x100002)), 1), (dict(drows=at(0x100001)), 1), (dict(ws=None), 1), (dict(wsb=100), 1),
    (dict(lens=at(0x200000)), 1), (dict(lens=at(0x20000c)), 1), (dict(lens=at(0x210000)), 1),
    (dict(rows=at(0x220008)), 1), (dict(desc=_desc(head_dim=72, cache_dtype=0)), 2),
    (dict(desc=_desc(head_dim=80, cache_dtype=0)), 2), (dict(desc=_desc(head_dim=64, cache_dtype=1)), 2),
])
def test_evict_refusals(lib, kw, status):
    assert _evict(lib, **kw) == status
    assert lib.pa_last_error_string().decode()


def test_evict_with_nothing_to_do(lib):
    assert _evict(lib, S=0, W=None, k=None) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    import paged_kv_cache_286_gb300 as pa
    x = torch.zeros(4, 4, 544, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        pa.cache_read(torch.zeros(4, dtype=torch.int64), x, x, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        pa.evict_keys(x, x, *[torch.zeros(1, dtype=torch.int32)] * 3, torch.zeros(1), torch.zeros(1), max_context_len=1,
                      max_keep_len=1, recent=0)
    with pytest.raises(ValueError, match="17"):
        pa.cache_desc(torch.zeros(4, 4, 540, dtype=torch.uint8))
    with pytest.raises(ValueError, match="head_dim"):
        pa.new_mxfp4_cache(4, 4, 96, device="cpu")
    assert pa.cache_desc(x).head_dim == 64 and pa.cache_desc(x).cache_dtype == 3


# ---- the block manager's evict -------------------------------------------------------------------
@pytest.fixture()
def bm(lib):
    from paged_kv_cache_286_gb300.block_manager import BlockManager
    return BlockManager(12)


def test_bm_evict_in_place_releases_the_rest(bm):
    bm.append(0, 70)                                   # 5 blocks
    old = bm.block_table(0).tolist()
    assert bm.evict(0, 33, 7).tolist() == old[:3] + [-1] * 4
    assert bm.num_tokens(0) == 33 and bm.num_free() == 9
    slots, _ = bm.append(0, 2)
    assert slots.tolist() == [old[2] * 16 + 1, old[2] * 16 + 2]


def test_bm_evict_leaves_shared_blocks_alone(bm):
    bm.append(0, 64)
    bm.fork(0, 1)
    old = bm.block_table(0).tolist()
    new = bm.evict(0, 20).tolist()
    assert len(new) == 2 and not set(new) & set(old)
    assert bm.block_table(1).tolist() == old and [bm.refcount(b) for b in old] == [1] * 4
    assert bm.num_free() == 12 - 4 - 2
    assert bm.evict(1, 20).tolist() == old[:2]         # alone now: in place


def test_bm_evict_takes_rewritten_blocks_out_of_the_prefix_cache(bm):
    toks = list(range(48))
    bm.append_tokens(0, toks)
    assert bm.cached_prefix(toks) == 48
    bm.evict(0, 16)
    assert bm.cached_prefix(toks) == 0                 # its first block is rewritten
    bm.append_tokens(0, list(range(100, 132)))         # no longer hashed
    bm.free(0)
    assert bm.num_free() == 12 and bm.cached_prefix(list(range(16))) == 0


def test_bm_evict_errors_change_nothing(bm):
    from paged_kv_cache_286_gb300.block_manager import NoSpace
    bm.append(0, 160)                                  # 10 of 12 blocks
    bm.fork(0, 1)
    table = bm.block_table(0).tolist()
    with pytest.raises(NoSpace):
        bm.evict(0, 40)                                # three fresh blocks are not there
    for bad in (lambda: bm.evict(9, 1), lambda: bm.evict(0, -1), lambda: bm.evict(0, 161), lambda: bm.evict(0, 40, 2)):
        with pytest.raises(ValueError):
            bad()
    assert bm.block_table(0).tolist() == table and bm.num_tokens(0) == 160 and bm.num_free() == 2
    assert bm.evict(0, 160).tolist() == table          # nothing to drop: nothing changes
    assert bm.evict(0, 0).tolist() == [] and bm.num_tokens(0) == 0
    assert bm.append(0, 1)[0].shape == (1,)
