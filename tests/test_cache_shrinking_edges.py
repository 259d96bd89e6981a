"""Host side of the cache-shrinking calls, edges: block tables of sequences evicted in one call."""

import random

import numpy as np
import pytest

pa_build = pytest.importorskip("paged_kv_cache_286_gb300.build")

BS = 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa_build.build()


def manager(blocks):
    from paged_kv_cache_286_gb300.block_manager import BlockManager
    return BlockManager(blocks)


# ---- several sequences evicted in one call -------------------------------------------------------
def check_plan(bm, seqs, keeps, before, new):
    """The tables are what one evict_keys call may take: no block written for a sequence is read or
    written for another, and an entry is the sequence's own at that place or nobody's."""
    held = {s: set(t) for s, t in before.items()}
    written = []
    for s, keep, row in zip(seqs, keeps, new):
        n = -(-keep // BS)
        row = row.tolist()
        assert all(b >= 0 for b in row[:n]) and all(b == -1 for b in row[n:])
        assert bm.block_table(s).tolist() == row[:n] and bm.num_tokens(s) == keep
        moves = keep < before_tokens[s]
        if not moves:
            assert row[:n] == before[s]
            continue
        for i, b in enumerate(row[:n]):
            if b != before[s][i]:
                assert all(b not in held[o] for o in held)
            assert all(b not in held[o] for o in held if o != s)
        written += row[:n]
    assert len(written) == len(set(written))


before_tokens = {}


def run_batch(bm, seqs, keeps, others=()):
    before = {s: bm.block_table(s).tolist() for s in list(seqs) + list(others)}
    before_tokens.clear()
    before_tokens.update({s: bm.num_tokens(s) for s in before})
    new = bm.evict_batch(seqs, keeps, 16)
    check_plan(bm, seqs, keeps, before, new)
    return before, new


def test_a_sequence_and_its_fork_evicted_together():
    bm = manager(16)
    bm.append(0, 80)
    bm.fork(0, 1)
    run_batch(bm, [0, 1], [60, 60])
    assert bm.num_free() == 16 - 8                      # the five shared blocks are free again
    assert all(bm.refcount(b) == 1 for s in (0, 1) for b in bm.block_table(s))


def test_released_blocks_are_not_handed_out_within_the_call():
    bm = manager(9)
    bm.append(0, 80)                                    # blocks 0 .. 4
    bm.append(1, 32)                                    # 5, 6
    bm.fork(1, 2)                                       # 7 and 8 are free
    run_batch(bm, [0, 1], [20, 20], others=[2])
    assert sorted(bm.block_table(1).tolist()) == [7, 8]
    bm = manager(7)                                     # none are free: 0's are not there for 1 yet
    from paged_kv_cache_286_gb300.block_manager import NoSpace
    bm.append(0, 80)
    bm.append(1, 32)
    bm.fork(1, 2)
    tables = bm.tables([0, 1, 2]).tolist()
    with pytest.raises(NoSpace):
        bm.evict_batch([0, 1], [20, 20])
    assert bm.tables([0, 1, 2]).tolist() == tables and bm.num_free() == 0
    assert [bm.num_tokens(s) for s in (0, 1, 2)] == [80, 32, 32]


def test_plans_of_random_batches():
    rng = random.Random(3)
    for _ in range(300):
        bm = manager(rng.choice([24, 40, 200]))
        from paged_kv_cache_286_gb300.block_manager import NoSpace
        seqs = []
        for s in range(rng.randrange(1, 8)):
            try:
                if seqs and rng.random() < 0.5:
                    bm.fork(rng.choice(seqs), s)
                    if rng.random() < 0.5:
                        bm.append(s, rng.randrange(1, 40))
                elif rng.random() < 0.5:
                    bm.append_tokens(s, [7] * rng.randrange(1, 90))     # prefixes shared through the cache
                else:
                    bm.append(s, rng.randrange(1, 90))
            except NoSpace:
                continue
            seqs.append(s)
        batch = [s for s in seqs if rng.random() < 0.8]
        rng.shuffle(batch)
        keeps = [rng.choice([0, bm.num_tokens(s), rng.randrange(bm.num_tokens(s) + 1)]) for s in batch]
        tables = {s: bm.block_table(s).tolist() for s in seqs}
        free = bm.num_free()
        try:
            before, _ = run_batch(bm, batch, keeps, [s for s in seqs if s not in batch])
        except NoSpace:
            assert {s: bm.block_table(s).tolist() for s in seqs} == tables and bm.num_free() == free
            continue
        held = {}
        for s in seqs:
            for b in bm.block_table(s).tolist():
                held[b] = held.get(b, 0) + 1
        assert all(bm.refcount(b) == held.get(b, 0) for b in range(bm.num_blocks))
        assert bm.num_free() == bm.num_blocks - len(held)
        for s in seqs:
            bm.free(s)
        assert bm.num_free() == bm.num_blocks


def test_batch_of_one_is_evict_and_of_none_is_nothing():
    plans = []
    for batch in (False, True):
        bm = manager(12)
        bm.append(0, 64)
        bm.fork(0, 1)
        bm.append(0, 30)
        plans.append((bm.evict_batch([0], [70], 7)[0] if batch else bm.evict(0, 70, 7)).tolist()
                     + [bm.num_free()] + bm.append(1, 1)[0].tolist())
        assert bm.evict_batch([], []).shape == (0, 1)
    assert plans[0] == plans[1]


def test_batch_refusals_change_nothing():
    bm = manager(12)
    bm.append(0, 64)
    bm.append(1, 20)
    for seqs, keeps, width in (([0, 0], [1, 1], 4), ([0, 9], [1, 1], 4), ([0, 1], [1, 21], 4), ([0, 1], [1, -1], 4),
                               ([1, 0], [1, 33], 2), ([0], [1, 2], 4)):
        with pytest.raises(ValueError):
            bm.evict_batch(seqs, keeps, width)
    assert [bm.num_tokens(s) for s in (0, 1)] == [64, 20] and bm.num_free() == 6
    import ctypes
    from paged_kv_cache_286_gb300 import _lib
    L = _lib.load()
    out, one = np.zeros(4, np.int32), np.zeros(1, np.int64)
    a = (one.ctypes.data, one.ctypes.data, 1, out.ctypes.data, 4)
    assert L.pa_bm_evict_batch(None, *a) == -2
    for i, bad in ((0, None), (1, None), (2, -1), (3, None), (4, -1)):
        b = list(a)
        b[i] = bad
        assert L.pa_bm_evict_batch(ctypes.c_void_p(bm._h), *b) == -2


# ---- after an eviction to nothing ----------------------------------------------------------------
def test_a_sequence_evicted_to_nothing_takes_no_cached_prefix():
    """Its next tokens follow those it dropped: blocks that hold the same tokens after the same prefix
    were computed over that prefix's keys, and blocks of a fresh prompt at other positions."""
    bm = manager(12)
    toks = list(range(48))
    bm.append_tokens(0, toks)                           # caches three blocks
    bm.append_tokens(1, toks[:16])
    bm.evict(1, 0)
    slots, pairs, hit = bm.append_tokens(1, toks[16:48])
    assert hit == 0 and len(slots) == 32 and pairs == []
    assert not set(bm.block_table(1).tolist()) & set(bm.block_table(0).tolist())
    bm.evict(1, 0)
    assert bm.append_tokens(1, toks)[2] == 0
    bm.append_tokens(2, toks)                           # an empty one still does
    assert bm.block_table(2).tolist() == bm.block_table(0).tolist()


# ---- workspaces ----------------------------------------------------------------------------------
def test_only_mxfp4_steps_have_room_for_bf16_copies():
    """48 decode tokens beside two chunks of 512, 32 q heads on 8 of 128 dims, contexts to 4,096."""
    torch = pytest.importorskip("torch")
    import paged_kv_cache_286_gb300 as pa
    L = pa.library()
    shape, bs = (50, 48 + 2 * 512, 32, 8, 128), 16
    BF16, E4M3, MXFP4 = 0, 1, 3
    pools = {BF16: torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16),
             E4M3: torch.zeros(4, 8, 16, 128, dtype=torch.uint8), MXFP4: torch.zeros(4, 8, 1088, dtype=torch.uint8)}
    for name in ("attention", "attention_key_weights"):
        plain = getattr(L, f"pa_{name}_workspace_size")(*shape, bs, 4096, 512)
        size_for = getattr(L, f"pa_{name}_workspace_size_for")
        py = getattr(pa, f"{name}_workspace_size")
        for dt in (BF16, E4M3):
            assert size_for(dt, *shape, bs, 4096, 512) == plain == py(*shape, 4096, 512, k_cache=pools[dt])
        mx = size_for(MXFP4, *shape, bs, 4096, 512)
        assert (256 << 20) <= mx - plain <= (257 << 20)
        assert mx == py(*shape, 4096, 512) == py(*shape, 4096, 512, k_cache=pools[MXFP4])
        # decode steps have none of it
        assert size_for(MXFP4, 50, 50, 32, 8, 128, bs, 4096, 1) == \
            getattr(L, f"pa_{name}_workspace_size")(50, 50, 32, 8, 128, bs, 4096, 1)


# ---- the scheduler -------------------------------------------------------------------------------
@pytest.mark.parametrize("prefix", [False, True])
def test_scheduler_refuses_to_plan_over_evicted_keys(prefix):
    """Its context lengths and slots count tokens."""
    from paged_kv_cache_286_gb300.scheduler import Request, Scheduler
    s = Scheduler(16, prefix_caching=prefix)
    s.submit(Request(0, 40, 8))
    s.submit(Request(1, 20, 8))
    for _ in range(3):
        assert s.step() is not None
    s.bm.evict(1, 20)
    with pytest.raises(RuntimeError, match="evicted"):
        s.step()
    assert s.step_no == 3
