"""The kernel launches that bench.py claims for a step, from its shape."""

import types

import pytest

import bench

torch = pytest.importorskip("torch")
pa_build = pytest.importorskip("paged_kv_cache_286_gb300.build")


@pytest.mark.parametrize("seqs,ctx,query,dtype,want", [
    (4, 80, 1, "bf16", 3),          # append, plan, split-KV: no sequence has two partitions
    (200, 128, 1, "bf16", 3),
    (1, 16, 1, "fp8_e4m3", 3),
    (4, 4096, 1, "bf16", 4),        # and the merge
    (4, 80, 40, "bf16", 4),         # and the prefill tiles
    (4, 4096, 512, "bf16", 5),
    (4, 4096, 512, "fp8_e4m3", 5),
])
def test_launches_per_step(seqs, ctx, query, dtype, want):
    import paged_kv_cache_286_gb300 as pa
    pa_build.build()
    w = types.SimpleNamespace(num_seqs=seqs, num_tokens=seqs * query, num_q_heads=32, num_kv_heads=8, head_dim=128,
                              max_context_len=ctx, max_query_len=query, cache_dtype=dtype)
    pool = torch.zeros(2, 8, 16, 128, dtype=torch.bfloat16 if dtype == "bf16" else torch.uint8)
    step = types.SimpleNamespace(w=w, pa=pa, k_cache=pool, has_prefill=lambda: query > 16)
    assert bench.DeviceWorkload.launches_per_step(step) == want
