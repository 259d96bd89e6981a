"""The cache-shrinking operators, measured: attention that accumulates each key's weight, eviction of
the keys of least weight, 4-bit (MXFP4) append and read-back, and attention over a 4-bit pool.

`own` false: `run` computes them in plain torch operations; true: through the library.
"""

import math

import numpy as np
import torch

own = False

BS = 16  # tokens per block of the pool


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _weights(name, lens, nq, hq, hkv, d, pool, lens_seed=1, decay=1.0, chunks=""):
    return dict(name=name, op="weights", lens=lens, nq=nq, chunks=chunks, hq=hq, hkv=hkv, d=d, pool=pool,
                lens_seed=lens_seed, decay=decay)


def _attend(name, lens, nq, hq, hkv, d, lens_seed=1, chunks=""):
    return dict(name=name, op="attend", lens=lens, nq=nq, chunks=chunks, hq=hq, hkv=hkv, d=d, pool="mxfp4",
                lens_seed=lens_seed)


def _evict(name, lens, hkv, d, keep, recent, lens_seed=1):
    return dict(name=name, op="evict", lens=lens, hkv=hkv, d=d, keep=keep, recent=recent, lens_seed=lens_seed)


def _append(name, tokens, run, hkv, d):
    return dict(name=name, op="append", tokens=tokens, run=run, hkv=hkv, d=d)


def listed():
    return [
        # a decode step of a few short requests: launches and latency
        _weights("weights tiny decode", "list:10,40,20,80", 1, 4, 4, 64, "bf16"),
        # a 7B-class decode step (multi-head attention), 64 requests
        _weights("weights MHA decode", "uniform:64:512:4096", 1, 32, 32, 128, "bf16", lens_seed=2),
        # a decode step over an E4M3 cache with grouped heads, 256 requests, weights that fade
        _weights("weights GQA E4M3 decode", "lognormal:256:1000:16:8192", 1, 32, 8, 128, "e4m3", lens_seed=3,
                 decay=0.96875),
        # decodes beside two prompt chunks, one of them after a cached prefix
        _weights("weights decodes + chunks", "uniform:48:256:4096", 1, 32, 8, 128, "bf16", lens_seed=4,
                 chunks="512:512,512:2560"),
        # a few short requests trimmed to their budget
        _evict("evict few short", "list:100,333,517,64", 4, 64, 48, 16),
        # 64 requests of a 7B-class cache halved, an odd budget
        _evict("evict MHA half", "uniform:64:512:4096", 32, 128, 1001, 128, lens_seed=2),
        # long documents cut to a sixteenth
        _evict("evict long", "fixed:16:32768", 8, 128, 2048, 512),
        # the new tokens of one decode step
        _append("append 4-bit decode", 64, 1, 8, 128),
        # a prompt of odd length
        _append("append 4-bit prompt", 8191, 8191, 32, 128),
        # a decode step with grouped heads, 256 requests
        _attend("attend 4-bit GQA decode", "lognormal:256:1000:16:8192", 1, 32, 8, 128, lens_seed=3),
        # long documents, one token each
        _attend("attend 4-bit long", "fixed:16:32768", 1, 32, 8, 128),
        # decodes beside a prompt chunk
        _attend("attend 4-bit chunk", "uniform:16:256:4096", 1, 32, 8, 128, lens_seed=4, chunks="512:2560"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "evict", "append", "attend", "attend"])
    hq, hkv = rng.choice([(4, 4), (8, 8), (16, 16), (32, 32), (8, 4), (32, 8), (16, 2), (32, 2), (12, 3), (24, 8)])
    seed = rng.randrange(1000)
    if op == "append":
        tokens = _logint(rng, 1, 8000)
        return dict(op=op, tokens=tokens, run=rng.choice([1, 5, 500, tokens]), hkv=hkv, d=rng.choice([64, 128]))
    # requests and their longest context: at most the largest listed sum of keys x kv heads
    s = _logint(rng, 1, 200)
    top = min(32768, max(40, int((2.0e6 if op == "evict" else 4.0e6) / (s * hkv))))
    hi = _logint(rng, 20, top)
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    lens = "uniform:%d:%d:%d" % (s, lo, hi)
    if op == "evict":
        keep = max(1, int(hi * rng.uniform(0.05, 0.8)))
        return dict(op=op, lens=lens, hkv=hkv, d=rng.choice([64, 128]), keep=keep,
                    recent=int(keep * rng.uniform(0.0, 0.7)), lens_seed=seed)
    nq = rng.choice([1, 1, 1, 1, 2, 4, 5])  # single tokens, or a few to verify
    chunks = ""
    if rng.random() < 0.4 and s <= 48 and hi <= 4096:
        n = _logint(rng, 17, 500)
        chunks = "%d:%d" % (n, n + rng.choice([0, 1, 777, 2048]))
    if op == "weights":
        pool = rng.choice(["bf16", "bf16", "e4m3", "mxfp4"])
        d = 128 if pool == "e4m3" else rng.choice([64, 128])
        return dict(op=op, lens=lens, nq=nq, chunks=chunks, hq=hq, hkv=hkv, d=d, pool=pool, lens_seed=seed,
                    decay=rng.choice([1.0, 0.96875, 0.5]))
    return dict(op=op, lens=lens, nq=nq, chunks=chunks, hq=hq, hkv=hkv, d=rng.choice([64, 128]), pool="mxfp4",
                lens_seed=seed)


def _lens(case):
    """(context lengths, query counts) of the case's sequences."""
    rng = np.random.default_rng(7000 + case["lens_seed"])
    kind, rest = case["lens"].split(":", 1)
    if kind == "list":
        lens = np.array([int(x) for x in rest.split(",")])
    else:
        p = [int(x) for x in rest.split(":")]
        if kind == "fixed":
            lens = np.full(p[0], p[1])
        elif kind == "uniform":
            lens = rng.integers(p[1], p[2] + 1, p[0])
        else:
            lens = np.clip(np.round(rng.lognormal(math.log(p[1]), 0.8, p[0])), p[2], p[3]).astype(np.int64)
    nq = np.minimum(case.get("nq", 1), lens)
    for c in filter(None, case.get("chunks", "").split(",")):
        n, l = (int(x) for x in c.split(":"))
        lens, nq = np.append(lens, l), np.append(nq, n)
    return lens.astype(np.int64), nq.astype(np.int64)


def _row_bytes(pool, d):
    return {"bf16": 2 * d, "e4m3": d, "mxfp4": d // 2 + d // 32}[pool]


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "append":  # bf16 K and V in, codes out; codes in, bf16 out
        n = case["tokens"] * hkv
        return {"bytes": n * 2 * (4 * d + 2 * _row_bytes("mxfp4", d)) + 16 * case["tokens"], "flops": 4 * n * d}
    lens, nq = _lens(case)
    keys = float(lens.sum()) * hkv
    if case["op"] == "evict":
        kept = float(np.minimum(lens, case["keep"]).sum()) * hkv
        return {"bytes": keys * 8 + kept * (4 + 4 * 2 * d), "flops": keys}
    pairs = float((nq * (lens - nq) + nq * (nq + 1) // 2).sum())  # (query, key) pairs
    n = keys * 2 * _row_bytes(case["pool"], d) + float(nq.sum()) * case["hq"] * d * 4
    if case["op"] == "weights":
        n += keys * 8
    return {"bytes": n, "flops": 4.0 * d * case["hq"] * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _encode(x):
    """float32 [..., D] -> (4-bit codes, scale bytes) of blocks of 32: a power of two two below that of
    the block's largest magnitude, and the nearest of 0 .5 1 1.5 2 3 4 6 (ties to the even code)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    byte = (((amax.view(torch.int32) >> 23) & 255) - 2).clamp(min=0)
    s = b * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)
    a = s.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code | (torch.signbit(s).int() << 3)
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def _pack(code, byte):
    """Codes and scale bytes [NB, H, 16, ...] -> the pool's [NB, H, tile] bytes: 16 rows of codes (16-bit
    words of four dims, word g * blocks + b holds dims 32 b + 4 g ..), then 16 rows of scale bytes."""
    nb, h, _, d = code.shape
    w = code.reshape(nb, h, 16, d // 32, 8, 2, 2).transpose(3, 4)
    w = w[..., 0] | (w[..., 1] << 4)
    return torch.cat([w.reshape(nb, h, -1), byte.reshape(nb, h, -1)], -1).contiguous()


def _decode(rows, byte):
    """The values of rows of packed codes [..., D / 2] and their scale bytes [..., D / 32]: float32 [..., D]."""
    w = rows.unflatten(-1, (8, -1, 2)).transpose(-2, -3)
    code = torch.stack([w & 15, w >> 4], -1).flatten(-3).int()
    a = code & 7
    v = torch.where(a < 5, 0.5 * a, torch.where(a == 7, 6.0, a - 2.0))
    v = torch.where(code > 7, -v, v)
    return (v * (byte.int() << 23).view(torch.float32).unsqueeze(-1)).flatten(-2)


def _unpack(pool):
    """The values of a 4-bit pool: [NB, H, tile] bytes -> float32 [NB, H, 16, D]."""
    d = pool.shape[2] * 2 // 17
    return _decode(pool[..., :8 * d].unflatten(-1, (16, -1)), pool[..., 8 * d:].unflatten(-1, (16, -1)))


def _randn(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(gen, kind, nb, hkv, d):
    if kind == "bf16":
        return torch.randn((nb, hkv, BS, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    x = _randn(gen, (nb, hkv, BS, d))
    if kind == "e4m3":
        return (x.float() / 0.0125).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _pack(*_encode(x.float()))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(100 + seed)
    rng = np.random.default_rng(seed)
    hkv, d = case["hkv"], case["d"]
    dev = lambda a, t: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    if case["op"] == "append":
        t = case["tokens"]
        per = min(case["run"], t)  # tokens of one request, in consecutive slots of its own blocks
        width = -(-per // BS) + 1
        nb = -(-t // per) * width
        first, i = rng.integers(0, BS, nb // width), np.arange(t)
        at = first[i // per] + i % per
        slots = rng.permutation(nb)[i // per * width + at // BS] * BS + at % BS
        st = dict(k=_randn(gen, (t, hkv, d)), v=_randn(gen, (t, hkv, d)),
                  slots=dev(slots, torch.int64),
                  k_cache=torch.zeros((nb, hkv, 17 * d // 2), dtype=torch.uint8, device="cuda"),
                  workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        return dict(st, case=case)
    lens, nq = _lens(case)
    S, blocks = len(lens), -(-lens // BS)
    width = int(blocks.max())
    nb = int(blocks.sum())
    evict = case["op"] == "evict"
    keep = np.minimum(lens, case["keep"]) if evict else lens
    kept_blocks = -(-keep // BS)
    total = nb + (int(kept_blocks.sum()) if evict else nb // 4 + 1)
    ids = rng.permutation(total)

    def table(counts, ids):
        t = np.full((S, width), -1, np.int32)
        t[np.arange(width)[None] < counts[:, None]] = ids[:counts.sum()]
        return t

    tables = table(blocks, ids)
    st = dict(case=case, tables=dev(tables, torch.int32), lens=dev(lens, torch.int32), lens_max=int(lens.max()))
    kind = case.get("pool", "bf16")
    st["k_cache"], st["v_cache"] = _pool(gen, kind, total, hkv, d), _pool(gen, kind, total, hkv, d)
    if case["op"] != "attend":
        st["row_len"] = int(lens.max()) + 5
        # what earlier steps left: few keys with much weight
        w = torch.rand((2 * S if evict else S, hkv, st["row_len"]), generator=gen, device="cuda").square_()
        st["key_weights"] = w.mul_(w).mul_(w)
    if evict:
        st.update(dst_tables=dev(table(kept_blocks, ids[nb:]), torch.int32),
                  keep=dev(np.full(S, case["keep"]), torch.int32), keep_max=int(keep.max()),
                  rows=dev(np.arange(S), torch.int32), dst_rows=dev(np.arange(S, 2 * S), torch.int32))
    else:
        qsl = np.concatenate([[0], np.cumsum(nq)])
        st.update(q=_randn(gen, (int(qsl[-1]), case["hq"], d)), qsl=dev(qsl, torch.int32), nq_max=int(nq.max()),
                  scale=d ** -0.5, k_scale=0.0125 if kind == "e4m3" else 1.0)
    if own:
        import paged_kv_cache_286_gb300 as pa
        if evict:
            n = pa.evict_workspace_size(S, hkv, st["lens_max"], st["keep_max"])
        else:
            f = pa.attention_workspace_size if case["op"] == "attend" else pa.attention_key_weights_workspace_size
            n = f(S, st["q"].shape[0], case["hq"], hkv, d, st["lens_max"], st["nq_max"])
        st["workspace"] = pa.new_workspace(n)
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_attend(s):
    import paged_kv_cache_286_gb300 as pa
    return pa.attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["qsl"], s["workspace"],
                        scale=s["scale"], max_context_len=s["lens_max"], max_query_len=s["nq_max"],
                        out_dtype=torch.bfloat16)


def _own_weights(s):
    import paged_kv_cache_286_gb300 as pa
    out = pa.attention_key_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["qsl"],
                                   s["key_weights"], s["workspace"], scale=s["scale"],
                                   max_context_len=s["lens_max"], max_query_len=s["nq_max"],
                                   decay=s["case"]["decay"], out_dtype=torch.bfloat16, k_scale=s["k_scale"],
                                   v_scale=s["k_scale"])
    return out, s["key_weights"]


def _own_evict(s):
    import paged_kv_cache_286_gb300 as pa
    kept, new_lens = pa.evict_keys(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["keep"],
                                   s["key_weights"], s["workspace"], max_context_len=s["lens_max"],
                                   max_keep_len=s["keep_max"], recent=s["case"]["recent"],
                                   dst_tables=s["dst_tables"], weight_rows=s["rows"],
                                   dst_weight_rows=s["dst_rows"])
    return kept, new_lens, s["key_weights"], s["k_cache"], s["v_cache"]


def _own_append(s):
    import paged_kv_cache_286_gb300 as pa
    pa.cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["workspace"])
    return pa.cache_read(s["slots"], s["k_cache"], s["v_cache"], s["workspace"], out_dtype=torch.bfloat16)


def _values(s, pool):
    """Keys or values of every sequence, float32 [S, Hkv, width * 16, D] (padding repeats block 0)."""
    t = s["tables"].clamp(min=0).long()
    g = pool[t]
    if pool.dtype == torch.bfloat16:
        g = g.float()
    elif pool.dim() == 4:
        g = g.view(torch.float8_e4m3fn).float() * s["k_scale"]
    else:
        g = _unpack(g.flatten(0, 1)).unflatten(0, t.shape)
    return g.transpose(1, 2).flatten(2, 3)


def _probabilities(s):
    """Softmax weights float32 [S, Hkv, n, G, L] of the padded queries, 0 where a query sees no key, and
    which padded queries there are."""
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    n = s["qsl"].diff()
    i = torch.arange(s["nq_max"], device="cuda")
    there = i < n[:, None]
    at = torch.where(there, s["qsl"][:-1, None] + i, 0).long()
    q = s["q"][at].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)       # [S, Hkv, n, G, D]
    k = _values(s, s["k_cache"])
    a = torch.matmul(q.flatten(2, 3) * s["scale"], k.transpose(-1, -2)).unflatten(2, q.shape[2:4])
    pos = (s["lens"] - n)[:, None] + i
    seen = there[:, :, None] & (torch.arange(k.shape[2], device="cuda") <= pos[:, :, None])
    a.masked_fill_(~seen[:, None, :, None], -math.inf)
    p = (a - a.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30), there


def _plain_out(s, p, there):
    o = torch.matmul(p.flatten(2, 3), _values(s, s["v_cache"])).unflatten(2, p.shape[2:4])
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)[there].to(torch.bfloat16)


def _plain_attend(s):
    return _plain_out(s, *_probabilities(s))


def _plain_weights(s):
    p, there = _probabilities(s)
    w = s["key_weights"]
    L = min(w.shape[2], p.shape[-1])
    old = w[..., :L]
    valid = torch.arange(L, device="cuda") < s["lens"][:, None, None]
    old.copy_(torch.where(valid, old * s["case"]["decay"] + p.sum((2, 3))[..., :L], old))
    return _plain_out(s, p, there), w


def _plain_evict(s):
    hkv, L = s["case"]["hkv"], s["lens_max"]
    lens = s["lens"][:, None, None]
    k = torch.minimum(s["keep"], s["lens"])[:, None, None]
    r = k.clamp(max=s["case"]["recent"])
    j = torch.arange(L, device="cuda")
    w = s["key_weights"][s["rows"].long()][..., :L]
    order = torch.where(w.isnan(), -math.inf, w).sort(dim=-1, descending=True, stable=True).indices
    cls = (j < lens).int() + ((j >= lens - r) & (j < lens))                      # kept anyway: 2, outside: 0
    order = order.gather(-1, cls.expand_as(w).gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)
    i = torch.arange(s["keep_max"], device="cuda")
    kept = torch.where(i < k, order[..., :s["keep_max"]], L).sort(-1).values
    there = i < k
    src = torch.where(there, kept, 0)
    # dst rows of the weights: the kept ones, then zeros up to the old length
    dst = s["key_weights"][s["dst_rows"].long()]
    moved = torch.nn.functional.pad(w.gather(-1, src), (0, max(0, dst.shape[2] - i.numel())))[..., :dst.shape[2]]
    jj = torch.arange(dst.shape[2], device="cuda")
    s["key_weights"][s["dst_rows"].long()] = torch.where(jj < k, moved, torch.where(jj < lens, 0.0, dst))
    head = torch.arange(hkv, device="cuda")[None, :, None].expand_as(src)
    from_b = s["tables"].long()[:, None].expand(-1, hkv, -1).gather(2, src // BS)
    to_b = s["dst_tables"].long()[:, None, :].expand(-1, hkv, -1).gather(2, (i // BS).expand_as(src))
    for pool in (s["k_cache"], s["v_cache"]):
        pool[to_b[there.expand_as(src)], head[there.expand_as(src)], (i % BS).expand_as(src)[there.expand_as(src)]] = \
            pool[from_b, head, src % BS][there.expand_as(src)]
    return (torch.where(there, kept, -1).int(), torch.minimum(s["keep"], s["lens"]), s["key_weights"], s["k_cache"],
            s["v_cache"])


def _plain_append(s):
    """The codes of each token written into its slot, and the values read back."""
    d, blk, off = s["case"]["d"], s["slots"] // BS, s["slots"] % BS

    def through(x, pool):
        code, byte = _encode(x.float())
        rows = code.unflatten(-1, (d // 32, 8, 2, 2)).transpose(2, 3)
        codes, scales = pool[..., :8 * d].unflatten(-1, (BS, -1)), pool[..., 8 * d:].unflatten(-1, (BS, -1))
        codes[blk, :, off] = (rows[..., 0] | (rows[..., 1] << 4)).flatten(2)
        scales[blk, :, off] = byte
        return _decode(codes[blk, :, off], scales[blk, :, off]).to(torch.bfloat16)

    return through(s["k"], s["k_cache"]), through(s["v"], s["v_cache"])


_plain = dict(weights=_plain_weights, attend=_plain_attend, evict=_plain_evict, append=_plain_append)
_own = dict(weights=_own_weights, attend=_own_attend, evict=_own_evict, append=_own_append)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------
def _decode64(pool, ids, h, n, k_scale):
    """The first n keys (or values) of kv head h in the blocks `ids`, float64 [n, D]."""
    x = pool[ids, h]
    if pool.dtype == torch.bfloat16:
        x = x.double()
    elif pool.dim() == 4:
        x = x.view(torch.float8_e4m3fn).float().double() * float(np.float32(k_scale))
    else:
        d = pool.shape[2] * 2 // 17
        code = torch.zeros((len(ids), BS, d), dtype=torch.long, device="cuda")
        for b in range(d // 32):
            for g in range(8):
                for e in range(4):
                    at = (g * (d // 32) + b) * 2 + e // 2
                    code[..., 32 * b + 4 * g + e] = (x[:, :8 * d].reshape(-1, BS, d // 2)[..., at] >> (4 * (e % 2))) & 15
        mag, exp = code & 1, (code >> 1) & 3
        v = torch.where(exp == 0, 0.5 * mag, (1 + 0.5 * mag) * 2.0 ** (exp - 1).double())
        v = torch.where(code >= 8, -v, v)
        e8 = x[:, 8 * d:].reshape(-1, BS, d // 32).double().repeat_interleave(32, -1)
        x = v * torch.exp2(e8 - 127)
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_append(x):
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent.double() - 3).clamp(min=-127)
    y = x * torch.exp2(-e)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return ((torch.round(y / step) * step).clamp(-6, 6) * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s["k"]), _exact_append(s["v"])
    lens, nq = _lens(case)
    if case["op"] == "evict":  # moves and choices: nothing is computed but the choice
        tables, dst = s["tables"].cpu().numpy(), s["dst_tables"].cpu().numpy()
        w = s["key_weights"].double()
        new = w.clone()
        k2, v2 = s["k_cache"].clone(), s["v_cache"].clone()
        S = len(lens)
        for i, L in enumerate(lens):
            k = min(int(L), case["keep"])
            r = min(case["recent"], k)
            best = w[i, :, :L - r].sort(dim=-1, descending=True, stable=True).indices[:, :k - r]
            kept = torch.cat([best.sort(-1).values, torch.arange(int(L) - r, int(L), device="cuda").expand(w.shape[1], r)], -1)
            new[S + i, :, :k] = w[i].gather(-1, kept)
            new[S + i, :, k:L] = 0
            at = torch.arange(k, device="cuda")
            tb, db = (torch.tensor(t[i], device="cuda").long() for t in (tables, dst))
            for h in range(w.shape[1]):
                for a, b in ((s["k_cache"], k2), (s["v_cache"], v2)):
                    b[db[at // BS], h, at % BS] = a[tb[kept[h] // BS], h, kept[h] % BS]
        return None, None, new, k2.float(), v2.float()
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pairs = float((nq * lens).sum()) * hq
    if pairs * d > 3e11 or float(lens.sum()) * hkv * d > 2e9:
        return None
    G = hq // hkv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    new = s["key_weights"].double() if case["op"] == "weights" else None
    tables, t0 = s["tables"].long(), 0
    for i, (L, n) in enumerate(zip(lens.tolist(), nq.tolist())):
        ids = tables[i, :-(-L // BS)]
        see = torch.arange(L, device="cuda")[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        for h in range(hkv):
            K, V = (_decode64(p, ids, h, L, s["k_scale"]) for p in (s["k_cache"], s["v_cache"]))
            a = torch.einsum("ngd,ld->gnl", s["q"][t0:t0 + n, h * G:(h + 1) * G].double(), K) * d ** -0.5
            p = torch.softmax(a.masked_fill(~see, -math.inf), -1)
            out[t0:t0 + n, h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", p, V)
            if new is not None:
                new[i, h, :L] = new[i, h, :L] * case["decay"] + p.sum((0, 1))
        t0 += n
    return out if new is None else (out, new)
