"""The paged-cache serving operators and the cases they are measured on.

Two entry points of kv_cache_append_gb300 work on a pool of cache blocks
[num_blocks, Hk, block_size, D] that a block table hands out to sequences:

* append_rotary_paged -- the new tokens' keys and queries are rotated to their
  positions, and the keys and values written into the pool. A pool in 8 bits
  (e4m3 or e5m2) has one scale for each (block, head), a power of two that
  grows when a new token needs it; the rows that the block held before are then
  rounded again to the larger step.
* attention_over_paged_cache -- packed queries attend the pool's blocks under
  the lower-right causal rule, with an optional cap on the scores
  (cap * tanh(s / cap)), a bias linear in the distance, and a sliding window.

With ``own`` false, ``run`` computes them in their plain form (elementary torch
operations); with ``own`` true it makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# 8-bit formats: explicit mantissa bits, least normal exponent, log2 of the
# power of two below the largest value (the largest is 1.75 times that)
EIGHT = {torch.float8_e4m3fn: (3, -6, 8), torch.float8_e5m2: (2, -14, 15)}


# ------------------------------------------------------------------ cases
def _append(name, dtype, pool, B, s, k, Hq, Hk, D, Dv, bs, rot=None, inter=False):
    c = {"op": "append", "dtype": dtype, "pool": pool, "B": B, "s_lo": s[0], "s_hi": s[1],
         "k_lo": k[0], "k_hi": k[1], "Hq": Hq, "Hk": Hk, "D": D, "Dv": Dv, "bs": bs,
         "rot": D if rot is None else rot, "inter": inter}
    return c if name is None else dict(c, name=name)


def _attend(name, dtype, pool, B, s, k, Hq, Hk, D, Dv, bs, cap=0.0, slopes=False, window=0):
    c = {"op": "attend", "dtype": dtype, "pool": pool, "B": B, "s_lo": s[0], "s_hi": s[1],
         "k_lo": k[0], "k_hi": k[1], "Hq": Hq, "Hk": Hk, "D": D, "Dv": Dv, "bs": bs,
         "cap": cap, "slopes": slopes, "window": window}
    return c if name is None else dict(c, name=name)


def listed():
    # s: new tokens of a sequence (lo, hi); k: slots in the cache before them
    return [
        # one user's next token: launch latency
        _append("append_one", "bf16", "bf16", 1, (1, 1), (1000, 1000), 32, 8, 128, 128, 16),
        # a decode batch (the grouped-query decode configuration)
        _append("append_decode", "bf16", "bf16", 64, (1, 1), (1024, 8190), 32, 8, 128, 128, 64),
        # prompts entering an empty or short cache, half of each head rotated
        _append("append_prompt", "f16", "f16", 8, (401, 1999), (0, 700), 32, 8, 128, 128, 64,
                rot=64, inter=True),
        # the decode batch on an 8-bit pool: most calls meet a part-filled block
        _append("append8_decode", "bf16", "e4m3", 64, (1, 1), (1024, 8190), 32, 8, 128, 128, 64),
        # prompts on an 8-bit pool, one KV head of wide keys (the long multi-query heads)
        _append("append8_prompt", "f16", "e4m3", 4, (1501, 7001), (100, 3001), 16, 1, 192, 128, 16),
        # one user's next token on an 8-bit cache
        _attend("attend8_one", "bf16", "e4m3", 1, (1, 1), (1000, 1000), 32, 8, 128, 128, 16),
        # the decode batch on an 8-bit cache
        _attend("attend8_decode", "bf16", "e4m3", 64, (1, 1), (1024, 8190), 32, 8, 128, 128, 64),
        # speculative decoding over very long contexts, one KV head for 16 query heads
        _attend("attend8_mqa", "f16", "e4m3", 8, (8, 8), (60000, 65528), 16, 1, 192, 128, 64),
        # prompts in chunks over an 8-bit cache
        _attend("attend8_prompt", "bf16", "e4m3", 4, (513, 2001), (0, 8190), 32, 8, 128, 128, 64),
        # short speculative steps, capped scores within a sliding window
        _attend("attend_capped_spec", "bf16", "bf16", 64, (1, 4), (64, 16380), 32, 8, 128, 128, 32,
                cap=50.0, window=4096),
        # chunked appends (the chunked configuration's heads) with a distance bias
        _attend("attend_biased_chunk", "f16", "f16", 2, (24, 40), (100, 2000), 8, 2, 64, 64, 16,
                slopes=True),
        # prompts with capped scores
        _attend("attend_capped_prompt", "bf16", "bf16", 3, (701, 2001), (0, 4000), 16, 4, 128, 128,
                128, cap=30.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(32, 8), (16, 1), (8, 2), (8, 8), (20, 4), (6, 2), (12, 1)])
    D, Dv = rng.choice([(128, 128), (64, 64), (192, 128), (80, 80), (96, 64), (256, 128), (40, 48)])
    bs = rng.choice([8, 16, 24, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f16", "f32"])
    pool = rng.choice([dtype, "e4m3", "e4m3", "e5m2"])
    B = _log(rng, 1, 96)
    wide = heads[1] * (D + Dv)
    if rng.random() < 0.4:  # append: up to about 30,000 tokens in all
        s_hi = _log(rng, 1, max(1, min(7000, 30000 // B)))
        s_lo = rng.randint(1, s_hi)
        k_hi = _log(rng, 1, max(1, min(8000, 20_000_000 // (B * wide))))
        rot = rng.choice([D, D, D // 2])
        return _append(None, dtype, pool, B, (s_lo, s_hi), (rng.randint(0, k_hi), k_hi), *heads,
                       D, Dv, bs, rot=rot, inter=rng.random() < 0.3)
    small = 8 if dtype == "f32" else 1
    k_hi = _log(rng, 1, max(1, min(60000, 500_000_000 // (B * wide * small))))
    # query rows: the plain form's scores stay under 2 GB, the work under the largest listed case's
    pairs = min(400_000_000, 1_500_000_000_000 // (4 * (D + Dv))) // small
    s_hi = max(1, min(2000, pairs // (B * heads[0] * (k_hi + 2000))))
    if rng.random() < 0.5:
        s_hi = min(s_hi, 8)
    s_hi = _log(rng, 1, s_hi)
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    window = rng.choice([0, 0, 0, rng.randint(1, 5000)])
    return _attend(None, dtype, pool, B, (rng.randint(1, s_hi), s_hi), (rng.randint(0, k_hi), k_hi),
                   *heads, D, Dv, bs, cap=cap, slopes=rng.random() < 0.25, window=window)


def _lens(case):
    """New tokens and earlier slots of each sequence: spread evenly over their
    ranges in an order of their own (prepare() deals them out by its seed)."""
    B = case["B"]
    s = [case["s_lo"] + int((case["s_hi"] - case["s_lo"] + 1) * ((i * 0.6180339887 + 0.999) % 1.0))
         for i in range(B)]
    k = [case["k_lo"] + int((case["k_hi"] - case["k_lo"] + 1) * ((i * 0.7548776662 + 0.999) % 1.0))
         for i in range(B)]
    return s, k


def work(case):
    c = case
    s, k = _lens(c)
    es = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]]
    ps = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "e5m2": 1}[c["pool"]]
    T, row = sum(s), c["Hk"] * (c["D"] + c["Dv"])
    if c["op"] == "append":
        # the queries in and out, the new rows in, the pool rows out, the angles
        n = T * (2 * c["Hq"] * c["D"] * es + row * (es + ps) + c["rot"] * 4)
        if ps == 1:  # each touched block's two scales, read and written
            n += sum((b + a - 1) // c["bs"] - a // c["bs"] + 1 for a, b in
                     zip(k, (x + y for x, y in zip(k, s)))) * c["Hk"] * 16
        return {"bytes": n, "flops": T * 3 * c["rot"] * (c["Hq"] + c["Hk"])}
    w = c["window"] or (1 << 60)
    slots = sum(min(a + n, w + n - 1) for a, n in zip(k, s))
    # visible (query, slot) pairs: row t of a sequence sees min(a + t + 1, w) slots
    pairs = 0
    for a, n in zip(k, s):
        full = max(0, min(n, w - a))  # rows that the window does not cut
        pairs += full * (a + 1) + full * (full - 1) // 2 + (n - full) * min(w, a + n)
    n = slots * row * ps + T * c["Hq"] * (c["D"] + c["Dv"]) * es
    if ps == 1:
        n += sum(-(-min(a + m, w + m - 1) // c["bs"]) for a, m in zip(k, s)) * c["Hk"] * 8
    return {"bytes": n, "flops": 2 * pairs * c["Hq"] * (c["D"] + c["Dv"])}


# ----------------------------------------------------------------- inputs
def _to_pool(x, dtype):
    """A pool of values in its type: (pool, scale for each block and head, or None)."""
    if dtype not in EIGHT:
        return x.to(dtype), None
    _, _, top = EIGHT[dtype]
    m, e = torch.frexp(x.abs().amax(dim=(2, 3)).double())
    scale = torch.exp2((e - 1 - top + (m > 0.875)).double()).float()
    return (x / scale[:, :, None, None]).to(dtype), scale


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    cpu = torch.Generator()
    cpu.manual_seed(int(seed))
    dt, pt = DTYPES[c["dtype"]], DTYPES[c["pool"]]
    B, Hq, Hk, D, Dv, bs = (c[n] for n in ("B", "Hq", "Hk", "D", "Dv", "bs"))
    s, k = _lens(c)
    order = torch.randperm(B, generator=cpu).tolist()
    s, k = [s[i] for i in order], [k[i] for i in order]
    total = [a + b for a, b in zip(s, k)]
    need = [-(-t // bs) for t in total]
    T, nb = sum(s), sum(need)
    num_blocks = nb + 3
    ids = torch.randperm(num_blocks, generator=cpu)[:nb]
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(s), 0)

    def pool_of(width):
        # blocks and heads differ in size, as keys and values of a trained model do
        x = torch.randn(num_blocks, Hk, bs, width, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(num_blocks, Hk, 1, 1, generator=g, device=dev))
        return _to_pool(x, pt)

    kp, ks = pool_of(D)
    vp, vs = pool_of(Dv)
    st = {"op": c["op"], "key_pool": kp, "value_pool": vp, "key_scale": ks, "value_scale": vs,
          "table": table.to(dev), "cu": cu.to(dev),
          "seqlens_k": torch.tensor(total, dtype=torch.int32, device=dev),
          "max_q": max(s), "max_k": max(total)}
    if c["op"] == "append":
        # the three projections leave one matrix; the operator takes its column ranges
        qkv = torch.randn(T, Hq * D + Hk * D + Hk * Dv, generator=g, device=dev).to(dt)
        st["query"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["key"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        st["value"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, Dv)
        R = c["rot"]
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
        ang = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["inter"] = c["inter"]
    else:
        # queries large enough that some rows look at few slots and a cap is felt
        st["query"] = (2.0 * torch.randn(T, Hq, D, generator=g, device=dev)).to(dt)
        st["cap"], st["window"], st["slopes"] = c["cap"], c["window"], None
        if c["slopes"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq)
    return st


# ---------------------------------------------------------------- plain form
def _rows(st):
    """Of each packed token: its sequence, and its slot in the cache."""
    tok = torch.arange(st["query"].shape[0], device=st["cu"].device, dtype=torch.int32)
    seq = torch.bucketize(tok, st["cu"][1:], right=True)
    ends = st["cu"][1:][seq]
    return seq, (st["seqlens_k"][seq] - (ends - tok)).long()


def _rotate(x, cos, sin, inter):
    h = cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _round8(x, dtype):
    """64-bit values rounded once, ties to even, to an 8-bit format, ending at its largest."""
    bits, low, top = EIGHT[dtype]
    _, e = torch.frexp(x)
    step = torch.exp2((torch.clamp(e - 1, min=low) - bits).double())
    y = torch.round(x / step) * step
    most = 1.75 * 2.0 ** top
    return y.clamp(-most, most).float().to(dtype)


def _plain_write8(pool, scale, x, blk, row, first, keep):
    """x [T, Hk, width] into rows (blk, row) of an 8-bit pool; `first` is each
    sequence's first touched block and `keep` how many of its rows it held."""
    _, _, top = EIGHT[pool.dtype]
    u8 = pool.view(torch.uint8)
    T, Hk, _ = x.shape
    most = torch.zeros(scale.shape, dtype=torch.float64, device=x.device)
    most.scatter_reduce_(0, blk[:, None].expand(T, Hk), x.abs().amax(-1), "amax")
    m, e = torch.frexp(most)
    want = torch.exp2((e - 1 - top + (m > 0.875)).clamp(-100, 100).double())
    want = torch.where(most > 0, want, 2.0 ** -100).float()
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
    touched[blk] = True
    held = torch.zeros_like(touched)
    held[first] = keep > 0
    new = torch.where(held[:, None], torch.maximum(scale, want), want)
    new = torch.where(touched[:, None], new, scale)
    # the rows that the first blocks held, at their new step
    ratio = (scale[first] / new[first])[:, :, None, None]
    old = pool[first].float()
    again = _round8((old * ratio).double(), pool.dtype).view(torch.uint8)
    mine = torch.arange(pool.shape[2], device=x.device)[None, :] < keep[:, None]
    u8[first] = torch.where(mine[:, None, :, None], again, u8[first])
    u8[blk, :, row] = _round8(x / new[blk].double()[..., None], pool.dtype).view(torch.uint8)
    scale.copy_(new)


def _plain_append(st):
    seq, pos = _rows(st)
    bs = st["key_pool"].shape[2]
    blk, row = st["table"][seq, pos // bs].long(), pos % bs
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    q = _rotate(st["query"].float(), cos, sin, st["inter"]).to(st["query"].dtype)
    if st["key_scale"] is None:
        k = _rotate(st["key"].float(), cos, sin, st["inter"])
        st["key_pool"][blk, :, row] = k.to(st["key_pool"].dtype)
        st["value_pool"][blk, :, row] = st["value"]
        return {"query": q, "key_pool": st["key_pool"], "value_pool": st["value_pool"]}
    # 64 bits: a value next to a border of the 8-bit grid must fall on its side
    k = _rotate(st["key"].double(), cos.double(), sin.double(), st["inter"])
    start = (st["seqlens_k"] - (st["cu"][1:] - st["cu"][:-1])).long()
    first = st["table"].gather(1, (start // bs)[:, None])[:, 0].long()
    _plain_write8(st["key_pool"], st["key_scale"], k, blk, row, first, start % bs)
    _plain_write8(st["value_pool"], st["value_scale"], st["value"].double(), blk, row, first,
                  start % bs)
    return {n: st[n] if n != "query" else q
            for n in ("query", "key_pool", "value_pool", "key_scale", "value_scale")}


def _plain_attend(st):
    q = st["query"]
    T, Hq, D = q.shape
    kp, vp, table = st["key_pool"], st["value_pool"], st["table"].long()
    B, (_, Hk, bs, Dv), S, K = table.shape[0], vp.shape, st["max_q"], st["max_k"]
    dev = q.device
    j = torch.arange(K, device=dev)
    n = st["cu"][1:] - st["cu"][:-1]
    live = j < st["seqlens_k"][:, None]
    blk = torch.where(live, table[:, (j // bs).clamp(max=table.shape[1] - 1)], 0)  # [B, K]

    def of(pool, scale):  # [B, Hk, K, width], slots past the end 0
        x = pool[blk.reshape(-1), :, (j % bs).repeat(B)] if scale is None else \
            pool.view(torch.uint8)[blk.reshape(-1), :, (j % bs).repeat(B)].view(pool.dtype)
        x = x.float().view(B, K, Hk, -1)
        if scale is not None:
            x *= scale[blk][..., None]
        x.masked_fill_(~live[..., None, None], 0.0)
        return x.transpose(1, 2)

    t = torch.arange(S, device=dev)
    rows = (st["cu"][:-1, None] + t).clamp(max=T - 1)  # [B, S]
    x = q.float()[rows].view(B, S, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    s = (x @ of(kp, st["key_scale"]).transpose(2, 3)).view(B, Hk, Hq // Hk, S, K)
    s *= 1.0 / math.sqrt(D)
    if st["cap"]:
        s = st["cap"] * torch.tanh(s / st["cap"])
    pos = (st["seqlens_k"] - n)[:, None] + t  # [B, S]
    far = pos[..., None] - j  # [B, S, K]
    if st["slopes"] is not None:
        s -= st["slopes"].view(1, Hk, Hq // Hk, 1, 1) * far[:, None, None].float()
    see = (far >= 0) & live[:, None]
    if st["window"]:
        see &= far < st["window"]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38))
    del s
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, -1, K) @ of(vp, st["value_scale"])).view(B, Hk, Hq // Hk, S, Dv) / total
    seq, _ = _rows(st)
    tok = torch.arange(T, device=dev) - st["cu"][seq]
    return o.permute(0, 3, 1, 2, 4).reshape(B, S, Hq, Dv)[seq, tok].to(q.dtype)


def run(state):
    st = state
    if own:
        import kv_cache_append_gb300 as kvc
        if st["op"] == "append":
            out = kvc.append_rotary_paged(
                st["query"], st["key"], st["value"], st["key_pool"], st["value_pool"],
                st["table"], st["cu"], st["seqlens_k"], st["cos"], st["sin"],
                key_scale=st["key_scale"], value_scale=st["value_scale"],
                interleaved=st["inter"], max_seqlen_q=st["max_q"])
            names = ("query", "key_pool", "value_pool", "key_scale", "value_scale")
            return {n: out[n] for n in names if out[n] is not None}
        return kvc.attention_over_paged_cache(
            st["query"], st["key_pool"], st["value_pool"], st["table"], st["cu"], st["seqlens_k"],
            key_scale=st["key_scale"], value_scale=st["value_scale"], softcap=st["cap"],
            alibi_slopes=st["slopes"], window=st["window"], max_seqlen_q=st["max_q"])
    return _plain_append(st) if st["op"] == "append" else _plain_attend(st)


# ------------------------------------------------------- 64 bits, one sequence at a time
def _exact_pool(st, which, b, lo, hi):
    """Slots lo..hi-1 of sequence b as the 64-bit values that the pool stands for: [hi-lo, Hk, width]."""
    pool, scale = st[which + "_pool"], st[which + "_scale"]
    bs = pool.shape[2]
    ids = st["table"][b, lo // bs:(hi + bs - 1) // bs].long()
    if scale is None:
        x = pool[ids].double()
    else:
        x = pool.view(torch.uint8)[ids].view(pool.dtype).double()
        x = x * scale[ids].double()[:, :, None, None]
    x = x.permute(0, 2, 1, 3).flatten(0, 1)
    at = lo - lo // bs * bs
    return x[at:at + hi - lo]


def _exact_attend(st):
    q, cu, kl = st["query"], st["cu"].tolist(), st["seqlens_k"].tolist()
    T, Hq, D = q.shape
    Hk, Dv = st["value_pool"].shape[1], st["value_pool"].shape[3]
    out = torch.zeros(T, Hq, Dv, dtype=torch.float64, device=q.device)
    for b, K in enumerate(kl):
        n = cu[b + 1] - cu[b]
        lo = max(0, K - n + 1 - st["window"]) if st["window"] else 0
        keys, vals = _exact_pool(st, "key", b, lo, K), _exact_pool(st, "value", b, lo, K)
        slot = torch.arange(lo, K, device=q.device)
        per = max(1, 300_000_000 // (Hq * (K - lo)))
        for t0 in range(0, n, per):
            t1 = min(n, t0 + per)
            at = torch.arange(K - n + t0, K - n + t1, device=q.device)
            hidden = slot[None] > at[:, None]
            if st["window"]:
                hidden |= slot[None] <= at[:, None] - st["window"]
            for h in range(Hq):
                s = q[cu[b] + t0:cu[b] + t1, h].double() @ keys[:, h * Hk // Hq].t() / math.sqrt(D)
                if st["cap"]:
                    s = st["cap"] * torch.tanh(s / st["cap"])
                if st["slopes"] is not None:
                    s = s + st["slopes"][h].double() * (slot[None] - at[:, None])
                a = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
                out[cu[b] + t0:cu[b] + t1, h] = a @ vals[:, h * Hk // Hq]
    return out


def _exact_append(st):
    cu, kl = st["cu"].tolist(), st["seqlens_k"].tolist()
    bs = st["key_pool"].shape[2]
    pos = torch.cat([torch.arange(K - (cu[b + 1] - cu[b]), K) for b, K in enumerate(kl)])
    pos = pos.to(st["query"].device)
    cos, sin = st["cos"].double()[pos][:, None], st["sin"].double()[pos][:, None]

    def turn(x):  # complex multiplication, pair by pair
        h, x = cos.shape[-1], x.double()
        z = x[..., :2 * h]
        z = z.unflatten(-1, (h, 2)) if st["inter"] else z.unflatten(-1, (2, h)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.complex(cos, sin)
        z = torch.view_as_real(z)
        z = z.flatten(-2) if st["inter"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., 2 * h:]], -1)

    out = {"query": turn(st["query"])}
    scales = {}
    for which, new in (("key", turn(st["key"])), ("value", st["value"].double())):
        pool, scale = st[which + "_pool"], st[which + "_scale"]
        held = pool.double()
        at = None if scale is None else scale.double().clone()
        for b, K in enumerate(kl):
            first = K - (cu[b + 1] - cu[b])
            for i in range(first // bs, -(-K // bs)):
                lo, hi = max(first, i * bs), min(K, (i + 1) * bs)
                x = new[cu[b] + lo - first:cu[b] + hi - first].transpose(0, 1)  # [Hk, rows, width]
                blk, r0, r1 = int(st["table"][b, i]), lo - i * bs, hi - i * bs
                if scale is None:
                    held[blk, :, r0:r1] = x
                    continue
                top = 1.75 * 2.0 ** EIGHT[pool.dtype][2]
                big = x.abs().flatten(1).amax(1)
                step = torch.exp2(torch.ceil(torch.log2(big / top)).clamp(-100, 100))
                step = torch.where(step * top < big, step * 2, step)
                step = torch.where(step * top / 2 >= big, step / 2, step)
                if r0:
                    step = torch.maximum(step, at[blk])
                    ratio = (at[blk] / step)[:, None, None]
                    held[blk, :, :r0] = _round8(held[blk, :, :r0] * ratio, pool.dtype).double()
                held[blk, :, r0:r1] = _round8(x / step[:, None, None], pool.dtype).double()
                at[blk] = step
        out[which + "_pool"] = held
        scales[which + "_scale"] = at
    if st["key_scale"] is not None:
        out.update(scales)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "append":
        bs = st["key_pool"].shape[2]
        if sum(st["seqlens_k"].tolist()) // bs > 200_000:
            return None
        return _exact_append(st)
    if case["op"] == "attend" and work(case)["flops"] > 4e12:
        return None
    return _exact_attend(st)
