"""append_rotary_paged against the 64-bit reference."""
import random

import pytest
import torch

import kv_cache_append_gb300 as kvc
import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
      "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def make(seed, dtype, pool, lens, Hq, Hk, D, Dv, bs, R, pad=0, spare=2, stride=None):
    """lens: (S, K) of each sequence. CPU tensors of one call; the pools hold
    earlier rows, in 8 bits with scales of their own."""
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    T = sum(s for s, _ in lens) + pad
    need = [max(1, -(-k // bs)) for _, k in lens]
    nb = sum(need) + spare
    ids = list(range(nb))
    r.shuffle(ids)
    table = torch.zeros(len(lens), max(need) + 1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)])
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor([s for s, _ in lens]), 0)
    kl = torch.tensor([k for _, k in lens], dtype=torch.int32)
    dt, pt = DT[dtype], DT[pool]

    def pool_of(w):
        x = torch.randn(nb, Hk, bs, w, generator=g)
        if pool not in ("e4m3", "e5m2"):
            return x.to(dt), None
        sc = 2.0 ** torch.randint(-9, -4, (nb, Hk), generator=g).float()
        return (x * 100).to(pt), sc

    kp, ks = pool_of(D)
    vp, vs = pool_of(Dv)
    q = torch.randn(T, Hq, D, generator=g).to(dt)
    k = (torch.randn(T, Hk, D, generator=g) * 3).to(dt)
    v = torch.randn(T, Hk, Dv, generator=g).to(dt)
    P = max(k for _, k in lens) + 1
    ang = torch.arange(P, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / max(R, 1))
    return dict(query=q, new_key=k, new_value=v, key_pool=kp, value_pool=vp, block_table=table,
                cu_seqlens_q=cu, seqlens_k=kl, cos=ang.cos().float(), sin=ang.sin().float(),
                key_scale=ks, value_scale=vs)


def on_gpu(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def check(x, got, interleaved, T=None):
    """T: packed rows of sequences (the rest must be left alone)."""
    want = ref.append(x["query"], x["new_key"], x["new_value"], x["key_pool"], x["value_pool"],
                      x["block_table"], x["cu_seqlens_q"], x["seqlens_k"], x["cos"], x["sin"],
                      x["key_scale"], x["value_scale"], interleaved)
    dt = x["query"].dtype
    T = x["query"].shape[0] if T is None else T
    # a turned element: two fp32 roundings of terms up to |x| + |y| (cos, sin <= 1),
    # then one rounding to the type (subnormal types: half their last step)
    big = x["query"].double().abs().amax(-1, keepdim=True)
    err = (got["query"].cpu().double() - want[0]).abs()[:T]
    assert (err <= (want[0].abs() * ref.UNIT[dt] * (1 + 2.0 ** -10) + big * 2.0 ** -22
                    + 2.0 ** -25)[:T]).all()
    if x["key_scale"] is None:
        live = want[1] != x["key_pool"].double()
        kbig = x["new_key"].double().abs().max()
        err = (got["key_pool"].cpu().double() - want[1]).abs()
        assert (err <= want[1].abs() * ref.UNIT[dt] * (1 + 2.0 ** -10)
                + kbig * 2.0 ** -22 + 2.0 ** -25)[live].all()
        assert torch.equal(got["key_pool"].cpu().double()[~live], want[1][~live])
        assert torch.equal(got["value_pool"].cpu().double(), want[2])
    else:  # rounded once from the exact value: equal
        for n, w in (("key_pool", want[1]), ("value_pool", want[2])):
            # (the pools' drawn values past the format's range are NaN codes, which stay)
            assert torch.allclose(got[n].cpu().double(), w, rtol=0, atol=0, equal_nan=True), n
        assert torch.equal(got["key_scale"].cpu().double(), want[3])
        assert torch.equal(got["value_scale"].cpu().double(), want[4])


LENS = [
    [(1, 1)],
    [(1, 1000)],
    [(5, 5), (0, 7), (1, 9), (17, 40)],
    [(0, 0), (33, 33), (2, 64), (64, 65)],
    [(130, 150), (3, 3)],
]


@pytest.mark.parametrize("lens", LENS, ids=[str(i) for i in range(len(LENS))])
@pytest.mark.parametrize("pool", ["same", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,Hq,Hk,D,Dv,bs,R,inter", [
    ("bf16", 8, 2, 64, 64, 16, 64, False),
    ("bf16", 4, 4, 128, 64, 32, 64, True),
    ("f16", 6, 1, 192, 128, 8, 192, False),
    ("f32", 4, 2, 40, 48, 24, 20, False),
    ("f16", 3, 3, 10, 7, 5, 6, True),
    ("bf16", 2, 1, 33, 1, 1, 0, False),
    ("f32", 2, 2, 256, 256, 64, 256, True),
])
def test_append(lens, pool, dtype, Hq, Hk, D, Dv, bs, R, inter):
    x = make(3, dtype, dtype if pool == "same" else pool, lens, Hq, Hk, D, Dv, bs, R)
    got = kvc.append_rotary_paged(**on_gpu(x), interleaved=inter)
    check(x, got, inter)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_many_tokens_per_block_and_strides(pool):
    """A prompt long enough for several tokens per thread block, the inputs
    column ranges of one projection, and padded rows behind the last sequence."""
    lens = [(900, 903), (1, 5), (2201, 2300)]
    x = make(5, "bf16", pool, lens, 4, 2, 32, 16, 16, 32, pad=37)
    g = on_gpu(x)
    T = x["query"].shape[0]
    wide = torch.cat([g[n].flatten(1) for n in ("query", "new_key", "new_value")], 1)
    at = [0, 128, 192, 224]
    for i, (n, w) in enumerate((("query", 32), ("new_key", 32), ("new_value", 16))):
        g[n] = wide[:, at[i]:at[i + 1]].view(T, -1, w)
        assert not g[n].is_contiguous()
    out = torch.full((T, 4, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    got = kvc.append_rotary_paged(**g, out_query=out)
    assert got["query"] is out
    check(x, got, False, T - 37)
    assert (out[T - 37:] == 7.0).all()


def test_head_major_inputs():
    """[B, H, S, D] tensors seen as packed rows of equal length."""
    x = make(7, "f16", "f16", [(6, 20)], 4, 2, 64, 64, 8, 64)
    g = on_gpu(x)
    for n in ("query", "new_key", "new_value"):
        g[n] = g[n].transpose(0, 1).contiguous().transpose(0, 1)
    check(x, kvc.append_rotary_paged(**g), False)


@pytest.mark.parametrize("pool", ["e4m3", "e5m2"])
def test_token_by_token_grows_the_scale(pool):
    """Tokens of growing size: the block's held rows are rounded again at each
    growth, as the reference does, and a new block starts from its own rows."""
    x = make(11, "f32", pool, [(1, 1), (1, 1)], 2, 2, 32, 32, 8, 32)
    x["key_scale"].fill_(2.0 ** 40)  # what an earlier owner left: not read
    x["block_table"] = torch.tensor([[1, 2], [3, 0]], dtype=torch.int32)
    ang = torch.arange(20, dtype=torch.float64)[:, None] * torch.rand(16, dtype=torch.float64)
    x["cos"], x["sin"] = ang.cos().float(), ang.sin().float()
    g = on_gpu(x)
    gen = torch.Generator().manual_seed(0)
    for step in range(12):
        x["seqlens_k"] = torch.tensor([step + 1, step + 1], dtype=torch.int32)
        for n in ("query", "new_key", "new_value"):
            x[n] = torch.randn(x[n].shape, generator=gen) * 1.7 ** (step if step < 6 else 12 - step)
        for n in ("query", "new_key", "new_value", "seqlens_k"):
            g[n] = x[n].cuda()
        got = kvc.append_rotary_paged(**g)
        check(x, got, False)
        for n in ("key_pool", "value_pool"):
            x[n] = got[n].cpu()
        for n in ("key_scale", "value_scale"):
            x[n] = got[n].cpu()


@pytest.mark.parametrize("pool", ["e4m3", "e5m2"])
def test_extreme_values(pool):
    """Zeros, the least and largest magnitudes, infinities and NaN."""
    x = make(13, "f32", pool, [(4, 4)], 1, 1, 16, 16, 4, 0)
    x["new_key"].zero_()
    x["new_value"][0] = 1e-38
    x["new_value"][1] = 3e38
    x["new_value"][2] = -3e38
    x["new_value"][3, 0, :8] = 0.0
    got = kvc.append_rotary_paged(**on_gpu(x))
    check(x, got, False)
    x["new_value"] = torch.randn(4, 1, 16)
    x["new_value"][1, 0, 3] = float("inf")
    x["new_value"][2, 0, 5] = float("-inf")
    x["new_value"][3, 0, 7] = float("nan")
    got = kvc.append_rotary_paged(**on_gpu(x))
    blk = int(x["block_table"][0, 0])
    v = got["value_pool"].cpu().float()[blk, 0]
    top = 1.75 * 2.0 ** ref.TOP[DT[pool]][2]
    assert v[1, 3] == top and v[2, 5] == -top and torch.isnan(v[3, 7])
    fin = x["new_value"][torch.isfinite(x["new_value"])].abs().max()
    assert float(got["value_scale"].cpu()[blk, 0]) == ref.least_scale(float(fin), DT[pool])


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_sequences_outside_the_contract_append_nothing(pool):
    """A bad length, a bad block id, too many positions: zero query rows, a
    status bit, pools untouched; the other sequences are served."""
    x = make(17, "bf16", pool, [(3, 10), (2, 6), (4, 4), (1, 12)], 2, 1, 32, 32, 4, 32)
    bad = {n: t if t is None else t.clone() for n, t in x.items()}
    bad["seqlens_k"][0] = 2                  # fewer than its rows
    bad["block_table"][1, 1] = 10 ** 6       # slots 4, 5
    bad["seqlens_k"][3] = 10 ** 6            # past the capacity
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvc.append_rotary_paged(**on_gpu(bad), status=status, max_seqlen_q=4)
    assert int(status) == kvc.DEV_OVERFLOW
    assert (got["query"][:5] == 0).all() and (got["query"][9:] == 0).all()
    keep = x["block_table"][2, 0]
    others = [i for i in range(x["key_pool"].shape[0]) if i != int(keep)]
    for n in ("key_pool", "value_pool"):
        assert torch.allclose(got[n].cpu().double()[others], x[n].double()[others], rtol=0, atol=0,
                              equal_nan=True)
    good = kvc.append_rotary_paged(**on_gpu(x), max_seqlen_q=4)
    assert torch.equal(good["query"][5:9], got["query"][5:9])
    assert torch.equal(good["key_pool"][keep].float(), got["key_pool"][keep].float())
    # more rows than the call said, positions past the tables, cu past the packed rows
    for change in (dict(max_seqlen_q=2), "cos", "cu"):
        z = {n: t if t is None else t.clone() for n, t in x.items()}
        kw = dict(max_seqlen_q=4)
        if change == "cos":
            z["cos"], z["sin"] = z["cos"][:9], z["sin"][:9]
        elif change == "cu":
            z["cu_seqlens_q"][4] = 50
        else:
            kw = change
        status.zero_()
        got = kvc.append_rotary_paged(**on_gpu(z), status=status, **kw)
        assert int(status) == kvc.DEV_OVERFLOW
        if change != "cu":  # sequences 0 and 2 (or 0 and 3) are outside
            assert (got["query"][:3] == 0).all()


def test_empty_and_refused_calls():
    x = on_gpu(make(19, "bf16", "e4m3", [(2, 3)], 2, 1, 32, 32, 4, 32))
    none = {**x, "query": x["query"][:0], "new_key": x["new_key"][:0],
            "new_value": x["new_value"][:0], "cu_seqlens_q": torch.zeros_like(x["cu_seqlens_q"])}
    before = x["key_pool"].float().clone()
    assert kvc.append_rotary_paged(**none)["query"].shape == (0, 2, 32)
    assert torch.equal(before, x["key_pool"].float())
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(**{**x, "key_scale": None})
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(**{**x, "cos": x["cos"].double(), "sin": x["sin"].double()})
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(**{**x, "new_key": x["new_key"].float()})
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(**{**x, "key_pool": x["key_pool"].transpose(1, 2)})
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(**{**x, "query": x["query"].requires_grad_()})
    with pytest.raises(kvc.KvcError):  # the turned queries onto the inputs
        q = x["query"].detach()
        kvc.append_rotary_paged(**{**x, "query": q}, out_query=q)


@pytest.mark.parametrize("pool", ["bf16", "e5m2"])
def test_side_stream_and_captured_graph(pool):
    """On a stream that is not the current device's default, and replayed from
    a captured graph on changed inputs."""
    x = make(23, "bf16", pool, [(1, 9), (1, 17)], 4, 2, 64, 64, 8, 64)
    g = on_gpu(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kvc.append_rotary_paged(**g, max_seqlen_q=1)
    side.synchronize()
    check(x, got, False)
    g = on_gpu(x)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(g["query"])
    with torch.cuda.graph(graph):
        kvc.append_rotary_paged(**g, max_seqlen_q=1, out_query=out)
    y = make(29, "bf16", pool, [(1, 9), (1, 17)], 4, 2, 64, 64, 8, 64)
    for n, t in y.items():
        if t is not None:
            g[n].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    check(y, {**g, "query": out}, False)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_tables_without_positions(pool):
    """cos / sin of no rows: every sequence is outside the contract; with no
    turned elements the tables' length does not matter."""
    x = on_gpu(make(23, "bf16", pool, [(3, 10), (1, 6)], 2, 1, 32, 32, 4, 32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = x["key_pool"].view(torch.uint8).clone()
    z = {**x, "cos": x["cos"][:0], "sin": x["sin"][:0]}
    got = kvc.append_rotary_paged(**z, status=status, max_seqlen_q=3)
    assert int(status) == kvc.DEV_OVERFLOW and (got["query"] == 0).all()
    assert torch.equal(x["key_pool"].view(torch.uint8), keep)
    status.zero_()
    z = {**x, "cos": x["cos"][:0, :0], "sin": x["sin"][:0, :0]}
    got = kvc.append_rotary_paged(**z, status=status, max_seqlen_q=3)
    assert int(status) == 0 and torch.equal(got["query"], x["query"])


def test_wide_integers_are_not_wrapped():
    x = on_gpu(make(24, "bf16", "bf16", [(2, 10), (1, 6)], 2, 1, 32, 32, 4, 32))
    keep = x["key_pool"].clone()
    y = {n: t.long() if n in ("block_table", "cu_seqlens_q", "seqlens_k") else t
         for n, t in x.items()}
    y["block_table"][0, 2] += 2 ** 32
    y["seqlens_k"][1] += 2 ** 33
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvc.append_rotary_paged(**y, status=status, max_seqlen_q=2)
    assert int(status) == kvc.DEV_OVERFLOW and (got["query"] == 0).all()
    assert torch.equal(x["key_pool"], keep)
