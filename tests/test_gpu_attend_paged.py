"""attention_over_paged_cache against the 64-bit reference, within bounds
derived from the taken kernel's arithmetic (paged_reference.attend)."""
import random

import pytest
import torch

import kv_cache_append_gb300 as kvc
import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
      "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def make(seed, dtype, pool, lens, Hq, Hk, D, Dv, bs, pad=0, qstd=2.0, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    T = sum(s for s, _ in lens) + pad
    need = [max(1, -(-k // bs)) for _, k in lens]
    nb = sum(need) + 2
    ids = list(range(nb))
    r.shuffle(ids)
    table = torch.full((len(lens), max(need) + 1), 10 ** 8, dtype=torch.int32)  # unused: never read
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)])
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor([s for s, _ in lens]), 0)
    kl = torch.tensor([k for _, k in lens], dtype=torch.int32)
    dt, pt = DT[dtype], DT[pool]

    def pool_of(w):
        x = torch.randn(nb, Hk, bs, w, generator=g, device="cuda")
        if pool not in ("e4m3", "e5m2"):
            return x.to(dt), None
        sc = 2.0 ** torch.randint(-7, -3, (nb, Hk), generator=g, device="cuda").float()
        if not spread:
            sc.fill_(2.0 ** -5)
        return (x * 32).to(pt), sc

    kp, ks = pool_of(D)
    vp, vs = pool_of(Dv)
    q = (torch.randn(T, Hq, D, generator=g, device="cuda") * qstd).to(dt)
    return dict(q=q, key_pool=kp, value_pool=vp, block_table=table.cuda(),
                cu_seqlens_q=cu.cuda(), seqlens_k=kl.cuda(), key_scale=ks, value_scale=vs)


def path_of(x, max_q):
    nb, Hk, bs, D = x["key_pool"].shape
    T, Hq, _ = x["q"].shape
    return kvc.attend_paged_path(kvc.make_paged_dims(
        x["block_table"].shape[0], T, max_q, Hq, Hk, D, x["value_pool"].shape[3], nb, bs,
        x["block_table"].shape[1], x["q"].dtype, x["key_pool"].dtype))


def check(x, got, max_q, scale=None, softcap=0.0, slopes=None, window=0, rows=None,
          telling=True):
    want, bound = ref.attend(x["q"], x["key_pool"], x["value_pool"], x["block_table"],
                             x["cu_seqlens_q"], x["seqlens_k"], x["key_scale"], x["value_scale"],
                             scale, softcap, slopes, window, path_of(x, max_q))
    live = ~torch.isnan(want)
    if rows is not None:
        live = live & rows[:, None, None]
    err = (got.double() - want).abs()
    worst = (err / bound.clamp(min=1e-300))[live]
    assert (err <= bound)[live].all(), f"{float(worst.max()):.3g} times the bound"
    if telling:
        # the bound takes every rounding at its worst; over a whole result they
        # are independent, and its relative error is about that of one weight (2^-8 at
        # most) and one score (2^-8 of a term, D of them of either sign)
        rel = float(err[live].norm() / want[live].norm())
        assert rel < (1e-5 if x["q"].dtype == torch.float32 else 2e-2), rel
    return float(worst.max())


LENS = {
    "one": [(1, 1)],
    "token": [(1, 700)],
    "decode": [(1, 1), (1, 127), (1, 128), (1, 129), (1, 1000), (0, 55), (1, 3000)],
    "spec": [(4, 4), (3, 131), (1, 1), (4, 640), (2, 129)],
    "chunk": [(40, 140), (33, 33), (1, 300), (24, 500)],
    "prompt": [(300, 300), (1, 77), (257, 900), (128, 129)],
}
SHAPES = [  # dtype, Hq, Hk, D, Dv, bs
    ("bf16", 8, 2, 128, 128, 64),
    ("f16", 16, 1, 192, 128, 16),
    ("bf16", 4, 2, 64, 64, 32),
    ("f16", 5, 5, 80, 48, 8),
    ("bf16", 12, 1, 256, 128, 24),
    ("f32", 6, 3, 40, 56, 24),
    ("f16", 2, 1, 33, 5, 3),
    ("bf16", 3, 1, 96, 200, 128),
]
MODS = {
    "plain": {},
    "cap": dict(softcap=5.0),
    "slopes": dict(slopes=True),
    "window": dict(window=150),
    "all": dict(softcap=20.0, slopes=True, window=37, scale=0.2),
}


@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("pool", ["same", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,Hq,Hk,D,Dv,bs", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
@pytest.mark.parametrize("lens", list(LENS))
def test_attend(lens, dtype, Hq, Hk, D, Dv, bs, pool, mod):
    x = make(1, dtype, dtype if pool == "same" else pool, LENS[lens], Hq, Hk, D, Dv, bs)
    kw = dict(MODS[mod])
    if kw.pop("slopes", False):
        kw["slopes"] = 0.5 ** torch.arange(1, Hq + 1, device="cuda").float()
    call = {("alibi_slopes" if n == "slopes" else n): v for n, v in kw.items()}
    max_q = max(s for s, _ in LENS[lens])
    got = kvc.attention_over_paged_cache(**x, **call, max_seqlen_q=max_q)
    check(x, got, max_q, **kw)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("S", [1, 3, 40])
def test_masked_places_never_enter(pool, S):
    """Infinities and NaN behind each sequence's end, before its window, in
    other blocks, and in the newest slot for the rows that do not see it."""
    x = make(2, "bf16", pool, [(S, 333), (S, 150 + S)], 4, 2, 64, 64, 16)
    kw = dict(window=100)
    max_q = S
    clean = kvc.attention_over_paged_cache(**x, **kw, max_seqlen_q=max_q)
    nanv = 0x7F if pool == "e4m3" else None
    for b, K in enumerate((333, 150 + S)):
        tb = x["block_table"][b].tolist()
        for p in ("key_pool", "value_pool"):
            t = x[p].view(torch.uint8) if nanv else x[p]
            val = nanv if nanv else float("nan")
            for j in list(range(0, K - S + 1 - 100)) + list(range(K, -(-K // 16) * 16)):
                t[tb[j // 16], :, j % 16] = val
            if S > 1:  # only the last row sees slot K - 1
                t[tb[(K - 1) // 16], :, (K - 1) % 16] = val
    got = kvc.attention_over_paged_cache(**x, **kw, max_seqlen_q=max_q)
    for b in range(2):
        n = S if S == 1 else S - 1
        assert torch.equal(got[b * S:b * S + n], clean[b * S:b * S + n])
        if S > 1:
            assert torch.isnan(got[b * S + S - 1]).all()


@pytest.mark.parametrize("pool", ["bf16", "e5m2"])
def test_infinite_value_in_one_column(pool):
    """One infinite value, seen by some rows only: it enters its own column of
    the rows that see it."""
    x = make(3, "bf16", pool, [(5, 70)], 2, 1, 64, 64, 16)
    clean = kvc.attention_over_paged_cache(**x, max_seqlen_q=5)
    blk = int(x["block_table"][0, 68 // 16])
    if pool == "bf16":
        x["value_pool"][blk, 0, 68 % 16, 9] = float("inf")
    else:
        x["value_pool"].view(torch.uint8)[blk, 0, 68 % 16, 9] = 0x7C
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=5)
    assert torch.equal(got[:3], clean[:3])  # rows at positions 65, 66, 67
    assert torch.isinf(got[3:, :, 9]).all()
    other = [i for i in range(64) if i != 9]
    check(x, got, 5, rows=torch.tensor([True] * 3 + [False] * 2, device="cuda"))
    assert torch.isfinite(got[3:][:, :, other]).all()
    err = (got[3:][:, :, other].double() - clean[3:][:, :, other].double()).abs()
    assert (err <= clean[3:].abs().double().amax() * 2.0 ** -6).all()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_one_slot_far_above_a_flat_rest(pool):
    """A slot that takes most of a row's weight, the rest spread over thousands of
    slots that together still matter: none of it may be rounded away."""
    K = 30000
    x = make(4, "bf16", pool, [(1, K)], 4, 1, 64, 64, 64, qstd=0.01, spread=False)
    x["q"][..., 0] = 1.0
    kp = x["key_pool"].view(torch.uint8).view(x["key_pool"].dtype)
    first = int(x["block_table"][0, 5])
    code = torch.tensor(83.0 if pool == "bf16" else 83.0 * 32).to(x["key_pool"].dtype)
    if pool == "e4m3":  # the largest code under a scale of its block
        x["key_scale"][first] = 2.0 ** -2
        kp[first] = (kp[first].float() / 8).to(kp.dtype)
        code = torch.tensor(332.0).to(kp.dtype)
    kp[first, 0, 3, 0] = code.to(kp.device)
    vf = x["value_pool"].float() + (1.0 if pool == "bf16" else 32.0)  # values with a mean
    x["value_pool"] = vf.to(x["value_pool"].dtype)
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=1)
    check(x, got, 1)


def test_values_of_very_different_scales():
    """Blocks whose value scales differ by 2^40: the weights' products keep their
    precision where the result lies."""
    for lo, hi in ((-60, -20), (20, 60)):
        x = make(5, "bf16", "e4m3", [(1, 600), (3, 900)], 4, 2, 64, 64, 32)
        sc = torch.randint(lo, hi, x["value_scale"].shape, device="cuda").float()
        x["value_scale"] = torch.exp2(sc)
        got = kvc.attention_over_paged_cache(**x, max_seqlen_q=3)
        want, bound = ref.attend(x["q"], x["key_pool"], x["value_pool"], x["block_table"],
                                 x["cu_seqlens_q"], x["seqlens_k"], x["key_scale"],
                                 x["value_scale"], path=path_of(x, 3))
        # relative to the row's largest result: terms below 2^-24 of it may go
        big = want.abs().amax(-1, keepdim=True)
        assert ((got.double() - want).abs() <= bound + big * 2.0 ** -6).all()


def test_scores_past_every_range():
    """Scores of thousands, and rows that meet ever larger ones: finite, exact
    weights on the largest."""
    x = make(6, "bf16", "bf16", [(2, 500)], 2, 1, 64, 64, 16, qstd=400.0)
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=2, scale=4.0)
    # scores up to 1e5: their fp32 rounding alone may move a weight by its own size
    check(x, got, 2, scale=4.0, telling=False)
    ramp = make(7, "f16", "f16", [(1, 2000)], 2, 1, 64, 64, 16)
    tb = ramp["block_table"][0].tolist()
    ramp["q"].fill_(1.0)
    for j in range(2000):
        ramp["key_pool"][tb[j // 16], 0, j % 16] = j / 64.0
    got = kvc.attention_over_paged_cache(**ramp, max_seqlen_q=1)
    check(ramp, got, 1)


@pytest.mark.parametrize("S", [1, 70])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_outside_the_contract_and_padding(pool, S):
    lens = [(S, 200 + S), (S, 90 + S), (S, 300 + S), (S, 130 + S)]
    x = make(8, "bf16", pool, lens, 4, 2, 64, 64, 16, pad=5)
    clean = kvc.attention_over_paged_cache(**x, max_seqlen_q=S)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = {n: t if t is None else t.clone() for n, t in x.items()}
    bad["seqlens_k"][0] = S - 1
    bad["block_table"][1, 2] = -1
    bad["seqlens_k"][3] = 10 ** 7
    out = torch.full_like(clean, 3.0)
    got = kvc.attention_over_paged_cache(**bad, max_seqlen_q=S, out=out, status=status)
    assert got is out and int(status) == kvc.DEV_OVERFLOW
    assert (out[:2 * S] == 0).all() and (out[3 * S:4 * S] == 0).all()
    assert torch.equal(out[2 * S:3 * S], clean[2 * S:3 * S])
    assert (out[4 * S:] == 3.0).all()
    status.zero_()
    out.fill_(3.0)  # a bad id that a window hides is not read
    far = {n: t if t is None else t.clone() for n, t in x.items()}
    far["block_table"][:, 0] = 10 ** 8
    kvc.attention_over_paged_cache(**far, max_seqlen_q=S, window=64, out=out, status=status)
    want = kvc.attention_over_paged_cache(**x, max_seqlen_q=S, window=64)
    assert int(status) == 0 and torch.equal(out[:4 * S], want[:4 * S])
    if S > 1:
        status.zero_()
        got = kvc.attention_over_paged_cache(**x, max_seqlen_q=S - 1, status=status)
        assert int(status) == kvc.DEV_OVERFLOW and (got[:4 * S] == 0).all()


@pytest.mark.parametrize("pool", ["f16", "e4m3"])
def test_strided_queries_streams_graphs_and_shared_workspace(pool):
    """Head-strided queries, a side stream, and two graphs that share a
    workspace, replayed in turn on changed inputs."""
    lens = [(1, 500), (1, 4000), (1, 77)]
    x = make(9, "f16", pool, lens, 8, 2, 64, 64, 16)
    want = kvc.attention_over_paged_cache(**x, max_seqlen_q=1)
    wide = torch.zeros(3, 8, 96, dtype=torch.float16, device="cuda")
    wide[..., 16:80] = x["q"]
    y = {**x, "q": wide[..., 16:80]}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kvc.attention_over_paged_cache(**y, max_seqlen_q=1)
    side.synchronize()
    assert torch.equal(got, want)
    nb, Hk, bs, D = x["key_pool"].shape
    need = kvc.attend_paged_workspace_bytes(kvc.make_paged_dims(
        3, 3, 1, 8, Hk, D, 64, nb, bs, x["block_table"].shape[1], torch.float16,
        x["key_pool"].dtype))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    z = make(10, "f16", pool, [(1, 900), (1, 1), (1, 2500)], 8, 2, 64, 64, 16)
    graphs, outs = [], []
    for t in (x, z):
        out = torch.empty_like(t["q"])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            kvc.attention_over_paged_cache(**t, max_seqlen_q=1, out=out, workspace=ws)
        graphs.append(gr)
        outs.append(out)
    wz = kvc.attention_over_paged_cache(**z, max_seqlen_q=1)
    for _ in range(3):
        ws.fill_(0xFF)
        for o in outs:
            o.zero_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], wz)
    with pytest.raises(kvc.KvcError):
        kvc.attention_over_paged_cache(**x, max_seqlen_q=1, workspace=ws[:need - 256])


@pytest.mark.parametrize("dtype,pool,D", [("bf16", "e4m3", 128), ("f16", "f16", 64),
                                          ("bf16", "bf16", 128), ("f16", "e5m2", 192)])
def test_many_tiles_and_units_a_block(dtype, pool, D):
    """Long runs: every ring, buffer and reference of a thread block is used many
    times over, and units end inside a block's run; the timeout bit stays clear."""
    lens = [(700, 5000), (1001, 1001), (330, 9000), (1, 4000)]
    x = make(21, dtype, pool, lens, 16, 4, D, 128, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=1001, status=status)
    assert int(status) == 0
    check(x, got, 1001)
    many = make(22, dtype, pool, [(1, 100 + 37 * i) for i in range(150)], 8, 8, D, 128, 64)
    got = kvc.attention_over_paged_cache(**many, max_seqlen_q=1, status=status)
    assert int(status) == 0
    check(many, got, 1)


def test_the_same_call_gives_the_same_bits():
    x = make(12, "bf16", "e4m3", [(1, 5000), (3, 700), (1, 12000)], 8, 2, 128, 128, 64)
    first = kvc.attention_over_paged_cache(**x, max_seqlen_q=3)
    for _ in range(5):
        assert torch.equal(kvc.attention_over_paged_cache(**x, max_seqlen_q=3), first)


def test_shared_blocks_and_long_offsets():
    """Sequences that share a prefix's blocks; and a pool past 2^32 bytes."""
    x = make(13, "bf16", "e4m3", [(1, 640), (1, 700)], 4, 2, 64, 64, 64)
    x["block_table"][1, :6] = x["block_table"][0, :6]
    check(x, kvc.attention_over_paged_cache(**x, max_seqlen_q=1), 1)
    nb, bs, w = 70000, 256, 256
    kp = torch.zeros(nb, 1, bs, w, dtype=torch.float8_e4m3fn, device="cuda")
    vp = torch.zeros(nb, 1, bs, 128, dtype=torch.float8_e4m3fn, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = [nb - 1, 3, nb - 2, 40000]
    for i in ids:
        kp[i] = torch.randn(1, bs, w, generator=g, device="cuda").to(kp.dtype)
        vp[i] = torch.randn(1, bs, 128, generator=g, device="cuda").to(vp.dtype)
    y = dict(q=torch.randn(1, 4, w, generator=g, device="cuda").bfloat16(), key_pool=kp,
             value_pool=vp, block_table=torch.tensor([ids], dtype=torch.int32, device="cuda"),
             cu_seqlens_q=torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
             seqlens_k=torch.tensor([1000], dtype=torch.int32, device="cuda"),
             key_scale=torch.full((nb, 1), 0.5, device="cuda"),
             value_scale=torch.full((nb, 1), 2.0, device="cuda"))
    check(y, kvc.attention_over_paged_cache(**y, max_seqlen_q=1), 1)


@pytest.mark.parametrize("pool", ["same", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_then_attend(dtype, pool):
    """The two as a serving loop uses them: a prompt, then tokens, each call's
    queries turned by the append and attended over the pool it wrote."""
    Hq, Hk, D, bs = 8, 2, 64, 16
    pt = DT[dtype if pool == "same" else pool]
    g = torch.Generator(device="cuda").manual_seed(5)
    nb = 24
    kp = torch.zeros(nb, Hk, bs, D, device="cuda").to(pt)
    vp = torch.zeros(nb, Hk, bs, D, device="cuda").to(pt)
    ks = vs = None
    if pool != "same":
        ks, vs = torch.ones(nb, Hk, device="cuda"), torch.ones(nb, Hk, device="cuda")
    table = torch.randperm(nb, generator=g, device="cuda")[:20].view(2, 10).int()
    ang = torch.arange(160, device="cuda").double()[:, None] * \
        10000.0 ** (-torch.arange(D // 2, device="cuda").double() * 2 / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    done = [0, 0]
    for new in ([70, 33], [1, 1], [1, 1], [4, 2], [0, 1], [1, 1]):
        T = sum(new)
        cu = torch.tensor([0, new[0], T], dtype=torch.int32, device="cuda")
        done = [a + b for a, b in zip(done, new)]
        kl = torch.tensor(done, dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(DT[dtype])
                   for h in (Hq, Hk, Hk))
        before = [t if t is None else t.cpu().clone() for t in (kp, vp, ks, vs)]
        got = kvc.append_rotary_paged(q, k, v, kp, vp, table, cu, kl, cos, sin, key_scale=ks,
                                      value_scale=vs, max_seqlen_q=max(new))
        want = ref.append(q.cpu(), k.cpu(), v.cpu(), before[0], before[1], table.cpu(), cu.cpu(),
                          kl.cpu(), cos.cpu(), sin.cpu(), before[2], before[3])
        if pool != "same":
            assert torch.equal(kp.cpu().double(), want[1]) and torch.equal(ks.cpu().double(), want[3])
        x = dict(q=got["query"], key_pool=kp, value_pool=vp, block_table=table, cu_seqlens_q=cu,
                 seqlens_k=kl, key_scale=ks, value_scale=vs)
        out = kvc.attention_over_paged_cache(**x, max_seqlen_q=max(new))
        check(x, out, max(new))


@pytest.mark.parametrize("S", [1, 40])
@pytest.mark.parametrize("dtype,pool", [("bf16", "e4m3"), ("f16", "f16")])
def test_unaligned_pools_queries_and_outputs(dtype, pool, S):
    """Tensors that start off a 16-byte boundary: the CUDA-core kernel, or (the
    output of few rows) the same one, within the same bounds."""
    x = make(31, dtype, pool, [(S, 300 + S), (S, S)], 4, 2, 64, 64, 16)

    def shifted(t, by):
        flat = torch.empty(t.numel() + by, dtype=torch.uint8 if t.element_size() == 1 else t.dtype,
                           device="cuda")
        flat[by:] = t.reshape(-1).view(flat.dtype)
        return flat[by:].view(t.dtype).view(t.shape)

    want, bound = ref.attend(x["q"], x["key_pool"], x["value_pool"], x["block_table"],
                             x["cu_seqlens_q"], x["seqlens_k"], x["key_scale"], x["value_scale"],
                             None, 0.0, None, 0, path_of(x, S))
    for name in ("key_pool", "value_pool", "q", "out"):
        y = dict(x)
        out = None
        if name == "out":
            out = shifted(torch.zeros_like(x["q"]), 1)
        else:
            y[name] = shifted(x[name], 1)
        got = kvc.attention_over_paged_cache(**y, max_seqlen_q=S, out=out)
        assert ((got.double() - want).abs() <= bound).all(), name


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("S", [1, 24])
def test_more_rows_announced_than_there_are(pool, S):
    """max_seqlen_q may be any bound on the rows: past the packed rows it changes nothing."""
    x = make(32, "bf16", pool, [(S, 500)], 4, 2, 64, 64, 16)
    want = kvc.attention_over_paged_cache(**x, max_seqlen_q=S)
    assert torch.equal(kvc.attention_over_paged_cache(**x, max_seqlen_q=10 ** 6), want)


def test_wide_integers_are_not_wrapped():
    x = make(33, "bf16", "bf16", [(1, 40), (1, 50)], 4, 2, 64, 64, 16)
    want = kvc.attention_over_paged_cache(**x, max_seqlen_q=1)
    y = {n: t.long() if n in ("block_table", "cu_seqlens_q", "seqlens_k") else t
         for n, t in x.items()}
    assert torch.equal(kvc.attention_over_paged_cache(**y, max_seqlen_q=1), want)
    y["block_table"][0, 1] += 2 ** 32
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvc.attention_over_paged_cache(**y, max_seqlen_q=1, status=status)
    assert int(status) == kvc.DEV_OVERFLOW
    assert (got[0] == 0).all() and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        kvc.attention_over_paged_cache(**{**x, "seqlens_k": x["seqlens_k"].bool()}, max_seqlen_q=1)


@pytest.mark.parametrize("pool", ["f16", "e5m2"])
def test_two_calls_at_once(pool):
    """Two streams, a workspace each, in turn over many rounds; and captured with
    their own workspaces into one graph's two branches."""
    x = make(34, "f16", pool, [(1, 3000), (1, 900), (1, 50)], 8, 2, 64, 64, 16)
    z = make(35, "f16", pool, [(60, 700), (33, 33)], 8, 2, 64, 64, 16)
    wx = kvc.attention_over_paged_cache(**x, max_seqlen_q=1)
    wz = kvc.attention_over_paged_cache(**z, max_seqlen_q=60)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(side[0]):
            got[0].append(kvc.attention_over_paged_cache(**x, max_seqlen_q=1))
        with torch.cuda.stream(side[1]):
            got[1].append(kvc.attention_over_paged_cache(**z, max_seqlen_q=60))
    torch.cuda.synchronize()
    assert all(torch.equal(o, wx) for o in got[0]) and all(torch.equal(o, wz) for o in got[1])
    ox, oz = torch.zeros_like(wx), torch.zeros_like(wz)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side[0].wait_stream(main)
        with torch.cuda.stream(side[0]):
            kvc.attention_over_paged_cache(**x, max_seqlen_q=1, out=ox)
        kvc.attention_over_paged_cache(**z, max_seqlen_q=60, out=oz)
        main.wait_stream(side[0])
    for _ in range(3):
        ox.zero_()
        oz.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ox, wx) and torch.equal(oz, wz)


@pytest.mark.parametrize("dtype,pool,D", [("bf16", "e4m3", 128), ("f16", "f16", 64),
                                          ("f16", "e5m2", 192)])
def test_many_short_units_a_block(dtype, pool, D):
    """Units of one to three tiles, several in each thread block: its groups work
    on up to three units at once; the same bits every time, the timeout bit clear."""
    r = random.Random(41)
    lens = [(s, s + r.randint(0, 260)) for s in (r.randint(9, 70) for _ in range(90))]
    x = make(41, dtype, pool, lens, 16, 4, D, 64, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=70, status=status)
    assert int(status) == 0
    check(x, got, 70)
    for _ in range(10):
        assert torch.equal(kvc.attention_over_paged_cache(**x, max_seqlen_q=70, status=status), got)
    assert int(status) == 0
    got = kvc.attention_over_paged_cache(**x, max_seqlen_q=70, window=100, softcap=8.0,
                                         status=status)
    assert int(status) == 0
    check(x, got, 70, window=100, softcap=8.0)
