"""64-bit reference of the packed, paged operators, one sequence and one slot
range at a time, and the error bounds their kernels are held to."""
import math

import torch

TOP = {torch.float8_e4m3fn: (3, -6, 8), torch.float8_e5m2: (2, -14, 15)}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def round8(x, dtype):
    """float64 -> the 8-bit format's values, one rounding, ties to even, saturating."""
    bits, low, top = TOP[dtype]
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=low) - bits)
    return (torch.round(x / step) * step).clamp(-1.75 * 2.0 ** top, 1.75 * 2.0 ** top)


def least_scale(amax, dtype):
    """2^e, e the least in [-100, 100] with amax <= 1.75 * 2^top * 2^e."""
    top = TOP[dtype][2]
    e = -100
    while e < 100 and amax > 1.75 * 2.0 ** (top + e):
        e += 1
    return 2.0 ** e


def rotate(x, cos, sin, interleaved):
    """x [..., D] float64, cos/sin [R/2] float64."""
    y = x.clone()
    h = cos.shape[-1]
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y[..., a] = x[..., a] * cos[i] - x[..., b] * sin[i]
        y[..., b] = x[..., b] * cos[i] + x[..., a] * sin[i]
    return y


def append(query, new_key, new_value, key_pool, value_pool, table, cu, kl, cos, sin,
           key_scale=None, value_scale=None, interleaved=False):
    """All on the CPU; returns float64 (query, key_pool, value_pool, key_scale,
    value_scale); 8-bit pools as their codes' values."""
    q = query.double().clone()
    bs = key_pool.shape[2]
    pools = {"k": key_pool.double().clone(), "v": value_pool.double().clone()}
    scales = {"k": None if key_scale is None else key_scale.double().clone(),
              "v": None if value_scale is None else value_scale.double().clone()}
    for b in range(table.shape[0]):
        s0, s1, K = int(cu[b]), int(cu[b + 1]), int(kl[b])
        start = K - (s1 - s0)
        new = {"k": [], "v": []}
        for t in range(s0, s1):
            j = start + t - s0
            q[t] = rotate(query[t].double(), cos[j].double(), sin[j].double(), interleaved)
            new["k"].append(rotate(new_key[t].double(), cos[j].double(), sin[j].double(),
                                   interleaved))
            new["v"].append(new_value[t].double())
        for w in "kv":
            pool, sc = pools[w], scales[w]
            j = start
            while j < K:
                blk, r0 = int(table[b, j // bs]), j % bs
                n = min(K - j, bs - r0)
                x = torch.stack(new[w][j - start:j - start + n])  # [n, Hk, width]
                for h in range(pool.shape[1]):
                    if sc is None:
                        pool[blk, h, r0:r0 + n] = x[:, h]
                        continue
                    fin = x[:, h][torch.isfinite(x[:, h])]
                    want = least_scale(float(fin.abs().max()) if fin.numel() else 0.0,
                                       key_pool.dtype)
                    if r0 and float(sc[blk, h]) > want:
                        want = float(sc[blk, h])
                    if r0:
                        pool[blk, h, :r0] = round8(pool[blk, h, :r0] * (float(sc[blk, h]) / want),
                                                   key_pool.dtype)
                    pool[blk, h, r0:r0 + n] = round8(x[:, h] / want, key_pool.dtype)
                    sc[blk, h] = want
                j += n
    return q, pools["k"], pools["v"], scales["k"], scales["v"]


def dense(pool, scale, table, b, K):
    """Slots [0, K) of sequence b as float64 [K, Hk, width]."""
    bs = pool.shape[2]
    ids = table[b, :(K + bs - 1) // bs].long()
    x = pool.view(torch.uint8)[ids].view(pool.dtype).double() if scale is not None \
        else pool[ids].double()
    if scale is not None:
        x = x * scale[ids].double()[:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(-1, pool.shape[1], pool.shape[3])[:K]


# Per kernel and pool kind: how far a query element (of the row's largest) and a
# weight (of itself) are off as the products see them, beyond fp32 arithmetic.
#   cores: fp32 throughout.
#   tensor cores, 8-bit pools: the row is scaled so that its largest element lies
#   in [2^7, 2^8), and an element is the sum of two e4m3 values (fp16: three), which hold
#   its bits down to e4m3's last step, 2^-9: off by 2^-10, 2^-17 of the largest. A
#   weight's fp16 rounding (2^-12) is the sum of three e5m2 values, two cut to 3 bits
#   and one rounded: 2^-9 more, or 2^-25 of the largest weight.
#   tensor cores, pools of the inputs' type: the query exact, a weight rounded to the type.
def operand_errors(path, q_dtype, eight):
    if path == "cores":
        return 0.0, 0.0
    if eight:
        return 2.0 ** -17, 2.0 ** -9 + 2.0 ** -11
    return 0.0, UNIT[q_dtype]


def attend(q, key_pool, value_pool, table, cu, kl, key_scale=None, value_scale=None, scale=None,
           softcap=0.0, slopes=None, window=0, path="cores"):
    """(out, bound) float64: the reference rows and how far a kernel of that
    path may be from each element. Rows of no sequence: NaN, bound 0."""
    T, Hq, D = q.shape
    Hk, Dv = value_pool.shape[1], value_pool.shape[3]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dev = q.device
    out = torch.full((T, Hq, Dv), float("nan"), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    eq, ew = operand_errors(path, q.dtype, key_scale is not None)
    u = 2.0 ** -24
    for b in range(table.shape[0]):
        s0, s1, K = int(cu[b]), int(cu[b + 1]), int(kl[b])
        if s1 == s0:
            continue
        k = dense(key_pool, key_scale, table, b, K)
        v = dense(value_pool, value_scale, table, b, K)
        pos = torch.arange(K - (s1 - s0), K, device=dev)[:, None]
        j = torch.arange(K, device=dev)[None]
        hide = j > pos
        if window:
            hide = hide | (j <= pos - window)
        for h in range(Hq):
            x, kh, vh = q[s0:s1, h].double(), k[:, h * Hk // Hq], v[:, h * Hk // Hq]
            kh = torch.where(torch.isfinite(kh), kh, torch.zeros_like(kh)) if bool(hide.any()) else kh
            s = scale * (x @ kh.t())
            # a score's error: the query's rounding, fp32 products and sums (D + 8
            # roundings of terms), and 2^-20 of its size for the cap, bias and base change
            err = scale * ((x.abs() @ kh.abs().t()) * ((D + 8) * u)
                           + eq * x.abs().amax(1, keepdim=True) * kh.abs().sum(1)[None])
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                err = err + softcap * 2.0 ** -21
            if slopes is not None:
                s = s - slopes[h].double() * (pos - j)
            err = (err + s.abs() * 2.0 ** -20).masked_fill(hide, 0.0).amax(1, keepdim=True)
            a = torch.softmax(s.masked_fill(hide, -math.inf), -1)
            vz = torch.where(torch.isfinite(vh), vh, torch.zeros_like(vh))
            o = a @ vz
            mass = a @ vz.abs()
            # a weight: exp of two scores' errors, its own rounding, exp2's and the
            # scale's (2^-18, with the sums over K slots in fp32, tiles at a time), and what
            # underflows: 2^-24 of the largest weight for each slot
            rel = torch.expm1(2 * err) + ew + 2.0 ** -18 + 8 * math.sqrt(K) * u
            lost = (a.amax(1, keepdim=True) * 2.0 ** -23) * \
                vz.abs().masked_fill(~torch.isfinite(vh), 0).sum(0)[None]
            out[s0:s1, h] = o
            bound[s0:s1, h] = mass * rel + lost + o.abs() * UNIT[q.dtype] + 2.0 ** -25
    return out, bound
