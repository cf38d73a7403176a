"""The packed, paged operators' C ABI on the CPU: sizes and arguments are
refused before anything is launched."""
import ctypes

import pytest
import torch

import kv_cache_append_gb300 as kvc
from kv_cache_append_gb300 import build as kbuild
from kv_cache_append_gb300 import paged

GOOD = dict(B=2, total_q=6, max_q=4, Hq=4, Hk=2, D=64, Dv=64, num_blocks=9, block_size=16,
            max_blocks=4, dtype=1, pool_dtype=1)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return paged._paged_library()


def dims(**kw):
    return kvc.make_paged_dims(**{**GOOD, **kw})


def ptr(i):
    return ctypes.c_void_p((i + 1) << 32)


def attend(lib, d, null=(), scale=0.125, softcap=0.0, window=0, ws=1 << 31, alias=None, st=(256, 64)):
    names = ["q", "kp", "vp", "ks", "vs", "table", "cu", "kl", "slopes", "out", "work"]
    p = {n: ptr(i) for i, n in enumerate(names)}
    if d is not None and d.pool_dtype < 3:
        p["ks"] = p["vs"] = None
    for n in null:
        p[n] = None
    if alias:
        p[alias[0]] = p[alias[1]]
    stp = (ctypes.c_int64 * 2)(*st)
    return lib.kvc_attend_paged(None if d is None else ctypes.byref(d), stp, p["q"], p["kp"],
                                p["vp"], p["ks"], p["vs"], p["table"], p["cu"], p["kl"], scale,
                                softcap, p["slopes"], window, p["out"], p["work"], ws, None, None)


def append(lib, d, null=(), R=64, P=100, inter=0, alias=None, st=(256, 64, 128, 64, 128, 64)):
    names = ["q", "k", "v", "table", "cu", "kl", "cos", "sin", "kp", "vp", "ks", "vs", "out"]
    p = {n: ptr(i) for i, n in enumerate(names)}
    if d is not None and d.pool_dtype < 3:
        p["ks"] = p["vs"] = None
    for n in null:
        p[n] = None
    if alias:
        p[alias[0]] = p[alias[1]]
    stp = (ctypes.c_int64 * 6)(*st)
    return lib.kvc_append_rotary_paged(None if d is None else ctypes.byref(d), R, P, inter, stp,
                                       *(p[n] for n in names), None, None)


BAD_DIMS = [
    (dict(B=0), -2), (dict(Hq=3), -2), (dict(D=0), -2), (dict(D=257), -2), (dict(Dv=300), -2),
    (dict(total_q=-1), -2), (dict(max_q=0), -2), (dict(num_blocks=0), -2),
    (dict(block_size=0), -2), (dict(max_blocks=0), -2), (dict(dtype=3), -3), (dict(dtype=9), -3),
    (dict(pool_dtype=2), -3), (dict(pool_dtype=5), -3), (dict(total_q=1 << 40), -2),
    (dict(max_blocks=1 << 28, block_size=16), -2), (dict(num_blocks=1 << 31), -2),
]


@pytest.mark.parametrize("change,code", BAD_DIMS, ids=[str(c) for c, _ in BAD_DIMS])
def test_bad_sizes(lib, change, code):
    d = dims(**change)
    assert attend(lib, d) == code
    assert append(lib, d) == code
    assert kvc.attend_paged_workspace_bytes(d) == 0
    with pytest.raises(ValueError):
        kvc.attend_paged_path(d)


@pytest.mark.parametrize("pool", [1, 3, 4])
def test_null_pointers(lib, pool):
    d = dims(pool_dtype=pool)
    assert attend(lib, None) == -1 and append(lib, None) == -1
    for n in ("q", "kp", "vp", "table", "cu", "kl", "out"):
        assert attend(lib, d, null=(n,)) == -1, n
        assert append(lib, d, null=(n,)) == -1, n
    for n in ("k", "v", "cos", "sin"):
        assert append(lib, d, null=(n,)) == -1, n
    if pool >= 3:
        for n in ("ks", "vs"):
            assert attend(lib, d, null=(n,)) == -1 and append(lib, d, null=(n,)) == -1
    assert attend(lib, d, null=("work",)) == -5


def test_scalars_strides_and_workspace(lib):
    d = dims()
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e300):
        assert attend(lib, d, scale=bad) == -4
    for bad in (-1.0, float("nan"), float("inf")):
        assert attend(lib, d, softcap=bad) == -4
    assert attend(lib, d, window=-1) == -2
    assert attend(lib, d, st=(-1, 64)) == -2
    assert attend(lib, d, ws=kvc.attend_paged_workspace_bytes(d) - 1) == -5
    assert append(lib, d, R=3) == -2 and append(lib, d, R=66) == -2 and append(lib, d, R=-2) == -2
    assert append(lib, d, inter=2) == -2 and append(lib, d, P=-1) == -2
    assert append(lib, d, st=(256, 64, 128, 64, 128, -64)) == -2


def test_overlaps(lib):
    d = dims(pool_dtype=3)
    for n in ("q", "kp", "vp", "ks", "vs", "table", "cu", "kl", "slopes", "work"):
        assert attend(lib, d, alias=("out", n)) == -6, n
    assert attend(lib, d, alias=("work", "kp")) == -6
    for n in ("q", "k", "v", "table", "cu", "kl", "cos", "sin", "kp", "vp", "ks", "vs"):
        assert append(lib, d, alias=("out", n)) == -6, n
    assert append(lib, d, alias=("vp", "kp")) == -6 and append(lib, d, alias=("ks", "vs")) == -6


def test_no_gpu_is_an_error_and_cpu_tensors_are_refused(lib):
    if not torch.cuda.is_available():
        assert attend(lib, dims()) in (-7, -8) and append(lib, dims()) in (-7, -8)
    q = torch.zeros(1, 2, 16)
    pool = torch.zeros(2, 1, 4, 16)
    t = torch.zeros(1, 1, dtype=torch.int32)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    kl = torch.tensor([1], dtype=torch.int32)
    with pytest.raises(ValueError):
        kvc.attention_over_paged_cache(q, pool, pool.clone(), t, cu, kl)
    with pytest.raises(ValueError):
        kvc.append_rotary_paged(q, q[:, :1], q[:, :1], pool, pool.clone(), t, cu, kl,
                                torch.zeros(4, 8), torch.zeros(4, 8))


def test_workspace_holds_for_every_size(lib):
    """Non-zero, whole 256-byte units, and no less for more rows."""
    last = 0
    for T in (0, 1, 7, 64, 4000):
        n = kvc.attend_paged_workspace_bytes(dims(total_q=T, max_q=max(T, 1)))
        assert n >= 256 and n % 256 == 0
        last = max(last, n)
    assert kvc.attend_paged_path(dims())


def test_scales_outside_fp32_and_blocks_past_31_bits(lib):
    d = dims()
    for bad in (1e-39, 1e-300, 3e38):
        assert attend(lib, d, scale=bad) == -4
        assert attend(lib, d, softcap=bad) == -4
    assert attend(lib, d, scale=1e10, softcap=1e-30) == -4
    e = dims(pool_dtype=3, block_size=1 << 25, max_blocks=1)
    assert append(lib, e) == -2


def test_rows_past_the_packed_ones_do_not_change_the_plan():
    for q in (4, 16):
        a, b = dims(B=1, total_q=q, max_q=q), dims(B=1, total_q=q, max_q=10 ** 6)
        assert kvc.attend_paged_path(a) == kvc.attend_paged_path(b)
        assert kvc.attend_paged_workspace_bytes(a) == kvc.attend_paged_workspace_bytes(b)
