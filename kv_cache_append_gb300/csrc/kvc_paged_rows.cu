// kvc_paged_rows.cu -- attention over a paged pool on the tensor cores, for
// units of many query rows: prompts, chunks, and steps of many heads per KV head.
//
// Query rows are the M dimension (128 rows r = t G + g of a KV head, a thread
// each), 128 slots a tile:
//
//   S  = Q K^T    (A = query rows, B = K tile, both from shared memory)
//   O += P V      (A = P from tensor memory, B = V tile read N-major)
//
// With 8-bit pools both products take the tiles as they lie in memory, the
// query rows as two e4m3 parts and the weights as three e5m2 parts (splits, scales
// and references as in kvc_paged_decode.cu): five products at twice the 16-bit
// rate against four halves, so the tensor-core time is 5/4 of 16-bit tiles', with
// half the memory traffic and no conversion of the cache.
//
// The softmax, not the products, is the longer part of a tile: two groups of 4
// warps take alternate tiles, each with its own S, O and row statistics, so
// that one group's softmax runs under the other's products; at a run's end the two
// halves of a row are joined out of tensor memory. P overwrites its S in place:
// the weights of 32 slots take 24 columns (16 of 16-bit weights), behind the 32
// score columns that are read next.
//
// Tensor memory: S at columns 0 and 128, O at 256 and 384. Warps: 8 softmax, an S
// issuer, a P.V issuer, a producer, and 4 that schedule the block's runs
// (kvc_paged_tc.cuh) and prepare the next run's query rows.
#include <algorithm>
#include <type_traits>

#include "kvc_paged_tc.cuh"

namespace kvc {
namespace {

constexpr int kTS = 128, kRows = 128;
constexpr int kSWarp = 8, kPvWarp = 9, kProdWarp = 10, kQWarp = 12;  // 12..15: query rows
constexpr int kThreads = 16 * 32;
constexpr uint32_t kColS = 0, kColO = 256;

struct Bars {
    uint32_t base;
    __device__ uint32_t k_full(int s) const { return base + 8u * s; }
    __device__ uint32_t k_empty(int s) const { return base + 64u + 8u * s; }
    __device__ uint32_t v_full(int s) const { return base + 128u + 8u * s; }
    __device__ uint32_t v_empty(int s) const { return base + 192u + 8u * s; }
    __device__ uint32_t item_full(int k) const { return base + 256u + 8u * k; }
    __device__ uint32_t item_empty(int k) const { return base + 272u + 8u * k; }
    __device__ uint32_t s_ready(int g) const { return base + 288u + 8u * g; }
    __device__ uint32_t p_ready(int g) const { return base + 304u + 8u * g; }
    __device__ uint32_t o_done(int g) const { return base + 320u + 8u * g; }
    __device__ uint32_t meet() const { return base + 336u; }
    __device__ uint32_t o_free() const { return base + 344u; }
    __device__ uint32_t drained() const { return base + 352u; }
};
constexpr int kTmemSlot = 360, kAbort = 364, kBad = 368 /* [2] */, kOdd = 376 /* [2] */;
constexpr int kStart = 512, kItems = 896, kXml = 1024;  // 2 KB of exchanged row statistics
constexpr int kScales = 3072, kScaleRing = 16;          // 8-bit pools: 16 tiles' scales

__device__ __forceinline__ void tc_mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 4 warps: lane 0 of the first walks the runs; all split the rows of the run.
template <typename T, int EB>
__device__ void query_warps(const PagedTcParams& p, unsigned char* smem, Bars bars,
                            const PagedStart* st, volatile int* abort) {
    const PagedAttendParams& a = p.a;
    const int lane = threadIdx.x & 31, qw = (threadIdx.x >> 5) - kQWarp;
    PagedItem* items = reinterpret_cast<PagedItem*>(smem + kItems);
    const int nkb = (a.D * EB + 127) / 128;
    constexpr int kBlk = kRows * 128;
    PagedWalk<kTS> w;  // each warp walks alike
    w.start(p, st);
    const long long unit0 = w.at - w.tt;
    PagedItem it;
    int unit_tiles = 0;
    bool more = w.next(p, it, unit_tiles);
    if (qw == 0 && lane == 0)
        paged_record(p, more && !(it.flags & kItemBegins) ? &it : nullptr, unit0, unit_tiles, w.per);
    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (k >= p.ni &&
            !warp_wait(bars.item_empty(kb), static_cast<uint32_t>((k / p.ni - 1) & 1), abort))
            return;
        if (!more) {
            if (qw == 0 && lane == 0) items[kb].flags = kItemDone;
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.item_full(kb), 1u);
            return;
        }
        unsigned char* sq = smem + p.off_q + kb * p.q_bytes;
        float* mul = reinterpret_cast<float*>(sq + 2 * nkb * kBlk);  // 8-bit pools
        const int R = it.S * a.G;
        if (qw == 0 && lane == 0) {
            items[kb] = it;
            *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 0;
        }
#pragma unroll 2
        for (int r = qw; r < kRows; r += 4) {
            const int rr = it.r0 + r;
            const bool live = rr < R;
            const T* q = static_cast<const T*>(a.q) +
                         static_cast<int64_t>(it.q0 + (live ? rr / a.G : 0)) * a.q_tok +
                         (static_cast<int64_t>(it.hk) * a.G + (live ? rr % a.G : 0)) * a.q_head;
            if (EB == 2) {
                for (int c = lane; c < nkb * 8; c += 32) {  // 16-byte chunks
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (live && c * 8 < a.D) v = *reinterpret_cast<const uint4*>(q + c * 8);
                    *reinterpret_cast<uint4*>(sq + (c >> 3) * kBlk + r * 128 +
                                              (((c & 7) ^ (r & 7)) << 4)) = v;
                }
            } else {
                float x[2][4];
                const float f = load_row_part<T>(q, a.D, live, lane, x);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c >= nkb) break;
                    uint32_t hi, lo;
                    split_row_part(x[c], f, hi, lo);
                    const int o = c * kBlk + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
                    *reinterpret_cast<uint32_t*>(sq + o) = hi;
                    *reinterpret_cast<uint32_t*>(sq + nkb * kBlk + o) = lo;
                }
                if (lane == 0) mul[r] = a.scale * (1.f / f);  // f is a power of two
            }
        }
        fence_async_shared();  // the query rows, for the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.item_full(kb), 1u);
        more = w.next(p, it, unit_tiles);
    }
}

template <int EB>
__device__ void producer_warp(const PagedTcParams& p, unsigned char* smem, Bars bars,
                              volatile int* abort) {
    const PagedAttendParams& a = p.a;
    const int lane = threadIdx.x & 31;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    StageScales* sc = reinterpret_cast<StageScales*>(smem + kScales);
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const uint32_t sK = smem_addr(smem + p.off_stage), kbytes = nkb * kTS * 128;
    const uint32_t sV = sK + p.ns * kbytes, vbytes = nvb * kTS * 128;
    int ck = 0, cv = 0;  // key and value tiles issued
    Ring kr, vr;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) break;
        for (int n = 0; n < it.nt; ++n) {
            if (ck >= p.ns && !warp_wait(bars.k_empty(kr.s), kr.ph ^ 1u, abort)) {
                ok = false;
                break;
            }
            const PagedBoxes x = paged_boxes<EB, kTS>(p, it, it.tile0 + n, sc + ck % kScaleRing);
            if (x.bad && lane == 0) {
                *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 1;
                if (a.status) atomicOr(a.status, KVC_DEV_OVERFLOW);
            }
            paged_load_boxes<EB, kTS>(p, &p.tk, x, sK + kr.s * kbytes, nkb, bars.k_full(kr.s));
            ++ck;
            kr.next(p.ns);
            if (cv >= p.nv && !warp_wait(bars.v_empty(vr.s), vr.ph ^ 1u, abort)) {
                ok = false;
                break;
            }
            paged_load_boxes<EB, kTS>(p, &p.tv, x, sV + vr.s * vbytes, nvb, bars.v_full(vr.s));
            ++cv;
            vr.next(p.nv);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.item_empty(kb), 1u);
    }
    // do not leave while issued copies may still write shared memory
    if (lane == 0) {
        for (int q = ck > p.ns ? ck - p.ns : 0; q < ck; ++q)
            mbar_drain(bars.k_full(q % p.ns), static_cast<uint32_t>((q / p.ns) & 1));
        for (int q = cv > p.nv ? cv - p.nv : 0; q < cv; ++q)
            mbar_drain(bars.v_full(q % p.nv), static_cast<uint32_t>((q / p.nv) & 1));
    }
}

// One thread: S of every tile, into its group's buffer once the group's last
// P (in the same columns) has been read.
template <typename T, int EB>
__device__ void s_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                         uint32_t tmem) {
    const PagedAttendParams& a = p.a;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    constexpr int kParts = EB == 1 ? 2 : 1, kBlk = kRows * 128;
    const int nkb = (a.D * EB + 127) / 128, ksteps = (a.D * EB + 31) / 32;
    const uint32_t sK0 = smem_addr(smem + p.off_stage);
    const uint32_t idesc = EB == 1 ? mma_idesc_f8(kRows, kTS, false, a.e5m2, false, false)
                                   : mma_idesc_f16(kRows, kTS, std::is_same<T, __nv_bfloat16>::value,
                                                   false, false);
    Ring kr;
    int c = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!mbar_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (items[kb].flags & kItemDone) break;
        const int nt = items[kb].nt;
        const uint32_t sQ = smem_addr(smem + p.off_q + kb * p.q_bytes);
        for (int n = 0; n < nt; ++n, ++c) {
            const int g = c & 1;
            if (!mbar_wait(bars.k_full(kr.s), kr.ph, abort) ||
                (c >= 2 && !mbar_wait(bars.o_done(g), static_cast<uint32_t>((c / 2 - 1) & 1), abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sK = sK0 + kr.s * nkb * kTS * 128;
            for (int part = 0; part < kParts; ++part)
                for (int i = 0; i < ksteps; ++i) {
                    const uint64_t da = smem_desc_sw128(
                        sQ + (part * nkb + (i >> 2)) * kBlk + (i & 3) * 32, 16, 1024);
                    const uint64_t db = smem_desc_sw128(sK + (i >> 2) * kTS * 128 + (i & 3) * 32, 16, 1024);
                    if (EB == 1)
                        tc_mma_f8(tmem + kColS + 128 * g, da, db, idesc, (part | i) != 0);
                    else
                        tc_mma(tmem + kColS + 128 * g, da, db, idesc, i != 0);
                }
            tc_commit(bars.s_ready(g));
            tc_commit(bars.k_empty(kr.s));
            kr.next(p.ns);
        }
        if (ok) tc_commit(bars.item_empty(kb));  // once the products have read the query rows
    }
    tc_commit(bars.drained());
    volatile int never = 0;
    mbar_wait(bars.drained(), 0u, &never);
}

// One thread: O += P V of every tile.
template <typename T, int EB>
__device__ void pv_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                          uint32_t tmem) {
    const PagedAttendParams& a = p.a;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const uint32_t sV0 = smem_addr(smem + p.off_stage) + p.ns * nkb * kTS * 128;
    const int N = (a.Dv + 15) / 16 * 16;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    Ring vr;
    int c = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!mbar_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (items[kb].flags & kItemDone) break;
        const int nt = items[kb].nt;
        // the last run's O has been read
        if (k > 0 && !mbar_wait(bars.o_free(), static_cast<uint32_t>((k - 1) & 1), abort)) break;
        for (int n = 0; n < nt; ++n, ++c) {
            const int g = c & 1;
            if (!mbar_wait(bars.v_full(vr.s), vr.ph, abort) ||
                !mbar_wait(bars.p_ready(g), static_cast<uint32_t>((c / 2) & 1), abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sV = sV0 + vr.s * nvb * kTS * 128;
            const uint32_t tP = tmem + kColS + 128 * g, tO = tmem + kColO + 128 * g;
            if (EB == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 32 slots per step
#pragma unroll
                    for (int part = 0; part < 3; ++part)
                        tc_mma_f8_ts(tO, tP + 24 * i + 8 * part,
                                     smem_desc_sw128(sV + i * 32 * 128, 16, 1024),
                                     mma_idesc_f8(kRows, N, true, a.e5m2, false, true),
                                     n >= 2 || (i | part) != 0);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 slots per step
                    tc_mma_ts(tO, tP + 8 * i, smem_desc_sw128(sV + i * 16 * 128, kTS * 128, 1024),
                              mma_idesc_f16(kRows, N, kBf16, true), n >= 2 || i != 0);
            }
            tc_commit(bars.o_done(g));
            tc_commit(bars.v_empty(vr.s));
            vr.next(p.nv);
        }
        if (ok) mbar_arrive(bars.item_empty(kb), 1u);
    }
    tc_commit(bars.drained());
    volatile int never = 0;
    mbar_wait(bars.drained(), 0u, &never);
}

// Columns past hi, and up to lo, masked.
__device__ __forceinline__ void hide_columns(float (&s)[32], int hi, int lo) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i > hi || i <= lo) s[i] = -INFINITY;
}

template <typename T, int EB, bool MOD>
__device__ void softmax_warps(const PagedTcParams& p, unsigned char* smem, Bars bars,
                              volatile int* abort, uint32_t tmem) {
    using St = Storage<T>;
    const PagedAttendParams& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 2;
    const int r = threadIdx.x & 127;  // query row (tensor-memory lane)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + 128 * g, tO = tmem + lanes + kColO;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    const StageScales* scales = reinterpret_cast<const StageScales*>(smem + kScales);
    float2* xml = reinterpret_cast<float2*>(smem + kXml);  // [2][128] (reference, sum)
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const int box = 31 - __clz(p.hh);
    unsigned char* sV0 = smem + p.off_stage + p.ns * nkb * kTS * 128;
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f;
    const float cap_out = a.softcap * kLog2e;
    int c = 0;       // tiles so far, both groups'
    int vs = 0;      // value stage of tile c
    uint32_t vph = 0;

    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) return;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) return;
        volatile int* odd = reinterpret_cast<volatile int*>(smem + kOdd + 4 * (k & 1));
        const int rr = it.r0 + r;
        const bool live = rr < it.S * a.G;
        const int lim = live ? it.K - it.S + rr / a.G : -1;
        const int low = a.window > 0 ? lim - a.window : -1;  // sees slots low < j <= lim
        float slope = 0.f;
        if (MOD && a.slopes && live) slope = a.slopes[it.hk * a.G + rr % a.G] * kLog2e;
        float mul = a.scale;
        if (EB == 1)
            mul = reinterpret_cast<const float*>(smem + p.off_q + kb * p.q_bytes + 2 * nkb * kRows * 128)[r];
        if (!MOD) mul *= kLog2e;
        float ref = -INFINITY, l = 0.f;
        bool any = false;  // this group has had a tile of the run
        for (int n = 0; n < it.nt; ++n, ++c) {
            const int stage = vs;
            const uint32_t sph = vph;
            if (++vs == p.nv) {
                vs = 0;
                vph ^= 1u;
            }
            if ((c & 1) != g) continue;
            if (!warp_wait(bars.s_ready(g), static_cast<uint32_t>((c / 2) & 1), abort)) return;
            tc_fence_after();
            const int j0 = (it.tile0 + n) * kTS;
            const bool edge = j0 + kTS - 1 > it.first || (a.window > 0 && j0 <= it.last - a.window);
            const StageScales* sc = scales + c % kScaleRing;
            // first pass: the row's largest score of the tile; with a cap or a bias
            // the scores go back to tensor memory. Both passes are loops of 32
            // columns: unrolled whole, their code would not fit the instruction cache
            float top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float s[32];
                tmem_ld32(tS + 32 * q, s);
                if (MOD) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float f = mul, lv = 0.f;
                        if (EB == 1) {
                            const float4 kv = sc->kv[(32 * q + e) >> box];
                            f *= kv.x;
                            lv = kv.z;
                        }
                        if (a.softcap > 0.f) {
                            // cap tanh(s / cap) = cap (1 - 2 / (1 + e^(2 s / cap)))
                            f *= cap_in;
#pragma unroll
                            for (int i = e; i < e + 8; ++i)
                                s[i] = fmaf(-2.f * cap_out, fast_rcp(1.f + fast_exp2(s[i] * f)),
                                            cap_out + lv);
                        } else {
                            f *= kLog2e;
#pragma unroll
                            for (int i = e; i < e + 8; ++i) s[i] = fmaf(s[i], f, lv);
                        }
                        if (a.slopes) {
                            const float far = slope * static_cast<float>(lim - j0 - 32 * q - e);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                s[e + i] += fmaf(slope, static_cast<float>(i), -far);
                        }
                    }
                }
                if (edge) hide_columns(s, lim - j0 - 32 * q, low - j0 - 32 * q);
                if (MOD) tmem_st32(tS + 32 * q, s);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float m = fmaxf(fmaxf(s[e], s[e + 1]), s[e + 2]);
                    m = fmaxf(fmaxf(m, s[e + 3]), s[e + 4]);
                    m = fmaxf(fmaxf(m, s[e + 5]), s[e + 6]);
                    m = fmaxf(m, s[e + 7]);
                    if (!MOD) {
                        float f = mul, lv = 0.f;
                        if (EB == 1) {
                            const float4 kv = sc->kv[(32 * q + e) >> box];
                            f = fmaxf(f * kv.x, 1e-37f);
                            lv = kv.z;
                        }
                        m = fmaf(m, f, lv);
                    }
                    top = fmaxf(top, m);
                }
            }
            float corr = 1.f;
            if (top > ref + RaiseAbove<EB>::v) {
                corr = ref == -INFINITY ? 0.f : fast_exp2(ref - top);
                l *= corr;
                ref = top;
            }
            if (__any_sync(0xffffffffu, corr != 1.f) && any) {
                // O is at rest: S of this tile was issued after the group's last product
                if (!warp_wait(bars.o_done(g), static_cast<uint32_t>((c / 2 - 1) & 1), abort)) return;
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < a.Dv; d += 16) {
                    float o[16];
                    tmem_ldn<16>(tO + 128 * g + d, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= corr;
                    tmem_stn<16>(tO + 128 * g + d, o);
                }
            }
            any = true;
            // the weights, over the scores (a row that saw nothing yet: all 2^-inf)
            const float off = ref == -INFINITY ? kWeightOffset : kWeightOffset - ref;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float s[32];
                tmem_ld32(tS + 32 * q, s);
                if (!MOD && edge) hide_columns(s, lim - j0 - 32 * q, low - j0 - 32 * q);
                uint32_t w[EB == 1 ? 24 : 16];
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float f = MOD ? 1.f : mul, lv = off, ivs = 1.f;
                    if (EB == 1) {
                        const float4 kv = sc->kv[(32 * q + e) >> box];
                        if (!MOD) {
                            f = fmaxf(f * kv.x, 1e-37f);
                            lv += kv.z;
                        }
                        ivs = kv.w;
                        sum = make_float2(0.f, 0.f);
                    }
                    float* x = s + e;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 v = fma2(make_float2(x[i], x[i + 1]), make_float2(f, f),
                                              make_float2(lv, lv));
                        x[i] = fast_exp2(v.x);
                        x[i + 1] = fast_exp2(v.y);
                        sum = add2(sum, make_float2(x[i], x[i + 1]));
                    }
                    if (EB == 1) {
                        l = fmaf(sum.x + sum.y, ivs, l);
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            uint32_t part[3];
                            split_weights(x[i], x[i + 1], x[i + 2], x[i + 3], part);
#pragma unroll
                            for (int k2 = 0; k2 < 3; ++k2) w[8 * k2 + (e + i) / 4] = part[k2];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i += 2) w[(e + i) / 2] = pack2<T>(x[i], x[i + 1]);
                    }
                }
                constexpr int kWords = EB == 1 ? 24 : 16;
#pragma unroll
                for (int i = 0; i < kWords; i += 8) tmem_st8_async(tS + kWords * q + i, w + i);
            }
            if (EB == 2) l += sum.x + sum.y;
            tmem_wait_st();
            if (edge) {  // thread r looks after slot r's value row
                if (!warp_wait(bars.v_full(stage), sph, abort)) return;
                const int j = j0 + r;
                unsigned char* vrow = sV0 + stage * nvb * kTS * 128 + r * 128;
                const bool some = j <= it.last && j >= it.lo;
                const bool all = j <= it.first && (a.window == 0 || j > it.last - a.window);
                if (!some) {
                    for (int b = 0; b < nvb; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(vrow + b * kTS * 128 + i * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                } else if (!all) {
                    for (int b = 0; b < nvb; ++b)
                        for (int i = 0; i < 32; ++i) {
                            uint32_t* x = reinterpret_cast<uint32_t*>(vrow + b * kTS * 128) +
                                          ((i + lane) & 31);
                            const uint32_t v = *x, u = clear_odd<EB, T>(v, a.e5m2);
                            if (u != v) {
                                *x = u;
                                *odd = k + 1;
                            }
                        }
                }
                fence_async_shared();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.p_ready(g), 1u);
        }
        // the run's end: both groups' last products
        // (a group without a tile of this run leaves the last run's to its readers)
        if (any) xml[g * 128 + r] = make_float2(ref, l);
        for (int h = 0; h < 2; ++h) {
            const int done = (c + 1 - h) / 2;  // tiles of group h so far
            if (done > 0 && !warp_wait(bars.o_done(h), static_cast<uint32_t>((done - 1) & 1), abort))
                return;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.meet(), 1u);
        if (!warp_wait(bars.meet(), static_cast<uint32_t>(k & 1), abort)) return;
        tc_fence_after();
        const float2 x0 = xml[r], x1 = xml[128 + r];
        const bool has0 = it.nt >= 2 || ((c - 1) & 1) == 0, has1 = it.nt >= 2 || ((c - 1) & 1) == 1;
        const float m = fmaxf(has0 ? x0.x : -INFINITY, has1 ? x1.x : -INFINITY);
        const float f0 = has0 ? (x0.x == m ? 1.f : fast_exp2(x0.x - m)) : 0.f;
        const float f1 = has1 ? (x1.x == m ? 1.f : fast_exp2(x1.x - m)) : 0.f;
        float sum = 0.f;
        if (has0) sum = fmaf(x0.y, f0, sum);
        if (has1) sum = fmaf(x1.y, f1, sum);
        const bool bad = *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) != 0;
        const bool odds = *odd == k + 1;
        const bool whole = (it.flags & kItemBegins) && (it.flags & kItemEnds);
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + ((it.flags & kItemBegins) ? 1 : 0);
        const int64_t row = static_cast<int64_t>(it.q0 + (live ? rr / a.G : 0)) * a.Hq +
                            it.hk * a.G + (live ? rr % a.G : 0);
        const float inv = __fdiv_rn(1.f, sum);
        // columns in runs of 16, the groups in turn
        for (int d = 16 * g; d < a.Dv; d += 32) {
            float o[16], o1[16];
            if (has0) tmem_ldn<16>(tO + d, o);
            if (has1) tmem_ldn<16>(tO + 128 + d, o1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = has0 ? o[i] * f0 : 0.f;
                if (has1) v = fmaf(o1[i], f1, v);
                o[i] = v;
            }
            if (odds && live) {  // what was cleared: from memory, into the rows that see it
                const int j1 = min(lim, (it.tile0 + it.nt) * kTS - 1);
                for (int j = max(low + 1, it.tile0 * kTS); j <= j1; ++j) {
                    if (j <= it.first && (a.window == 0 || j > it.last - a.window)) {
                        j = max(j, it.first);
                        continue;
                    }
                    const int id = a.table[it.b * a.max_blocks + j / a.bs];
                    if (id < 0 || id >= a.num_blocks) continue;
                    const int64_t e =
                        ((static_cast<int64_t>(id) * a.Hk + it.hk) * a.bs + j % a.bs) * a.Dv + d;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (d + i >= a.Dv) break;
                        const float v = EB == 1
                                            ? from_eight(static_cast<const uint8_t*>(a.vp)[e + i], a.e5m2)
                                            : St::to_float(static_cast<const T*>(a.vp)[e + i]);
                        if (!(fabsf(v) < INFINITY)) o[i] += v;
                    }
                }
            }
            if (live && whole) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = bad ? 0u : pack2<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
                T* dst = static_cast<T*>(a.out) + row * a.Dv + d;
                *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                if (d + 8 < a.Dv) *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            } else if (live) {
                float* dst = p.part_acc + (slot * kRows + r) * a.Dv + d;
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    if (d + i < a.Dv)
                        *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
            __syncwarp();
        }
        if (!whole && live && g == 0) {
            p.part_ml[2 * (slot * kRows + r)] = m;
            p.part_ml[2 * (slot * kRows + r) + 1] = bad ? -1.f : sum;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bars.o_free(), 1u);
            mbar_arrive(bars.item_empty(kb), 1u);
        }
    }
}

template <typename T, int EB, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const __grid_constant__ PagedTcParams p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const Bars bars{smem_addr(smem)};
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kAbort);
    PagedStart* st = reinterpret_cast<PagedStart*>(smem + kStart);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.ns; ++s) {
            mbar_init(bars.k_full(s), 1u);
            mbar_init(bars.k_empty(s), 1u);
        }
        for (int s = 0; s < p.nv; ++s) {
            mbar_init(bars.v_full(s), 1u);
            mbar_init(bars.v_empty(s), 1u);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(bars.item_full(k), 4u);         // the query warps
            mbar_init(bars.item_empty(k), 3u + 8u);   // producer, both issuers, softmax warps
            mbar_init(bars.s_ready(k), 1u);
            mbar_init(bars.p_ready(k), 4u);
            mbar_init(bars.o_done(k), 1u);
        }
        mbar_init(bars.meet(), 8u);
        mbar_init(bars.o_free(), 8u);
        mbar_init(bars.drained(), 2u);
        *abort = 0;
        *reinterpret_cast<volatile int*>(smem + kOdd) = 0;
        *reinterpret_cast<volatile int*>(smem + kOdd + 4) = 0;
        fence_mbar_init();
    }
    if (warp == kSWarp) {
        tmem_alloc(smem_addr(smem + kTmemSlot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    paged_plan<T, kTS, kThreads>(p, st);  // with block barriers
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTmemSlot);
    launch_dependents();

    // 184 registers for a softmax thread, 72 for the others (8 warps x 184 + 8 x 72 =
    // the launch's 16 x 128)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        softmax_warps<T, EB, MOD>(p, smem, bars, abort, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kSWarp) {
            if ((threadIdx.x & 31) == 0) s_issuer<T, EB>(p, smem, bars, abort, tmem);
        } else if (warp == kPvWarp) {
            if ((threadIdx.x & 31) == 0) pv_issuer<T, EB>(p, smem, bars, abort, tmem);
        } else if (warp == kProdWarp) {
            producer_warp<EB>(p, smem, bars, abort);
        } else if (warp >= kQWarp) {
            query_warps<T, EB>(p, smem, bars, st, abort);
        }
    }
    tc_fence_before();
    __syncthreads();  // every thread reaches this exactly once: all waits are bounded
    if (warp == kSWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort && p.a.status) atomicOr(p.a.status, KVC_DEV_TIMEOUT);
}

template <typename T, int EB, bool MOD>
cudaError_t launch_t(const PagedTcParams& p, size_t smem, cudaStream_t stream) {
    auto kern = paged_rows_kernel<T, EB, MOD>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.ctas), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}
template <typename T, int EB>
cudaError_t launch_eb(const PagedTcParams& p, size_t smem, cudaStream_t stream) {
    return p.a.softcap > 0.f || p.a.slopes ? launch_t<T, EB, true>(p, smem, stream)
                                           : launch_t<T, EB, false>(p, smem, stream);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedTcParams& p, int dtype, int pool_dtype, size_t smem,
                              cudaStream_t stream) {
    if (pool_dtype == dtype)
        return dtype == KVC_BF16 ? launch_eb<__nv_bfloat16, 2>(p, smem, stream)
                                 : launch_eb<__half, 2>(p, smem, stream);
    return dtype == KVC_BF16 ? launch_eb<__nv_bfloat16, 1>(p, smem, stream)
                             : launch_eb<__half, 1>(p, smem, stream);
}

}  // namespace kvc
