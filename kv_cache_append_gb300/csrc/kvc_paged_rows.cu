// kvc_paged_rows.cu -- attention over a paged pool on the tensor cores, for
// units of many query rows: prompts, chunks, and steps of many heads per KV head.
//
// Query rows are the M dimension (128 rows r = t G + g of a KV head, a thread
// each), 128 slots a tile:
//
//   S  = Q K^T    (A = query rows, B = K tile, both from shared memory)
//   O += P V      (A = P from tensor memory, B = V tile read N-major)
//
// With 8-bit pools both products take the tiles as they lie in memory, the query
// rows as two e4m3 parts (fp16: three) and the weights as three e5m2 parts (splits,
// scales and references as in kvc_paged_decode.cu): five or six products at twice
// the 16-bit rate against four halves, so the tensor-core time is 5/4 (3/2) of 16-bit
// tiles', with half the memory traffic and no conversion of the cache. (Value tiles
// turned into fp16 by four more warps, with weights of one part, took 1156 us where the
// parts took 1020, in this kernel's state of that time: the conversion, 2300 cycles a
// tile, then was the longest stage.)
//
// The softmax, not the products, is the longer part of a tile, and a tile's chain
// (S, softmax, P V, the next S into the same columns) is longer still: three groups
// of 4 warps take the tiles in turn, each with its S in tensor memory, so that
// two tiles' softmax run under one tile's products and barriers. O is one for all of them,
// so a row has one reference: tile n's warp reads what tile n - 1's warp of the
// same rows left before it makes its weights (a decision comes after the first of a
// tile's two passes, and raising is rare), and each group measures its sum by the
// reference it last saw. P overwrites its S in place: the weights of 32 slots take 24
// columns (16 of 16-bit weights), behind the 32 score columns that are read next.
//
// Tensor memory: S of the groups at columns 0, 128 and 256, O at 384. Warps: 12
// softmax, an S issuer, a P.V issuer, a producer of key tiles and one of value tiles,
// and 4 that schedule the block's runs (kvc_paged_tc.cuh) and prepare the next
// run's query rows.
//
// Measured, 32 heads on 8 of 128, four prompts of 513 to 2001 tokens over up to 8190
// slots (617 GFLOP): e4m3 pool 752 us, 820 TFLOP/s, bf16 pool 640 us; bounded by the
// softmax warps' instruction fetch and issue (a tile takes about 2600 cycles where its
// products take 1280 and 1024) and by a unit's start and end, the time of about 7 tiles.
#include <algorithm>
#include <type_traits>

#include "kvc_paged_tc.cuh"

namespace kvc {
namespace {

constexpr int kTS = 128, kRows = 128;
constexpr int kGroups = 3;                 // of 4 softmax warps, tiles in turn
constexpr int kSoft = 4 * kGroups;
constexpr int kSWarp = 12, kPvWarp = 13, kKWarp = 14, kVWarp = 15, kQWarp = 16;  // 16..19: query rows
constexpr int kThreads = 20 * 32;
constexpr uint32_t kColS = 0, kColO = 384;  // S buffers of the three groups, O

struct Bars {
    uint32_t base;
    __device__ uint32_t k_full(int s) const { return base + 8u * s; }
    __device__ uint32_t k_empty(int s) const { return base + 64u + 8u * s; }
    __device__ uint32_t v_full(int s) const { return base + 128u + 8u * s; }
    __device__ uint32_t v_empty(int s) const { return base + 192u + 8u * s; }
    __device__ uint32_t item_full(int k) const { return base + 256u + 8u * k; }
    __device__ uint32_t item_empty(int k) const { return base + 272u + 8u * k; }
    __device__ uint32_t s_ready(int g) const { return base + 288u + 8u * g; }
    __device__ uint32_t p_ready(int g) const { return base + 312u + 8u * g; }
    __device__ uint32_t o_done(int g) const { return base + 336u + 8u * g; }
    // per 32 rows and group: one barrier for all would let a group that is two tiles
    // ahead of the decisions take an old phase for the one it waits for
    __device__ uint32_t decide(int w, int g) const { return base + 360u + 8u * (3 * w + g); }
    __device__ uint32_t meet(int k) const { return base + ((k & 1) ? 528u : 456u); }
    __device__ uint32_t o_free() const { return base + 464u; }
    __device__ uint32_t drained() const { return base + 472u; }
    // the run is known (its query rows are not ready yet)
    __device__ uint32_t item_known(int k) const { return base + 480u + 8u * k; }
};
constexpr int kTmemSlot = 496, kAbort = 500, kBad = 504 /* [2] */, kOdd = 512 /* [3] */;
constexpr int kStart = 576, kItems = 896;
// exchanged between the groups, for three runs in turn: a row's reference [3][128],
// each group's sum and the reference it is measured by [3][3][128]
constexpr int kXr = 1024, kXl = 2560;
constexpr int kScales = 11776, kScaleRing = 16;  // 8-bit pools: 16 tiles' scales

// Tile c's group (c % 3) and the parity of its use of that group's barriers.
struct Turn {
    int g = 0;
    uint32_t ph = 0;
    __device__ void next() {
        if (++g == kGroups) {
            g = 0;
            ph ^= 1u;
        }
    }
};

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
    const int before = w.tt - w.lead;  // of the unit's tiles, in earlier blocks
    PagedItem it;
    int unit_tiles = 0;
    bool more = w.next(p, it, unit_tiles);
    if (qw == 0 && lane == 0)
        paged_record(p, more && !(it.flags & kItemBegins) ? &it : nullptr, before, unit_tiles, w.per);
    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (k >= p.ni &&
            !warp_wait(bars.item_empty(kb), static_cast<uint32_t>((k / p.ni - 1) & 1), abort))
            return;
        if (!more) {
            if (qw == 0 && lane == 0) {
                items[kb].flags = kItemDone;
                mbar_arrive(bars.item_known(kb), 1u);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.item_full(kb), 1u);
            return;
        }
        unsigned char* sq = smem + p.off_q + kb * p.q_bytes;
        float* mul = reinterpret_cast<float*>(sq + QueryParts<T, EB>::v * nkb * kBlk);  // 8-bit pools
        if (qw == 0 && lane == 0) {
            items[kb] = it;
            *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 0;
            mbar_arrive(bars.item_known(kb), 1u);
        }
        prepare_rows<T, EB, kRows, 128>(p, it, sq, nkb, kBlk, 32 * qw + lane, EB == 1 ? mul : nullptr);
        fence_async_shared();  // the query rows, for the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.item_full(kb), 1u);
        more = w.next(p, it, unit_tiles);
    }
}

// Two warps: the key tiles (with the scales) and the value tiles.
template <int EB, bool KEYS>
__device__ void producer_warp(const PagedTcParams& p, unsigned char* smem, Bars bars,
                              volatile int* abort) {
    const PagedAttendParams& a = p.a;
    const int lane = threadIdx.x & 31;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    StageScales* sc = reinterpret_cast<StageScales*>(smem + kScales);
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const int stages = KEYS ? p.ns : p.nv;
    const uint32_t bytes = (KEYS ? nkb : nvb) * kTS * 128;
    const uint32_t base = smem_addr(smem + p.off_stage) + (KEYS ? 0 : p.ns * nkb * kTS * 128);
    int c = 0;  // tiles issued
    Ring ring;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_known(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) break;
        constexpr bool kScaled = EB == 1 && KEYS;
        int id = feed_id<kTS>(p, it, it.tile0);
        int id1 = it.nt > 1 ? feed_id<kTS>(p, it, it.tile0 + 1) : kNoBox;
        float fs = 1.f, fs1 = 1.f;
        if (kScaled) fs = feed_scale(p, it, id);
        for (int n = 0; n < it.nt; ++n) {
            const int tile = it.tile0 + n;
            const int id2 = n + 2 < it.nt ? feed_id<kTS>(p, it, tile + 2) : kNoBox;
            if (kScaled) fs1 = feed_scale(p, it, id1);
            if (c >= stages &&
                !warp_wait(KEYS ? bars.k_empty(ring.s) : bars.v_empty(ring.s), ring.ph ^ 1u, abort)) {
                ok = false;
                break;
            }
            if (KEYS && __any_sync(0xffffffffu, feed_bad(p, id)) && lane == 0) {
                *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 1;
                if (a.status) atomicOr(a.status, KVC_DEV_OVERFLOW);
            }
            if (kScaled) feed_store(sc + c % kScaleRing, fs);
            const uint32_t to = base + ring.s * bytes;
            feed_copy<EB, kTS>(p, it, tile, id, to, KEYS ? nkb : 0, to, KEYS ? 0 : nvb,
                               KEYS ? bars.k_full(ring.s) : bars.v_full(ring.s));
            id = id1;
            id1 = id2;
            fs = fs1;
            ++c;
            ring.next(stages);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.item_empty(kb), 1u);
    }
    // do not leave while issued copies may still write shared memory
    if (lane == 0)
        for (int q = c > stages ? c - stages : 0; q < c; ++q)
            mbar_drain(KEYS ? bars.k_full(q % stages) : bars.v_full(q % stages),
                       static_cast<uint32_t>((q / stages) & 1));
}

// One warp: S of every tile, into its group's buffer once the group's last
// P (in the same columns) has been read.
template <typename T, int EB>
__device__ void s_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                         uint32_t tmem) {
    const PagedAttendParams& a = p.a;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    constexpr int kParts = QueryParts<T, EB>::v, kBlk = kRows * 128;
    const int nkb = (a.D * EB + 127) / 128, ksteps = (a.D * EB + 31) / 32;
    const uint32_t sK0 = smem_addr(smem + p.off_stage);
    const uint32_t idesc = EB == 1 ? mma_idesc_f8(kRows, kTS, false, a.e5m2, false, false)
                                   : mma_idesc_f16(kRows, kTS, std::is_same<T, __nv_bfloat16>::value,
                                                   false, false);
    Ring kr;
    Turn turn;
    int c = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (uniform(items[kb].flags) & kItemDone) break;
        const int nt = uniform(items[kb].nt);
        const uint32_t sQ = smem_addr(smem + p.off_q + kb * p.q_bytes);
        for (int n = 0; n < nt; ++n, ++c) {
            const int g = turn.g;
            if (!warp_wait(bars.k_full(kr.s), kr.ph, abort) ||
                (c >= kGroups && !warp_wait(bars.o_done(g), turn.ph ^ 1u, abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sK = sK0 + kr.s * nkb * kTS * 128;
            const uint32_t tS = tmem + kColS + 128 * g;
            if (elect_one()) {
                for (int b = 0; b < nkb; ++b) {
                    // column block b of both; 32 bytes of a row per instruction, 2 in
                    // the descriptor's address field
                    const uint64_t db = smem_desc_sw128(sK + b * kTS * 128, 16, 1024);
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        const uint64_t da = smem_desc_sw128(sQ + (part * nkb + b) * kBlk, 16, 1024);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (4 * b + i >= ksteps) break;
                            if (EB == 1)
                                tc_mma_f8(tS, da + 2 * i, db + 2 * i, idesc, (b | part | i) != 0);
                            else
                                tc_mma(tS, da + 2 * i, db + 2 * i, idesc, (b | i) != 0);
                        }
                    }
                }
                tc_commit(bars.s_ready(g));
                tc_commit(bars.k_empty(kr.s));
            }
            __syncwarp();
            kr.next(p.ns);
            turn.next();
        }
        if (ok && elect_one()) tc_commit(bars.item_empty(kb));  // once the products have read the query rows
    }
    if (elect_one()) tc_commit(bars.drained());
    __syncwarp();
    volatile int never = 0;
    warp_wait(bars.drained(), 0u, &never);
}

// One warp: O += P V of every tile.
template <typename T, int EB>
__device__ void pv_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                          uint32_t tmem) {
    const PagedAttendParams& a = p.a;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const uint32_t sV0 = smem_addr(smem + p.off_stage) + p.ns * nkb * kTS * 128;
    const int N = (a.Dv + 15) / 16 * 16;
    const uint32_t idesc = EB == 1 ? mma_idesc_f8(kRows, N, true, a.e5m2, false, true)
                                   : mma_idesc_f16(kRows, N, std::is_same<T, __nv_bfloat16>::value, true);
    Ring vr;
    Turn turn;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (uniform(items[kb].flags) & kItemDone) break;
        const int nt = uniform(items[kb].nt);
        // the last run's O has been read
        if (k > 0 && !warp_wait(bars.o_free(), static_cast<uint32_t>((k - 1) & 1), abort)) break;
        for (int n = 0; n < nt; ++n) {
            const int g = turn.g;
            if (!warp_wait(bars.v_full(vr.s), vr.ph, abort) ||
                !warp_wait(bars.p_ready(g), turn.ph, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sV = sV0 + vr.s * nvb * kTS * 128;
            const uint32_t tP = tmem + kColS + 128 * g, tO = tmem + kColO;
            const uint64_t dv = smem_desc_sw128(sV, kTS * 128, 1024);
            if (elect_one()) {
                if (EB == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 slots per step
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            tc_mma_f8_ts(tO, tP + 24 * i + 8 * part,
                                         dv + i * (32 * 128 / 16), idesc, (n | i | part) != 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 slots per step
                        tc_mma_ts(tO, tP + 8 * i, dv + i * (16 * 128 / 16), idesc, (n | i) != 0);
                }
                tc_commit(bars.o_done(g));
                tc_commit(bars.v_empty(vr.s));
            }
            __syncwarp();
            vr.next(p.nv);
            turn.next();
        }
        if (ok && elect_one()) mbar_arrive(bars.item_empty(kb), 1u);
        __syncwarp();
    }
    if (elect_one()) tc_commit(bars.drained());
    __syncwarp();
    volatile int never = 0;
    warp_wait(bars.drained(), 0u, &never);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Columns past hi, and up to lo, masked.
__device__ __forceinline__ void hide_columns(float (&s)[32], int hi, int lo) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i > hi || i <= lo) s[i] = -INFINITY;
}

// WIDE (8-bit pools): the boxes have 32 slots or more, so 32 columns share their scales.
template <typename T, int EB, bool MOD, bool WIDE>
__device__ void softmax_warps(const PagedTcParams& p, unsigned char* smem, Bars bars,
                              volatile int* abort, uint32_t tmem) {
    using St = Storage<T>;
    const PagedAttendParams& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 2, wq = warp & 3;
    const int r = threadIdx.x & 127;  // query row (tensor-memory lane)
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + 128 * g, tO = tmem + lanes + kColO;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + kItems);
    const StageScales* scales = reinterpret_cast<const StageScales*>(smem + kScales);
    const int nkb = (a.D * EB + 127) / 128, nvb = (a.Dv * EB + 127) / 128;
    const int box = 31 - __clz(p.hh);
    unsigned char* sV0 = smem + p.off_stage + p.ns * nkb * kTS * 128;
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f;
    const float cap_out = a.softcap * kLog2e;
    int c = 0;      // tiles so far, all groups'
    Turn turn;      // tile c's group
    Ring vr;        // and value stage

    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) return;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) return;
        // a group that is done with its tiles goes on to the next run, at most two ahead
        // of the last group: run k - 3's exchange buffers are free once all met in run k - 2
        if (k >= 2 && !warp_wait(bars.meet(k), static_cast<uint32_t>((k >> 1) - 1) & 1u, abort)) return;
        const int k3 = k % 3;
        volatile int* odd = reinterpret_cast<volatile int*>(smem + kOdd + 4 * k3);
        const int rr = it.r0 + r;
        const bool live = rr < it.S * a.G;
        const int lim = live ? it.K - it.S + rr / a.G : -1;
        const int low = a.window > 0 ? lim - a.window : -1;  // sees slots low < j <= lim
        float slope = 0.f;
        if (MOD && a.slopes && live) slope = a.slopes[it.hk * a.G + rr % a.G] * kLog2e;
        float mul = a.scale;
        if (EB == 1)
            mul = reinterpret_cast<const float*>(smem + p.off_q + kb * p.q_bytes +
                                                 QueryParts<T, EB>::v * nkb * kRows * 128)[r];
        if (!MOD) mul *= kLog2e;
        // the row's reference is one for all groups: tile n's warp reads what tile n -
        // 1's left, and may raise it
        float* xr = reinterpret_cast<float*>(smem + kXr) + k3 * 128 + r;
        float2* xl = reinterpret_cast<float2*>(smem + kXl) + k3 * 3 * 128 + r;
        float ref = -INFINITY, l = 0.f;  // the reference that this group's sum is measured by
        for (int n = 0; n < it.nt; ++n, ++c) {
            const int stage = vr.s, tg = turn.g;
            const uint32_t sph = vr.ph, tph = turn.ph;
            vr.next(p.nv);
            turn.next();
            if (tg != g) continue;
            if (!warp_wait(bars.s_ready(g), tph, abort)) return;
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
                if (MOD || EB == 2 || WIDE) {
                    float m = max3(s[0], s[1], s[2]);
#pragma unroll
                    for (int e = 3; e < 31; e += 2) m = max3(m, s[e], s[e + 1]);
                    m = fmaxf(m, s[31]);
                    if (!MOD) {
                        float f = mul, lv = 0.f;
                        if (EB == 1) {
                            const float4 kv = sc->kv[(32 * q) >> box];
                            f = fmaxf(f * kv.x, 1e-37f);
                            lv = kv.z;
                        }
                        m = fmaf(m, f, lv);
                    }
                    top = fmaxf(top, m);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float m = max3(s[e], s[e + 1], s[e + 2]);
                        m = max3(m, s[e + 3], s[e + 4]);
                        m = max3(m, s[e + 5], s[e + 6]);
                        m = fmaxf(m, s[e + 7]);
                        const float4 kv = sc->kv[(32 * q + e) >> box];
                        top = fmaxf(top, fmaf(m, fmaxf(mul * kv.x, 1e-37f), kv.z));
                    }
                }
            }
            // the last tile's decision, then this one's; a raised reference also
            // rescales O, at rest between the two tiles' products
            const int pg = g == 0 ? kGroups - 1 : g - 1;  // tile c - 1's group and parity
            const uint32_t pph = g == 0 ? tph ^ 1u : tph;
            // (a run's first tile waits too: no group's decisions are two ahead of another's)
            if (c > 0 && !warp_wait(bars.decide(wq, pg), pph, abort)) return;
            const float was = n > 0 ? *xr : -INFINITY;
            const bool raise = top > was + RaiseAbove<EB>::v;
            const float now = raise ? top : was;
            if (n == 0 || raise) *xr = now;
            const bool some = __any_sync(0xffffffffu, raise && was != -INFINITY);
            if (lane == 0) mbar_arrive(bars.decide(wq, g), 1u);
            if (now != ref) {
                if (ref != -INFINITY) l *= fast_exp2(ref - now);
                ref = now;
            }
            if (some) {
                if (!warp_wait(bars.o_done(pg), pph, abort)) return;
                tc_fence_after();
                const float corr = raise && was != -INFINITY ? fast_exp2(was - now) : 1.f;
#pragma unroll 1
                for (int d = 0; d < a.Dv; d += 16) {
                    float o[16];
                    tmem_ldn<16>(tO + d, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= corr;
                    tmem_stn<16>(tO + d, o);
                }
            }
            // the weights, over the scores (a row that saw nothing yet: all 2^-inf)
            const float off = ref == -INFINITY ? kWeightOffset : kWeightOffset - ref;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float s[32];
                tmem_ld32(tS + 32 * q, s);
                if (!MOD && edge) hide_columns(s, lim - j0 - 32 * q, low - j0 - 32 * q);
                uint32_t w[EB == 1 ? 24 : 16];
                float f = MOD ? 1.f : mul, lv = off, ivs = 1.f;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (EB == 1 && (e == 0 || !WIDE)) {
                        const float4 kv = sc->kv[(32 * q + e) >> box];
                        if (!MOD) {
                            f = fmaxf(mul * kv.x, 1e-37f);
                            lv = off + kv.z;
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
                        if (e == 24 || !WIDE) l = fmaf(sum.x + sum.y, ivs, l);
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
                const bool some_see = j <= it.last && j >= it.lo;
                const bool all_see = j <= it.first && (a.window == 0 || j > it.last - a.window);
                if (!all_see && clean_value_row<EB, T>(vrow, nvb, kTS * 128, some_see, a.e5m2))
                    *odd = k + 1;
                fence_async_shared();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.p_ready(g), 1u);
        }
        // the run's end: the group of its last tile (turn's predecessor) writes the
        // result; the others go on
        xl[128 * g] = make_float2(l, ref);
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.meet(k), 1u);
        const int pg = turn.g == 0 ? kGroups - 1 : turn.g - 1;
        if (g != pg) {
            if (lane == 0) mbar_arrive(bars.item_empty(kb), 1u);
            continue;
        }
        if (!warp_wait(bars.o_done(pg), turn.g == 0 ? turn.ph ^ 1u : turn.ph, abort) ||
            !warp_wait(bars.meet(k), static_cast<uint32_t>((k >> 1) & 1), abort))
            return;
        tc_fence_after();
        const float m = *xr;
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < kGroups; ++h) {
            const float2 x = xl[128 * h];
            if (x.x != 0.f) sum = fmaf(x.x, x.y == m ? 1.f : fast_exp2(x.y - m), sum);
        }
        const bool bad = *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) != 0;
        const bool odds = *odd == k + 1;
        const bool whole = (it.flags & kItemBegins) && (it.flags & kItemEnds);
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + ((it.flags & kItemBegins) ? 1 : 0);
        const int64_t row = static_cast<int64_t>(it.q0 + (live ? rr / a.G : 0)) * a.Hq +
                            it.hk * a.G + (live ? rr % a.G : 0);
        const float inv = __fdiv_rn(1.f, sum);
#pragma unroll 1
        for (int d = 0; d < a.Dv; d += 16) {
            float o[16];
            tmem_ldn<16>(tO + d, o);
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
        if (!whole && live) {
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
            mbar_init(bars.item_known(k), 1u);
            mbar_init(bars.item_full(k), 4u);         // the query warps
            mbar_init(bars.item_empty(k), 4u + kSoft);  // producers, issuers, softmax warps
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(bars.s_ready(g), 1u);
            mbar_init(bars.p_ready(g), 4u);
            mbar_init(bars.o_done(g), 1u);
        }
        for (int w = 0; w < 4; ++w)
            for (int g = 0; g < kGroups; ++g) mbar_init(bars.decide(w, g), 1u);
        mbar_init(bars.meet(0), kSoft);
        mbar_init(bars.meet(1), kSoft);
        mbar_init(bars.o_free(), 4u);  // the group that read it
        mbar_init(bars.drained(), 2u);
        *abort = 0;
        *reinterpret_cast<volatile int*>(smem + kOdd) = 0;
        *reinterpret_cast<volatile int*>(smem + kOdd + 4) = 0;
        *reinterpret_cast<volatile int*>(smem + kOdd + 8) = 0;
        fence_mbar_init();
        prefetch_map(&p.tk);
        prefetch_map(&p.tv);
    }
    if (warp == kSWarp) {
        tmem_alloc(smem_addr(smem + kTmemSlot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    paged_plan<T, kTS, kThreads>(p, st);  // with block barriers
    tc_fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile int*>(smem + kTmemSlot));
    launch_dependents();

    // 120 registers for a softmax thread, 56 for the others: 12 warps x 120 + 8 x 56 <=
    // the launch's 20 x 96
    if (warp < kSoft) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        if (EB == 2 || p.hh >= 32)
            softmax_warps<T, EB, MOD, true>(p, smem, bars, abort, tmem);
        else
            softmax_warps<T, EB, MOD, EB == 2>(p, smem, bars, abort, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kSWarp) {
            s_issuer<T, EB>(p, smem, bars, abort, tmem);
        } else if (warp == kPvWarp) {
            pv_issuer<T, EB>(p, smem, bars, abort, tmem);
        } else if (warp == kKWarp) {
            producer_warp<EB, true>(p, smem, bars, abort);
        } else if (warp == kVWarp) {
            producer_warp<EB, false>(p, smem, bars, abort);
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
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern));
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
