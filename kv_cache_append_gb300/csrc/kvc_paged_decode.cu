// kvc_paged_decode.cu -- attention over a paged pool on the tensor cores, for
// units (sequence, KV head) of at most 16 query rows: decode and short
// speculative steps.
//
// A step reads each visible cache row once and does 2 R (D + Dv) operations on
// it: memory bounds it once the arithmetic is off the CUDA cores. As in the
// decode kernel of the step, a tile's 128 slots are the M dimension of both
// products, the unit's rows (padded to N = 16) the N dimension:
//
//   S^T  = K Q^T      (A = K tile as TMA wrote it, B = query rows)
//   O^T += V^T P^T    (A = V tile read M-major, B = P^T from shared memory)
//
// 8-bit pools go to the tensor cores as they lie in memory (kind::f8f6f4), with
// no conversion: the other operand is split into 8-bit parts, and the
// products of all parts add up in the same accumulator.
//   Query rows: x 2^k as two e4m3 parts, three for fp16, k from the row's largest
//   element (2^7..2^8 then): exact, but for what is under 2^-17 of that element.
//   Weights: three e5m2 parts of an fp16 value (split_weights): 2^-9 of the weight
//   over 16 octaves below the largest, 2^-25 of the largest under that. (e4m3 parts
//   end at 2^-10: they would drop the flat rest behind one dominant slot of
//   a long context.)
// The key scale of a slot's block multiplies its scores. The value scale goes into
// the weight: w = 2^(s + log2 vs - ref), and the row sum takes w / vs, so one
// reference per row bounds the weights whatever the blocks' scales are.
// The further parts cost nothing that matters: the tensor cores are idle most of
// the time.
//
// Warps: one or two groups of 4 softmax warps (a thread owns a slot, for all rows
// or for its group's half of them), one S issuer, one P.V issuer,
// one producer (block-table look-ups, scales, TMA boxes), one scheduler, which walks
// the block's runs (kvc_paged_tc.cuh) and splits the next run's query rows
// while the others work on the current one. 8-bit tiles of D = Dv = 128 are 32
// KB, so two blocks fit an SM with three stages each and cover each
// other's softmax latency; 16-bit tiles take one block an SM.
//
// A slot that no row sees has its value row set to zero in the tile. A
// slot that some rows see and others do not (the newest tokens, a window's edge)
// could carry an infinity or NaN into the rows that do not: its thread then
// clears those elements in the tile and the unit's epilogue adds them, from
// memory, to the rows that see them.
//
// Measured: 64 tokens over 1024 to 8190 slots, 32 heads on 8 of 128, e4m3 pool (602 MB):
// 108.5 us, 5550 GB/s, bounded by DRAM and about 10 us of start and tail (4.2 GB of
// cache: 6580 GB/s); 64 sequences of 1 to 4 tokens, cap, window 4096, bf16 pool (935 MB):
// 172 us, 5430 GB/s, bounded by a tile's softmax chain with three stages an SM.
#include <algorithm>
#include <type_traits>

#include "kvc_paged_tc.cuh"

namespace kvc {
namespace {

constexpr int kTS = 128;
// SG groups of 4 softmax warps (each takes NR / SG of the unit's rows for all 128
// slots), then the S issuer, the P.V issuer, the producer and the scheduler.
template <int SG>
struct Roles {
    static constexpr int soft = 4 * SG, s = soft, pv = soft + 1, prod = soft + 2;
    static constexpr int threads = (soft + 4) * 32;
};
struct Bars {
    uint32_t base;
    __device__ uint32_t full(int s) const { return base + 8u * s; }
    __device__ uint32_t empty(int s) const { return base + 64u + 8u * s; }
    __device__ uint32_t item_full(int k) const { return base + 128u + 8u * k; }
    __device__ uint32_t item_empty(int k) const { return base + 160u + 8u * k; }
    __device__ uint32_t s_ready(int b) const { return base + 192u + 8u * b; }
    __device__ uint32_t s_free(int b) const { return base + 208u + 8u * b; }
    __device__ uint32_t p_ready(int b) const { return base + 224u + 8u * b; }
    __device__ uint32_t o_done(int b) const { return base + 240u + 8u * b; }
    __device__ uint32_t meet(int g) const { return base + 256u + 8u * g; }
    __device__ uint32_t drained() const { return base + 272u; }
    // the run is known (its query rows are not ready yet)
    __device__ uint32_t item_known(int k) const { return base + 280u + 8u * k; }
};
constexpr int kTmemSlot = 312, kAbort = 316, kBad = 320 /* [4] */, kOdd = 336 /* [2] */;
// from 512: PagedStart (read before the first tile is loaded), then the stages'
// StageScales; then the items and their rows' data

// What a run holds besides the query rows: per row the factor of its
// products, its position (-1: no row) and its bias slope (times log2 e).
struct RowData {
    float mul[32];  // (16 rows; a whole warp writes the rest)
    int lim[32];
    float slope[32];
};

constexpr int DN = 16;  // a unit's rows padded: N of the products
template <int EB>
struct Shape {
    static constexpr int kWParts = EB == 1 ? 3 : 1;        // of a weight
    static constexpr int nblk = DN * 128;                  // a 128-byte column block of Q or P^T
    static constexpr int pblks = EB == 1 ? 1 : 2;          // column blocks of 128 weights
    static constexpr int pbytes = kWParts * pblks * nblk;  // one P^T buffer
    static constexpr int npt = EB == 2 ? 2 : 1;  // P^T buffers (one leaves 8-bit pools a third stage)
    static constexpr uint32_t col_o = 2 * DN;
    static constexpr uint32_t cols = 64;
};

template <int NR, bool MAX>
__device__ __forceinline__ float reduce_rows(const float (&v)[NR]) {
    // reduce-scatter over the warp: row (lane >> (5 - log2 NR))'s result
    const int lane = threadIdx.x & 31;
    float a[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) a[i] = v[i];
    int o = 16;
#pragma unroll
    for (int h = NR / 2; h >= 1; h /= 2, o /= 2) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float keep = up ? a[i + h] : a[i];
            const float send = up ? a[i] : a[i + h];
            const float got = __shfl_xor_sync(0xffffffffu, send, o);
            a[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
#pragma unroll
    for (; o >= 1; o /= 2) {
        const float got = __shfl_xor_sync(0xffffffffu, a[0], o);
        a[0] = MAX ? fmaxf(a[0], got) : a[0] + got;
    }
    return a[0];
}

template <typename T, int EB>
__device__ void sched_warp(const PagedTcParams& p, unsigned char* smem, Bars bars,
                           const PagedStart* st, volatile int* abort) {
    using S = Shape<EB>;
    const PagedAttendParams& a = p.a;
    const int lane = threadIdx.x & 31;
    PagedItem* items = reinterpret_cast<PagedItem*>(smem + p.off_item);
    const int nkb = (a.D * EB + 127) / 128;
    PagedWalk<kTS> w;
    w.start(p, st);
    const int before = w.tt - w.lead;  // of the unit's tiles, in earlier blocks
    PagedItem it;
    int unit_tiles = 0;
    bool more = w.next(p, it, unit_tiles);
    if (lane == 0)
        paged_record(p, more && !(it.flags & kItemBegins) ? &it : nullptr, before, unit_tiles, w.per);
    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (k >= p.ni &&
            !warp_wait(bars.item_empty(kb), static_cast<uint32_t>((k / p.ni - 1) & 1), abort))
            return;
        if (!more) {
            if (lane == 0) {
                items[kb].flags = kItemDone;
                mbar_arrive(bars.item_known(kb), 1u);
                mbar_arrive(bars.item_full(kb), 1u);
            }
            return;
        }
        unsigned char* sq = smem + p.off_q + kb * p.q_bytes;
        RowData* rd = reinterpret_cast<RowData*>(smem + p.off_item + 128) + kb;
        const int R = it.S * a.G;
        if (lane == 0) {
            items[kb] = it;
            *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 0;
            mbar_arrive(bars.item_known(kb), 1u);
        }
        {
            const int r = it.r0 + lane;
            const bool live = lane < p.RG && r < R;
            rd->lim[lane] = live ? it.K - it.S + r / a.G : -1;
            rd->slope[lane] = live && a.slopes ? a.slopes[it.hk * a.G + r % a.G] * kLog2e : 0.f;
        }
        prepare_rows<T, EB, DN, 32>(p, it, sq, nkb, S::nblk, lane, rd->mul);
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
    const uint32_t stage0 = smem_addr(smem + p.off_stage);
    StageScales* sc = reinterpret_cast<StageScales*>(smem + 512);
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + p.off_item);
    const int nkb = (a.D * EB + 127) / 128;
    const int nvb = EB == 1 ? 1 : 2;  // value columns padded to 128: the boxes past them read zeros
    int issued = 0;
    Ring ring;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_known(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) break;
        int id = feed_id<kTS>(p, it, it.tile0);
        int id1 = it.nt > 1 ? feed_id<kTS>(p, it, it.tile0 + 1) : kNoBox;
        float fs = 1.f, fs1 = 1.f;
        if (EB == 1) fs = feed_scale(p, it, id);
        for (int n = 0; n < it.nt; ++n) {
            const int tile = it.tile0 + n;
            const int id2 = n + 2 < it.nt ? feed_id<kTS>(p, it, tile + 2) : kNoBox;
            if (EB == 1) fs1 = feed_scale(p, it, id1);
            if (issued >= p.ns && !warp_wait(bars.empty(ring.s), ring.ph ^ 1u, abort)) {
                ok = false;
                break;
            }
            if (__any_sync(0xffffffffu, feed_bad(p, id)) && lane == 0) {
                *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) = 1;
                if (a.status) atomicOr(a.status, KVC_DEV_OVERFLOW);
            }
            if (EB == 1) feed_store(sc + ring.s, fs);
            const uint32_t sK = stage0 + static_cast<uint32_t>(ring.s) * p.stage_bytes;
            feed_copy<EB, kTS>(p, it, tile, id, sK, nkb, sK + static_cast<uint32_t>(nkb * kTS * 128), nvb,
                               bars.full(ring.s));
            id = id1;
            id1 = id2;
            fs = fs1;
            ++issued;
            ring.next(p.ns);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.item_empty(kb), 1u);
    }
    // do not leave while issued copies may still write shared memory
    if (lane == 0)
        for (int q = issued > p.ns ? issued - p.ns : 0; q < issued; ++q)
            mbar_drain(bars.full(q % p.ns), static_cast<uint32_t>((q / p.ns) & 1));
}

// One warp: S^T of every tile.
template <typename T, int EB>
__device__ void s_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                         uint32_t tmem) {
    using S = Shape<EB>;
    const PagedAttendParams& a = p.a;
    const uint32_t stage0 = smem_addr(smem + p.off_stage);
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + p.off_item);
    const int nkb = (a.D * EB + 127) / 128;
    const int ksteps = (a.D * EB + 31) / 32;  // 32 bytes of a row per instruction
    const uint32_t idesc = EB == 1 ? mma_idesc_f8(kTS, DN, a.e5m2, false, false, false)
                                   : mma_idesc_f16(kTS, DN, std::is_same<T, __nv_bfloat16>::value,
                                                   false, false);
    Ring ring;
    int c = 0;  // tiles so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (uniform(items[kb].flags) & kItemDone) break;
        const int nt = uniform(items[kb].nt);
        const uint32_t sQ = smem_addr(smem + p.off_q + kb * p.q_bytes);
        for (int n = 0; n < nt; ++n, ++c) {
            const int sb = c & 1;
            if (!warp_wait(bars.full(ring.s), ring.ph, abort) ||
                (c >= 2 && !warp_wait(bars.s_free(sb), static_cast<uint32_t>((c / 2 - 1) & 1), abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sK = stage0 + static_cast<uint32_t>(ring.s) * p.stage_bytes;
            if (elect_one()) {
                for (int b = 0; b < nkb; ++b) {
                    // column block b of both; 32 bytes of a row per instruction, 2 in
                    // the descriptor's address field
                    const uint64_t da = smem_desc_sw128(sK + b * kTS * 128, 16, 1024);
#pragma unroll
                    for (int part = 0; part < QueryParts<T, EB>::v; ++part) {
                        const uint64_t db = smem_desc_sw128(sQ + (part * nkb + b) * S::nblk, 16, 1024);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (4 * b + i >= ksteps) break;
                            if (EB == 1)
                                tc_mma_f8(tmem + sb * DN, da + 2 * i, db + 2 * i, idesc, (b | part | i) != 0);
                            else
                                tc_mma(tmem + sb * DN, da + 2 * i, db + 2 * i, idesc, (b | i) != 0);
                        }
                    }
                }
                tc_commit(bars.s_ready(sb));
            }
            __syncwarp();
            ring.next(p.ns);
        }
        if (ok && elect_one()) tc_commit(bars.item_empty(kb));  // once the products have read the query rows
    }
    if (elect_one()) tc_commit(bars.drained());
    __syncwarp();
    volatile int never = 0;
    warp_wait(bars.drained(), 0u, &never);
}

// One warp: O^T += V^T P^T of every tile; releases the stages.
template <typename T, int EB>
__device__ void pv_issuer(const PagedTcParams& p, unsigned char* smem, Bars bars, volatile int* abort,
                          uint32_t tmem) {
    using S = Shape<EB>;
    const PagedAttendParams& a = p.a;
    const uint32_t stage0 = smem_addr(smem + p.off_stage);
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + p.off_item);
    const int nkb = (a.D * EB + 127) / 128;
    const uint32_t idesc = EB == 1 ? mma_idesc_f8(128, DN, a.e5m2, true, true, false)
                                   : mma_idesc_f16(128, DN, std::is_same<T, __nv_bfloat16>::value, false,
                                                   true);
    Ring ring;
    int c = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) break;
        if (uniform(items[kb].flags) & kItemDone) break;
        const int nt = uniform(items[kb].nt);
        for (int n = 0; n < nt; ++n, ++c) {
            const int pb = c % S::npt;
            if (!warp_wait(bars.full(ring.s), ring.ph, abort) ||
                !warp_wait(bars.p_ready(pb), static_cast<uint32_t>((c / S::npt) & 1), abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sV = stage0 + static_cast<uint32_t>(ring.s) * p.stage_bytes +
                                static_cast<uint32_t>(nkb * kTS * 128);
            const uint32_t sP = smem_addr(smem + p.off_p) + pb * S::pbytes;
            if (elect_one()) {
                const uint64_t da = smem_desc_sw128(sV, kTS * 128, 1024);
                const uint64_t db = smem_desc_sw128(sP, 16, 1024);
                const uint32_t tO = tmem + S::col_o;
                if (EB == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 slots per step
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            tc_mma_f8(tO, da + i * (32 * 128 / 16), db + part * (S::nblk / 16) + 2 * i,
                                      idesc, (n | part | i) != 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 slots per step
                        tc_mma(tO, da + i * (16 * 128 / 16), db + (i >> 2) * (S::nblk / 16) + 2 * (i & 3),
                               idesc, (n | i) != 0);
                }
                tc_commit(bars.o_done(pb));
                tc_commit(bars.empty(ring.s));
            }
            __syncwarp();
            ring.next(p.ns);
        }
        if (ok && elect_one()) mbar_arrive(bars.item_empty(kb), 1u);
        __syncwarp();
    }
    if (elect_one()) tc_commit(bars.drained());
    __syncwarp();
    volatile int never = 0;
    warp_wait(bars.drained(), 0u, &never);
}

template <typename T, int EB, int NRT, int SG, bool MOD>
__device__ void softmax_warps(const PagedTcParams& p, unsigned char* smem, Bars bars,
                              volatile int* abort, uint32_t tmem, const PagedStart* st) {
    constexpr int NR = NRT / SG;  // rows of this thread's group
    using S = Shape<EB>;
    using St = Storage<T>;
    const PagedAttendParams& a = p.a;
    const int t = threadIdx.x & 127;  // slot of the tile; value column of O^T
    const int g = threadIdx.x >> 7, r0 = g * NR;  // group, its first row
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16) + r0;
    const PagedItem* items = reinterpret_cast<const PagedItem*>(smem + p.off_item);
    const StageScales* scales = reinterpret_cast<const StageScales*>(smem + 512);
    // the group's exchange: values [2][NR][4], flags [2][4]
    float* xval = reinterpret_cast<float*>(smem + p.off_x + g * (2 * NR * 16 + 32));
    int* xflag = reinterpret_cast<int*>(xval + 2 * NR * 4);
    unsigned char* pt = smem + p.off_p;
    const int nkb = (a.D * EB + 127) / 128;
    constexpr int nvb = EB == 1 ? 1 : 2;
    constexpr int kGroup = 32 / NR;  // lanes that end a reduction with one row
    const int box = 31 - __clz(p.hh);
    Ring ring;
    int c = 0;        // tiles so far
    uint32_t rv = 0;  // meetings so far
    float mref[NR], lsum[NR];

    // The 4 warps meet (a bounded wait, unlike bar.sync); what each wrote to
    // exchange buffer rv % 2 before is visible to all after.
    auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.meet(g), 1u);
        const bool ok = warp_wait(bars.meet(g), rv & 1u, abort);
        ++rv;
        return ok;
    };
    auto wait_pv = [&](int i) -> bool {  // product i has finished
        return warp_wait(bars.o_done(i % S::npt), static_cast<uint32_t>((i / S::npt) & 1), abort);
    };
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f;
    const float cap_out = a.softcap * kLog2e;

    for (int k = 0;; ++k) {
        const int kb = k % p.ni;
        if (!warp_wait(bars.item_full(kb), static_cast<uint32_t>((k / p.ni) & 1), abort)) return;
        const PagedItem it = items[kb];
        if (it.flags & kItemDone) return;
        const RowData* rd = reinterpret_cast<const RowData*>(smem + p.off_item + 128) + kb;
        // set behind this run's first meeting, read behind its last
        volatile int* odd = reinterpret_cast<volatile int*>(smem + kOdd + 4 * (k & 1));
        if (threadIdx.x == 0) *odd = 0;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            mref[r] = -INFINITY;
            lsum[r] = 0.f;
        }
        for (int n = 0; n < it.nt; ++n, ++c) {
            const int sb = c & 1;
            if (!warp_wait(bars.full(ring.s), ring.ph, abort) ||
                !warp_wait(bars.s_ready(sb), static_cast<uint32_t>((c / 2) & 1), abort))
                return;
            tc_fence_after();
            float sv[NR];
            tmem_ldn<NR>(trow + sb * DN, sv);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.s_free(sb), 1u);
            float ksc = 1.f, ivs = 1.f, lv = 0.f;  // key scale, 1 / value scale, its log2
            if (EB == 1) {
                const float4 kv = scales[ring.s].kv[t >> box];
                ksc = kv.x;
                lv = kv.z;
                ivs = kv.w;
            }
            const int j0 = (it.tile0 + n) * kTS, j = j0 + t;
            // a tile with a slot that some row does not see
            const bool edge = j0 + kTS - 1 > it.first || (a.window > 0 && j0 <= it.last - a.window);
            if (!MOD) ksc *= kLog2e;
            uint32_t seen = 0xffffffffu;
            if (edge) {
                seen = 0u;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int lim = rd->lim[r0 + r];
                    if (j <= lim && (a.window == 0 || j > lim - a.window)) seen |= 1u << r;
                }
            }
            bool need = false;
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const float4 m4 = *reinterpret_cast<const float4*>(rd->mul + r0 + r);
                const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = sv[r + e] * (m[e] * ksc);
                    if (MOD) {
                        if (a.softcap > 0.f) {
                            // cap tanh(s / cap) = cap (1 - 2 / (1 + e^(2 s / cap)))
                            const float ex = fast_exp2(s * cap_in);
                            s = cap_out - __fdividef(2.f * cap_out, 1.f + ex);
                            if (!(ex < INFINITY)) s = ex == ex ? cap_out : ex;
                        } else {
                            s *= kLog2e;
                        }
                        s -= rd->slope[r0 + r + e] * static_cast<float>(rd->lim[r0 + r + e] - j);
                    }
                    s += lv;
                    if (!((seen >> (r + e)) & 1u)) s = -INFINITY;
                    sv[r + e] = s;
                    need |= s > mref[r + e] + RaiseAbove<EB>::v;
                }
            }
            // the references are raised for the whole tile or not at all
            const uint32_t bf = rv & 1u;
            const int wneed = __any_sync(0xffffffffu, need);
            if (lane == 0) xflag[bf * 4 + warp] = wneed;
            if (!meet()) return;
            const int4 fl = *reinterpret_cast<const int4*>(xflag + bf * 4);
            bool rescale = false;
            float corr[NR];
            if (fl.x | fl.y | fl.z | fl.w) {
                const uint32_t bm = rv & 1u;
                const float mine = reduce_rows<NR, true>(sv);
                if ((lane & (kGroup - 1)) == 0) xval[(bm * NR + lane / kGroup) * 4 + warp] = mine;
                if (!meet()) return;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float4 q4 = *reinterpret_cast<const float4*>(xval + (bm * NR + r) * 4);
                    const float top = fmaxf(fmaxf(q4.x, q4.y), fmaxf(q4.z, q4.w));
                    corr[r] = 1.f;
                    if (top > mref[r] + RaiseAbove<EB>::v) {
                        if (mref[r] != -INFINITY) {
                            corr[r] = fast_exp2(mref[r] - top);
                            rescale = true;
                        }
                        lsum[r] *= corr[r];
                        mref[r] = top;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                // a row that saw nothing yet has no reference: every slot of it is masked
                sv[r] = sv[r] == -INFINITY ? 0.f : fast_exp2(sv[r] - mref[r] + kWeightOffset);
                lsum[r] = EB == 1 ? fmaf(sv[r], ivs, lsum[r]) : lsum[r] + sv[r];
            }
            if (c >= S::npt && !wait_pv(c - S::npt)) return;
            unsigned char* pb = pt + (c % S::npt) * S::pbytes;
            if (EB == 1) {
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    uint32_t part[3];
                    split_weights(sv[r], sv[r + 1], sv[r + 2], sv[r + 3], part);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int rr = r0 + r + e;
                        unsigned char* o = pb + rr * 128 + (((t >> 4) ^ (rr & 7)) << 4) + (t & 15);
#pragma unroll
                        for (int k2 = 0; k2 < 3; ++k2)
                            o[k2 * S::nblk] = static_cast<unsigned char>(part[k2] >> (8 * e));
                    }
                }
            } else {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    *reinterpret_cast<T*>(pb + (t >> 6) * S::nblk + (r0 + r) * 128 +
                                          ((((t & 63) >> 3) ^ ((r0 + r) & 7)) << 4) + (t & 7) * 2) =
                        St::from_float(sv[r]);
            }
            if (edge && g == 0) {
                unsigned char* vrow = smem + p.off_stage + static_cast<int64_t>(ring.s) * p.stage_bytes +
                                      nkb * kTS * 128 + t * 128;
                const bool some_see = j <= it.last && j >= it.lo;
                const bool all_see = j <= it.first && (a.window == 0 || j > it.last - a.window);
                if (!all_see && clean_value_row<EB, T>(vrow, nvb, kTS * 128, some_see, a.e5m2)) *odd = 1;
            }
            if (rescale && n > 0) {
                // O^T is at rest: the previous product has finished, this tile's
                // waits for p_ready
                if (!wait_pv(c - 1)) return;
                tc_fence_after();
                float ov[NR];
                tmem_ldn<NR>(trow + S::col_o, ov);
#pragma unroll
                for (int r = 0; r < NR; ++r) ov[r] *= corr[r];
                tmem_stn<NR>(trow + S::col_o, ov);
            }
            fence_async_shared();  // the weights and cleared value rows, for the tensor cores
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.p_ready(c % S::npt), 1u);
            ring.next(p.ns);
        }
        // the run's end: O^T column r is row r's weighted values
        if (!wait_pv(c - 1)) return;
        tc_fence_after();
        float ov[NR];
        tmem_ldn<NR>(trow + S::col_o, ov);
        tc_fence_before();
        const uint32_t bm = rv & 1u;
        const float mine = reduce_rows<NR, false>(lsum);
        if ((lane & (kGroup - 1)) == 0) xval[(bm * NR + lane / kGroup) * 4 + warp] = mine;
        if (!meet()) return;
        if (*odd && t < a.Dv) {  // what was cleared: from memory, into the rows that see it
            const int j1 = min(it.last, (it.tile0 + it.nt) * kTS - 1);
            for (int j = max(it.lo, it.tile0 * kTS); j <= j1; ++j) {
                if (j <= it.first && (a.window == 0 || j > it.last - a.window)) {
                    // seen by all: to the next slot that is not (behind the first row, if any)
                    j = max(j, it.first);
                    continue;
                }
                const int id = a.table[it.b * a.max_blocks + j / a.bs];
                if (id < 0 || id >= a.num_blocks) continue;
                const int64_t e = ((static_cast<int64_t>(id) * a.Hk + it.hk) * a.bs + j % a.bs) * a.Dv + t;
                const float v = EB == 1 ? from_eight(static_cast<const uint8_t*>(a.vp)[e], a.e5m2)
                                        : St::to_float(static_cast<const T*>(a.vp)[e]);
                if (fabsf(v) < INFINITY) continue;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int lim = rd->lim[r0 + r];
                    if (j <= lim && (a.window == 0 || j > lim - a.window)) ov[r] += v;
                }
            }
        }
        const bool bad = *reinterpret_cast<volatile int*>(smem + kBad + 4 * kb) != 0;
        const bool whole = (it.flags & kItemBegins) && (it.flags & kItemEnds);
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + ((it.flags & kItemBegins) ? 1 : 0);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int lim = rd->lim[r0 + r];
            if (lim < 0) continue;
            const float4 q4 = *reinterpret_cast<const float4*>(xval + (bm * NR + r) * 4);
            const float l = (q4.x + q4.y) + (q4.z + q4.w);
            if (whole) {
                const int rr = it.r0 + r0 + r;
                const int64_t row = static_cast<int64_t>(it.q0 + rr / a.G) * a.Hq + it.hk * a.G + rr % a.G;
                if (t < a.Dv)
                    static_cast<T*>(a.out)[row * a.Dv + t] =
                        St::from_float(bad ? 0.f : __fdiv_rn(ov[r], l));
            } else {
                if (t < a.Dv) p.part_acc[(slot * p.RG + r0 + r) * a.Dv + t] = ov[r];
                if (t == r) {
                    p.part_ml[2 * (slot * p.RG + r0 + r)] = mref[r];
                    p.part_ml[2 * (slot * p.RG + r0 + r) + 1] = bad ? -1.f : l;
                }
            }
        }
        // the run's row data and flags are read; the next meeting or product
        // does not reuse them before every warp has arrived here
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.item_empty(kb), 1u);
    }
}

template <typename T, int EB, int NR, int SG, bool MOD>
__global__ void __launch_bounds__(Roles<SG>::threads, EB == 1 ? 2 : 1)
    paged_decode_kernel(const __grid_constant__ PagedTcParams p) {
    using S = Shape<EB>;
    using R = Roles<SG>;
    constexpr int kThreads = R::threads;
    extern __shared__ __align__(1024) unsigned char smem[];
    const Bars bars{smem_addr(smem)};
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kAbort);
    PagedStart* st = reinterpret_cast<PagedStart*>(smem + 512);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.ns; ++s) {
            mbar_init(bars.full(s), 1u);
            mbar_init(bars.empty(s), 1u);
        }
        for (int k = 0; k < p.ni; ++k) {
            mbar_init(bars.item_known(k), 1u);
            mbar_init(bars.item_full(k), 1u);
            mbar_init(bars.item_empty(k), 3u + R::soft);  // producer, both issuers, softmax warps
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bars.s_ready(b), 1u);
            mbar_init(bars.s_free(b), R::soft);
            mbar_init(bars.p_ready(b), R::soft);
            mbar_init(bars.o_done(b), 1u);
        }
        for (int g = 0; g < SG; ++g) mbar_init(bars.meet(g), 4u);
        mbar_init(bars.drained(), 2u);
        *abort = 0;
        fence_mbar_init();
        prefetch_map(&p.tk);
        prefetch_map(&p.tv);
    }
    // weights of rows past the unit's stay zero: clear the buffers once
    for (int i = threadIdx.x; i < S::npt * S::pbytes / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem + p.off_p)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_async_shared();
    if (warp == R::s) {
        tmem_alloc(smem_addr(smem + kTmemSlot), S::cols);
        tmem_relinquish();
    }
    tc_fence_before();
    paged_plan<T, kTS, kThreads>(p, st);  // with block barriers
    tc_fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile int*>(smem + kTmemSlot));
    launch_dependents();

    if (warp < R::soft) {
        softmax_warps<T, EB, NR, SG, MOD>(p, smem, bars, abort, tmem, st);
    } else if (warp == R::s) {
        s_issuer<T, EB>(p, smem, bars, abort, tmem);
    } else if (warp == R::pv) {
        pv_issuer<T, EB>(p, smem, bars, abort, tmem);
    } else if (warp == R::prod) {
        producer_warp<EB>(p, smem, bars, abort);
    } else {
        sched_warp<T, EB>(p, smem, bars, st, abort);
    }
    tc_fence_before();
    __syncthreads();  // every thread reaches this exactly once: all waits are bounded
    if (warp == R::s) {
        tc_fence_after();
        tmem_dealloc(tmem, S::cols);
    }
    if (threadIdx.x == 0 && *abort && p.a.status) atomicOr(p.a.status, KVC_DEV_TIMEOUT);
}

// Block (c, y): the unit whose second block is c, 8 / WPR of its rows. WPR warps
// take a row's partials in turn, a lane four value columns, eight loads under way.
constexpr int kMergeWarps = 8;
template <typename T, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ PagedTcParams p) {
    __shared__ float4 sh[kMergeWarps][32];
    __shared__ float shl[kMergeWarps];
    grid_dependency_wait();
    const PagedAttendParams& a = p.a;
    const PagedRec rec = p.rec[blockIdx.x];
    if (!rec.valid || static_cast<int>(blockIdx.x) != rec.c0 + 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * (kMergeWarps / WPR) + warp / WPR, part = warp % WPR;
    const int n = rec.c1 - rec.c0 + 1;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    auto slot = [&](int k) -> int64_t {
        return (2 * static_cast<int64_t>(rec.c0 + k) + (k == 0 ? 1 : 0)) * p.RG + r;
    };
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int bad = 0;
    if (r < rec.rows) {
        float m = -INFINITY;
        for (int k = lane; k < n; k += 32) {
            const float2 x = ml[slot(k)];
            if (x.y < 0.f) bad = 1;
            if (x.y != 0.f) m = fmaxf(m, x.x);
        }
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        bad = __any_sync(0xffffffffu, bad);
        constexpr int kAhead = 8;
        for (int k0 = part; k0 < n; k0 += kAhead * WPR) {
            float4 v[kAhead];
            float2 x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = k0 + i * WPR;
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                x[i] = make_float2(0.f, 0.f);
                if (k < n) {
                    x[i] = ml[slot(k)];
                    if (4 * lane < a.Dv)
                        v[i] = *reinterpret_cast<const float4*>(p.part_acc + slot(k) * a.Dv + 4 * lane);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (x[i].y == 0.f) continue;
                const float f = x[i].x == m ? 1.f : fast_exp2(x[i].x - m);
                l = fmaf(x[i].y, f, l);
                acc.x = fmaf(v[i].x, f, acc.x);
                acc.y = fmaf(v[i].y, f, acc.y);
                acc.z = fmaf(v[i].z, f, acc.z);
                acc.w = fmaf(v[i].w, f, acc.w);
            }
        }
    }
    if (WPR > 1) {
        sh[warp][lane] = acc;
        if (lane == 0) shl[warp] = l;
        __syncthreads();
        if (part != 0) return;
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
            const float4 v = sh[warp + w][lane];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
            l += shl[warp + w];
        }
    }
    if (r < rec.rows && 4 * lane < a.Dv) {
        const int rr = rec.r0 + r;
        const int64_t row = static_cast<int64_t>(rec.q0 + rr / a.G) * a.Hq + rec.hk * a.G + rr % a.G;
        T* o = static_cast<T*>(a.out) + row * a.Dv + 4 * lane;
        const float x[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = Storage<T>::from_float(bad ? 0.f : __fdiv_rn(x[e], l));
    }
}

template <typename T, int EB, int NR, int SG, bool MOD>
cudaError_t launch_t(const PagedTcParams& p, size_t smem, cudaStream_t stream) {
    auto kern = paged_decode_kernel<T, EB, NR, SG, MOD>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern));
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.ctas), Roles<SG>::threads, smem, stream>>>(p);
    return cudaGetLastError();
}
template <typename T, int EB, int NR>
cudaError_t launch_nr(const PagedTcParams& p, size_t smem, cudaStream_t stream) {
    // where a block has the SM to itself, two softmax groups from 8 rows on (an 8-bit
    // pool's two blocks an SM cover each other's softmax, 4 rows are too few to divide)
    constexpr int SG = EB == 2 && NR >= 8 ? 2 : 1;
    return p.a.softcap > 0.f || p.a.slopes ? launch_t<T, EB, NR, SG, true>(p, smem, stream)
                                           : launch_t<T, EB, NR, SG, false>(p, smem, stream);
}
template <typename T, int EB>
cudaError_t launch_eb(const PagedTcParams& p, int nr, size_t smem, cudaStream_t stream) {
    switch (nr) {
        case 4: return launch_nr<T, EB, 4>(p, smem, stream);
        case 8: return launch_nr<T, EB, 8>(p, smem, stream);
        default: return launch_nr<T, EB, 16>(p, smem, stream);
    }
}

}  // namespace

cudaError_t launch_paged_decode(const PagedTcParams& p, int dtype, int pool_dtype, int nr,
                                size_t smem, cudaStream_t stream) {
    if (pool_dtype == dtype)
        return dtype == KVC_BF16 ? launch_eb<__nv_bfloat16, 2>(p, nr, smem, stream)
                                 : launch_eb<__half, 2>(p, nr, smem, stream);
    return dtype == KVC_BF16 ? launch_eb<__nv_bfloat16, 1>(p, nr, smem, stream)
                             : launch_eb<__half, 1>(p, nr, smem, stream);
}

template <typename T>
static cudaError_t launch_merge_t(const PagedTcParams& p, cudaStream_t stream) {
    // few rows: more warps for each (a long context's unit can have hundreds of partials)
    const int wpr = p.RG <= 16 ? 4 : 1, per = kMergeWarps / wpr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), static_cast<unsigned>((p.RG + per - 1) / per));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return wpr == 4 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 4>, p)
                    : cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, 1>, p);
}

cudaError_t launch_paged_merge(const PagedTcParams& p, int dtype, cudaStream_t stream) {
    if (p.ctas < 2) return cudaSuccess;
    return dtype == KVC_BF16 ? launch_merge_t<__nv_bfloat16>(p, stream)
                             : launch_merge_t<__half>(p, stream);
}

}  // namespace kvc
