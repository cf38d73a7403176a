// kvc_paged_tc.cuh -- what the tensor-core kernels of the paged attention
// share (kvc_paged_decode.cu, kvc_paged_rows.cu): the even split of the work, the
// tile producer and the tensor-core forms for 8-bit operands.
//
// Work. A unit is (sequence, group of up to RG query rows, KV head); rows r =
// t G + g of a KV head are grouped in order. Its tiles are the runs of TS slots
// (aligned to TS) from its first visible slot to its last. All units' tiles in
// order (sequence, group, head) are one list; block c of the grid takes tiles [c per,
// (c + 1) per). The start of a unit (its query rows, its first tile's latency, its
// result) counts as p.lead further tiles before the first, which no block works on
// (in a list that has a block for every tile, as none).
// Every block computes the list's length itself from cu_seqlens and seqlens_k (one
// pass over B sequences), so a call is one launch, whatever the lengths, and all blocks
// have about the same to do. A unit that lies
// within one block is finished there; of a unit cut between blocks each block
// leaves a partial (at most two per block: the tail of a unit in slot 0, the
// head of one in slot 1), which paged_merge_kernel joins.
#pragma once

#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "kvc_launch.h"
#include "kvc_paged.cuh"
#include "kvc_pipeline.cuh"
#include "kvc_tcgen05.cuh"

namespace kvc {

// A kernel's dynamic shared memory limit, raised to the block's most once per device.
struct SmemLimit {
    std::atomic<uint64_t> done{0};
    cudaError_t raise(const void* kern) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1u)) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
        return e;
    }
};

// D[tmem] (+)= A[smem] * B[smem], kind::f8f6f4: 8-bit operands (each of its
// own format), fp32 accumulate, 32 elements of K per instruction.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Instruction descriptor of a kind::f8f6f4 product with fp32 accumulation.
__device__ __forceinline__ uint32_t mma_idesc_f8(int M, int N, bool a_e5m2, bool b_e5m2,
                                                 bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) |
           ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// One lane of a converged warp. The issuing warps run as a whole, on values that
// are the same in all lanes, and only the tensor-core instructions stand behind
// this: their operands are then uniform registers. (Issued by a lone thread of a
// diverged warp, an instruction took 130 to 270 cycles, and the issue, not the products,
// bounded the kernels.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
// A value that all lanes hold, as one the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// The slots that query rows [r0, r0 + RG) of a sequence see, and their tiles.
struct PagedGroup {
    int first, last;  // positions of the group's first and last row
    int lo;           // first slot any of them sees (the last is `last`)
    int tile0, nt;
};
template <int TS>
__device__ __forceinline__ PagedGroup paged_group(const PagedTcParams& p, int S, int K, int i) {
    const PagedAttendParams& a = p.a;
    const int RG = p.RG;
    PagedGroup g;
    const int R = S * a.G, r0 = i * RG;
    g.first = K - S + r0 / a.G;
    g.last = K - S + (min(R, r0 + RG) - 1) / a.G;
    g.lo = a.window > 0 ? max(0, g.first - a.window + 1) : 0;
    g.tile0 = g.lo / TS;
    g.nt = g.last / TS - g.tile0 + 1;
    return g;
}
__device__ __forceinline__ int paged_groups(const PagedAttendParams& a, int RG, int S) {
    return (S * a.G + RG - 1) / RG;
}

// A run of tiles of one unit, as the scheduling warp hands it to the others.
struct PagedItem {
    int b, q0, S, K;
    int r0, hk;          // the group's first row, KV head
    int first, last, lo; // as PagedGroup
    int tile0, nt;       // the run
    int flags;
};
constexpr int kItemBegins = 1;  // the run starts the unit
constexpr int kItemEnds = 2;    // the run ends the unit
constexpr int kItemDone = 4;    // no more runs

// Where a block's run of the tile list starts, found by all threads of it.
constexpr int kPlanWarps = 20;  // of a block, at most
struct PagedStart {
    long long total, per;
    int lead;       // places of the list that a unit's start takes
    int b;          // sequence of the block's first place
    long long off;  // its place within the sequence
    long long sums[kPlanWarps];
    int units[kPlanWarps];
};
static_assert(sizeof(PagedStart) <= 320, "the kernels keep 320 bytes for it");

template <int TS>
__device__ __forceinline__ long long paged_seq_tiles(const PagedTcParams& p, int64_t b, int* invalid,
                                                      int* units) {
    const PagedAttendParams& a = p.a;
    const PagedSeq s = paged_seq(a.cu, a.kl, b, a.total_q, a.max_q, a.M);
    if (!s.ok) *invalid = 1;
    *units = 0;
    if (!s.ok || s.S == 0) return 0;
    long long n = 0;
    const int ng = paged_groups(a, p.RG, s.S);
    for (int i = 0; i < ng; ++i) n += paged_group<TS>(p, s.S, s.K, i).nt;
    *units = ng * a.Hk;
    return n * a.Hk;
}

// All threads; ends with a block barrier. Where a sequence lies outside the
// contract, block c also writes the zero rows of sequences c, c + grid, ...
template <typename T, int TS, int THREADS>
__device__ __forceinline__ void paged_plan(const PagedTcParams& p, PagedStart* st) {
    const PagedAttendParams& a = p.a;
    const int64_t B = a.B;
    const int64_t per_thread = (B + THREADS - 1) / THREADS;
    const int64_t b0 = min(B, threadIdx.x * per_thread), b1 = min(B, b0 + per_thread);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long mine = 0;
    int invalid = 0, mine_u = 0;
    for (int64_t b = b0; b < b1; ++b) {
        int u;
        mine += paged_seq_tiles<TS>(p, b, &invalid, &u);
        mine_u += u;
    }
    long long incl = mine;
    int incl_u = mine_u;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        const int u = __shfl_up_sync(0xffffffffu, incl_u, o);
        if (lane >= o) {
            incl += v;
            incl_u += u;
        }
    }
    static_assert(THREADS / 32 <= kPlanWarps, "a sum for every warp");
    if (lane == 31) {
        st->sums[warp] = incl;
        st->units[warp] = incl_u;
    }
    invalid = __syncthreads_or(invalid);
    long long before = 0, total = 0;
    int before_u = 0, total_u = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const long long v = st->sums[w];
        const int u = st->units[w];
        if (w < warp) {
            before += v;
            before_u += u;
        }
        total += v;
        total_u += u;
    }
    // a block for every tile: nothing to level, and each takes one
    const int lead = total <= p.ctas ? 0 : p.lead;
    total += static_cast<long long>(lead) * total_u;
    before += static_cast<long long>(lead) * (before_u + incl_u - mine_u);
    const long long tiles = mine;
    mine += static_cast<long long>(lead) * mine_u;
    const long long per = total < (1ll << 31)
                              ? (static_cast<uint32_t>(total) + p.ctas - 1) / static_cast<uint32_t>(p.ctas)
                              : (total + p.ctas - 1) / p.ctas;
    const long long at = static_cast<long long>(blockIdx.x) * per;
    long long cur = before + incl - tiles;
    if (threadIdx.x == 0) {
        st->total = total;
        st->per = per;
        st->lead = lead;
    }
    if (per_thread == 1 && at >= cur && at < cur + mine) {
        st->b = static_cast<int>(b0);
        st->off = at - cur;
    } else if (at >= cur && at < cur + mine) {
        for (int64_t b = b0; b < b1; ++b) {
            int u;
            long long n = paged_seq_tiles<TS>(p, b, &invalid, &u);
            n += static_cast<long long>(lead) * u;
            if (at < cur + n) {
                st->b = static_cast<int>(b);
                st->off = at - cur;
                break;
            }
            cur += n;
        }
    }
    if (invalid) {
        for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
            const PagedSeq s = paged_seq(a.cu, a.kl, b, a.total_q, a.max_q, a.M);
            if (s.ok) continue;
            if (threadIdx.x == 0 && a.status) atomicOr(a.status, KVC_DEV_OVERFLOW);
            const int64_t n = static_cast<int64_t>(s.S) * a.Hq * a.Dv;
            T* o = static_cast<T*>(a.out) + static_cast<int64_t>(s.q0) * a.Hq * a.Dv;
            for (int64_t i = threadIdx.x; i < n; i += THREADS) o[i] = Storage<T>::from_float(0.f);
        }
    }
    __syncthreads();
}

// The scheduling warp's walk over its block's runs (all lanes alike).
template <int TS>
struct PagedWalk {
    long long left = 0;  // places to hand out
    long long per = 1;
    int lead = 0;
    int b = 0, i = 0, hk = 0, tt = 0;  // next tile: sequence, group, head, tile of the unit
    PagedSeq s{};
    int ng = 0;

    __device__ void load(const PagedTcParams& p) {
        s = paged_seq(p.a.cu, p.a.kl, b, p.a.total_q, p.a.max_q, p.a.M);
        ng = s.ok ? paged_groups(p.a, p.RG, s.S) : 0;
    }
    __device__ void start(const PagedTcParams& p, const PagedStart* st) {
        per = st->per;
        lead = st->lead;
        left = min(per, st->total - static_cast<long long>(blockIdx.x) * per);
        if (left <= 0) return;
        b = st->b;
        load(p);
        // the group of tile `off`: 32 groups at a time
        long long off = st->off;
        const int lane = threadIdx.x & 31;
        for (i = 0;; i += 32) {
            long long n = 0;
            if (i + lane < ng)
                n = static_cast<long long>(paged_group<TS>(p, s.S, s.K, i + lane).nt + lead) * p.a.Hk;
            long long incl = n;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const uint32_t in = __ballot_sync(0xffffffffu, off < incl);
            if (in) {
                const int l = __ffs(in) - 1;
                off -= __shfl_sync(0xffffffffu, incl - n, l);
                i += l;
                break;
            }
            off -= __shfl_sync(0xffffffffu, incl, 31);
            if (i + 32 >= ng) {  // not reached: off lies within the sequence
                left = 0;
                return;
            }
        }
        const int n = paged_group<TS>(p, s.S, s.K, i).nt + lead;
        hk = off < (1ll << 31) ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(n))
                               : static_cast<int>(off / n);
        tt = static_cast<int>(off - static_cast<long long>(hk) * n);
    }
    // The next run into `it`; false at the end.
    __device__ bool next(const PagedTcParams& p, PagedItem& it, int& unit_tiles) {
        if (left <= 0) return false;
        while (ng == 0 || i >= ng) {
            ++b;
            if (b >= p.a.B) return false;
            i = 0;
            load(p);
        }
        const PagedGroup g = paged_group<TS>(p, s.S, s.K, i);
        const int take = static_cast<int>(min(static_cast<long long>(g.nt + lead - tt), left));
        left -= take;
        // its tiles among these places (none: they are the block's last)
        const int t0 = max(tt - lead, 0), t1 = tt + take - lead;
        if (t1 <= 0) return false;
        it.b = b; it.q0 = s.q0; it.S = s.S; it.K = s.K;
        it.r0 = i * p.RG; it.hk = hk;
        it.first = g.first; it.last = g.last; it.lo = g.lo;
        it.tile0 = g.tile0 + t0; it.nt = t1 - t0;
        it.flags = (t0 == 0 ? kItemBegins : 0) | (t1 == g.nt ? kItemEnds : 0);
        unit_tiles = g.nt;
        tt += take;
        if (tt == g.nt + lead) {
            tt = 0;
            if (++hk == p.a.Hk) {
                hk = 0;
                ++i;
            }
        }
        return true;
    }
};

// The record of a block whose first run continues a unit: which unit, and the
// blocks it lies in. Written for every block at every call.
__device__ __forceinline__ void paged_record(const PagedTcParams& p, const PagedItem* it, int before,
                                             int unit_tiles, long long per) {
    PagedRec r{};
    if (it) {
        // `before` of the unit's tiles lie in earlier blocks; each block has a run of per
        const uint32_t run = static_cast<uint32_t>(min(per, 1ll << 30));
        r.valid = 1;
        r.q0 = it->q0; r.r0 = it->r0; r.hk = it->hk;
        r.rows = min(p.RG, it->S * p.a.G - it->r0);
        r.c0 = static_cast<int>(blockIdx.x - (before + run - 1) / run);
        r.c1 = static_cast<int>(blockIdx.x + (unit_tiles - before - 1) / run);
    }
    p.rec[blockIdx.x] = r;
}

// Of each box of a tile: key scale, value scale, its log2 and its inverse.
constexpr int kMaxBoxes = 16;
struct StageScales {
    float4 kv[kMaxBoxes];
};

// What a producer warp feeds a run's tiles from: box `lane % 16` of a tile is hh
// slots of one pool block; lanes below 16 stand for its keys, the others for its values.
// Block ids are read two tiles ahead and scales one, so no tile waits for a look-up,
// and each lane issues its own box's copies (with the look-ups in line a tile took 1700
// cycles before its first copy went out; copies issued in turn by one lane, with the
// boxes' places handed round, took 1900 for four: either bounded the kernels).
constexpr int kNoBox = -0x7fffffff;  // the box holds no visible slot: not read
__device__ __forceinline__ int feed_box() { return threadIdx.x & 15; }
__device__ __forceinline__ bool feed_values() { return (threadIdx.x & 16) != 0; }

template <int TS>
__device__ __forceinline__ int feed_id(const PagedTcParams& p, const PagedItem& it, int tile) {
    const int at = feed_box() * p.hh, slot = tile * TS + at;
    if (at >= TS || slot + p.hh <= it.lo || slot > it.last) return kNoBox;
    return p.a.table[it.b * p.a.max_blocks + p.block_of(slot)];
}
__device__ __forceinline__ bool feed_bad(const PagedTcParams& p, int id) {
    return id != kNoBox && (id < 0 || id >= p.a.num_blocks);
}
// The box's key or value scale (of one that is not read: anything finite).
__device__ __forceinline__ float feed_scale(const PagedTcParams& p, const PagedItem& it, int id) {
    if (id < 0 || id >= p.a.num_blocks) return 1.f;
    const int64_t u = static_cast<int64_t>(id) * p.a.Hk + it.hk;
    return (feed_values() ? p.a.vs : p.a.ks)[u];
}
__device__ __forceinline__ void feed_store(StageScales* sc, float s) {
    float* kv = reinterpret_cast<float*>(&sc->kv[feed_box()]);
    if (!feed_values()) {
        kv[0] = s;
    } else {
        kv[1] = s;
        kv[2] = __log2f(s);
        kv[3] = __fdividef(1.f, s);
    }
}
// The copies of a tile's keys (nkb column blocks of 128 bytes for each box), values
// (nvb) or both (block 0 in place of a bad id), announced on `full`.
template <int EB, int TS>
__device__ __forceinline__ void feed_copy(const PagedTcParams& p, const PagedItem& it, int tile, int id,
                                          uint32_t sK, int nkb, uint32_t sV, int nvb, uint32_t full) {
    constexpr int kElems = 128 / EB;  // elements of a column block
    const bool values = feed_values();
    const int nb = values ? nvb : nkb;
    // (the vote also orders the lanes' scales before the arrive that publishes the tile)
    const int n = __popc(__ballot_sync(0xffffffffu, id != kNoBox && !values));
    if ((threadIdx.x & 31) == 0)
        mbar_arrive_expect_tx(full, static_cast<uint32_t>(n * (nkb + nvb) * p.hh * 128));
    __syncwarp();
    if (id != kNoBox) {
        const int at = feed_box() * p.hh, slot = tile * TS + at;
        const int y = slot - p.block_of(slot) * p.a.bs;
        const int z = (feed_bad(p, id) ? 0 : id) * p.a.Hk + it.hk;
        const uint32_t to = (values ? sV : sK) + static_cast<uint32_t>(at * 128);
        const CUtensorMap* map = values ? &p.tv : &p.tk;
        for (int k = 0; k < nb; ++k) tma_load_3d(to + k * TS * 128, map, kElems * k, y, z, full);
    }
    __syncwarp();
}

// Parts of a query element for the 8-bit products, e4m3 each: 4 + 4 significant bits
// hold a bfloat16, 4 + 4 + 4 an fp16 value (with two, fp16 scores were off by 2^-9
// of their terms, ten times the rounding of an fp16 result).
template <typename T, int EB>
struct QueryParts {
    static constexpr int v = EB == 2 ? 1 : std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
};

// A run's query rows into the swizzled operand layout, by THREADS threads, one or
// two for a row (rows past the unit's are zero). 8-bit products: the parts one after
// the other, of the row times the power of two that takes its largest element into
// [2^7, 2^8) (what is under 2^-17 of that is lost); mul[r] is the score scale over
// that power. (128 rows of 192: a warp for a row at a time needed a reduction and a
// division for each, 45 us. 128 rows of 128 take 18,000 cycles, most of them latency of the
// four warps' loads and conversions; eight threads a row, with four rows' or the next row's
// loads ahead, spilled and were slower: 34.0 against 32.6 us for a unit of 16 tiles.)
template <typename T, int EB, int ROWS, int THREADS>
__device__ __forceinline__ void prepare_rows(const PagedTcParams& p, const PagedItem& it,
                                             unsigned char* sq, int nkb, int blk, int tid, float* mul) {
    constexpr int kPerRow = THREADS / ROWS;
    static_assert(kPerRow == 1 || (kPerRow == 2 && THREADS == 32), "one thread for a row, or two lanes");
    const PagedAttendParams& a = p.a;
    const int r = tid % ROWS, part = tid / ROWS;
    const int R = min(p.RG, it.S * a.G - it.r0);
    const bool live = r < R;
    const int rr = it.r0 + (live ? r : 0), t = rr / a.G;
    const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(it.q0 + t) * a.q_tok +
                 (static_cast<int64_t>(it.hk) * a.G + (rr - t * a.G)) * a.q_head;
    const int nch = nkb * 8;  // 16-byte chunks of a row in shared memory
    unsigned char* dst = sq + r * 128;
    if (EB == 2) {
#pragma unroll 4
        for (int c = part; c < nch; c += kPerRow) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live && c * 8 < a.D) v = *reinterpret_cast<const uint4*>(q + c * 8);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * blk + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        if (mul && part == 0) mul[r] = a.scale;
        return;
    }
    // eight elements, in one load where every row starts on a 16-byte boundary
    const bool wide = ((reinterpret_cast<uintptr_t>(a.q) | static_cast<uintptr_t>(2 * a.q_tok) |
                        static_cast<uintptr_t>(2 * a.q_head)) & 15u) == 0u;
    auto words = [&](int d) {
        if (!live || d >= a.D) return make_uint4(0u, 0u, 0u, 0u);
        if (wide) return *reinterpret_cast<const uint4*>(q + d);
        const uint2 x = *reinterpret_cast<const uint2*>(q + d), y = *reinterpret_cast<const uint2*>(q + d + 4);
        return make_uint4(x.x, x.y, y.x, y.y);
    };
    constexpr uint32_t kInf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    // the largest magnitude, as its 16 bits, of either half of the words
    uint32_t top = 0;
#pragma unroll 4
    for (int c = part; c < 2 * nch; c += kPerRow) {
        const uint4 v = words(c * 8);
        const uint32_t m = 0x7fff7fffu;
        top = __vmaxu2(__vmaxu2(top, v.x & m), __vmaxu2(v.y & m, __vmaxu2(v.z & m, v.w & m)));
    }
    uint32_t big = max(top & 0xffffu, top >> 16);
    if (kPerRow == 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, 16));
    const bool odd = big >= kInf;  // infinities or NaN: the largest finite one
    if (__any_sync(0xffffffffu, odd)) {
        uint32_t fin = 0;
#pragma unroll 1
        for (int c = part; c < 2 * nch; c += kPerRow) {
            const uint4 v = words(c * 8);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const uint32_t x = (w[h >> 1] >> (16 * (h & 1))) & 0x7fffu;
                if (x < kInf) fin = max(fin, x);
            }
        }
        if (kPerRow == 2) fin = max(fin, __shfl_xor_sync(0xffffffffu, fin, 16));
        big = fin;
    }
    const unsigned short raw = static_cast<unsigned short>(big);
    const float bigf = Storage<T>::to_float(*reinterpret_cast<const T*>(&raw));
    int e2 = 7 - (static_cast<int>(__float_as_uint(bigf) >> 23) - 127);
    e2 = max(-120, min(120, e2));
    const float f = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
#pragma unroll 1
    for (int c = part; c < nch; c += kPerRow) {
        constexpr int NP = QueryParts<T, 1>::v;
        uint32_t w[NP][4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const uint4 v = words(c * 16 + e * 4);
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
            // in fp16, which holds the scaled elements down to 2^-32 of the largest
            __half2 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const T* x = reinterpret_cast<const T*>(&vw[k]);
                float y0 = Storage<T>::to_float(x[0]) * f, y1 = Storage<T>::to_float(x[1]) * f;
                if (odd) {  // no infinity: NaN
                    if (!(fabsf(y0) < INFINITY)) y0 = __uint_as_float(0x7fffffffu);
                    if (!(fabsf(y1) < INFINITY)) y1 = __uint_as_float(0x7fffffffu);
                }
                y[k] = __floats2half2_rn(y0, y1);
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[k] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(y[k]), __NV_SATFINITE,
                                                      __NV_E4M3);
                    if (n + 1 < NP)  // what is left, exactly
                        y[k] = __hsub2(y[k], __half2(__nv_cvt_fp8x2_to_halfraw2(
                                                 static_cast<__nv_fp8x2_storage_t>(h[k]), __NV_E4M3)));
                }
                w[n][e] = h[0] | (h[1] << 16);
                w[n][e + 1] = h[2] | (h[3] << 16);
            }
        }
        unsigned char* o = dst + (c >> 3) * blk + (((c & 7) ^ (r & 7)) << 4);
#pragma unroll
        for (int n = 0; n < NP; ++n)
            *reinterpret_cast<uint4*>(o + n * nkb * blk) = make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]);
    }
    if (part == 0) mul[r] = a.scale * __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
}

// Four weights as three e5m2 parts each (a word of four codes per part). e5m2
// is the upper byte of fp16, so from the weights in fp16 the first two parts are
// cut off by a mask, each difference is exact, and the last is rounded: 3 + 3 + 3
// significant bits. A weight from 2^-8 to 2^15.75 is off by at most 2^-9 of
// itself (and fp16's 2^-12), any other by 2^-17.
__device__ __forceinline__ void split_weights(float a, float b, float c, float d, uint32_t* part) {
    const __half2 w0 = __floats2half2_rn(a, b), w1 = __floats2half2_rn(c, d);
    const uint32_t m = 0xff00ff00u;
    const uint32_t u0 = *reinterpret_cast<const uint32_t*>(&w0);
    const uint32_t u1 = *reinterpret_cast<const uint32_t*>(&w1);
    const uint32_t h0 = u0 & m, h1 = u1 & m;
    const __half2 r0 = __hsub2(w0, *reinterpret_cast<const __half2*>(&h0));
    const __half2 r1 = __hsub2(w1, *reinterpret_cast<const __half2*>(&h1));
    const uint32_t v0 = *reinterpret_cast<const uint32_t*>(&r0);
    const uint32_t v1 = *reinterpret_cast<const uint32_t*>(&r1);
    const uint32_t g0 = v0 & m, g1 = v1 & m;
    const __half2 q0 = __hsub2(r0, *reinterpret_cast<const __half2*>(&g0));
    const __half2 q1 = __hsub2(r1, *reinterpret_cast<const __half2*>(&g1));
    part[0] = __byte_perm(u0, u1, 0x7531);
    part[1] = __byte_perm(v0, v1, 0x7531);
    part[2] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(q0), __NV_SATFINITE, __NV_E5M2) |
              (static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(q1),
                                                                __NV_SATFINITE, __NV_E5M2)) << 16);
}
// Of the 8-bit kernels a weight is 2^(s - ref + 8), and a row's reference is
// raised when a score exceeds it by more than 7.75: weights stay under e5m2's
// largest, 57344. 16-bit weights have the room of fp16 above 2^8.
constexpr float kWeightOffset = 8.f;
template <int EB>
struct RaiseAbove {
    static constexpr float v = EB == 1 ? 7.75f : 7.f;
};

// A word of 8- or 16-bit elements with those that are an infinity or NaN cleared.
template <int EB, typename T>
__device__ __forceinline__ uint32_t clear_odd(uint32_t w, bool e5m2) {
    uint32_t keep = 0xffffffffu;
    if (EB == 2) {
        const uint32_t inf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
        if ((w & 0x7fffu) >= inf) keep &= 0xffff0000u;
        if (((w >> 16) & 0x7fffu) >= inf) keep &= 0x0000ffffu;
    } else {
        const uint32_t inf = e5m2 ? 0x7cu : 0x7fu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (((w >> (8 * i)) & 0x7fu) >= inf) keep &= ~(0xffu << (8 * i));
    }
    return w & keep;
}

// Nonzero when one of a word's elements is an infinity or NaN.
template <int EB, typename T>
__device__ __forceinline__ uint32_t has_odd(uint32_t w, bool e5m2) {
    // the exponent (and for e4m3 the whole magnitude) all ones: one more carries out of it
    const uint32_t field = EB == 2 ? (std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u)
                                   : (e5m2 ? 0x7c7c7c7cu : 0x7f7f7f7fu);
    const uint32_t one = EB == 2 ? (std::is_same<T, __nv_bfloat16>::value ? 0x00800080u : 0x04000400u)
                                 : (e5m2 ? 0x04040404u : 0x01010101u);
    return ((w & field) + one) & (EB == 2 ? 0x80008000u : 0x80808080u);
}

// A slot's value row in shared memory (eight 16-byte chunks in each of nvb column
// blocks): cleared where no query row sees the slot, and of infinities and NaN where
// some do and some do not; true where there were any of those.
template <int EB, typename T>
__device__ __forceinline__ bool clean_value_row(unsigned char* row, int nvb, int block_bytes, bool some,
                                                bool e5m2) {
    bool found = false;
    for (int b = 0; b < nvb; ++b) {
        uint4* v = reinterpret_cast<uint4*>(row + b * block_bytes);
        if (!some) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 w = v[(i + threadIdx.x) & 7];
            any |= has_odd<EB, T>(w.x, e5m2) | has_odd<EB, T>(w.y, e5m2) | has_odd<EB, T>(w.z, e5m2) |
                   has_odd<EB, T>(w.w, e5m2);
        }
        if (any) {
            found = true;
            uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll 1
            for (int i = 0; i < 32; ++i) w[i] = clear_odd<EB, T>(w[i], e5m2);
        }
    }
    return found;
}

}  // namespace kvc
