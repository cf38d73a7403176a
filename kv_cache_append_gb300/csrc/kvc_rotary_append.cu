// kvc_rotary_append.cu -- append of packed new tokens to a paged pool, with the
// rotary position embedding applied on the way ("ClikaRT::ops::
// attention_over_cache" names RoPE and quantised-scale options of its cache;
// "Fixed-capacity KV cache", Task: append adds the new steps after the stored
// ones).
//
// Token t of sequence b sits at position j = K_b - S_b + t. The first R
// elements of a query or key row are R/2 pairs (x, y), turned by row j of the
// tables: (x cos - y sin, y cos + x sin); pairs are (d, d + R/2), or
// (2d, 2d + 1) when interleaved. The rest is copied.
//
// One launch: the first blocks rotate the queries (and, for pools of the
// inputs' type, write the keys and values, each a pure stream: every byte is
// read and written once); with an 8-bit pool the remaining blocks each take one
// (sequence, touched pool block, head, keys or values): a pass over the block's
// new rows for the largest absolute value, the block's scale, and a second pass
// that rounds and stores.
//
// 8-bit pools: the scale is 2^e, e the least with amax <= 1.75 * 2^top * 2^e,
// never below the scale of rows that the block already holds; a power of two
// makes x / scale exact, so each value is rounded once, and re-rounding held
// rows to a larger scale loses only bits below the format's subnormal step.
// A rotated value is formed exactly (two products as head and tail, their sum
// rounded to odd in fp32), so the one rounding to 8 bits is that of the exact
// value, whatever order or fusion the products are taken in.
//
// Measured (device time): one token 4.2 us and 64 tokens 4.9 us (7.9 us into an e4m3
// pool), the launch and two dependent look-ups; 9600 f16 prompt tokens, 32 query heads on 8
// of 128: 54.5 us, 4590 GB/s, bounded by each block's look-up before its one round of loads;
// 16600 tokens, 16 query heads on one of 192 into an e4m3 pool: 73.5 us, 3980 GB/s,
// bounded by the issue of the exact products and the barrier between the passes.
#include <algorithm>

#include "kvc_launch.h"
#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kAppThreads = 256;

// x*c - y*s, rounded to odd: nothing that a later rounding to 22 bits or fewer
// depends on is lost.
__device__ __forceinline__ float rot_odd(float x, float c, float y, float s) {
    const float p = __fmul_rn(x, c), pe = __fmaf_rn(x, c, -p);
    const float q = __fmul_rn(y, s), qe = __fmaf_rn(y, s, -q);
    const float d = __fsub_rn(p, q);
    if (!(fabsf(d) < INFINITY)) return d;
    const float bb = __fsub_rn(d, p);  // two-sum of p and -q: d + e exactly
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, bb)), __fadd_rn(q, bb));
    const float lo = __fadd_rn(e, __fsub_rn(pe, qe));
    const float hi = __fadd_rn(d, lo);
    const float r = __fsub_rn(lo, __fsub_rn(hi, d));
    uint32_t bits = __float_as_uint(hi);
    if (r != 0.f && (bits & 1u) == 0u) {
        if (hi == 0.f) return r;
        bits += ((r > 0.f) == (hi > 0.f)) ? 1u : 0xffffffffu;
    }
    return __uint_as_float(bits);
}

template <int BYTES>
struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<1> { using type = uint8_t; };

template <typename T, int VE>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
    using W = typename Word<VE * sizeof(T)>::type;
    const W w = *reinterpret_cast<const W*>(p);
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = Storage<T>::to_float(e[i]);
}
template <typename T, int VE>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
    using W = typename Word<VE * sizeof(T)>::type;
    W w;
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = Storage<T>::from_float(f[i]);
    *reinterpret_cast<W*>(p) = w;
}
template <int VE, bool E5M2>
__device__ __forceinline__ void store_eight(uint8_t* p, const float* f) {
    if constexpr (VE == 1) {
        *p = static_cast<uint8_t>(to_eight2<E5M2>(f[0], 0.f));
    } else {
        using W = typename Word<VE>::type;
        W w;
        uint16_t* h = reinterpret_cast<uint16_t*>(&w);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            h[i] = static_cast<uint16_t>(to_eight2<E5M2>(f[2 * i], f[2 * i + 1]));
        *reinterpret_cast<W*>(p) = w;
    }
}
template <int VE>
__device__ __forceinline__ void load_angles(const float* p, float* f) {
    if constexpr (VE % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VE; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = __ldg(p + i);
    }
}

// One job of a row: a chunk of VE pairs, rotated, at elements o0.. and o1..; or
// (behind the rotated part, and in value rows) one chunk of VE elements, copied
// (o1 < 0). EXACT: values rounded to odd.
template <typename T, int VE, bool EXACT>
__device__ __forceinline__ void row_job(const AppendParams& p, const T* src, int j, bool rotate,
                                        const float* cosr, const float* sinr, float* y, int& o0,
                                        int& o1) {
    const int h = p.half, npair = rotate ? h / VE : 0;
    if (j >= npair) {
        o0 = (rotate ? 2 * h : 0) + (j - npair) * VE;
        o1 = -1;
        load_vec<T, VE>(src + o0, y);
        return;
    }
    float x[2 * VE], c[VE], s[VE];
    o0 = p.interleaved ? 2 * j * VE : j * VE;
    o1 = p.interleaved ? o0 + VE : h + j * VE;
    load_vec<T, VE>(src + o0, x);
    load_vec<T, VE>(src + o1, x + VE);
    load_angles<VE>(cosr + j * VE, c);
    load_angles<VE>(sinr + j * VE, s);
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            y[2 * i] = EXACT ? rot_odd(a, c[i], b, s[i]) : fmaf(a, c[i], -b * s[i]);
            y[2 * i + 1] = EXACT ? rot_odd(b, c[i], -a, s[i]) : fmaf(b, c[i], a * s[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float a = x[i], b = x[VE + i];
            y[i] = EXACT ? rot_odd(a, c[i], b, s[i]) : fmaf(a, c[i], -b * s[i]);
            y[VE + i] = EXACT ? rot_odd(b, c[i], -a, s[i]) : fmaf(b, c[i], a * s[i]);
        }
    }
}

// The sequence is within the contract, its block ids aside.
__device__ __forceinline__ bool append_ok(const AppendParams& p, const PagedSeq& s) {
    return s.ok && (s.S == 0 || s.K <= p.num_pos);
}
// A block id of its new slots lies outside the pool (all threads of the block take
// part; the answer is the same for all).
__device__ __forceinline__ bool append_bad_ids(const AppendParams& p, int64_t b, const PagedSeq& s) {
    int bad = 0;
    if (s.S > 0) {
        const int i0 = (s.K - s.S) / p.bs, i1 = (s.K - 1) / p.bs;
        for (int i = i0 + threadIdx.x; i <= i1; i += blockDim.x) {
            const int id = p.table[b * p.max_blocks + i];
            bad |= id < 0 || id >= p.num_blocks;
        }
    }
    return __syncthreads_or(bad);
}

// Rows of `heads` heads for each of the block's tokens: a thread takes one job of
// the rows of p.hg heads (kHeads, or one where tokens are few), whose loads are
// all under way together and share the angles (one row at a time a prompt ran at 38% of
// the copy bandwidth, now at 69%), and steps over such groups, so that nothing is
// divided in the loop.
constexpr int kHeads = 4;
template <typename T, int VE, typename Dst>
__device__ __forceinline__ void token_rows(const AppendParams& p, const T* src, int64_t tok0, int nt,
                                           int heads, int jobs, int64_t st_tok, int64_t st_head,
                                           bool rotate, const int* pos, bool zero_bad, int first, Dst dst_of) {
    using W = typename Word<VE * sizeof(T)>::type;
    const int groups = (heads + p.hg - 1) / p.hg;  // of a token
    const int step = blockDim.x / jobs;
    // the work starts at thread `first`: behind what the rows before have left idle
    int tid = threadIdx.x - first;
    if (tid < 0) tid += blockDim.x;
    int g = tid / jobs;
    if (g >= step) return;
    const int j = tid - g * jobs;
    const int npair = rotate ? p.half / VE : 0;
    const bool turn = j < npair;
    int o0, o1 = 0;
    if (!turn) {
        o0 = (rotate ? 2 * p.half : 0) + (j - npair) * VE;
    } else {
        o0 = p.interleaved ? 2 * j * VE : j * VE;
        o1 = p.interleaved ? o0 + VE : p.half + j * VE;
    }
    int i = 0;
    for (;;) {
        while (g >= groups) {
            g -= groups;
            ++i;
        }
        if (i >= nt) return;
        const int at = pos[i];  // -1: outside the contract, -2: of no sequence
        if (at >= 0 || (at == -1 && zero_bad)) {
            const int h0 = g * p.hg, n = min(p.hg, heads - h0);
            const T* row = src + (tok0 + i) * st_tok + h0 * st_head;
            W x0[kHeads], x1[kHeads];
#pragma unroll
            for (int u = 0; u < kHeads; ++u)
                if (u < n) {
                    x0[u] = *reinterpret_cast<const W*>(row + u * st_head + o0);
                    if (turn) x1[u] = *reinterpret_cast<const W*>(row + u * st_head + o1);
                }
            float c[VE], sn[VE];
            if (turn && at >= 0) {  // (a row outside the contract reads no angles: there may be none)
                const int64_t a = static_cast<int64_t>(at) * p.half + j * VE;
                load_angles<VE>(p.cos + a, c);
                load_angles<VE>(p.sin + a, sn);
            }
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
                if (u >= n) break;
                T* dst = dst_of(i, h0 + u);
                if (at < 0) {
                    float z[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) z[e] = 0.f;
                    store_vec<T, VE>(dst + o0, z);
                    if (turn) store_vec<T, VE>(dst + o1, z);
                } else if (!turn) {
                    *reinterpret_cast<W*>(dst + o0) = x0[u];
                } else {
                    const T* e0 = reinterpret_cast<const T*>(&x0[u]);
                    const T* e1 = reinterpret_cast<const T*>(&x1[u]);
                    float y[2 * VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        auto el = [&](int k) {
                            return Storage<T>::to_float(k < VE ? e0[k] : e1[k - VE]);
                        };
                        if (p.interleaved) {
                            const float a = el(2 * e), b = el(2 * e + 1);
                            y[2 * e] = fmaf(a, c[e], -b * sn[e]);
                            y[2 * e + 1] = fmaf(b, c[e], a * sn[e]);
                        } else {
                            const float a = el(e), b = el(VE + e);
                            y[e] = fmaf(a, c[e], -b * sn[e]);
                            y[VE + e] = fmaf(b, c[e], a * sn[e]);
                        }
                    }
                    store_vec<T, VE>(dst + o0, y);
                    store_vec<T, VE>(dst + o1, y + VE);
                }
            }
        }
        g += step;
    }
}

// Blocks [0, p.tok_blocks): p.tpb tokens each.
template <typename T, bool EIGHT, int VE>
__device__ void append_tokens(const AppendParams& p) {
    __shared__ int64_t dst_row[kMaxTokensPerBlock];  // pool row (of head 0) of the token's slot
    __shared__ int pos[kMaxTokensPerBlock];          // position; -1: outside the contract, -2: no sequence
    __shared__ int seq[kMaxTokensPerBlock];
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tpb;
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.tpb), p.total_q - tok0));
    if (static_cast<int>(threadIdx.x) < nt) {
        // the first sequence whose end lies past the token
        const int tok = static_cast<int>(tok0) + threadIdx.x;
        int lo = 0, hi = static_cast<int>(p.B);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid + 1] <= tok) lo = mid + 1; else hi = mid;
        }
        seq[threadIdx.x] = lo;
    }
    __syncthreads();
    PagedSeq s{};
    bool ok = false;
    for (int i = 0; i < nt; ++i) {
        const int b = seq[i];
        if (i == 0 || b != seq[i - 1]) {
            if (b < p.B) s = paged_seq(p.cu, p.kl, b, p.total_q, p.max_q, p.M);
            ok = b < p.B && append_ok(p, s) && !append_bad_ids(p, b, s);
        }
        if (static_cast<int>(threadIdx.x) == i) {
            const int t = static_cast<int>(tok0) + i - s.q0;
            const bool mine = b < p.B && s.rows_ok && t >= 0 && t < s.S;
            const int j = s.K - s.S + t;
            pos[i] = !mine ? -2 : ok ? j : -1;
            if (mine && ok)
                dst_row[i] = (static_cast<int64_t>(p.table[b * p.max_blocks + j / p.bs]) * p.Hk) * p.bs +
                             j % p.bs;
            else if (mine && p.status)
                atomicOr(p.status, KVC_DEV_OVERFLOW);
        }
    }
    __syncthreads();
    const int jr = (p.half + (p.D - 2 * p.half)) / VE, jv = p.Dv / VE;
    token_rows<T, VE>(p, static_cast<const T*>(p.query), tok0, nt, p.Hq, jr, p.st[0], p.st[1], true,
                      pos, true, 0, [&](int i, int h) {
                          return static_cast<T*>(p.out_query) + ((tok0 + i) * p.Hq + h) * p.D;
                      });
    if (EIGHT) return;
    const int kv_groups = nt * ((p.Hk + p.hg - 1) / p.hg);
    const int k_at = nt * ((p.Hq + p.hg - 1) / p.hg) * jr % blockDim.x;
    const int v_at = (k_at + kv_groups * jr) % blockDim.x;
    token_rows<T, VE>(p, static_cast<const T*>(p.new_key), tok0, nt, p.Hk, jr, p.st[2], p.st[3], true,
                      pos, false, k_at, [&](int i, int h) {
                          return static_cast<T*>(p.key_pool) +
                                 (dst_row[i] + static_cast<int64_t>(h) * p.bs) * p.D;
                      });
    token_rows<T, VE>(p, static_cast<const T*>(p.new_value), tok0, nt, p.Hk, jv, p.st[4], p.st[5],
                      false, pos, false, v_at, [&](int i, int h) {
                          return static_cast<T*>(p.value_pool) +
                                 (dst_row[i] + static_cast<int64_t>(h) * p.bs) * p.Dv;
                      });
}

// One (sequence, touched block, head, keys or values) of an 8-bit pool.
template <typename T, bool E5M2, int VE>
__device__ void append_block8(const AppendParams& p, int64_t unit_index) {
    __shared__ uint32_t red[kAppThreads / 32];
    const int which = static_cast<int>(unit_index & 1);  // 0: keys, 1: values
    int hk, ib;
    int64_t b;
    if (p.units8 < (int64_t(1) << 31)) {
        const uint32_t i = static_cast<uint32_t>(unit_index) >> 1, j = i / p.Hk;
        hk = static_cast<int>(i - j * p.Hk);
        const uint32_t q = j / static_cast<uint32_t>(p.seq_blocks);
        ib = static_cast<int>(j - q * static_cast<uint32_t>(p.seq_blocks));
        b = q;
    } else {
        const int64_t i = unit_index >> 1, j = i / p.Hk;
        hk = static_cast<int>(i - j * p.Hk);
        b = j / p.seq_blocks;
        ib = static_cast<int>(j - b * p.seq_blocks);
    }
    const PagedSeq s = paged_seq(p.cu, p.kl, b, p.total_q, p.max_q, p.M);
    if (!append_ok(p, s)) {
        if (threadIdx.x == 0 && ib == 0 && p.status) atomicOr(p.status, KVC_DEV_OVERFLOW);
        return;
    }
    if (s.S == 0) return;
    const int start = s.K - s.S;
    const int i = start / p.bs + ib;
    const int lo = max(start, i * p.bs), hi = min(s.K, (i + 1) * p.bs);
    const int width = which ? p.Dv : p.D;
    const int jn = which ? p.Dv / VE : (p.half + (p.D - 2 * p.half)) / VE;
    const T* src0 = static_cast<const T*>(which ? p.new_value : p.new_key) + hk * p.st[which ? 5 : 3] +
                    (s.q0 + (lo - start)) * p.st[which ? 4 : 2];
    const int64_t tstride = p.st[which ? 4 : 2];
    const int njobs = max(0, hi - lo) * jn;
    auto job = [&](int w, float* y, int& row, int& o0, int& o1) {
        row = w / jn;
        const int64_t a = static_cast<int64_t>(lo + row) * p.half;
        row_job<T, VE, true>(p, src0 + row * tstride, w - row * jn, !which, p.cos + a, p.sin + a, y,
                             o0, o1);
    };
    auto largest = [&](const float* y, int o1, uint32_t most) {  // finite |value|, as its bits
#pragma unroll
        for (int e = 0; e < 2 * VE; ++e) {
            const uint32_t v = __float_as_uint(y[e]) & 0x7fffffffu;
            if ((e < VE || o1 >= 0) && v < 0x7f800000u) most = max(most, v);
        }
        return most;
    };
    // a thread's first jobs stay in registers for the second pass (all there is for
    // small pool blocks); the rest is formed again, out of L1
    constexpr int kKeep = 2;
    const int nth = blockDim.x;
    float y[kKeep][2 * VE];
    int row[kKeep], o0[kKeep], o1[kKeep];
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int w = threadIdx.x + u * nth;
        if (w < njobs) {
            job(w, y[u], row[u], o0[u], o1[u]);
            most = largest(y[u], o1[u], most);
        }
    }
    for (int w = threadIdx.x + kKeep * nth; w < njobs; w += nth) {
        float z[2 * VE];
        int r, a0, a1;
        job(w, z, r, a0, a1);
        most = largest(z, a1, most);
    }
    if (append_bad_ids(p, b, s)) {
        if (threadIdx.x == 0 && ib == 0 && p.status) atomicOr(p.status, KVC_DEV_OVERFLOW);
        return;
    }
    if (lo >= hi) return;
    const int64_t unit = static_cast<int64_t>(p.table[b * p.max_blocks + i]) * p.Hk + hk;
    float* sp = (which ? p.value_scale : p.key_scale) + unit;
    const int held = lo - i * p.bs;  // rows that the block already holds
    const float old = held ? *sp : 0.f;
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int w = 0; w < nth / 32; ++w) most = max(most, red[w]);
    int e = static_cast<int>(most >> 23) - 127 - Eight<E5M2>::top +
            ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(-100, min(100, e));
    float scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    if (held && old > scale) scale = old;
    const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0u;
    const float inv = 1.f / scale;  // exact for a power of two
    uint8_t* base = static_cast<uint8_t*>(which ? p.value_pool : p.key_pool) + unit * p.bs * width;
    if (held && old != scale) {  // the held rows, at the larger scale
        const float f = __fdiv_rn(old, scale);
        const int n = held * width;
        for (int w = 2 * threadIdx.x; w + 1 < n; w += 2 * nth) {
            const float2 v = from_eight2<E5M2>(base[w] | (static_cast<uint32_t>(base[w + 1]) << 8));
            const uint32_t c = to_eight2<E5M2>(v.x * f, v.y * f);
            base[w] = static_cast<uint8_t>(c);
            base[w + 1] = static_cast<uint8_t>(c >> 8);
        }
        if ((n & 1) && threadIdx.x == 0)
            base[n - 1] = static_cast<uint8_t>(
                to_eight2<E5M2>(from_eight(base[n - 1], E5M2) * f, 0.f));
    }
    base += static_cast<int64_t>(held) * width;
    auto put = [&](float* z, int r, int a0, int a1) {
#pragma unroll
        for (int k = 0; k < 2 * VE; ++k) z[k] = pow2 ? z[k] * inv : __fdiv_rn(z[k], scale);
        store_eight<VE, E5M2>(base + static_cast<int64_t>(r) * width + a0, z);
        if (a1 >= 0) store_eight<VE, E5M2>(base + static_cast<int64_t>(r) * width + a1, z + VE);
    };
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
        if (static_cast<int>(threadIdx.x) + u * nth < njobs) put(y[u], row[u], o0[u], o1[u]);
    for (int w = threadIdx.x + kKeep * nth; w < njobs; w += nth) {
        float z[2 * VE];
        int r, a0, a1;
        job(w, z, r, a0, a1);
        put(z, r, a0, a1);
    }
    if (threadIdx.x == 0) *sp = scale;
}

template <typename T, int KIND, int VE>  // KIND 0: a pool of the inputs' type, 1: e4m3, 2: e5m2
__global__ void __launch_bounds__(kAppThreads, 3) append_rotary_kernel(const __grid_constant__ AppendParams p) {
    if (blockIdx.x < p.tok_blocks) {
        append_tokens<T, KIND != 0, VE>(p);
        if (blockIdx.x == 0 && p.status)  // sequences whose packed rows are no rows of the tensor
            for (int64_t b = threadIdx.x; b < p.B; b += blockDim.x)
                if (!paged_seq(p.cu, p.kl, b, p.total_q, p.max_q, p.M).ok)
                    atomicOr(p.status, KVC_DEV_OVERFLOW);
    } else if constexpr (KIND != 0) {
        for (int64_t i = blockIdx.x - p.tok_blocks; i < p.units8; i += gridDim.x - p.tok_blocks) {
            append_block8<T, KIND == 2, VE>(p, i);
            __syncthreads();  // the reduction buffer is read before the next unit fills it
        }
    }
}

template <typename T, int VE>
cudaError_t launch_ve(const AppendParams& p, int kind, unsigned grid, cudaStream_t stream) {
    switch (kind) {
        case 0: append_rotary_kernel<T, 0, VE><<<grid, p.threads, 0, stream>>>(p); break;
        case 1: append_rotary_kernel<T, 1, VE><<<grid, p.threads, 0, stream>>>(p); break;
        default: append_rotary_kernel<T, 2, VE><<<grid, p.threads, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rotary(const AppendParams& p, int dtype, int kind, int ve,
                                 cudaStream_t stream) {
    const int64_t rest = std::min<int64_t>(p.units8, int64_t(1) << 24);
    const unsigned grid = static_cast<unsigned>(p.tok_blocks + rest);
    if (grid == 0) return cudaSuccess;
    if (dtype == KVC_F32)
        return ve == 4 ? launch_ve<float, 4>(p, kind, grid, stream)
                       : launch_ve<float, 1>(p, kind, grid, stream);
    if (dtype == KVC_BF16)
        return ve == 8   ? launch_ve<__nv_bfloat16, 8>(p, kind, grid, stream)
               : ve == 4 ? launch_ve<__nv_bfloat16, 4>(p, kind, grid, stream)
                         : launch_ve<__nv_bfloat16, 1>(p, kind, grid, stream);
    return ve == 8   ? launch_ve<__half, 8>(p, kind, grid, stream)
           : ve == 4 ? launch_ve<__half, 4>(p, kind, grid, stream)
                     : launch_ve<__half, 1>(p, kind, grid, stream);
}

}  // namespace kvc
