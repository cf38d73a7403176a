// kvc_paged_attend.cu -- attention of packed queries over a paged pool on the
// CUDA cores: any type, widths up to 256, any block size ("ClikaRT::ops::
// attention_over_cache": paged block pool, softcap, sliding-window and
// quantised-scale options).
//
// Query row (t, h) of sequence b sits at p = K_b - S_b + t and sees the slots
// j <= p, j > p - window. s = scale q.k_j, with the key block's scale; then
// cap tanh(s / cap), then - slope_h (p - j); out = softmax(s) . v, with the value
// block's scale folded into the weight.
//
// A block of 4 warps takes 8 query rows of one KV head and one split of the
// slots; a warp takes every fourth run of slots. Per slot: lanes over the width
// hold the 8 rows' products, a reduce-scatter leaves row r's score in lanes
// 4r..4r+3, which keep that row's running maximum and sum (fp32); the weights
// go back to all lanes by shuffles. About 100 instructions a slot and 8 rows:
// issue-bound. This kernel serves fp32 and the sizes that the tensor-core kernels
// do not take, so a warp's simple form was kept: 64 tokens over 1024 to 8190 slots of
// an e4m3 pool, 32 heads on 8 of 128, took 2507 us where the decode kernel takes 109.
#include <algorithm>

#include "kvc_launch.h"
#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kRows = 8;   // query rows of a block
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <typename P>
__device__ __forceinline__ float pool_value(const P* p, bool) {
    return Storage<P>::to_float(*p);
}
template <>
__device__ __forceinline__ float pool_value<uint8_t>(const uint8_t* p, bool e5m2) {
    return from_eight(*p, e5m2);
}

// s * scale in natural units -> capped, biased, in base 2
__device__ __forceinline__ float score2(const PagedAttendParams& p, float s, float slope, int dist) {
    if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
    if (p.slopes) s -= slope * static_cast<float>(dist);
    return s * kLog2e;
}

template <typename T, typename P, int ND>  // lanes hold ND elements each: widths up to 32 ND
__global__ void __launch_bounds__(kThreads)
    paged_attend_kernel(const __grid_constant__ PagedAttendParams p) {
    __shared__ float sh_ml[kWarps][kRows][2];
    __shared__ float sh_acc[kWarps][kRows][32 * ND];
    __shared__ int sh_bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hk = blockIdx.y % p.Hk, split = blockIdx.y / p.Hk;
    const int64_t chunks = (p.max_q * p.G + kRows - 1) / kRows;
    for (int64_t unit = blockIdx.x; unit < p.B * chunks; unit += gridDim.x) {
        __syncthreads();
        if (threadIdx.x == 0) sh_bad = 0;
        __syncthreads();
        const int64_t b = unit / chunks;
        const int64_t r0 = (unit - b * chunks) * kRows;
        const PagedSeq s = paged_seq(p.cu, p.kl, b, p.total_q, p.max_q, p.M);
        if (!s.ok) {  // zero rows, flagged
            if (threadIdx.x == 0 && p.status) atomicOr(p.status, KVC_DEV_OVERFLOW);
            if (split == 0)
                for (int64_t r = r0; r < static_cast<int64_t>(s.S) * p.G; r += chunks * kRows)
                    for (int e = threadIdx.x; e < kRows * p.Dv; e += kThreads) {
                        const int64_t rr = r + e / p.Dv;
                        if (rr >= static_cast<int64_t>(s.S) * p.G) continue;
                        const int64_t row = (s.q0 + rr / p.G) * p.Hq + hk * p.G + rr % p.G;
                        static_cast<T*>(p.out)[row * p.Dv + e % p.Dv] = Storage<T>::from_float(0.f);
                    }
            continue;
        }
        const int64_t R = static_cast<int64_t>(s.S) * p.G;
        if (r0 >= R) continue;
        const int nr = static_cast<int>(min(static_cast<int64_t>(kRows), R - r0));
        float qf[kRows][ND];
        int lim[kRows];
        const int base = s.K - s.S;
        int lim_lo = 0x7fffffff, lim_hi = -1;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            lim[r] = -1;
#pragma unroll
            for (int i = 0; i < ND; ++i) qf[r][i] = 0.f;
            if (r < nr) {
                const int t = static_cast<int>((r0 + r) / p.G), g = static_cast<int>((r0 + r) % p.G);
                lim[r] = base + t;
                lim_lo = min(lim_lo, lim[r]);
                lim_hi = max(lim_hi, lim[r]);
                const T* q = static_cast<const T*>(p.q) + (s.q0 + t) * p.q_tok +
                             (static_cast<int64_t>(hk) * p.G + g) * p.q_head;
#pragma unroll
                for (int i = 0; i < ND; ++i)
                    if (lane + 32 * i < p.D) qf[r][i] = Storage<T>::to_float(q[lane + 32 * i]);
            }
        }
        const int own = lane >> 2;  // the row whose statistics this lane keeps
        const int own_lim = base + static_cast<int>((r0 + own) / p.G);
        const bool own_live = own < nr;
        const float slope = p.slopes && own_live ? p.slopes[hk * p.G + (r0 + own) % p.G] : 0.f;
        float m = -INFINITY, l = 0.f;
        float acc[kRows][ND];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < ND; ++i) acc[r][i] = 0.f;
        const int first = p.window > 0 ? max(0, lim_lo - p.window + 1) : 0;
        const int64_t a0 = first + static_cast<int64_t>(split) * p.split_len;
        const int j_end = p.nsplit > 1 ? static_cast<int>(min(static_cast<int64_t>(lim_hi) + 1,
                                                              a0 + p.split_len))
                                       : lim_hi + 1;
        int blk = -1, id = 0;
        float ksc = 1.f, vsc = 1.f;
        bool bad = false;
        for (int64_t j64 = a0 + warp; j64 < j_end; j64 += kWarps) {
            const int j = static_cast<int>(j64);
            if (j / p.bs != blk) {
                blk = j / p.bs;
                id = p.table[b * p.max_blocks + blk];
                if (id < 0 || id >= p.num_blocks) {
                    bad = true;
                    id = 0;
                }
                if (p.ks) {
                    ksc = p.ks[static_cast<int64_t>(id) * p.Hk + hk];
                    vsc = p.vs[static_cast<int64_t>(id) * p.Hk + hk];
                }
            }
            const int64_t row = (static_cast<int64_t>(id) * p.Hk + hk) * p.bs + j % p.bs;
            const P* kr = static_cast<const P*>(p.kp) + row * p.D;
            float part[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) part[r] = 0.f;
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                const float k = lane + 32 * i < p.D ? pool_value<P>(kr + lane + 32 * i, p.e5m2) : 0.f;
#pragma unroll
                for (int r = 0; r < kRows; ++r) part[r] = fmaf(qf[r][i], k, part[r]);
            }
            // reduce-scatter: row r's sum in lanes 4r..4r+3
#pragma unroll
            for (int h = kRows / 2, o = 16; h >= 1; h /= 2, o /= 2) {
                const bool up = (lane & o) != 0;
#pragma unroll
                for (int i = 0; i < h; ++i) {
                    const float keep = up ? part[i + h] : part[i];
                    const float send = up ? part[i] : part[i + h];
                    part[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
            float sc = part[0];
            sc += __shfl_xor_sync(0xffffffffu, sc, 2);
            sc += __shfl_xor_sync(0xffffffffu, sc, 1);
            const bool see = own_live && j <= own_lim && (p.window == 0 || j > own_lim - p.window);
            float pw = 0.f, corr = 1.f;
            if (see) {
                const float s2 = score2(p, sc * (p.scale * ksc), slope, own_lim - j);
                if (s2 > m) {
                    corr = fast_exp2(m - s2);
                    l *= corr;
                    m = s2;
                }
                pw = s2 == -INFINITY ? 0.f : fast_exp2(s2 - m);
                l += pw;
                if (p.vs) pw *= vsc;
            }
            if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float c = __shfl_sync(0xffffffffu, corr, 4 * r);
#pragma unroll
                    for (int i = 0; i < ND; ++i) acc[r][i] *= c;
                }
            }
            const uint32_t vis = __ballot_sync(0xffffffffu, see);
            const P* vr = static_cast<const P*>(p.vp) + row * p.Dv;
            float v[ND];
#pragma unroll
            for (int i = 0; i < ND; ++i)
                v[i] = lane + 32 * i < p.Dv ? pool_value<P>(vr + lane + 32 * i, p.e5m2) : 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float w = __shfl_sync(0xffffffffu, pw, 4 * r);
                if ((vis >> (4 * r)) & 1u) {  // a masked slot's value never enters, NaN or not
#pragma unroll
                    for (int i = 0; i < ND; ++i) acc[r][i] = fmaf(w, v[i], acc[r][i]);
                }
            }
        }
        if (bad) sh_bad = 1;
        if ((lane & 3) == 0) {
            sh_ml[warp][own][0] = m;
            sh_ml[warp][own][1] = l;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < ND; ++i) sh_acc[warp][r][lane + 32 * i] = acc[r][i];
        __syncthreads();
        if (sh_bad && threadIdx.x == 0 && p.status) atomicOr(p.status, KVC_DEV_OVERFLOW);
        for (int r = warp; r < nr; r += kWarps) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (sh_ml[w][r][1] != 0.f) mm = fmaxf(mm, sh_ml[w][r][0]);
            float f[kWarps], ll = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = sh_ml[w][r][1] != 0.f
                           ? (sh_ml[w][r][0] == mm ? 1.f : fast_exp2(sh_ml[w][r][0] - mm)) : 0.f;
                ll += sh_ml[w][r][1] * f[w];
            }
            const int64_t row = (s.q0 + (r0 + r) / p.G) * p.Hq + hk * p.G + (r0 + r) % p.G;
            const int64_t prow = split * p.total_q * p.Hq + row;
            if (p.nsplit > 1 && lane == 0) {
                p.part_ml[2 * prow] = mm;
                p.part_ml[2 * prow + 1] = sh_bad ? -1.f : ll;
            }
            const float inv = 1.f / ll;
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                const int d = lane + 32 * i;
                if (d >= p.Dv) continue;
                float a = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (f[w] != 0.f) a += sh_acc[w][r][d] * f[w];
                if (p.nsplit > 1)
                    p.part_acc[prow * p.Dv + d] = a;
                else
                    static_cast<T*>(p.out)[row * p.Dv + d] =
                        Storage<T>::from_float(sh_bad ? 0.f : a * inv);
            }
        }
    }
}

// One warp per query row: the splits' partials joined (l < 0: zero row).
template <typename T>
__global__ void __launch_bounds__(256) paged_merge_rows_kernel(const __grid_constant__ PagedAttendParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t rows = p.total_q * p.Hq;
    if (row >= rows) return;
    // the row's sequence: rows behind the last one are left as they were
    const int tok = static_cast<int>(row / p.Hq);
    int64_t lo = 0, hi = p.B;  // the first sequence whose end lies past the token
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] <= tok) lo = mid + 1; else hi = mid;
    }
    if (lo >= p.B) return;
    const PagedSeq s = paged_seq(p.cu, p.kl, lo, p.total_q, p.max_q, p.M);
    if (!s.rows_ok || tok < s.q0 || !s.ok) return;
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    for (int k = 0; k < p.nsplit; ++k) {
        const float lk = p.part_ml[2 * (k * rows + row) + 1];
        if (lk < 0.f) bad = true;
        if (lk != 0.f) m = fmaxf(m, p.part_ml[2 * (k * rows + row)]);
    }
    for (int k = 0; k < p.nsplit; ++k) {
        const float lk = p.part_ml[2 * (k * rows + row) + 1], mk = p.part_ml[2 * (k * rows + row)];
        if (lk != 0.f) l += lk * (mk == m ? 1.f : fast_exp2(mk - m));
    }
    const float inv = 1.f / l;
    for (int d = lane; d < p.Dv; d += 32) {
        float a = 0.f;
        for (int k = 0; k < p.nsplit; ++k) {
            const float lk = p.part_ml[2 * (k * rows + row) + 1], mk = p.part_ml[2 * (k * rows + row)];
            if (lk != 0.f)
                a += p.part_acc[(k * rows + row) * p.Dv + d] * (mk == m ? 1.f : fast_exp2(mk - m));
        }
        static_cast<T*>(p.out)[row * p.Dv + d] = Storage<T>::from_float(bad ? 0.f : a * inv);
    }
}

template <typename T, typename P>
cudaError_t launch_nd(const PagedAttendParams& p, dim3 grid, cudaStream_t stream) {
    const int w = std::max(p.D, p.Dv);
    if (w <= 64)
        paged_attend_kernel<T, P, 2><<<grid, kThreads, 0, stream>>>(p);
    else if (w <= 128)
        paged_attend_kernel<T, P, 4><<<grid, kThreads, 0, stream>>>(p);
    else
        paged_attend_kernel<T, P, 8><<<grid, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    const int64_t warps = p.total_q * p.Hq;
    paged_merge_rows_kernel<T><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_pool(const PagedAttendParams& p, bool eight, dim3 grid, cudaStream_t stream) {
    return eight ? launch_nd<T, uint8_t>(p, grid, stream) : launch_nd<T, T>(p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_attend(const PagedAttendParams& p, int dtype, int pool_dtype,
                                cudaStream_t stream) {
    const int64_t units = p.B * ((p.max_q * p.G + kRows - 1) / kRows);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(units, int64_t(1) << 20)),
                    static_cast<unsigned>(p.Hk * p.nsplit));
    const bool eight = pool_dtype != dtype;
    if (dtype == KVC_F32) return launch_pool<float>(p, eight, grid, stream);
    if (dtype == KVC_BF16) return launch_pool<__nv_bfloat16>(p, eight, grid, stream);
    return launch_pool<__half>(p, eight, grid, stream);
}

}  // namespace kvc
