// kvc_paged.cuh -- what the kernels of the packed, paged operators share:
// append_rotary_paged (kvc_rotary_append.cu) and attend_paged
// (kvc_paged_attend.cu, kvc_paged_decode.cu, kvc_paged_rows.cu).
//
// T = total_q packed tokens; sequence b owns rows cu_seqlens_q[b] ..
// cu_seqlens_q[b+1]-1, S_b of them, its last S_b of seqlens_k[b] = K_b cached
// positions. Slot j of sequence b is row j % block_size of pool block
// block_table[b, j / block_size].
#pragma once

#include <cuda_fp8.h>

#include "kvc_internal.cuh"

namespace kvc {

struct PagedSeq {
    int q0, S, K;  // first packed row, query rows, cached positions
    bool rows_ok;  // its packed rows lie inside [0, total_q)
    bool ok;       // within the contract (its block ids aside)
};

__device__ __forceinline__ PagedSeq paged_seq(const int32_t* cu, const int32_t* kl, int64_t b,
                                              int64_t total_q, int64_t max_q, int64_t M) {
    PagedSeq s;
    const int a = cu[b], e = cu[b + 1], k = kl[b];
    s.q0 = a;
    s.rows_ok = a >= 0 && e >= a && e <= total_q;
    s.S = s.rows_ok ? e - a : 0;
    s.K = k;
    s.ok = s.rows_ok && s.S <= max_q && s.S <= k && k <= M;
    return s;
}

// ------------------------------------------------------------ 8-bit formats
// Both formats' largest value is 1.75 * 2^top.
template <bool E5M2>
struct Eight {
    static constexpr int top = E5M2 ? 15 : 8;
    static constexpr __nv_fp8_interpretation_t kind = E5M2 ? __NV_E5M2 : __NV_E4M3;
};

// Two values to two codes (the first in the low byte), ties to even, ending
// at the largest value; NaN stays NaN.
template <bool E5M2>
__device__ __forceinline__ uint32_t to_eight2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, Eight<E5M2>::kind);
}

// Two codes to their values (exact: fp16 holds every value of both formats).
template <bool E5M2>
__device__ __forceinline__ float2 from_eight2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w),
                                                     Eight<E5M2>::kind);
    return __half22float2(__half2(h));
}

__device__ __forceinline__ float from_eight(uint8_t w, bool e5m2) {
    return e5m2 ? from_eight2<true>(w).x : from_eight2<false>(w).x;
}

}  // namespace kvc
