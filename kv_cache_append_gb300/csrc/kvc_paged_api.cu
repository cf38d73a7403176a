// kvc_paged_api.cu -- C entry points of the packed, paged operators
// (include/kvc.h): argument checks and launch plans. Nothing here allocates or
// synchronises.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "kvc_launch.h"

namespace kvc {
namespace {

// Splits and grids are planned for this many SMs, so that the workspace size
// does not depend on the device.
constexpr int64_t kPlanSms = 152;
constexpr int64_t kMaxInt = int64_t(1) << 30;

struct Range {
    uintptr_t lo, hi;
};
Range range_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + static_cast<uintptr_t>(bytes > 0 && p ? bytes : 0)};
}
bool overlaps(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int elem(int32_t dtype) {
    return dtype == KVC_F32 ? 4 : (dtype == KVC_E4M3 || dtype == KVC_E5M2) ? 1 : 2;
}
bool eight(const kvc_paged_dims& d) { return d.pool_dtype != d.dtype; }

int check_paged(const kvc_paged_dims* dims) {
    if (!dims) return KVC_E_NULL;
    const kvc_paged_dims& d = *dims;
    if (d.dtype < KVC_F32 || d.dtype > KVC_F16 ||
        (d.pool_dtype != d.dtype && d.pool_dtype != KVC_E4M3 && d.pool_dtype != KVC_E5M2))
        return KVC_E_DTYPE;
    if (d.B < 1 || d.total_q < 0 || d.max_q < 0 || d.Hq < 1 || d.Hk < 1 || d.Hq % d.Hk != 0 ||
        d.D < 1 || d.Dv < 1 || d.D > 256 || d.Dv > 256 || d.num_blocks < 1 || d.block_size < 1 ||
        d.max_blocks < 1 || (d.total_q > 0 && d.max_q < 1))
        return KVC_E_SHAPE;
    // device code counts rows, slots and blocks in 31 bits, bytes in 64
    if (d.B > kMaxInt || d.Hq > 65535 || d.num_blocks > kMaxInt / d.Hk ||
        d.block_size > kMaxInt || d.max_blocks > kMaxInt / d.block_size ||
        d.total_q > kMaxInt / d.Hq || d.max_q > kMaxInt / d.Hq || d.B > kMaxInt / d.Hq)
        return KVC_E_SHAPE;
    return KVC_OK;
}

int64_t span(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t w, int64_t es) {
    return n0 < 1 ? 0 : ((n0 - 1) * s0 + (n1 - 1) * s1 + w) * es;
}

bool current_is_gb300() {
    static std::atomic<uint64_t> known{0};  // devices found to be sm_103
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    if (dev < 64 && (known.load(std::memory_order_relaxed) >> dev & 1u)) return true;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        major != 10 || minor != 3)
        return false;
    if (dev < 64) known.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return true;
}

// No sequence has more rows than there are.
int64_t most_rows(const kvc_paged_dims& d) { return std::min(d.max_q, d.total_q); }

// The CUDA-core kernel's splits of the slots: enough blocks for every SM to
// hold a few, each with 256 slots or more of the capacity.
struct CorePlan {
    int64_t nsplit, split_len, bytes;
};
CorePlan core_plan(const kvc_paged_dims& d) {
    const int64_t G = d.Hq / d.Hk, M = d.max_blocks * d.block_size;
    const int64_t blocks = std::max<int64_t>(1, d.B * ((most_rows(d) * G + 7) / 8) * d.Hk);
    CorePlan c;
    c.nsplit = std::max<int64_t>(1, std::min({(4 * kPlanSms + blocks - 1) / blocks, M / 256,
                                              int64_t(64), 65535 / d.Hk}));
    c.split_len = (M + c.nsplit - 1) / c.nsplit;
    c.bytes = c.nsplit > 1 ? c.nsplit * d.total_q * d.Hq * (d.Dv + 2) * 4 : 0;
    return c;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// The tensor-core kernels: 16-bit queries, rows of whole 16-byte words, keys up
// to 256 and values up to 128 wide, blocks of a multiple of 8 slots (a box
// then starts on an 8-row swizzle atom).
struct TcPlan {
    bool ok = false;
    int nr = 0;  // decode kernel: rows a unit is padded to; 0: the rows kernel
    size_t smem = 0;
    int64_t bytes = 0, off_ml = 0, off_acc = 0;
    PagedTcParams p;
};
// Units of up to this many query rows take the decode kernel. 64 sequences of 1024 to
// 8190 slots, 8 KV heads: at 16 rows decode 212 us and rows 252 on an 8-bit pool (230
// and 247 on bf16), at 32 rows 312 and 252 (262 and 254).
constexpr int64_t kDecodeRows = 16;
// What the start of a unit takes of a block's time, in tiles: its first tile's latency,
// its query rows, its result and the tiles at its mask's edge. Not counted, the blocks
// with the most unit starts are the last to end. Rows kernel, at 0, 3, 6, 8 and 12
// tiles: 32 prompts of 20 to 300 tokens over up to 4000 slots, 32 heads on 8, e4m3 646,
// 411, 339, 339 and 356 us (bf16 685, 433, 346, 307, 295); 4 of 513 to 2001 over up to
// 8190, 902, 822, 783, 772 and 767. Decode kernel, at 0, 1, 2 and 3: 64 tokens over 1024
// to 8190 slots, e4m3 113.5, 110.3, 108.4 and 109.7 us; 200 over 100 to 2000 at 1, 2 and 3
// 128.8, 121.0 and 117.5; 64 sequences of 1 to 4 tokens, cap, bf16 198, 185, 176 and 172.
constexpr int kLeadRows = 8, kLeadDecode = 3;
constexpr int64_t kSmemSm = 228 * 1024, kSmemBlock = 227 * 1024, kSmemReserved = 1024;

// 8-bit parts of a query element: bf16 2, fp16 3
int64_t query_parts(const kvc_paged_dims& d) { return !eight(d) ? 1 : d.dtype == KVC_BF16 ? 2 : 3; }

// records of the blocks, then their partials
void tc_workspace(const kvc_paged_dims& d, TcPlan* t) {
    const PagedTcParams& p = t->p;
    t->off_ml = up(p.ctas * static_cast<int64_t>(sizeof(PagedRec)), 256);
    t->off_acc = t->off_ml + up(int64_t(2) * p.ctas * p.RG * 8, 256);
    t->bytes = t->off_acc + int64_t(2) * p.ctas * p.RG * d.Dv * 4;
    t->ok = true;
}

TcPlan tc_plan(const kvc_paged_dims& d) {
    TcPlan t;
    const int64_t es = elem(d.pool_dtype), R = most_rows(d) * (d.Hq / d.Hk);
    if (d.dtype == KVC_F32 || d.D * es % 16 != 0 || d.Dv * es % 16 != 0 || d.Dv > 128 ||
        d.block_size % 8 != 0 || d.total_q < 1)
        return t;
    std::memset(&t.p, 0, sizeof(t.p));
    PagedTcParams& p = t.p;
    // exact for slots below 2^30: with l = ceil(log2 d), m = ceil(2^(30 + l) / d), the
    // excess m d - 2^(30 + l) < d <= 2^l takes slot m / 2^(30 + l) less than 1 / d up
    int l = 0;
    while ((int64_t(1) << l) < d.block_size) ++l;
    p.lead = R > kDecodeRows ? kLeadRows : kLeadDecode;
    p.bs_shift = static_cast<uint32_t>(30 + l);
    p.bs_mul = static_cast<uint32_t>(((int64_t(1) << (30 + l)) + d.block_size - 1) / d.block_size);
    if (R > kDecodeRows) {
        // groups of 128 rows: query buffers, then rings of key and value tiles
        const int64_t parts = query_parts(d), nkb = (d.D * es + 127) / 128, nvb = (d.Dv * es + 127) / 128;
        const int64_t kb = nkb * 128 * 128, vb = nvb * 128 * 128;
        p.RG = 128;
        p.hh = 128;
        while (d.block_size % p.hh != 0) p.hh /= 2;
        p.off_q = es == 1 ? 16384 : 12288;  // behind the scales of 16 tiles, or none
        p.q_bytes = static_cast<int>(parts * kb + (es == 1 ? 1024 : 0));
        // the next run's query rows are prepared ahead where that leaves three tiles
        int64_t room = kSmemBlock - p.off_q - 2 * p.q_bytes;
        p.ni = room >= 3 * (kb + vb) ? 2 : 1;
        room = kSmemBlock - p.off_q - p.ni * p.q_bytes;
        const int64_t pairs = std::min<int64_t>(8, room / (kb + vb));
        if (pairs < 1) return t;
        room -= pairs * (kb + vb);
        p.ns = static_cast<int>(pairs < 8 && room >= kb ? pairs + 1 : pairs);
        if (p.ns > pairs) room -= kb;
        p.nv = static_cast<int>(pairs < 8 && room >= vb ? pairs + 1 : pairs);
        if (p.ns < 2) return t;
        p.off_stage = p.off_q + p.ni * p.q_bytes;
        t.smem = static_cast<size_t>(p.off_stage + p.ns * kb + p.nv * vb);
        p.ctas = static_cast<int>(kPlanSms);
        tc_workspace(d, &t);
        return t;
    }
    t.nr = R <= 4 ? 4 : R <= 8 ? 8 : 16;
    const int64_t dn = 16, parts = query_parts(d);
    const int64_t nkb = (d.D * es + 127) / 128, nvb = es == 1 ? 1 : 2, nblk = dn * 128;
    p.RG = t.nr;
    p.hh = 128;
    while (d.block_size % p.hh != 0) p.hh /= 2;
    p.stage_bytes = static_cast<int>((nkb + nvb) * 128 * 128);
    p.q_bytes = static_cast<int>(parts * nkb * nblk);
    const int64_t npt = es == 2 ? 2 : 1;
    p.ni = parts == 3 && nkb == 1 ? 1 : 2;  // (one query buffer leaves fp16 a third stage)
    auto layout = [&](int64_t stages, int64_t cap) {  // scales, items, exchange, queries, weights, stages
        p.off_item = static_cast<int>(512 + std::max<int64_t>(320, stages * 256));
        p.off_x = p.off_item + 128 + 2 * 384;
        p.off_q = static_cast<int>(up(p.off_x + 2 * t.nr * 16 + 64, 1024));
        p.off_p = p.off_q + p.ni * p.q_bytes;
        p.off_stage = static_cast<int>(p.off_p + npt * (es == 1 ? 3 : 2) * nblk);
        p.ns = static_cast<int>(std::min(stages, (cap - p.off_stage) / p.stage_bytes));
    };
    // two blocks an SM where each still has two stages or more
    int64_t blocks = es == 1 ? 2 : 1;
    if (blocks == 2) {
        layout(3, kSmemSm / 2 - kSmemReserved);
        if (p.ns < 2) blocks = 1;
    }
    if (blocks == 1) layout(8, kSmemBlock);
    if (p.ns < 2) return t;
    t.smem = static_cast<size_t>(p.off_stage + int64_t(p.ns) * p.stage_bytes);
    p.ctas = static_cast<int>(kPlanSms * blocks);
    tc_workspace(d, &t);
    return t;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// A pool as [num_blocks * Hk][block_size][width], boxes of 128 bytes x hh slots.
bool pool_map(CUtensorMap* map, const void* base, const kvc_paged_dims& d, int64_t width, int hh) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const int64_t es = elem(d.pool_dtype);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(d.block_size),
                                static_cast<cuuint64_t>(d.num_blocks * d.Hk)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width * es),
                                   static_cast<cuuint64_t>(d.block_size * width * es)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(hh), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : d.dtype == KVC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace kvc

extern "C" {

int kvc_append_rotary_paged(const kvc_paged_dims* dims, int64_t rotary_dim, int64_t num_positions,
                            int32_t interleaved, const int64_t* strides, const void* query,
                            const void* new_key, const void* new_value, const int32_t* block_table,
                            const int32_t* cu_seqlens_q, const int32_t* seqlens_k, const float* cos,
                            const float* sin, void* key_pool, void* value_pool, float* key_scale,
                            float* value_scale, void* out_query, int32_t* dev_status,
                            void* stream_ptr) {
    using namespace kvc;
    const int rc = check_paged(dims);
    if (rc != KVC_OK) return rc;
    const kvc_paged_dims d = *dims;
    const int64_t T = d.total_q, es = elem(d.dtype), ps = elem(d.pool_dtype);
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > d.D || num_positions < 0 ||
        num_positions > kMaxInt || (interleaved != 0 && interleaved != 1))
        return KVC_E_SHAPE;
    // a block's 8-bit rows are counted in 31 bits
    if (eight(d) && d.block_size > kMaxInt / std::max(d.D, d.Dv)) return KVC_E_SHAPE;
    const int64_t half = rotary_dim / 2;
    if (!strides || !block_table || !cu_seqlens_q || !seqlens_k || !key_pool || !value_pool ||
        (T > 0 && (!query || !new_key || !new_value || !out_query)) ||
        (half > 0 && num_positions > 0 && (!cos || !sin)) ||
        (eight(d) ? (!key_scale || !value_scale) : (key_scale || value_scale)))
        return KVC_E_NULL;
    for (int i = 0; i < 6; ++i)
        if (strides[i] < 0 || strides[i] > (int64_t(1) << 40)) return KVC_E_SHAPE;
    const int64_t rows = d.num_blocks * d.Hk * d.block_size;
    const Range ins[] = {
        range_of(query, span(T, strides[0], d.Hq, strides[1], d.D, es)),
        range_of(new_key, span(T, strides[2], d.Hk, strides[3], d.D, es)),
        range_of(new_value, span(T, strides[4], d.Hk, strides[5], d.Dv, es)),
        range_of(block_table, d.B * d.max_blocks * 4),
        range_of(cu_seqlens_q, (d.B + 1) * 4),
        range_of(seqlens_k, d.B * 4),
        range_of(cos, num_positions * half * 4),
        range_of(sin, num_positions * half * 4),
    };
    const Range outs[] = {
        range_of(key_pool, rows * d.D * ps),
        range_of(value_pool, rows * d.Dv * ps),
        range_of(out_query, T * d.Hq * d.D * es),
        range_of(key_scale, d.num_blocks * d.Hk * 4),
        range_of(value_scale, d.num_blocks * d.Hk * 4),
    };
    for (int i = 0; i < 5; ++i) {
        for (const Range& r : ins)
            if (overlaps(outs[i], r)) return KVC_E_ALIAS;
        for (int k = 0; k < i; ++k)
            if (overlaps(outs[i], outs[k])) return KVC_E_ALIAS;
    }
    if (!current_is_gb300()) return KVC_E_DEVICE;
    if (T == 0) return KVC_OK;

    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = d.B; p.total_q = T; p.max_q = most_rows(d); p.M = d.max_blocks * d.block_size;
    p.max_blocks = d.max_blocks; p.num_blocks = static_cast<int>(d.num_blocks);
    p.Hq = static_cast<int>(d.Hq); p.Hk = static_cast<int>(d.Hk);
    p.D = static_cast<int>(d.D); p.Dv = static_cast<int>(d.Dv); p.bs = static_cast<int>(d.block_size);
    p.half = static_cast<int>(half); p.num_pos = half ? static_cast<int>(num_positions) : 0x7fffffff;
    p.interleaved = interleaved;
    std::copy(strides, strides + 6, p.st);
    p.query = query; p.new_key = new_key; p.new_value = new_value;
    p.table = block_table; p.cu = cu_seqlens_q; p.kl = seqlens_k; p.cos = cos; p.sin = sin;
    p.key_pool = key_pool; p.value_pool = value_pool;
    p.key_scale = key_scale; p.value_scale = value_scale;
    p.out_query = out_query; p.status = dev_status;
    // the widest access (16 bytes of a 16-bit type, or 8, or one element) that
    // every row, stride and pointer allows
    int ve = es == 2 ? 8 : 4;
    auto fits = [&](int64_t v) {
        bool ok = half % v == 0 && (d.D - rotary_dim) % v == 0 && d.Dv % v == 0 && d.D % v == 0 &&
                  aligned(cos, 16) && aligned(sin, 16) && aligned(key_pool, v * ps) &&
                  aligned(value_pool, v * ps) && aligned(out_query, v * es) &&
                  aligned(query, v * es) && aligned(new_key, v * es) && aligned(new_value, v * es);
        for (int i = 0; i < 6; ++i) ok = ok && strides[i] % v == 0;
        return ok;
    };
    while (ve > 1 && !fits(ve)) ve = ve == 8 ? 4 : 1;
    // a block per token while blocks are few; then as many tokens as leave two rounds
    // of blocks on every SM (three of 256 threads at a time), so that the look-up of a
    // token's sequence and slot is paid for once per block's worth of loads: 9600
    // prompt tokens took 121 us at one token, 61 at four and 57 at eight
    p.tpb = static_cast<int>(std::min<int64_t>(kMaxTokensPerBlock,
                                               (T + 6 * kPlanSms - 1) / (6 * kPlanSms)));
    p.tok_blocks = static_cast<unsigned>((T + p.tpb - 1) / p.tpb);
    p.hg = T <= 2 * kPlanSms ? 1 : 4;
    // 8-bit pools: small blocks, more of them on an SM (their two passes meet at barriers)
    p.threads = eight(d) && std::max(d.D - half, d.Dv) / ve <= 128 ? 128 : 256;
    if (eight(d)) {
        p.seq_blocks = std::min<int64_t>((p.max_q + d.block_size - 2) / d.block_size + 1, d.max_blocks);
        p.units8 = d.B * p.seq_blocks * d.Hk * 2;
    }
    return launch_append_rotary(p, d.dtype, d.pool_dtype == KVC_E4M3 ? 1 : d.pool_dtype == KVC_E5M2 ? 2 : 0,
                                ve, static_cast<cudaStream_t>(stream_ptr)) == cudaSuccess
               ? KVC_OK : KVC_E_CUDA;
}

const char* kvc_attend_paged_path(const kvc_paged_dims* dims) {
    if (kvc::check_paged(dims) != KVC_OK) return nullptr;
    const kvc::TcPlan t = kvc::tc_plan(*dims);
    return !t.ok ? "cores" : t.nr ? "decode" : "rows";
}

size_t kvc_attend_paged_workspace_bytes(const kvc_paged_dims* dims) {
    if (kvc::check_paged(dims) != KVC_OK) return 0;
    // enough for either kernel: which one runs also depends on the pointers
    return static_cast<size_t>(
        kvc::up(std::max(kvc::core_plan(*dims).bytes, kvc::tc_plan(*dims).bytes), 256) + 256);
}

int kvc_attend_paged(const kvc_paged_dims* dims, const int64_t* q_strides, const void* q,
                     const void* key_pool, const void* value_pool, const float* key_scale,
                     const float* value_scale, const int32_t* block_table,
                     const int32_t* cu_seqlens_q, const int32_t* seqlens_k, double scale,
                     double softcap, const float* alibi_slopes, int64_t window, void* out,
                     void* workspace, size_t workspace_bytes, int32_t* dev_status,
                     void* stream_ptr) {
    using namespace kvc;
    const int rc = check_paged(dims);
    if (rc != KVC_OK) return rc;
    const kvc_paged_dims d = *dims;
    const int64_t T = d.total_q, es = elem(d.dtype), ps = elem(d.pool_dtype);
    if (window < 0) return KVC_E_SHAPE;
    if (!q_strides || !key_pool || !value_pool || !block_table || !cu_seqlens_q || !seqlens_k ||
        (T > 0 && (!q || !out)) ||
        (eight(d) ? (!key_scale || !value_scale) : (key_scale || value_scale)))
        return KVC_E_NULL;
    if (!(scale > 0.0) || !std::isfinite(scale) || !(softcap >= 0.0) || !std::isfinite(softcap) ||
        softcap > FLT_MAX / 4)
        return KVC_E_SCALE;
    // what the kernels form of them stays a finite, normal fp32 value
    if (scale < FLT_MIN || scale > FLT_MAX / 4 ||
        (softcap > 0.0 && (softcap < FLT_MIN || scale / softcap > FLT_MAX / 4)))
        return KVC_E_SCALE;
    for (int i = 0; i < 2; ++i)
        if (q_strides[i] < 0 || q_strides[i] > (int64_t(1) << 40)) return KVC_E_SHAPE;
    const size_t need = kvc_attend_paged_workspace_bytes(dims);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return KVC_E_WORKSPACE;
    const int64_t rows = d.num_blocks * d.Hk * d.block_size;
    const Range ins[] = {
        range_of(q, span(T, q_strides[0], d.Hq, q_strides[1], d.D, es)),
        range_of(key_pool, rows * d.D * ps),
        range_of(value_pool, rows * d.Dv * ps),
        range_of(key_scale, d.num_blocks * d.Hk * 4),
        range_of(value_scale, d.num_blocks * d.Hk * 4),
        range_of(block_table, d.B * d.max_blocks * 4),
        range_of(cu_seqlens_q, (d.B + 1) * 4),
        range_of(seqlens_k, d.B * 4),
        range_of(alibi_slopes, d.Hq * 4),
    };
    const Range o = range_of(out, T * d.Hq * d.Dv * es);
    const Range w = range_of(workspace, static_cast<int64_t>(need));
    if (overlaps(o, w)) return KVC_E_ALIAS;
    for (const Range& r : ins)
        if (overlaps(o, r) || overlaps(w, r)) return KVC_E_ALIAS;
    if (!current_is_gb300()) return KVC_E_DEVICE;
    if (T == 0) return KVC_OK;

    const CorePlan c = core_plan(d);
    PagedAttendParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = d.B; p.total_q = T; p.max_q = most_rows(d); p.M = d.max_blocks * d.block_size;
    p.max_blocks = d.max_blocks; p.num_blocks = static_cast<int>(d.num_blocks);
    p.Hq = static_cast<int>(d.Hq); p.Hk = static_cast<int>(d.Hk); p.G = static_cast<int>(d.Hq / d.Hk);
    p.D = static_cast<int>(d.D); p.Dv = static_cast<int>(d.Dv); p.bs = static_cast<int>(d.block_size);
    p.q_tok = q_strides[0]; p.q_head = q_strides[1];
    p.q = q; p.kp = key_pool; p.vp = value_pool; p.ks = key_scale; p.vs = value_scale;
    p.table = block_table; p.cu = cu_seqlens_q; p.kl = seqlens_k; p.slopes = alibi_slopes;
    p.scale = static_cast<float>(scale); p.softcap = static_cast<float>(softcap);
    p.window = window >= p.M ? 0 : static_cast<int>(window);
    p.out = out; p.status = dev_status; p.e5m2 = d.pool_dtype == KVC_E5M2;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    TcPlan t = tc_plan(d);
    // the tensor-core kernels read query rows in words of 8 bytes (split into
    // 8-bit parts) or 16 (copied)
    const int64_t qw = eight(d) ? 8 : 16;
    if (t.ok && (t.nr || aligned(out, 16)) && aligned(key_pool, 16) && aligned(value_pool, 16) && aligned(q, qw) &&
        q_strides[0] * es % qw == 0 && q_strides[1] * es % qw == 0 &&
        pool_map(&t.p.tk, key_pool, d, d.D, t.p.hh) && pool_map(&t.p.tv, value_pool, d, d.Dv, t.p.hh)) {
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        t.p.a = p;
        t.p.rec = reinterpret_cast<PagedRec*>(ws);
        t.p.part_ml = reinterpret_cast<float*>(ws + t.off_ml);
        t.p.part_acc = reinterpret_cast<float*>(ws + t.off_acc);
        cudaError_t e = t.nr ? launch_paged_decode(t.p, d.dtype, d.pool_dtype, t.nr, t.smem, stream)
                             : launch_paged_rows(t.p, d.dtype, d.pool_dtype, t.smem, stream);
        if (e == cudaSuccess) e = launch_paged_merge(t.p, d.dtype, stream);
        return e == cudaSuccess ? KVC_OK : KVC_E_CUDA;
    }
    p.nsplit = static_cast<int>(c.nsplit); p.split_len = static_cast<int>(c.split_len);
    p.part_ml = static_cast<float*>(workspace);
    p.part_acc = p.part_ml + 2 * c.nsplit * T * d.Hq;
    return launch_paged_attend(p, d.dtype, d.pool_dtype, stream) == cudaSuccess ? KVC_OK : KVC_E_CUDA;
}

}  // extern "C"
