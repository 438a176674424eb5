// sv_attend.cu -- host side of spec_verify_attention: checks, the choice of kernel, the
// workspace.
#include "sv_attend.cuh"

#include <cstring>
#include <mutex>

namespace sv {
namespace {

constexpr double kLog2e = 1.4426950408889634;

// Rows of a cache head's tile: 16, 32 or 128 where that holds a sequence's rows, else 256.
// A tile too small reads the cache once more, one too large computes rows that are not
// there.  64 sequences behind 4096 (8 cache heads of 128), us with tiles of 16 / 32 / 128 / 256:
//    16 rows   175 /  180 / 199 / 204        36 rows   490 / 349 / 211 / 217
//    20 rows   331 /  186 / 199 / 204       128 rows  1278 / 697 / 224 / 228
//    32 rows   333 /  190 / 201 / 204       132 rows  1437 / 859 / 398 / 239
// (Of calls of some 20 us, 36 rows take 14.7 us in tiles of 32 and 18.0 in one of 128.)
// Over a cache held in 8 bits the borders are the same: 64 sequences x 8 tokens behind 1.5-8k (32 rows)
// take 226 us in a tile of 32 and 436 in one of 128; 2 x 6 tokens behind 90-131k (48 rows) 128 in two of
// 32 and 121 in one of 128; two chunks of 2048 (8192 rows) 1741 in tiles of 32 and 462 in tiles of 256.
int row_tile(int64_t N, int64_t group) {
    const int64_t rows = N * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}

int check_attention(int64_t B, int64_t N, int64_t q_heads, int64_t kv_heads, int64_t dim) {
    if (B < 0 || N < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads) return SV_EINVAL;
    if (dim != 64 && dim != 128) return SV_EUNSUPPORTED;
    if (B > SV_MAX_BATCH || q_heads > 65536 || q_heads / kv_heads > SV_MAX_GROUP || N > kMaxRows ||
        N * (q_heads / kv_heads) > kMaxRows)
        return SV_ETOO_LARGE;
    return SV_OK;
}

struct Workspace {
    size_t cut, ml, o, total;
};
Workspace workspace(int64_t dim, int rm) {
    Workspace w;
    w.cut = 0;
    w.ml = align_up(sizeof(Cut) * kMaxCtas, 256);
    w.o = align_up(w.ml + (size_t)2 * kMaxCtas * rm * 8, 256);
    w.total = align_up(w.o + (size_t)2 * kMaxCtas * rm * dim * 4, 256);
    return w;
}

int sm_count(int dev) {
    static int counts[64];
    static std::mutex mu;
    int n = 0;
    if (dev < 0 || dev >= 64)
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!counts[dev] && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) counts[dev] = n;
    return counts[dev];
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's encoder of tensor maps, fetched through the runtime (no link-time dependency)
EncodeFn encoder() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (EncodeFn)f;
    });
    return fn;
}

// pages as [pages][heads][dim / 64][page_size][64]
bool encode(CUtensorMap* m, const void* base, const AttendArgs& p, int64_t sp, int64_t sh, int64_t ss, int box,
            int parts) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[5] = {64, (cuuint64_t)p.a.cache.page_size, (cuuint64_t)p.a.dim / 64,
                                (cuuint64_t)p.a.kv_heads, (cuuint64_t)p.a.cache.pages};
    // a stride that no second element uses may be anything: give the encoder a plain one
    if (p.a.kv_heads == 1) sh = ss;
    if (p.a.cache.pages == 1) sp = ss;
    const cuuint64_t strides[4] = {(cuuint64_t)ss * 2, 128, (cuuint64_t)sh * 2, (cuuint64_t)sp * 2};
    const cuuint32_t boxes[5] = {64, (cuuint32_t)box, (cuuint32_t)parts, 1, 1}, ones[5] = {1, 1, 1, 1, 1};
    return fn(m, p.a.dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
              const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pages of codes as [pages][heads][page_size][dim]
bool encode8(CUtensorMap* m, const void* base, const AttendArgs& p, int64_t sp, int64_t sh, int64_t ss, int box) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)p.a.dim, (cuuint64_t)p.a.cache.page_size, (cuuint64_t)p.a.kv_heads,
                                (cuuint64_t)p.a.cache.pages};
    if (p.a.kv_heads == 1) sh = ss;
    if (p.a.cache.pages == 1) sp = ss;
    const cuuint64_t strides[3] = {(cuuint64_t)ss, (cuuint64_t)sh, (cuuint64_t)sp};
    const cuuint32_t boxes[4] = {(cuuint32_t)p.a.dim, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, boxes, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, p.a.dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_codes(CUtensorMap* keys, CUtensorMap* values, const AttendArgs& p, int box) {
    const sv_paged_cache& c = p.a.cache;
    return encode8(keys, c.k_pages, p, c.k_stride_page, c.k_stride_head, c.k_stride_slot, box) &&
           encode8(values, c.v_pages, p, c.v_stride_page, c.v_stride_head, c.v_stride_slot, box);
}

bool encode_pages(CUtensorMap* keys, CUtensorMap* values, const AttendArgs& p, int box, int parts) {
    const sv_paged_cache& c = p.a.cache;
    return encode(keys, c.k_pages, p, c.k_stride_page, c.k_stride_head, c.k_stride_slot, box, parts) &&
           encode(values, c.v_pages, p, c.v_stride_page, c.v_stride_head, c.v_stride_slot, box, parts);
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_verify_attention_workspace_size(int64_t B, int64_t N, int64_t q_heads, int64_t kv_heads,
                                                       int64_t dim) {
    if (check_attention(B, N, q_heads, kv_heads, dim) != SV_OK) return 0;
    return workspace(dim, row_tile(N, q_heads / kv_heads)).total;
}

namespace {

// sinks: positions that a window leaves in sight; scales: of a cache held in 8 bits, or null
int attend(const sv_attention_args* args, int64_t sinks, const sv_cache_scales* scales, void* stream) {
    if (!args || args->struct_size != sizeof(sv_attention_args)) return SV_EINVAL;
    const sv_attention_args& a = *args;
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) return SV_EUNSUPPORTED;
    int rc = check_attention(a.B, a.N, a.q_heads, a.kv_heads, a.dim);
    if (rc != SV_OK) return rc;
    if (a.window < 0 || a.max_context < 0 || !(a.scale > 0.0) || a.scale > 1e30) return SV_EINVAL;
    if (a.B == 0) return SV_OK;
    if (bad_rows(a.q, a.q_stride_b, a.q_stride_n, a.q_stride_h) ||
        bad_rows(a.out, a.o_stride_b, a.o_stride_n, a.o_stride_h))
        return SV_EINVAL;
    // two output rows on the same memory would race
    if ((a.q_heads > 1 && a.o_stride_h < a.dim) || (a.N > 1 && a.o_stride_n < a.dim) ||
        (a.B > 1 && a.o_stride_b < a.dim))
        return SV_EINVAL;
    rc = check_cache(a.cache, a.B, a.kv_heads, a.dim, scales ? 1 : 2);
    if (rc == SV_OK && scales) rc = check_scales(*scales, a.cache, a.kv_heads);
    if (rc != SV_OK) return rc;
    const int group = (int)(a.q_heads / a.kv_heads);
    const int rm = row_tile(a.N, group);
    const Workspace w = workspace(a.dim, rm);
    if (!a.workspace || a.workspace_bytes < (int64_t)w.total) return SV_EWORKSPACE;
    if ((uintptr_t)a.workspace & 255u) return SV_EINVAL;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SV_ECUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SV_ECUDA;
    AttendArgs p;
    memset(&p, 0, sizeof p);
    p.a = a;
    p.group = group;
    p.group_inv = group > 1 ? (uint32_t)(((1ull << 32) + group - 1) / group) : 0u;
    p.page_shift = -1;
    for (int i = 4; i <= 16; ++i)
        if (a.cache.page_size == (int64_t)1 << i) p.page_shift = i;
    p.max_row_tiles = (int)((a.N * group + rm - 1) / rm);
    p.qscale = (float)(a.scale * kLog2e);
    p.capacity = a.cache.pages_per_seq * a.cache.page_size;
    if (p.capacity > 0x7FFFFF00) p.capacity = 0x7FFFFF00;  // positions are 32-bit
    if (a.window > 0) {  // (positions are below 0x7FFFFF00)
        p.sinks = (int)(sinks < 0x7FFFFF00 ? sinks : 0x7FFFFF00);
        p.sink_tiles = (p.sinks + kKeyTile - 1) / kKeyTile;
    }
    if (scales) p.sc = *scales;
    char* ws = (char*)a.workspace;
    p.cut = (Cut*)(ws + w.cut);
    p.part_ml = (float*)(ws + w.ml);
    p.part_o = (float*)(ws + w.o);
    // never more CTAs than tiles: a bound from what the host knows of the lengths
    const int64_t ctx = a.max_context > 0 && a.max_context < p.capacity ? a.max_context : p.capacity;
    const double tiles = (double)a.B * a.kv_heads * (double)((a.N * group + rm - 1) / rm) *
                         (double)((ctx + kKeyTile - 1) / kKeyTile + 1);
    p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    if (tiles < p.ctas) p.ctas = (int)tiles;
    cudaStream_t s = (cudaStream_t)stream;
    p.wait_ns = a.wait_limit_ns ? a.wait_limit_ns : kWaitLimitNs;
    const auto launch = rm >= 128 ? (scales ? launch_attend_tiles_8bit : p.sinks ? launch_attend_tiles_sinks : launch_attend_tiles)
                                  : (scales ? launch_attend_rows_8bit : p.sinks ? launch_attend_rows_sinks : launch_attend_rows);
    const cudaError_t e = launch((int)a.dtype, (int)a.dim, rm >= 128 ? rm : rm / 16, p, s);
    if (e != cudaSuccess) return SV_ECUDA;
    if (launch_attend_join((int)a.dtype, (int)a.dim, rm, p, s) != cudaSuccess) return SV_ECUDA;
    return SV_OK;
}

}  // namespace

extern "C" int spec_verify_attention(const sv_attention_args* args, void* stream) {
    return attend(args, 0, nullptr, stream);
}

extern "C" int spec_verify_attention_ex(const sv_attention_args* args, const sv_attention_options* options,
                                        void* stream) {
    if (!options) return attend(args, 0, nullptr, stream);
    if (options->struct_size != sizeof(sv_attention_options) || options->sinks < 0) return SV_EINVAL;
    return attend(args, options->sinks, options->scales.k ? &options->scales : nullptr, stream);
}
