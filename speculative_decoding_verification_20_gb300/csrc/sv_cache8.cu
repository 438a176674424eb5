// sv_cache8.cu -- reading back what a cache held in 8 bits stands for (spec_verify_read_cache).
//
// A block has four positions; a thread takes 16 codes of a head's row, keys or values, of each and
// writes 16 numbers.  The call is bound by its bytes (1 read, 2 written an element), small
// ones by the chain lengths -> page id -> codes, which the four go through together.
#include <cuda_runtime.h>

#include <type_traits>

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {
namespace {

constexpr int kReadThreads = 128, kReadRows = 4;

// A code times a scale of 24 bits has 28, and is rounded once: the product is cut to 24 bits, and its last bit set where
// something may be missing.  That is the exact product's rounding if that is not itself in the middle between two
// results (9 bits; fp16: 12): a scale of more significant bits than these gives none that is, since a product's odd part
// is a multiple of the scale's; with one of fewer the product has 16 at most, and nothing is cut off (of a bf16 result
// below 2^-134 something may be, and does not matter).
template <typename T>
__device__ __forceinline__ uint32_t last_bit(float scale) {
    constexpr uint32_t kBelow = std::is_same<T, __half>::value ? 0xFFFu : 0x7FFFu;
    return (__float_as_uint(scale < 1.0f ? scale * 0x1p64f : scale) & kBelow) != 0;  // (subnormal ones have fewer)
}
__device__ __forceinline__ float product_cut(float code, float scale, uint32_t last) {
    return __uint_as_float(__float_as_uint(__fmul_rz(code, scale)) | last);
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ sv_read_args a) {
    const unsigned groups = (unsigned)((a.N + kReadRows - 1) / kReadRows);
    const int b = (int)(blockIdx.x / groups), i0 = (int)(blockIdx.x % groups) * kReadRows;
    const int H = (int)a.kv_heads, per = (int)a.dim / 16;
    const SeqLens sl = seq_lens(a.cache, b, (int)a.N, a.cache.pages_per_seq * a.cache.page_size);
    if (sl.bad && threadIdx.x == 0 && i0 == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_LENGTH);
    int64_t page[kReadRows], slot[kReadRows];
    bool nan[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        page[i] = -1;  // (nothing to read)
        slot[i] = 0;
        nan[i] = sl.bad;
        if (i0 + i >= sl.n) continue;
        const int pos = sl.past + i0 + i, at = pos / (int)a.cache.page_size;
        page[i] = a.cache.page_table[b * a.cache.page_table_stride + at];
        slot[i] = pos - at * (int)a.cache.page_size;
        nan[i] = page[i] < 0 || page[i] >= a.cache.pages;
        if (nan[i]) {
            page[i] = -1;
            if (threadIdx.x == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_PAGE);
        }
    }
    for (int x = threadIdx.x; x < 2 * H * per; x += kReadThreads) {
        const bool keys = x < H * per;
        const int y = keys ? x : x - H * per, h = y / per, c = y % per * 16;
        const uint8_t* base = keys ? (const uint8_t*)a.cache.k_pages + h * a.cache.k_stride_head
                                   : (const uint8_t*)a.cache.v_pages + h * a.cache.v_stride_head;
        const float* scales = keys ? a.scales.k + h * a.scales.k_stride_head : a.scales.v + h * a.scales.v_stride_head;
        const int64_t sp = keys ? a.cache.k_stride_page : a.cache.v_stride_page;
        const int64_t ss = keys ? a.cache.k_stride_slot : a.cache.v_stride_slot;
        const int64_t scp = keys ? a.scales.k_stride_page : a.scales.v_stride_page;
        uint4 q[kReadRows];
        float s[kReadRows];
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            if (page[i] < 0) continue;
            q[i] = *reinterpret_cast<const uint4*>(base + page[i] * sp + slot[i] * ss + c);
            s[i] = scales[page[i] * scp + slot[i] / SV_SCALE_BLOCK];
        }
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            if (i0 + i >= a.N) break;
            const uint32_t none = nan[i] ? Pair<T>::pack(NAN, NAN) : 0u;
            uint32_t w[8] = {none, none, none, none, none, none, none, none};
            if (page[i] >= 0) {
                const uint32_t last = last_bit<T>(s[i]);
                const uint32_t qs[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = e4m3_pair(qs[e / 2] >> (e % 2 * 16));
                    w[e] = Pair<T>::pack(product_cut(f.x, s[i], last), product_cut(f.y, s[i], last));
                }
            }
            T* dst = (T*)(keys ? a.k_out : a.v_out) + (((int64_t)b * a.N + i0 + i) * H + h) * a.dim + c;
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

}  // namespace
}  // namespace sv

extern "C" int spec_verify_read_cache(const sv_read_args* args, void* stream) {
    if (!args || args->struct_size != sizeof(sv_read_args)) return SV_EINVAL;
    const sv_read_args& a = *args;
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) return SV_EUNSUPPORTED;
    if (a.B < 0 || a.N < 1 || a.kv_heads < 1 || a.dim < 16 || a.dim % 16) return SV_EINVAL;
    if (a.dim > SV_MAX_HEAD_DIM || a.B > SV_MAX_BATCH || a.N > 0x7FFFFFFF || a.kv_heads > 65536 ||
        (double)a.B * a.N > 2147483647.0)
        return SV_ETOO_LARGE;
    if (a.B == 0) return SV_OK;
    if (!a.k_out || !a.v_out || (((uintptr_t)a.k_out | (uintptr_t)a.v_out) & 15u)) return SV_EINVAL;
    int rc = sv::check_cache(a.cache, a.B, a.kv_heads, a.dim, 1);
    if (rc == SV_OK) rc = sv::check_scales(a.scales, a.cache, a.kv_heads);
    if (rc != SV_OK) return rc;
    const unsigned grid = (unsigned)(a.B * ((a.N + sv::kReadRows - 1) / sv::kReadRows));
    cudaStream_t s = (cudaStream_t)stream;
    if (a.dtype == SV_BF16)
        sv::read_kernel<__nv_bfloat16><<<grid, sv::kReadThreads, 0, s>>>(a);
    else
        sv::read_kernel<__half><<<grid, sv::kReadThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
