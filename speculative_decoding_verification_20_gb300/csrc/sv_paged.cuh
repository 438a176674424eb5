// sv_paged.cuh -- what the rotary and the attention kernels share: 16-bit element
// types, a sequence's lengths, and checks of a paged cache's description.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify_target.h"

namespace sv {

#ifdef __CUDACC__
__device__ __forceinline__ float2 to_float2(__nv_bfloat162 h) { return __bfloat1622float2(h); }
__device__ __forceinline__ float2 to_float2(__half2 h) { return __half22float2(h); }

template <typename T>
struct Pair;  // two elements in one 32-bit word
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// Cached and new tokens of a sequence.  bad: lengths that no result can be given
// for (n is 0 then); capacity: positions that the page table can address.
struct SeqLens {
    int past, n;
    bool bad;
};
__device__ __forceinline__ SeqLens seq_lens(const sv_paged_cache& c, int b, int N, int64_t capacity) {
    SeqLens s;
    s.past = c.cache_lens[b];
    s.n = c.num_new ? c.num_new[b] : N;
    s.bad = s.past < 0 || s.n < 0 || s.n > N || (int64_t)s.past + s.n > capacity;
    if (s.bad) s.past = s.n = 0;
    return s;
}
#endif  // __CUDACC__

// host checks of the cache's description (dim: elements of a head's row)
inline int check_cache(const sv_paged_cache& c, int64_t B, int64_t kv_heads, int64_t dim) {
    if (!c.k_pages || !c.v_pages || !c.page_table || !c.cache_lens) return SV_EINVAL;
    if (c.pages < 1 || c.page_size < 16 || c.page_size % 16 || c.pages_per_seq < 1) return SV_EINVAL;
    if (c.pages > 0x7FFFFFFF || c.page_size > 65536 || c.pages_per_seq > 0x7FFFFFFF) return SV_ETOO_LARGE;
    if (c.page_table_stride < 0 || (B > 1 && c.page_table_stride < c.pages_per_seq)) return SV_EINVAL;
    if (((uintptr_t)c.k_pages | (uintptr_t)c.v_pages) & 15u) return SV_EINVAL;
    const int64_t st[6] = {c.k_stride_page, c.k_stride_head, c.k_stride_slot,
                           c.v_stride_page, c.v_stride_head, c.v_stride_slot};
    for (int64_t x : st)
        if (x < 0 || x % 8) return SV_EINVAL;
    if (c.k_stride_slot < dim || c.v_stride_slot < dim) return SV_EINVAL;
    if (kv_heads > 1 && (c.k_stride_head < dim || c.v_stride_head < dim)) return SV_EINVAL;
    return SV_OK;
}

inline bool bad_rows(const void* p, int64_t sb, int64_t sn, int64_t sh) {
    return !p || ((uintptr_t)p & 15u) || sb < 0 || sn < 0 || sh < 0 || sb % 8 || sn % 8 || sh % 8;
}

}  // namespace sv
