// sv_rotate.cu -- rotary positions on a round's queries and keys, the rotated keys and
// the values written to their pages (spec_verify_rotate_append).
//
// A rotation mixes two elements of a head, so a thread takes 8 + 8 of them: elements
// (8j .., rot_dim/2 + 8j ..) of a half-split head, or 16 neighbours of an interleaved
// one.  Either way they are two 16-byte vectors and 8 pairs whose cosines and sines lie
// together in the table.  Past rot_dim, and for v, the 16 elements are copied.
//
// A block has one token; a thread keeps its place j in the head and goes over the heads
// of q, k and v, kHeads at a time, so that it reads its 16 cosines and sines once and has
// 2 kHeads loads in flight.  (One head a thread, with the token found by a division for
// each, took 35 us for two chunks of 4096 tokens, 4.4 TB/s; this form takes 28 us, 5.45 TB/s;
// two heads in flight 29.0, six 30.8, blocks of 256 threads 37.6 us.)  The call is bound by
// reading q, k, v and writing q', k', v' once; small ones by the chain lengths -> page id ->
// store.
#include <cuda_runtime.h>

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {
namespace {

constexpr int kRThreads = 128;
constexpr int kHeads = 4;  // heads that a thread has in flight

template <typename T>
__device__ __forceinline__ void rotate16(uint4& x0, uint4& x1, const float (&cs)[8], const float (&sn)[8],
                                         bool interleaved) {
    uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    if (interleaved) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const float2 f = Pair<T>::unpack(w[p]);
            w[p] = Pair<T>::pack(f.x * cs[p] - f.y * sn[p], f.y * cs[p] + f.x * sn[p]);
        }
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float2 f = Pair<T>::unpack(w[p]), g = Pair<T>::unpack(w[p + 4]);
            w[p] = Pair<T>::pack(f.x * cs[2 * p] - g.x * sn[2 * p], f.y * cs[2 * p + 1] - g.y * sn[2 * p + 1]);
            w[p + 4] = Pair<T>::pack(g.x * cs[2 * p] + f.x * sn[2 * p], g.y * cs[2 * p + 1] + f.y * sn[2 * p + 1]);
        }
    }
    x0 = make_uint4(w[0], w[1], w[2], w[3]);
    x1 = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T>
__global__ void __launch_bounds__(kRThreads) rotate_kernel(const __grid_constant__ sv_rotate_args a) {
    const int per = (int)a.dim / 16;          // threads of a head
    const int sets = kRThreads / per;         // heads at once
    const int j = threadIdx.x % per, set = threadIdx.x / per;
    const int b = (int)(blockIdx.x / (unsigned)a.N), i = (int)(blockIdx.x % (unsigned)a.N);
    const int64_t table_cap = a.cache.pages_per_seq * a.cache.page_size;
    const SeqLens sl = seq_lens(a.cache, b, (int)a.N, a.table_len < table_cap ? a.table_len : table_cap);
    const bool live = i < sl.n;
    if (sl.bad && threadIdx.x == 0 && i == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_LENGTH);
    if (set >= sets) return;
    const int half = (int)a.rot_dim / 2, Hq = (int)a.q_heads, Hkv = (int)a.kv_heads;
    const bool turns = 16 * j < a.rot_dim;
    const int e0 = turns && !a.interleaved ? 8 * j : 16 * j;
    const int e1 = turns && !a.interleaved ? half + 8 * j : 16 * j + 8;
    const int pos = sl.past + i;
    int page = -1;
    int64_t in_page = 0;
    if (live) {
        const int at = pos / (int)a.cache.page_size;
        page = a.cache.page_table[b * a.cache.page_table_stride + at];
        in_page = pos - at * (int)a.cache.page_size;
        if (page < 0 || page >= a.cache.pages) {
            page = -1;
            if (threadIdx.x == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_PAGE);
        }
    }
    const int heads = live ? Hq + 2 * Hkv : Hq;
    auto source = [&](int h) -> const T* {
        if (h < Hq) return (const T*)a.q + b * a.q_stride_b + i * a.q_stride_n + h * a.q_stride_h;
        if (h < Hq + Hkv) return (const T*)a.k + b * a.k_stride_b + i * a.k_stride_n + (h - Hq) * a.k_stride_h;
        return (const T*)a.v + b * a.v_stride_b + i * a.v_stride_n + (h - Hq - Hkv) * a.v_stride_h;
    };
    auto target = [&](int h) -> T* {
        if (h < Hq) return (T*)a.q_out + b * a.o_stride_b + i * a.o_stride_n + h * a.o_stride_h;
        if (page < 0) return nullptr;
        if (h < Hq + Hkv)
            return (T*)a.cache.k_pages + page * a.cache.k_stride_page + (h - Hq) * a.cache.k_stride_head +
                   in_page * a.cache.k_stride_slot;
        return (T*)a.cache.v_pages + page * a.cache.v_stride_page + (h - Hq - Hkv) * a.cache.v_stride_head +
               in_page * a.cache.v_stride_slot;
    };
    float cs[8], sn[8];
    if (live && turns) {
        const float4* c4 = reinterpret_cast<const float4*>(a.table + (int64_t)pos * a.rot_dim + 8 * j);
        const float4* s4 = reinterpret_cast<const float4*>(a.table + (int64_t)pos * a.rot_dim + half + 8 * j);
        *reinterpret_cast<float4*>(cs) = __ldg(c4);
        *reinterpret_cast<float4*>(cs + 4) = __ldg(c4 + 1);
        *reinterpret_cast<float4*>(sn) = __ldg(s4);
        *reinterpret_cast<float4*>(sn + 4) = __ldg(s4 + 1);
    }
    for (int h0 = set; h0 < heads; h0 += kHeads * sets) {
        uint4 x0[kHeads], x1[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * sets;
            const uint32_t w = sl.bad ? Pair<T>::pack(NAN, NAN) : 0u;  // rows without a token
            x0[k] = x1[k] = make_uint4(w, w, w, w);
            if (h < heads && live) {
                const T* src = source(h);
                x0[k] = *reinterpret_cast<const uint4*>(src + e0);
                x1[k] = *reinterpret_cast<const uint4*>(src + e1);
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * sets;
            if (h >= heads) break;
            if (live && turns && h < Hq + Hkv) rotate16<T>(x0[k], x1[k], cs, sn, a.interleaved != 0);
            T* dst = target(h);
            if (!dst) continue;
            *reinterpret_cast<uint4*>(dst + e0) = x0[k];
            *reinterpret_cast<uint4*>(dst + e1) = x1[k];
        }
    }
}

}  // namespace
}  // namespace sv

extern "C" int spec_verify_rotate_append(const sv_rotate_args* args, void* stream) {
    if (!args || args->struct_size != sizeof(sv_rotate_args)) return SV_EINVAL;
    const sv_rotate_args& a = *args;
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) return SV_EUNSUPPORTED;
    if (a.B < 0 || a.N < 1 || a.q_heads < 1 || a.kv_heads < 1 || a.dim < 16 || a.dim % 16) return SV_EINVAL;
    if (a.rot_dim < 16 || a.rot_dim % 16 || a.rot_dim > a.dim || a.table_len < 0) return SV_EINVAL;
    if (a.dim > SV_MAX_HEAD_DIM || a.B > SV_MAX_BATCH || a.N > 0x7FFFFFFF || a.q_heads > 65536 || a.kv_heads > 65536)
        return SV_ETOO_LARGE;
    if (a.B == 0) return SV_OK;
    if (sv::bad_rows(a.q, a.q_stride_b, a.q_stride_n, a.q_stride_h) ||
        sv::bad_rows(a.q_out, a.o_stride_b, a.o_stride_n, a.o_stride_h) ||
        sv::bad_rows(a.k, a.k_stride_b, a.k_stride_n, a.k_stride_h) ||
        sv::bad_rows(a.v, a.v_stride_b, a.v_stride_n, a.v_stride_h) || !a.table || ((uintptr_t)a.table & 15u))
        return SV_EINVAL;
    // two output rows on the same memory would race
    if ((a.q_heads > 1 && a.o_stride_h < a.dim) || (a.N > 1 && a.o_stride_n < a.dim) ||
        (a.B > 1 && a.o_stride_b < a.dim))
        return SV_EINVAL;
    const int rc = sv::check_cache(a.cache, a.B, a.kv_heads, a.dim);
    if (rc != SV_OK) return rc;
    if ((double)a.B * a.N > 2147483647.0) return SV_ETOO_LARGE;
    const unsigned grid = (unsigned)(a.B * a.N);
    cudaStream_t s = (cudaStream_t)stream;
    if (a.dtype == SV_BF16)
        sv::rotate_kernel<__nv_bfloat16><<<grid, sv::kRThreads, 0, s>>>(a);
    else
        sv::rotate_kernel<__half><<<grid, sv::kRThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
