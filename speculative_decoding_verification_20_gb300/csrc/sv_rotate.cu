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
//
// Into a cache held in 8 bits the token's blocks do q alone, and further blocks of the same
// launch take one head's keys or values of 16 positions each, which share a scale: live
// elements of the block, new and held, in registers; their largest across the block; codes
// and scale written.  A key next to the border between two codes goes to one or the other:
// its rotation is formed to 1.5 steps of 32 bits, and where that leaves the side of a border
// open (one element in 60000) without error and rounded to odd, so that the one rounding to a
// code that follows is that of the exact value.  The instructions bound chunks: with the exact
// form throughout, two chunks of 4096 tokens took 42 us; now 38.  (A warp for 16 positions, four rounds each,
// took 19 us for 256 x 8 tokens with its values in registers, 29 formed twice, where a block
// for them takes 17: the chain of one thread's work is what counts.)
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

// 8-bit cache: blocks of 16 positions that the N new tokens of a sequence can touch
__host__ __device__ inline int64_t touched_blocks(int64_t N) { return (N + SV_SCALE_BLOCK - 2) / SV_SCALE_BLOCK + 1; }

// (hi + lo) rounded to odd: hi is the sum rounded to nearest, lo what is missing; of the two numbers
// around the exact one the odd one, from which a second rounding to fewer bits is the right one
__device__ __forceinline__ float to_odd(float hi, float lo) {
    if (lo == 0.0f || !isfinite(hi)) return hi;
    if (hi == 0.0f) return lo;
    const int w = __float_as_int(hi);
    return w & 1 ? hi : __int_as_float(w + ((lo > 0.0f) == (hi > 0.0f) ? 1 : -1));
}
// a + b and its rounding error (the error is exact whatever the sizes)
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
    const float s = __fadd_rn(a, b), bv = __fsub_rn(s, a), av = __fsub_rn(s, bv);
    err = __fadd_rn(__fsub_rn(b, bv), __fsub_rn(a, av));
    return s;
}
// a c + b s, rounded to odd: products and their errors, then the sum and its own.  (The products'
// errors may be steps of a smaller sum: they go into it before what is missing is looked at.)
__device__ __forceinline__ float dot2_odd(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
    const float pe = __fmaf_rn(a, c, -p), qe = __fmaf_rn(b, s, -q);
    float e, f, g, h;
    const float sum = two_sum(p, q, e);
    const float errors = two_sum(pe, qe, f);
    const float low = two_sum(e, errors, g);
    const float hi = two_sum(sum, low, h);
    return to_odd(hi, h != 0.0f ? h : __fadd_rn(g, f));
}
// A held code times its scale, rounded to odd: 28 bits where the scale is no power of two.  (The error of a
// small product is formed 2^64 times as large, so that it does not fall below 32-bit numbers.)
__device__ __forceinline__ float product_odd(float code, float scale) {
    const float p = __fmul_rn(code, scale), up = scale < 1.0f ? 0x1p64f : 1.0f;
    return p == 0.0f ? p : to_odd(p, __fmaf_rn(code, scale * up, -(p * up)));
}

// dot2_odd's sum to 1.5 steps (an exact product's error added behind the other product).
__device__ __forceinline__ float dot2(float a, float c, float b, float s) {
    const float w = __fmul_rn(b, s), e = __fmaf_rn(b, s, -w);
    return __fadd_rn(__fmaf_rn(a, c, w), e);
}
// Whether a number 3 steps away may get another code or scale: borders between codes, among them those below
// 2^-6 scale, and 448 powers of two, have zeros in their low 19 bits.
__device__ __forceinline__ bool near_border(float x) { return ((__float_as_uint(x) + 4u) & 0x7FFFFu) <= 8u; }

// One head's keys or values of a block of 16 positions, by a CTA of the launch: item x of
// [B][touched blocks][2 kv_heads].
// ITER: rounds of the block's threads over the 16 positions.
template <typename T, int ITER>
__device__ __forceinline__ void append8(const sv_rotate_args& a, const sv_cache_scales& sc, unsigned x) {
    constexpr int kTok = SV_SCALE_BLOCK;
    __shared__ float s_top[kRThreads / 32];
    const int t = threadIdx.x, Hkv = (int)a.kv_heads;
    const unsigned nb = (unsigned)touched_blocks(a.N);
    const int item = (int)(x % (2u * Hkv));
    const unsigned rest = x / (2u * Hkv);
    const int b = (int)(rest / nb);
    const bool keys = item < Hkv;
    const int h = keys ? item : item - Hkv;
    const int64_t table_cap = a.cache.pages_per_seq * a.cache.page_size;
    const SeqLens sl = seq_lens(a.cache, b, (int)a.N, a.table_len < table_cap ? a.table_len : table_cap);
    const int p0 = (sl.past / kTok + (int)(rest % nb)) * kTok;  // the block's first position
    if (sl.n == 0 || p0 >= sl.past + sl.n) return;
    const int at = p0 / (int)a.cache.page_size;
    const int page = a.cache.page_table[b * a.cache.page_table_stride + at];
    const int64_t slot = p0 - at * (int)a.cache.page_size;
    if (page < 0 || page >= a.cache.pages) {
        if (t == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_PAGE);
        return;
    }
    const int64_t cache_slot = keys ? a.cache.k_stride_slot : a.cache.v_stride_slot;
    uint8_t* codes = keys ? (uint8_t*)a.cache.k_pages + page * a.cache.k_stride_page + h * a.cache.k_stride_head
                          : (uint8_t*)a.cache.v_pages + page * a.cache.v_stride_page + h * a.cache.v_stride_head;
    codes += slot * cache_slot;
    float* scale_at = (keys ? sc.k + page * sc.k_stride_page + h * sc.k_stride_head
                            : sc.v + page * sc.v_stride_page + h * sc.v_stride_head) + slot / kTok;
    const float held_scale = p0 < sl.past ? *scale_at : 1.0f;
    const int per = (int)a.dim / 16, sets = kRThreads / per, half = (int)a.rot_dim / 2;
    const int j = t % per, set = t / per;
    const bool turns = keys && 16 * j < a.rot_dim;
    const int e0 = turns && !a.interleaved ? 8 * j : 16 * j;
    const int e1 = turns && !a.interleaved ? half + 8 * j : 16 * j + 8;
    float v[ITER][16];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int tok = set + i * sets, pos = p0 + tok;
#pragma unroll
        for (int e = 0; e < 16; ++e) v[i][e] = 0.0f;
        if (set >= sets || tok >= kTok || pos >= sl.past + sl.n) continue;
        if (pos < sl.past) {
            const uint8_t* src = codes + tok * cache_slot;
            const uint2 w0 = *reinterpret_cast<const uint2*>(src + e0), w1 = *reinterpret_cast<const uint2*>(src + e1);
            const uint32_t w[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = e4m3_pair(w[e / 2] >> (e % 2 * 16));
                v[i][2 * e] = f.x * held_scale, v[i][2 * e + 1] = f.y * held_scale;
            }
            if (__float_as_int(held_scale) & 0x7FFFFF) {  // a scale that the caller set, no power of two
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = e4m3_pair(w[e / 2] >> (e % 2 * 16));
                    v[i][2 * e] = product_odd(f.x, held_scale), v[i][2 * e + 1] = product_odd(f.y, held_scale);
                }
            }
        } else {
            const int64_t n = pos - sl.past;
            const T* src = keys ? (const T*)a.k + b * a.k_stride_b + n * a.k_stride_n + h * a.k_stride_h
                                : (const T*)a.v + b * a.v_stride_b + n * a.v_stride_n + h * a.v_stride_h;
            const uint4 x0 = *reinterpret_cast<const uint4*>(src + e0), x1 = *reinterpret_cast<const uint4*>(src + e1);
            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = Pair<T>::unpack(w[e]);
                v[i][2 * e] = f.x, v[i][2 * e + 1] = f.y;
            }
            if (turns) {
                float cs[8], sn[8];
                const float4* c4 = reinterpret_cast<const float4*>(a.table + (int64_t)pos * a.rot_dim + 8 * j);
                const float4* s4 = reinterpret_cast<const float4*>(a.table + (int64_t)pos * a.rot_dim + half + 8 * j);
                *reinterpret_cast<float4*>(cs) = __ldg(c4);
                *reinterpret_cast<float4*>(cs + 4) = __ldg(c4 + 1);
                *reinterpret_cast<float4*>(sn) = __ldg(s4);
                *reinterpret_cast<float4*>(sn + 4) = __ldg(s4 + 1);
                // pairs (e, e + 8) from here on
                if (a.interleaved) {
                    float r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = v[i][e];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = r[2 * e], v[i][e + 8] = r[2 * e + 1];
                }
                bool open = false;
                float r[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[e] = dot2(v[i][e], cs[e], -v[i][e + 8], sn[e]);
                    r[e + 8] = dot2(v[i][e + 8], cs[e], v[i][e], sn[e]);
                    open |= near_border(r[e]) | near_border(r[e + 8]);
                }
                if (open) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        r[e] = dot2_odd(v[i][e], cs[e], -v[i][e + 8], sn[e]);
                        r[e + 8] = dot2_odd(v[i][e + 8], cs[e], v[i][e], sn[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) v[i][e] = a.interleaved ? r[e / 2 + e % 2 * 8] : r[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (fabsf(v[i][e]) < INFINITY)
                top = fmaxf(top, fabsf(v[i][e]));
            else
                v[i][e] = NAN;  // (the conversion alone would make the largest value of an infinity)
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (t % 32 == 0) s_top[t / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRThreads / 32; ++w) top = fmaxf(top, s_top[w]);
    // the least power of two s with top <= 448 s = 1.75 2^8 s: from top's exponent and fraction bits
    const int bits = __float_as_int(top);
    const int k = max((bits >> 23) - 127 - ((bits & 0x7FFFFF) <= 0x600000 ? 8 : 7), -126);
    const float scale = top > 0.0f ? __int_as_float((k + 127) << 23) : 1.0f;
    const float inv = top > 0.0f ? __int_as_float((127 - k) << 23) : 1.0f;
    if (t == 0) *scale_at = scale;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int tok = set + i * sets, pos = p0 + tok;
        if (set >= sets || tok >= kTok || pos >= sl.past + sl.n || (pos < sl.past && scale == held_scale)) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = to_e4m3(v[i][4 * e] * inv, v[i][4 * e + 1] * inv) |
                                           to_e4m3(v[i][4 * e + 2] * inv, v[i][4 * e + 3] * inv) << 16;
        uint8_t* dst = codes + tok * cache_slot;
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + e1) = make_uint2(w[2], w[3]);
    }
}

// ITER: of append8, for a cache held in 8 bits (0: 16 bits)
template <typename T, int ITER>
__global__ void __launch_bounds__(kRThreads, 8) rotate_kernel(const __grid_constant__ sv_rotate_args a,
                                                           const __grid_constant__ sv_cache_scales sc) {
    constexpr bool E8 = ITER > 0;
    unsigned token = blockIdx.x;
    if constexpr (E8) {
        // (the appending blocks first: their chain is the longer one)
        const unsigned appends = gridDim.x - (unsigned)(a.B * a.N);
        if (blockIdx.x < appends) {
            append8<T, ITER>(a, sc, blockIdx.x);
            return;
        }
        token -= appends;
    }
    const int per = (int)a.dim / 16;          // threads of a head
    const int sets = kRThreads / per;         // heads at once
    const int j = threadIdx.x % per, set = threadIdx.x / per;
    const int b = (int)(token / (unsigned)a.N), i = (int)(token % (unsigned)a.N);
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
    if (!E8 && live) {
        const int at = pos / (int)a.cache.page_size;
        page = a.cache.page_table[b * a.cache.page_table_stride + at];
        in_page = pos - at * (int)a.cache.page_size;
        if (page < 0 || page >= a.cache.pages) {
            page = -1;
            if (threadIdx.x == 0 && a.row_status) atomicOr(a.row_status + b, SV_ROW_BAD_PAGE);
        }
    }
    const int heads = live && !E8 ? Hq + 2 * Hkv : Hq;
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

namespace {

// scales: of a cache held in 8 bits, or null
int rotate_append(const sv_rotate_args* args, const sv_cache_scales* scales, void* stream) {
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
    int rc = sv::check_cache(a.cache, a.B, a.kv_heads, a.dim, scales ? 1 : 2);
    if (rc == SV_OK && scales) rc = sv::check_scales(*scales, a.cache, a.kv_heads);
    if (rc != SV_OK) return rc;
    const double blocks = (double)a.B * a.N + (scales ? 2.0 * a.B * sv::touched_blocks(a.N) * a.kv_heads : 0.0);
    if (blocks > 2147483647.0) return SV_ETOO_LARGE;
    const unsigned grid = (unsigned)blocks;
    cudaStream_t s = (cudaStream_t)stream;
    const sv_cache_scales none = {};
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        // a block has 16 positions of up to 128 elements in one round
        const auto kernel = !scales ? sv::rotate_kernel<T, 0> : a.dim <= 128 ? sv::rotate_kernel<T, 1> : sv::rotate_kernel<T, 2>;
        kernel<<<grid, sv::kRThreads, 0, s>>>(a, scales ? *scales : none);
    };
    if (a.dtype == SV_BF16)
        launch(__nv_bfloat16());
    else
        launch(__half());
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}

}  // namespace

extern "C" int spec_verify_rotate_append(const sv_rotate_args* args, void* stream) {
    return rotate_append(args, nullptr, stream);
}

extern "C" int spec_verify_rotate_append_ex(const sv_rotate_args* args, const sv_rotate_options* options, void* stream) {
    if (options && options->struct_size != sizeof(sv_rotate_options)) return SV_EINVAL;
    return rotate_append(args, options && options->scales.k ? &options->scales : nullptr, stream);
}
