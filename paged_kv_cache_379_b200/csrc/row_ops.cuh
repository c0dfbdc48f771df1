// row_ops.cuh -- per-row work between the projection and the cache:
//   row_kernel         RMS norm of each query / key head, position rotation, and
//                      the write of K and V rows into a bf16, FP8 or 4-bit cache
//                      (any part of that alone: norm + rotation only, or the
//                      4-bit cache write only),
//   dequantize_blocks_int4_kernel  whole 4-bit blocks back to bf16 blocks.
//
// 4-bit cache: one record per (block, KV head), [num_blocks, num_kv_heads, record]:
//   BS rows of D/2 code bytes (dim 2i in the low nibble of byte i, dim 2i+1 in
//   the high one), then BS pairs (scale, zero) of bf16.  A code c of row o stands
//   for zero_o + scale_o * c.  The record of one head of a block is contiguous
//   (1088 bytes at D = 128, BS = 16), so the decode fetches it with one bulk copy.
// A row is quantised against its own minimum and maximum:
//   zero = min x (a bf16 value already), scale = bf16(fp32(max r) - fp32(min r)),
//   r = fp32(1/15)  (the two products keep max - min from overflowing),
//   code = clamp(rint(fp32(fp32(x - zero) * fp32(1 / scale))), 0, 15).
// Every step is one correctly rounded fp32 operation, so the codes are defined
// bit for bit.  A row of range below 2^-126 * 15 or so has scale 0 and codes 0
// (its values are its minimum); a row holding a NaN or an infinity stands for
// NaN throughout (zero = NaN, scale 0, codes 0): it shows up, it is not hidden.
// Included once, by pagedkv.cu.
#pragma once

#include "cache_ops.cuh"
#include "common.cuh"

namespace pakv {

constexpr int kCacheNone = 0, kCacheBf16 = 1, kCacheFp8 = 2, kCacheInt4 = 3;

struct RowParams {
    const __nv_bfloat16 *query, *key, *value;       // token t's heads start at t * stride
    int64_t q_stride, k_stride, v_stride;           // elements
    __nv_bfloat16 *query_out, *key_out;             // key_out: nullptr = not wanted
    int64_t qo_stride, ko_stride;
    const __nv_bfloat16 *q_weight, *k_weight;       // [D] or nullptr (no scaling by a weight)
    float eps;
    const float *cos_sin;                           // [max_position, rot]: rot/2 cosines, then rot/2 sines
    int rot, max_position;
    const int64_t *positions;                       // [T]
    const int64_t *slots;                           // [T], or nullptr: the newest position of each sequence
    const int32_t *block_tables, *seq_lens;         // (slots == nullptr)
    int64_t *slots_out;                             // (slots == nullptr) receives the slots, or nullptr
    int max_blocks;
    void *key_cache, *value_cache;
    int num_heads, num_kv_heads, rows;              // rows of one token: Hq + Hkv (+ Hkv with a cache)
    int block_size;
    int64_t num_slots;
    float k_inv, v_inv;                             // inverse scales of an FP8 cache
    int units, chunks;                              // warps of work; per token
};

__device__ __forceinline__ int int4_record_bytes(int block_size, int d) { return block_size * (d / 2 + 4); }

__device__ __forceinline__ void unpack8(const uint4 &w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Quantises a row spread over LPR neighbouring lanes, 8 values each: this lane's
// 8 codes, and the row's packed (scale, zero) pair (the same in every lane).
template <int LPR>
__device__ __forceinline__ uint32_t quantise_row_int4(const float *x, uint32_t &pair)
{
    float lo = x[0], hi = x[0];
    bool finite = fabsf(x[0]) <= 3.402823466e38f;
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
        finite &= fabsf(x[e]) <= 3.402823466e38f;
    }
    if (!finite) hi = INFINITY;  // fmin and fmax would drop a NaN
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    constexpr float r15 = 1.0f / 15.0f;
    float scale = __bfloat162float(__float2bfloat16_rn(__fsub_rn(__fmul_rn(hi, r15), __fmul_rn(lo, r15))));
    float zero = lo + 0.0f;  // -0 and +0 are one minimum
    float inv = 0.f;
    if (!(hi < INFINITY)) {
        scale = 0.f;
        zero = __uint_as_float(0x7FC00000u);
    } else if (scale >= 1.17549435e-38f) {
        inv = __frcp_rn(scale);
    } else {
        scale = 0.f;
    }
    uint32_t codes = 0;
    if (scale > 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = fminf(__fmul_rn(__fsub_rn(x[e], zero), inv), 15.f);
            // adding 2^23 rounds to the nearest integer, ties to even
            codes |= (__float_as_uint(__fadd_rn(t, 8388608.f)) & 15u) << (4 * e);
        }
    }
    pair = pack_bf16x2(scale, zero);
    return codes;
}

// A warp takes U * (32 / LPR) rows of one token (LPR = D / 8 lanes a row, 16
// bytes a lane), so the token's cosines and sines are loaded once for all of
// them and every lane has U loads in flight.  Bound by HBM: each row is read and
// written once.
template <int D, int CACHE, bool ROPE, bool INTERLEAVED>
__global__ void __launch_bounds__(256) row_kernel(const RowParams p)
{
    constexpr int LPR = D / 8;
    constexpr int GPW = 32 / LPR;
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const int gl = lane % LPR, grp = lane / LPR;
    const int unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    // With ROPE the kernel writes queries (and keys), which the kernels after it
    // may read before their own griddepcontrol.wait: it never lets them start early.
    if constexpr (!ROPE) pdl_launch_dependents();
    if (unit >= p.units) return;
    const int t = unit / p.chunks;
    const int c = unit - t * p.chunks;

    float cs[8], sn[8];
    int half = 0;  // lanes per rotated half (half-split pairs)
    bool turned = false;
    if constexpr (ROPE) {
        const int64_t pos = p.positions[t];
        if (pos < 0 || pos >= p.max_position) return;  // padding: nothing is written
        const float *row = p.cos_sin + pos * p.rot;
        if constexpr (INTERLEAVED) {
            turned = gl * 8 < p.rot;
            if (turned) {
                *reinterpret_cast<float4 *>(cs) = *reinterpret_cast<const float4 *>(row + gl * 4);
                *reinterpret_cast<float4 *>(sn) = *reinterpret_cast<const float4 *>(row + p.rot / 2 + gl * 4);
            }
        } else {
            half = p.rot / 16;
            turned = gl < 2 * half;
            if (turned) {
                const int i = (gl < half ? gl : gl - half) * 8;
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    *reinterpret_cast<float4 *>(cs + e) = *reinterpret_cast<const float4 *>(row + i + e);
                    *reinterpret_cast<float4 *>(sn + e) = *reinterpret_cast<const float4 *>(row + p.rot / 2 + i + e);
                }
            }
        }
    }
    int64_t slot = -1;
    if constexpr (CACHE != kCacheNone) {
        if (p.slots) {
            slot = p.slots[t];
        } else {
            const int64_t pos = (int64_t)p.seq_lens[t] - 1;
            if (pos >= 0 && pos / p.block_size < p.max_blocks) {
                const int32_t b = p.block_tables[(int64_t)t * p.max_blocks + pos / p.block_size];
                if (b >= 0) slot = (int64_t)b * p.block_size + pos % p.block_size;
            }
            if (c == 0 && lane == 0 && p.slots_out) p.slots_out[t] = slot;
        }
        if (slot >= p.num_slots) slot = -1;
    }

    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int r = (c * U + i) * GPW + grp;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= p.rows) continue;
        const __nv_bfloat16 *src;
        if (r < p.num_heads)
            src = p.query + t * p.q_stride + (int64_t)r * D;
        else if (r < p.num_heads + p.num_kv_heads)
            src = p.key + t * p.k_stride + (int64_t)(r - p.num_heads) * D;
        else
            src = p.value + t * p.v_stride + (int64_t)(r - p.num_heads - p.num_kv_heads) * D;
        raw[i] = *reinterpret_cast<const uint4 *>(src + gl * 8);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int r = (c * U + i) * GPW + grp;
        const bool is_q = r < p.num_heads;
        const bool is_k = !is_q && r < p.num_heads + p.num_kv_heads;
        const int h = is_q ? r : (is_k ? r - p.num_heads : r - p.num_heads - p.num_kv_heads);
        if constexpr (ROPE) {
            float x[8], y[8];
            unpack8(raw[i], x);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float rms = rsqrtf(ss * (1.0f / D) + p.eps);
            const __nv_bfloat16 *w = is_q ? p.q_weight : p.k_weight;
            float wf[8];
            if (w) {
                unpack8(*reinterpret_cast<const uint4 *>(w + gl * 8), wf);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) wf[e] = 1.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * rms * wf[e];
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    y[e] = turned ? x[e] * cs[e / 2] - x[e + 1] * sn[e / 2] : x[e];
                    y[e + 1] = turned ? x[e + 1] * cs[e / 2] + x[e] * sn[e / 2] : x[e + 1];
                }
            } else {
                // the pair's other element sits `half` lanes away in the row's lane group
                const int other = grp * LPR + (gl < half ? gl + half : gl - half);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float o = __shfl_sync(0xffffffffu, x[e], turned ? other : lane);
                    y[e] = turned ? (gl < half ? x[e] * cs[e] - o * sn[e] : x[e] * cs[e] + o * sn[e]) : x[e];
                }
            }
            if (is_q || is_k) raw[i] = pack8(y);  // rounded to bf16 once; V rows stay as they are
        }
        const bool live = r < p.rows;
        if (live && is_q) *reinterpret_cast<uint4 *>(p.query_out + t * p.qo_stride + (int64_t)h * D + gl * 8) = raw[i];
        if (live && is_k && p.key_out)
            *reinterpret_cast<uint4 *>(p.key_out + t * p.ko_stride + (int64_t)h * D + gl * 8) = raw[i];
        if constexpr (CACHE == kCacheBf16) {
            if (live && !is_q && slot >= 0)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_k ? p.key_cache : p.value_cache) +
                                           (slot * p.num_kv_heads + h) * D + gl * 8) = raw[i];
        } else if constexpr (CACHE == kCacheFp8) {
            if (live && !is_q && slot >= 0) {
                float x[8];
                unpack8(raw[i], x);
                const float inv = is_k ? p.k_inv : p.v_inv;
                uint32_t w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[e] = f32x2_to_e4m3x2(__fmul_rn(x[4 * e], inv), __fmul_rn(x[4 * e + 1], inv)) |
                           ((uint32_t)f32x2_to_e4m3x2(__fmul_rn(x[4 * e + 2], inv), __fmul_rn(x[4 * e + 3], inv)) << 16);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_k ? p.key_cache : p.value_cache) +
                                           (slot * p.num_kv_heads + h) * D + gl * 8) = make_uint2(w[0], w[1]);
            }
        } else if constexpr (CACHE == kCacheInt4) {
            // a warp of query rows only has nothing to quantise
            if (__any_sync(0xffffffffu, live && !is_q)) {
                float x[8];
                unpack8(raw[i], x);
                uint32_t pair;
                const uint32_t codes = quantise_row_int4<LPR>(x, pair);
                if (live && !is_q && slot >= 0) {
                    const int64_t block = slot / p.block_size;
                    const int o = (int)(slot - block * p.block_size);
                    uint8_t *rec = static_cast<uint8_t *>(is_k ? p.key_cache : p.value_cache) +
                                   (block * p.num_kv_heads + h) * int4_record_bytes(p.block_size, D);
                    *reinterpret_cast<uint32_t *>(rec + o * (D / 2) + gl * 4) = codes;
                    if (gl == 0) *reinterpret_cast<uint32_t *>(rec + p.block_size * (D / 2) + o * 4) = pair;
                }
            }
        }
    }
}

// Blocks of a 4-bit cache back to bf16 blocks [num_ids, BS, Hkv, D]: one warp per
// (listed block, KV head, cache), D / 8 lanes a row.  value = fma(scale, code, zero)
// in fp32, rounded to bf16.
template <int D>
__global__ void __launch_bounds__(256)
    dequantize_blocks_int4_kernel(__nv_bfloat16 *__restrict__ key_out, __nv_bfloat16 *__restrict__ value_out,
                                  const uint8_t *__restrict__ key_cache, const uint8_t *__restrict__ value_cache,
                                  const int32_t *__restrict__ ids, int64_t units, int num_kv_heads, int block_size,
                                  int num_blocks)
{
    constexpr int LPR = D / 8;
    constexpr int GPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int gl = lane % LPR, grp = lane / LPR;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (unit >= units) return;
    const int64_t i = unit / (2 * num_kv_heads);
    const int r = (int)(unit - i * 2 * num_kv_heads);
    const int h = r >> 1;
    const int64_t block = ids[i];
    if (block < 0 || block >= num_blocks) return;  // not a block: its rows are left as they were
    const uint8_t *rec = ((r & 1) ? value_cache : key_cache) +
                         (block * num_kv_heads + h) * int4_record_bytes(block_size, D);
    __nv_bfloat16 *out = ((r & 1) ? value_out : key_out) + (i * block_size * num_kv_heads + h) * D + gl * 8;
#pragma unroll 4
    for (int o = grp; o < block_size; o += GPW) {
        const uint32_t codes = *reinterpret_cast<const uint32_t *>(rec + o * (D / 2) + gl * 4);
        const float2 sz = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(rec + block_size * (D / 2) + o * 4));
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(sz.x, (float)((codes >> (4 * e)) & 15u), sz.y);
        *reinterpret_cast<uint4 *>(out + (int64_t)o * num_kv_heads * D) = pack8(x);
    }
}

}  // namespace pakv
