// row_ops.cuh -- per-row work between the projection and the cache:
//   row_kernel         RMS norm of each query / key head, position rotation, and
//                      the write of K and V rows into a bf16, FP8 or 4-bit cache
//                      (or no cache),
//   store_int4_kernel  the 4-bit cache write alone,
//   dequantize_blocks_int4_kernel  whole 4-bit blocks back to bf16 blocks.
//
// 4-bit cache: one record per (block, KV head), [num_blocks, num_kv_heads, record]:
//   BS rows of D/2 code bytes (dim 2i in the low nibble of byte i, dim 2i+1 in
//   the high one), then BS pairs (scale, zero) of bf16.  A code c of row o stands
//   for zero_o + scale_o * c.  The record of one head of a block is contiguous
//   (1088 bytes at D = 128, BS = 16), so the decode's 16-byte copies cover whole lines.
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
    int block_size, block_shift;                    // block_size = 1 << block_shift (4-bit cache)
    int64_t num_slots;
    float k_inv, v_inv;                             // inverse scales of an FP8 cache
    int num_tokens;
    uint32_t num_rows, div_mul, div_shift;          // row / rows = umulhi(row, div_mul) >> div_shift (row < 2^31)
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

__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Minimum and negated maximum of 8 values as one pair of bf16; a NaN prevails.
__device__ __forceinline__ uint32_t low_high(const uint4 &raw)
{
    constexpr uint32_t kSigns = 0x80008000u;
    const uint32_t a = min_nan_bf16x2(min_nan_bf16x2(raw.x, raw.y), min_nan_bf16x2(raw.z, raw.w));
    const uint32_t b = min_nan_bf16x2(min_nan_bf16x2(raw.x ^ kSigns, raw.y ^ kSigns),
                                      min_nan_bf16x2(raw.z ^ kSigns, raw.w ^ kSigns));
    return min_nan_bf16x2(prmt(a, b, 0x5410u), prmt(a, b, 0x7632u));
}

// A row's quantisation, from low_high over it: its packed (scale, zero) pair, and what the codes need.
struct RowQuant {
    uint32_t pair;
    float zero, inv;  // inv 0: all codes are 0
    bool wide;        // max - min overflows
};
__device__ __forceinline__ RowQuant row_quant(uint32_t both)
{
    const float2 mm = unpack_bf16x2(both);
    const float lo = mm.x, hi = -mm.y;
    constexpr float r15 = 1.0f / 15.0f;
    float scale = __bfloat162float(__float2bfloat16_rn(__fsub_rn(__fmul_rn(hi, r15), __fmul_rn(lo, r15))));
    RowQuant q;
    q.zero = lo + 0.0f;  // -0 and +0 are one minimum
    if (!(hi < INFINITY && lo > -INFINITY)) {
        scale = 0.f;
        q.zero = __uint_as_float(0x7FC00000u);
    }
    if (scale < 1.17549435e-38f) scale = 0.f;
    q.inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    q.wide = hi - lo == INFINITY;
    q.pair = pack_bf16x2(scale, q.zero);
    return q;
}

// The codes of 8 values, packed.  The quotient stays below 15.06 (the scale is
// within 2^-8 of range / 15), unless x - zero overflows.  Adding 2^23 rounds to the
// nearest integer, ties to even: the sum's bits are 0x4B000000 + code.
__device__ __forceinline__ uint32_t codes8(const uint4 &raw, const RowQuant &q)
{
    constexpr uint32_t kBias = 0x4B000000u * 0x11111111u;
    uint32_t codes = 0;
    if (q.inv == 0.f) return 0u;
    if (!q.wide) {
        float x[8];
        unpack8(raw, x);
#pragma unroll
        for (int e = 7; e >= 0; --e)
            codes = codes * 16u + __float_as_uint(__fadd_rn(__fmul_rn(__fsub_rn(x[e], q.zero), q.inv), 8388608.f));
    } else {
#pragma unroll 1
        for (int e = 7; e >= 0; --e) {
            const float2 v = unpack_bf16x2(u4_word(raw, e >> 1));
            const float t = fminf(__fmul_rn(__fsub_rn(e & 1 ? v.y : v.x, q.zero), q.inv), 15.f);
            codes = codes * 16u + __float_as_uint(__fadd_rn(t, 8388608.f));
        }
    }
    return codes - kBias;
}

// Quantises a row spread over LPR neighbouring lanes, 8 values each.
template <int LPR>
__device__ __forceinline__ uint32_t quantise_row_int4(const uint4 &raw, uint32_t &pair)
{
    uint32_t both = low_high(raw);
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1)
        both = min_nan_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, off));
    const RowQuant q = row_quant(both);
    pair = q.pair;
    return codes8(raw, q);
}

// The slot of the newest position of sequence t (-1: none).
__device__ __forceinline__ int64_t newest_slot(const RowParams &p, int t)
{
    const int64_t pos = (int64_t)p.seq_lens[t] - 1;
    if (pos < 0 || pos >> p.block_shift >= p.max_blocks) return -1;
    const int32_t b = p.block_tables[(int64_t)t * p.max_blocks + (pos >> p.block_shift)];
    return b < 0 ? -1 : ((int64_t)b << p.block_shift) + (pos & (p.block_size - 1));
}

// K and V rows into a 4-bit cache, D / 32 lanes a row and 32 values a lane: what a
// row costs as a whole (its scale, its reciprocal) is shared by 8 or 16 rows of a
// warp, and a lane's codes are one 16-byte store.  16384 tokens of 8 + 8 heads (85 MB
// with the codes) take about 17 us, 13 at the measured copy rate, bound by issue
// slots (74 % used; 8 values a lane: 27 us).
template <int D>
__global__ void __launch_bounds__(128) store_int4_kernel(const RowParams p)
{
    constexpr int LPR = D / 32;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t idx = blockIdx.x * 128 + threadIdx.x;
    const int gl = threadIdx.x % LPR;
    const uint32_t row = min(idx / LPR, p.num_rows - 1);  // a surplus lane takes part in the shuffles only
    const bool live = idx / LPR < p.num_rows;
    const int t = (int)(__umulhi(row, p.div_mul) >> p.div_shift);
    const int r = (int)(row - (uint32_t)t * p.rows);
    const bool is_k = r < p.num_kv_heads;
    const int h = is_k ? r : r - p.num_kv_heads;
    const uint4 *src = reinterpret_cast<const uint4 *>(is_k ? p.key + t * p.k_stride : p.value + t * p.v_stride) +
                       h * (D / 8) + gl * 4;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = src[i];
    int64_t slot = p.slots ? p.slots[t] : newest_slot(p, t);
    if (p.slots_out && live && r == 0 && gl == 0) p.slots_out[t] = slot;
    if (slot >= p.num_slots) slot = -1;
    uint32_t both = min_nan_bf16x2(min_nan_bf16x2(low_high(raw[0]), low_high(raw[1])),
                                   min_nan_bf16x2(low_high(raw[2]), low_high(raw[3])));
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1)
        both = min_nan_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, off));
    const RowQuant q = row_quant(both);
    const uint4 codes = make_uint4(codes8(raw[0], q), codes8(raw[1], q), codes8(raw[2], q), codes8(raw[3], q));
    if (!live || slot < 0) return;
    const int o = (int)(slot & (p.block_size - 1));
    const int64_t rec = ((slot >> p.block_shift) * p.num_kv_heads + h) * int4_record_bytes(p.block_size, D);
    uint8_t *dst = static_cast<uint8_t *>(is_k ? p.key_cache : p.value_cache) + rec;
    *reinterpret_cast<uint4 *>(dst + o * (D / 2) + gl * 16) = codes;
    if (gl == 0) *reinterpret_cast<uint32_t *>(dst + p.block_size * (D / 2) + o * 4) = q.pair;
}

// A warp takes U * (32 / LPR) rows of one token (LPR = D / 8 lanes a row, 16
// bytes a lane), so the token's cosines and sines are loaded once for all of
// them and every lane has U loads in flight.  Each row is read and written once:
// 16384 tokens of 32 + 8 + 8 heads (407 MB) take 75 us, 83 % of the measured copy
// rate; beside that bound, instructions (the norm's and the rotation's, ~150 for two
// rows) take two thirds of the issue slots.  Half-split pairs over the whole head, whose
// partners come by shuffles, take 91 us (an FP8 cache as much); a 4-bit cache, quantised
// with 8 values a lane, 99 us interleaved and 126 half-split.  One step's 128 tokens: 3.3
// us (4-bit 3.8), launch and latency.
template <int D, int CACHE, bool INTERLEAVED, int U>
__global__ void __launch_bounds__(256) row_kernel(const RowParams p)
{
    constexpr int LPR = D / 8;
    constexpr int GPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int gl = lane % LPR, grp = lane / LPR;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);  // token
    const int c = blockIdx.y;                           // its U * GPW rows
    pdl_wait();
    // It writes queries (and keys), which the kernels after it may read before their
    // own griddepcontrol.wait: it never lets them start early.
    if (t >= p.num_tokens) return;

    float cs[8], sn[8];
    int half = 0;  // lanes per rotated half (half-split pairs)
    bool turned = false;
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) return;  // padding: nothing is written
    const float *row = p.cos_sin + pos * p.rot;
    if constexpr (INTERLEAVED) {
        if (gl * 8 < p.rot) {
            *reinterpret_cast<float4 *>(cs) = *reinterpret_cast<const float4 *>(row + gl * 4);
            *reinterpret_cast<float4 *>(sn) = *reinterpret_cast<const float4 *>(row + p.rot / 2 + gl * 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] = 1.f, sn[e] = 0.f;
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
            if (gl < half) {  // the first of a pair: a cos - b sin
#pragma unroll
                for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
        }
    }
    int64_t slot = -1;
    if constexpr (CACHE != kCacheNone) {
        slot = p.slots[t];
        if (slot >= p.num_slots) slot = -1;
    }

    // Rows of a token: queries, keys, values.  Addresses are a token's base and the row.
    const int r0 = c * U * GPW + grp, nq = p.num_heads, nqk = nq + p.num_kv_heads;
    const __nv_bfloat16 *qs = p.query + t * p.q_stride + gl * 8;
    const __nv_bfloat16 *ks = p.key + t * p.k_stride + gl * 8;
    const __nv_bfloat16 *vs = CACHE == kCacheNone ? nullptr : p.value + t * p.v_stride + gl * 8;
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int r = r0 + i * GPW;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.rows)
            raw[i] = *reinterpret_cast<const uint4 *>(r < nq ? qs + r * D : r < nqk ? ks + (r - nq) * D
                                                                                    : vs + (r - nqk) * D);
    }
    // 4-bit cache: the row's codes and pair in head 0's records; a head is `record` bytes further on
    const uint32_t record = CACHE == kCacheInt4 ? (uint32_t)int4_record_bytes(p.block_size, D) : 0u;
    uint8_t *krec = nullptr, *vrec = nullptr;
    int pair_at = 0;
    if constexpr (CACHE == kCacheInt4) {
        const int o = (int)(slot & (p.block_size - 1));
        const int64_t at = (slot >> p.block_shift) * ((int64_t)p.num_kv_heads * record) + o * (D / 2) + gl * 4;
        krec = static_cast<uint8_t *>(p.key_cache) + at;
        vrec = static_cast<uint8_t *>(p.value_cache) + at;
        pair_at = (p.block_size - o) * (D / 2) + o * 4;  // from the row's first byte
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int r = r0 + i * GPW;
        const bool is_q = r < nq;
        const bool is_k = !is_q && r < nqk;
        const int h = is_q ? r : (is_k ? r - nq : r - nqk);
        // values only pass through: a warp of them has nothing to do here
        if (__any_sync(0xffffffffu, is_q || is_k)) {
            float x[8], y[8];
            unpack8(raw[i], x);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float rms = rsqrtf(ss * (1.0f / D) + p.eps);
            const __nv_bfloat16 *w = is_q ? p.q_weight : p.k_weight;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= rms;
            if (w) {
                float wf[8];
                unpack8(*reinterpret_cast<const uint4 *>(w + gl * 8), wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= wf[e];
            }
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    y[e] = x[e] * cs[e / 2] - x[e + 1] * sn[e / 2];
                    y[e + 1] = x[e + 1] * cs[e / 2] + x[e] * sn[e / 2];
                }
            } else {
                // the pair's other element sits `half` lanes away in the row's lane group
                const int other = !turned ? lane : grp * LPR + (gl < half ? gl + half : gl - half);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = fmaf(__shfl_sync(0xffffffffu, x[e], other), sn[e], x[e] * cs[e]);
            }
            // rounded to bf16 once; value rows of a mixed warp stay as they are
            if (is_q || is_k) raw[i] = pack8(y);
        }
        const bool live = r < p.rows;
        if (live && is_q) *reinterpret_cast<uint4 *>(p.query_out + t * p.qo_stride + h * D + gl * 8) = raw[i];
        if constexpr (CACHE == kCacheNone) {
            if (live && is_k) *reinterpret_cast<uint4 *>(p.key_out + t * p.ko_stride + h * D + gl * 8) = raw[i];
        } else if constexpr (CACHE == kCacheBf16) {
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
                uint32_t pair;
                const uint32_t codes = quantise_row_int4<LPR>(raw[i], pair);
                if (live && !is_q && slot >= 0) {
                    uint8_t *rec = (is_k ? krec : vrec) + (uint64_t)(uint32_t)h * record;
                    *reinterpret_cast<uint32_t *>(rec) = codes;
                    if (gl == 0) *reinterpret_cast<uint32_t *>(rec + pair_at) = pair;
                }
            }
        }
    }
}

// Blocks of a 4-bit cache back to bf16 blocks [num_ids, BS, Hkv, D]: one warp per
// (listed block, KV head, cache), D / 8 lanes a row and 8 values a lane (so that a store covers whole lines; 16 a lane: 22.6
// instead of 15.6 us for 1024 blocks of 16x8x128, the copies and all).  value =
// bf16(scale * code + zero), rounded once: a code in the low bits of 128.0 is 128 +
// code exactly, the difference code, and the packed multiply-add rounds its exact result.
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
    // It writes rows that the append kernels after it may read before their own
    // griddepcontrol.wait: it never lets them start early.
    pdl_wait();
    if (unit >= units) return;
    const int64_t i = unit / (2 * num_kv_heads);
    const int r = (int)(unit - i * 2 * num_kv_heads);
    const int h = r >> 1;
    const int64_t block = ids[i];
    if (block < 0 || block >= num_blocks) return;  // not a block: its rows are left as they were
    const uint8_t *rec = ((r & 1) ? value_cache : key_cache) +
                         (block * num_kv_heads + h) * int4_record_bytes(block_size, D);
    __nv_bfloat16 *out = ((r & 1) ? value_out : key_out) + (i * block_size * num_kv_heads + h) * D + gl * 8;
    const __nv_bfloat162 bias = __floats2bfloat162_rn(128.f, 128.f);
#pragma unroll 4
    for (int o = grp; o < block_size; o += GPW) {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(rec + o * (D / 2) + gl * 4);
        const uint32_t pair = *reinterpret_cast<const uint32_t *>(rec + block_size * (D / 2) + o * 4);
        const uint32_t s2 = prmt(pair, pair, 0x1010u), z2 = prmt(pair, pair, 0x3232u);
        const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162 *>(&s2);
        const __nv_bfloat162 zero = *reinterpret_cast<const __nv_bfloat162 *>(&z2);
        uint32_t v[4];  // dims (j, j + 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t m = ((c >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
            const __nv_bfloat162 x = __hfma2(scale, __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), bias), zero);
            v[j] = *reinterpret_cast<const uint32_t *>(&x);
        }
        *reinterpret_cast<uint4 *>(out + (int64_t)o * num_kv_heads * D) =
            make_uint4(prmt(v[0], v[1], 0x5410u), prmt(v[2], v[3], 0x5410u), prmt(v[0], v[1], 0x7632u),
                       prmt(v[2], v[3], 0x7632u));
    }
}

}  // namespace pakv
