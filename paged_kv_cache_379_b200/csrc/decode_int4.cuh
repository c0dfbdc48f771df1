// decode_int4.cuh -- single-query paged decode attention over a 4-bit cache
// (format: row_ops.cuh).  With k_t = z_t + s_t c_t (scale, zero, codes of token
// t's key row) and likewise for the values,
//     x_t = scale * (s_t (q . c_t) + z_t sum(q)),   p_t = exp(x_t - m),
//     out = (sum_t p_t s'_t c'_t + sum_t p_t z'_t) / sum_t p_t,
// so a row's scale and zero meet its 64 bytes of codes only in per-token scalars.
// Included once, by pagedkv.cu.
#pragma once

#include "common.cuh"
#include "row_ops.cuh"

namespace pakv {

struct Int4DecodeParams {
    __nv_bfloat16 *out;                 // [B, Hq, D]
    const __nv_bfloat16 *query;         // [B, Hq, D]
    const uint8_t *key_cache, *value_cache;
    const int32_t *block_tables;        // [B, max_blocks]
    const int32_t *seq_lens;            // [B]
    void *workspace;
    float scale_log2;                   // scale * log2(e)
    int num_seqs, num_heads, num_kv_heads, group, max_blocks, num_blocks;
};

// One CTA per (KV head, sequence); warp w takes tokens w, w + 4, ...; a lane
// holds D / 32 dims of every query head of the group.
template <int D>
__global__ void __launch_bounds__(128) decode_int4_simple_kernel(const Int4DecodeParams p, int block_size)
{
    constexpr int E = D / 32;
    constexpr int GMAX = 16;
    __shared__ float sm_o[4][D], sm_m[4], sm_l[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, s = blockIdx.y;
    pdl_wait();
    const int L = min(p.seq_lens[s], p.max_blocks * block_size);
    const int G = p.group;
    const __nv_bfloat16 *q = p.query + ((int64_t)s * p.num_heads + (int64_t)h * G) * D + lane * E;
    float qf[GMAX][E], o[GMAX][E], m[GMAX], l[GMAX];
#pragma unroll
    for (int g = 0; g < GMAX; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            o[g][e] = 0.f;
            qf[g][e] = g < G ? __bfloat162float(q[g * D + e]) * p.scale_log2 : 0.f;
        }
    }
    for (int t = warp; t < L; t += 4) {
        const int block = p.block_tables[(int64_t)s * p.max_blocks + t / block_size];
        const bool bad = block < 0 || block >= p.num_blocks;
        if (bad) record_status(kStatusBadBlock);
        const int row = t % block_size;
        const int64_t rec = ((int64_t)(bad ? 0 : block) * p.num_kv_heads + h) * int4_record_bytes(block_size, D);
        float kf[E], vf[E];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t *r = (kv ? p.value_cache : p.key_cache) + rec;
            const float2 sz = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(r + block_size * (D / 2) + row * 4));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint8_t byte = r[row * (D / 2) + (lane * E + e) / 2];
                (kv ? vf : kf)[e] = bad ? NAN : fmaf(sz.x, (float)((byte >> (4 * (e & 1))) & 15), sz.y);
            }
        }
#pragma unroll
        for (int g = 0; g < GMAX; ++g) {
            if (g >= G) break;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(qf[g][e], kf[e], x);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            const float mn = fmaxf(m[g], x);
            const float corr = m[g] == -INFINITY ? 0.f : exp2f(m[g] - mn);
            const float w = exp2f(x - mn);
            m[g] = mn;
            l[g] = l[g] * corr + w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] = fmaf(w, vf[e], o[g][e] * corr);
        }
    }
#pragma unroll
    for (int g = 0; g < GMAX; ++g) {
        if (g >= G) break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[g][e];
        if (lane == 0) {
            sm_m[warp] = m[g];
            sm_l[warp] = l[g];
        }
        __syncthreads();
        const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
        if (threadIdx.x < D) {
            float acc = 0.f, den = 0.f;
            for (int w = 0; w < 4; ++w) {
                if (sm_l[w] == 0.f) continue;  // a warp without a token
                const float c = exp2f(sm_m[w] - M);
                den = fmaf(c, sm_l[w], den);
                acc = fmaf(c, sm_o[w][threadIdx.x], acc);
            }
            p.out[((int64_t)s * p.num_heads + (int64_t)h * G + g) * D + threadIdx.x] =
                __float2bfloat16_rn(den == 0.f ? 0.f : acc / den);
        }
    }
}

}  // namespace pakv
