// batch_ops.cuh -- a step's block tables, lengths, positions and slots built on
// the GPU from the requests' lengths (the device counterpart of the host pool's
// per-step work), and the return of finished requests' blocks:
//   prepare_batch_kernel   one CTA: sums over the requests, the decision whether
//                          the step fits, the new blocks, lengths and row starts
//                          (and, for small steps, the per-token arrays),
//   fill_tokens_kernel     the per-token arrays of large steps,
//   release_blocks_kernel  one CTA: pushes the blocks of marked requests.
// For request s with c cached and n new tokens, have = ceil(c / bs), need =
// ceil((c + n) / bs) - have, before_s = the sum of need over the requests before
// it; its new logical block have + j is free[num_free - 1 - before_s - j]: the
// order in which a pool that pops its free list's end would hand them out.  All
// integer work, bound by launch and load latency; every sum is 64 bits wide.
// Included once, by pagedkv.cu.
#pragma once

#include "common.cuh"

namespace pakv {

struct BatchParams {
    int32_t *block_tables;                          // [B, max_blocks], new entries written
    const int32_t *context_lens, *query_lens;       // [B]
    const int32_t *free_blocks, *num_free;
    int32_t *seq_lens, *q_start, *seq_ids;          // seq_ids: nullptr = not wanted
    int64_t *positions, *slots;
    int32_t *num_free_out, *status;
    int num_seqs, max_blocks, num_tokens, block_size, num_blocks, free_capacity;
};

constexpr int kBatchThreads = 1024;
// per-token arrays of up to this many rows are filled by the one CTA itself
constexpr int kBatchFusedTokens = 4096;
// requests whose row starts fit the shared-memory copy
constexpr int kBatchSmemSeqs = 4096;

// Inclusive scan of two 64-bit values over the CTA; returns the totals too.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t &ta, int64_t &tb)
{
    __shared__ int64_t sa[kBatchThreads / 32], sb[kBatchThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) {
            a += x;
            b += y;
        }
    }
    __syncthreads();  // the arrays may still be read by the previous scan
    if (lane == 31) {
        sa[warp] = a;
        sb[warp] = b;
    }
    __syncthreads();
    int64_t x = sa[lane], y = sb[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) {
            x += u;
            y += v;
        }
    }
    const int64_t pa = __shfl_sync(0xffffffffu, x, warp ? warp - 1 : 0), pb = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
    if (warp) {
        a += pa;
        b += pb;
    }
    ta = __shfl_sync(0xffffffffu, x, 31);
    tb = __shfl_sync(0xffffffffu, y, 31);
}

// Row t of the per-token arrays.  `starts`: q_start, in shared or global memory.
__device__ __forceinline__ void fill_token(const BatchParams &p, const int32_t *starts, int t)
{
    int64_t pos = -1, slot = -1;
    int s = -1;
    if (t < starts[p.num_seqs]) {
        int lo = 0, hi = p.num_seqs;  // the last request that starts at or before t (empty ones share its start)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= t) lo = mid; else hi = mid;
        }
        s = lo;
        pos = (int64_t)p.seq_lens[s] - p.query_lens[s] + (t - starts[s]);
        const int64_t b = pos / p.block_size;
        const int32_t block = p.block_tables[(int64_t)s * p.max_blocks + b];
        if (block >= 0) slot = (int64_t)block * p.block_size + (pos - b * p.block_size);
    }
    if (p.seq_ids) p.seq_ids[t] = s;
    if (p.positions) p.positions[t] = pos;
    if (p.slots) p.slots[t] = slot;
}

__global__ void __launch_bounds__(kBatchThreads) prepare_batch_kernel(const BatchParams p, int fused)
{
    __shared__ int32_t s_have[kBatchThreads], s_need[kBatchThreads];
    __shared__ int64_t s_before[kBatchThreads];
    __shared__ int32_t s_start[kBatchSmemSeqs + 1];
    __shared__ int s_bad, s_bad_block;
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = s_bad_block = 0;
    pdl_wait();  // its outputs are read early by later kernels: they are never let start before it ends
    __syncthreads();
    const int bs = p.block_size;
    const int64_t cap = (int64_t)p.max_blocks * bs;
    const int64_t nf = p.num_free[0];

    // does the step fit?
    int64_t need_sum = 0, tok_sum = 0;
    bool bad = nf < 0 || nf > p.free_capacity;
    for (int s = tid; s < p.num_seqs; s += kBatchThreads) {
        const int64_t c = p.context_lens[s], n = p.query_lens[s];
        if (c < 0 || n < 0 || c + n > cap) {
            bad = true;
            continue;
        }
        need_sum += (c + n + bs - 1) / bs - (c + bs - 1) / bs;
        tok_sum += n;
    }
    if (bad) s_bad = 1;
    int64_t need_total, tok_total;
    block_scan2(need_sum, tok_sum, need_total, tok_total);
    __syncthreads();
    const int status = s_bad || tok_total > p.num_tokens ? PA_ERR_BAD_SHAPE
                                                         : (need_total > nf ? PA_ERR_POOL_EXHAUSTED : PA_OK);
    const bool ok = status == PA_OK;

    int64_t carry_need = 0, carry_tok = 0;
    for (int base = 0; base < p.num_seqs; base += kBatchThreads) {
        const int s = base + tid;
        int64_t c = 0, n = 0, need = 0, have = 0;
        if (s < p.num_seqs) {
            c = p.context_lens[s];
            n = ok ? p.query_lens[s] : 0;
            have = (c + bs - 1) / bs;
            need = ok ? (c + n + bs - 1) / bs - have : 0;
        }
        int64_t a = need, b = n, ta, tb;
        block_scan2(a, b, ta, tb);
        const int64_t before = carry_need + a - need, start = carry_tok + b - n;
        carry_need += ta;
        carry_tok += tb;
        s_have[tid] = (int)have;
        s_need[tid] = (int)need;
        s_before[tid] = before;
        if (s < p.num_seqs) {
            // a step that does not fit adds nothing: the lengths stay the cached ones
            p.seq_lens[s] = (int32_t)(ok ? c + n : (c < 0 ? 0 : (c > cap ? cap : c)));
            p.q_start[s] = (int32_t)start;
            if (s < kBatchSmemSeqs) s_start[s] = (int32_t)start;
        }
        __syncthreads();
        // the new blocks: a warp per request, its lanes over the request's blocks
        const int count = min(kBatchThreads, p.num_seqs - base);
        for (int i = tid >> 5; i < count; i += kBatchThreads / 32) {
            const int m = s_need[i];
            const int64_t top = nf - 1 - s_before[i];
            int32_t *row = p.block_tables + (int64_t)(base + i) * p.max_blocks + s_have[i];
            for (int j = tid & 31; j < m; j += 32) {
                int32_t id = p.free_blocks[top - j];
                if (id < 0 || id >= p.num_blocks) {
                    id = -1;
                    s_bad_block = 1;
                }
                row[j] = id;
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.q_start[p.num_seqs] = (int32_t)carry_tok;
        if (p.num_seqs <= kBatchSmemSeqs) s_start[p.num_seqs] = (int32_t)carry_tok;
        p.num_free_out[0] = (int32_t)(nf - carry_need);
        p.status[0] = ok && s_bad_block ? PA_ERR_BAD_BLOCK : status;
    }
    if (!fused) return;
    __syncthreads();
    for (int t = tid; t < p.num_tokens; t += kBatchThreads)
        fill_token(p, p.num_seqs <= kBatchSmemSeqs ? s_start : p.q_start, t);
}

__global__ void __launch_bounds__(256) fill_tokens_kernel(const BatchParams p)
{
    __shared__ int32_t s_start[kBatchSmemSeqs + 1];
    pdl_wait();
    const int32_t *starts = p.q_start;
    if (p.num_seqs <= kBatchSmemSeqs) {
        for (int s = threadIdx.x; s <= p.num_seqs; s += blockDim.x) s_start[s] = p.q_start[s];
        starts = s_start;
        __syncthreads();
    }
    const int t0 = blockIdx.x * 1024 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t0 + i * 256 < p.num_tokens) fill_token(p, starts, t0 + i * 256);
}

// The blocks of every marked request go back on the free list in request order,
// each row's blocks in order; the row's entries become -1 and its length 0.
__global__ void __launch_bounds__(kBatchThreads)
    release_blocks_kernel(int32_t *__restrict__ block_tables, int num_seqs, int max_blocks, int32_t *__restrict__ seq_lens,
                          const int32_t *__restrict__ release, int32_t *__restrict__ free_blocks,
                          int32_t *__restrict__ num_free, int free_capacity, int block_size, int num_blocks,
                          int32_t *__restrict__ status)
{
    __shared__ int32_t s_have[kBatchThreads];
    __shared__ int64_t s_before[kBatchThreads];
    __shared__ int s_bad, s_bad_block;
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = s_bad_block = 0;
    pdl_wait();
    __syncthreads();
    const int64_t cap = (int64_t)max_blocks * block_size;
    const int64_t nf = num_free[0];
    int64_t sum = 0, zero = 0, total, unused;
    bool bad = nf < 0 || nf > free_capacity, bad_block = false;
    for (int s = tid; s < num_seqs; s += kBatchThreads) {
        if (!release[s]) continue;
        const int64_t n = seq_lens[s];
        if (n < 0 || n > cap)
            bad = true;
        else
            sum += (n + block_size - 1) / block_size;
    }
    if (bad) s_bad = 1;
    block_scan2(sum, zero, total, unused);
    __syncthreads();
    if (!s_bad) {
        // every id is looked at before anything is pushed
        for (int s = tid >> 5; s < num_seqs; s += kBatchThreads / 32) {
            if (!release[s]) continue;
            const int n = (int)(((int64_t)seq_lens[s] + block_size - 1) / block_size);
            for (int j = tid & 31; j < n; j += 32) {
                const int32_t id = block_tables[(int64_t)s * max_blocks + j];
                bad_block |= id < 0 || id >= num_blocks;
            }
        }
        if (bad_block) s_bad_block = 1;
    }
    __syncthreads();
    const int code = s_bad || nf + total > free_capacity ? PA_ERR_BAD_SHAPE : (s_bad_block ? PA_ERR_BAD_BLOCK : PA_OK);
    if (code == PA_OK) {
        int64_t carry = 0;
        for (int base = 0; base < num_seqs; base += kBatchThreads) {
            const int s = base + tid;
            int64_t have = 0;
            if (s < num_seqs && release[s]) have = ((int64_t)seq_lens[s] + block_size - 1) / block_size;
            int64_t a = have, b = 0, ta, tb;
            block_scan2(a, b, ta, tb);
            s_have[tid] = (int)have;
            s_before[tid] = carry + a - have;
            carry += ta;
            if (s < num_seqs && release[s]) seq_lens[s] = 0;
            __syncthreads();
            const int count = min(kBatchThreads, num_seqs - base);
            for (int i = tid >> 5; i < count; i += kBatchThreads / 32) {
                int32_t *row = block_tables + (int64_t)(base + i) * max_blocks;
                for (int j = tid & 31; j < s_have[i]; j += 32) {
                    free_blocks[nf + s_before[i] + j] = row[j];
                    row[j] = -1;
                }
            }
            __syncthreads();
        }
        if (tid == 0) num_free[0] = (int32_t)(nf + total);
    }
    if (tid == 0) status[0] = code;
}

}  // namespace pakv
