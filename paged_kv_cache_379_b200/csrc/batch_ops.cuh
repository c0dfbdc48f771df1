// batch_ops.cuh -- a step's block tables, lengths, positions and slots built on
// the GPU from the requests' lengths (the device counterpart of the host pool's
// per-step work), and the return of finished requests' blocks:
//   prepare_batch_kernel   sums over the requests, the decision whether the step
//                          fits, the new blocks, lengths and row starts, and the
//                          per-token arrays.  Every CTA goes through the requests;
//                          CTA r fills rows 2048 r .. and the tables of every
//                          grid-th request.  One CTA alone where an output is an
//                          input (a CTA must not write what another still reads),
//   fill_tokens_kernel     the per-token arrays where one CTA would fill too many,
//   release_blocks_kernel  one CTA: pushes the blocks of marked requests.
// For request s with c cached and n new tokens, have = ceil(c / bs), need =
// ceil((c + n) / bs) - have, before_s = the sum of need over the requests before
// it; its new logical block have + j is free[num_free - 1 - before_s - j]: the
// order in which a pool that pops its free list's end would hand them out.  All
// integer work, bound by launch and load latency (256 requests of one token 6 us, 64
// prompt chunks of 73 K rows 7 us; one CTA and a second launch for the rows 11 us, one
// cluster of 8 CTAs 17 to 19 us); every sum is 64 bits wide.
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
    uint32_t div_mul, div_shift;                    // n / block_size = umulhi(n, mul) >> shift for n < 2^31 (mul 0: 1)
};

constexpr int kBatchThreads = 1024;
// rows of the per-token arrays that a CTA of several, and that one alone, fills
constexpr int kBatchRows = 2 * kBatchThreads, kBatchFusedTokens = 4 * kBatchThreads;
// requests whose sums fit the shared-memory copy
constexpr int kBatchSmemSeqs = 2048;

__device__ __forceinline__ uint32_t div_block(const BatchParams &p, uint32_t n)
{
    return p.div_mul ? __umulhi(n, p.div_mul) >> p.div_shift : n;
}

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

// The request that row t belongs to: the last one that starts at or before it
// (empty ones share its start).
template <typename F>
__device__ __forceinline__ int request_of(F start, int num_seqs, int t)
{
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void write_token(const BatchParams &p, int t, int s, int64_t pos, int32_t block)
{
    if (p.seq_ids) p.seq_ids[t] = s;
    if (p.positions) p.positions[t] = pos;
    if (p.slots) {
        const uint32_t at = (uint32_t)pos;
        p.slots[t] = block < 0 ? -1 : (int64_t)block * p.block_size + (at - div_block(p, at) * p.block_size);
    }
}

// Row t from what has been written: the tables, the lengths and q_start.
__device__ __forceinline__ void fill_token(const BatchParams &p, int t)
{
    if (t >= p.q_start[p.num_seqs]) {
        write_token(p, t, -1, -1, -1);
        return;
    }
    const int s = request_of([&](int i) { return p.q_start[i]; }, p.num_seqs, t);
    // positions stay below max_blocks * block_size, which fits 31 bits; query_lens may be overwritten by now
    const int64_t pos = (int64_t)p.seq_lens[s] - p.q_start[s + 1] + t;
    write_token(p, t, s, pos, p.block_tables[(int64_t)s * p.max_blocks + div_block(p, (uint32_t)pos)]);
}

__global__ void __launch_bounds__(kBatchThreads) prepare_batch_kernel(const BatchParams p, int fused)
{
    __shared__ int32_t s_start[kBatchSmemSeqs + 1], s_ctx[kBatchSmemSeqs], s_have[kBatchSmemSeqs], s_before[kBatchSmemSeqs];
    __shared__ int s_bad, s_bad_block;
    const int tid = threadIdx.x;
    const bool near = p.num_seqs <= kBatchSmemSeqs;  // every request has its own place in the copies
    if (tid == 0) s_bad = s_bad_block = 0;
    pdl_wait();  // its outputs are read early by later kernels: they are never let start before it ends
    __syncthreads();
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    const int64_t nf = p.num_free[0];
    auto blocks_of = [&](int64_t len) { return len > 0 ? (int)div_block(p, (uint32_t)len - 1u) + 1 : 0; };

    // does the step fit?
    int64_t need_sum = 0, tok_sum = 0;
    bool bad = nf < 0 || nf > p.free_capacity;
    for (int s = tid; s < p.num_seqs; s += kBatchThreads) {
        const int64_t c = p.context_lens[s], n = p.query_lens[s];
        if (c < 0 || n < 0 || c + n > cap) {
            bad = true;
            continue;
        }
        need_sum += blocks_of(c + n) - blocks_of(c);
        tok_sum += n;
    }
    if (bad) s_bad = 1;
    int64_t need_total, tok_total;
    block_scan2(need_sum, tok_sum, need_total, tok_total);
    __syncthreads();
    const int status = s_bad || tok_total > p.num_tokens ? PA_ERR_BAD_SHAPE
                                                         : (need_total > nf ? PA_ERR_POOL_EXHAUSTED : PA_OK);
    const bool ok = status == PA_OK;
    // the k-th block that the step takes, checked: an entry outside the cache counts as none
    auto taken = [&](int64_t k) {
        const int32_t id = p.free_blocks[nf - 1 - k];
        return id < 0 || id >= p.num_blocks ? -1 : id;
    };

    int64_t carry_need = 0, carry_tok = 0;
    for (int base = 0; base < p.num_seqs; base += kBatchThreads) {
        const int s = base + tid, at = near ? base : 0;
        int64_t c = 0, n = 0;
        int need = 0, have = 0;
        if (s < p.num_seqs) {
            c = p.context_lens[s];
            if (ok) {
                n = p.query_lens[s];
                have = blocks_of(c);
                need = blocks_of(c + n) - have;
            }
        }
        int64_t a = need, b = n, ta, tb;
        block_scan2(a, b, ta, tb);
        const int64_t before = carry_need + a - need, start = carry_tok + b - n;
        carry_need += ta;
        carry_tok += tb;
        if (s < p.num_seqs) {
            s_start[at + tid] = (int32_t)start;
            s_ctx[at + tid] = (int32_t)c;
            s_have[at + tid] = have;
            s_before[at + tid] = (int32_t)before;  // ok: below num_free
            if (blockIdx.x == 0) {
                // a step that does not fit adds nothing: the lengths stay the cached ones
                p.seq_lens[s] = (int32_t)(ok ? c + n : (c < 0 ? 0 : (c > cap ? cap : c)));
                p.q_start[s] = (int32_t)start;
            }
        }
        const int count = min(kBatchThreads, p.num_seqs - base);
        __syncthreads();
        // the new blocks: a warp per request, its lanes over the request's blocks
        for (int i = (tid >> 5) * gridDim.x + blockIdx.x; i < count; i += kBatchThreads / 32 * gridDim.x) {
            const int64_t first = s_before[at + i];
            const int m = (int)((i + 1 < count ? s_before[at + i + 1] : carry_need) - first);
            int32_t *row = p.block_tables + (int64_t)(base + i) * p.max_blocks + s_have[at + i];
            for (int j = tid & 31; j < m; j += 32) row[j] = taken(first + j);
        }
        if (blockIdx.x == 0) {
            const int64_t end = carry_need;
            for (int64_t k = carry_need - ta + tid; k < end; k += kBatchThreads)
                if (taken(k) < 0) s_bad_block = 1;
        }
        __syncthreads();
    }
    if (tid == 0 && near) s_start[p.num_seqs] = (int32_t)carry_tok;
    if (tid == 0 && blockIdx.x == 0) {
        p.q_start[p.num_seqs] = (int32_t)carry_tok;
        p.num_free_out[0] = (int32_t)(nf - carry_need);
        p.status[0] = ok && s_bad_block ? PA_ERR_BAD_BLOCK : status;
    }
    if (!fused) return;
    __syncthreads();
    // 64 bits: the step past the last rows may pass 31
    const int64_t t0 = (int64_t)blockIdx.x * kBatchRows;
    const int t1 = gridDim.x > 1 ? (int)min((int64_t)p.num_tokens, t0 + kBatchRows) : p.num_tokens;
    for (int64_t row = t0 + tid; row < t1; row += kBatchThreads) {
        const int t = (int)row;
        if (!near) {  // one CTA: all of it is its own
            fill_token(p, t);
        } else if (t >= (int)carry_tok) {
            write_token(p, t, -1, -1, -1);
        } else {
            const int s = request_of([&](int i) { return s_start[i]; }, p.num_seqs, t);
            const int pos = s_ctx[s] + (t - s_start[s]);
            const int b = (int)div_block(p, (uint32_t)pos);
            write_token(p, t, s, pos, b < s_have[s] ? p.block_tables[(int64_t)s * p.max_blocks + b]
                                                    : taken((int64_t)s_before[s] + b - s_have[s]));
        }
    }
}

__global__ void __launch_bounds__(256) fill_tokens_kernel(const BatchParams p)
{
    pdl_wait();
    const int t0 = blockIdx.x * 1024 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t0 + i * 256 < p.num_tokens) fill_token(p, t0 + i * 256);
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
