// decode_int4.cuh -- single-query paged decode attention over a 4-bit cache
// (format: row_ops.cuh).  With k_t = z_t + s_t c_t (scale, zero, codes of token
// t's key row) and v_t = z'_t + s'_t c'_t,
//     x_t = scale * (s_t (q . c_t) + z_t sum(q)),   p_t = 2^(x_t log2 e - m),
//     out = (sum_t (p_t s'_t) c'_t + sum_t p_t z'_t) / sum_t p_t,
// so a row's scale and zero meet its codes only in per-token scalars, and the
// codes go to the tensor cores as they are: a nibble in bits 0-3 of a half word is
// the fp16 subnormal c 2^-24, one in bits 4-7 is 16 c 2^-24, so one AND gives two
// exact operands.  In the key product the 16 goes into the query, which is exact in
// fp16 (as a 16-bit integer on the byte product 42.0 instead of 44.6 us for the
// grouped-query batch, but every entry off by up to 2^-15 of a head's largest, times its
// code: one entry 2^10 times the others cost 2 % of the result); in the value product it
// comes out of the accumulator.
//
// Work: a unit is one sequence and KV head, a stage 32 of its tokens.  The weight of
// all units is cut into equal ranges, one for each warp of the grid, so a long
// sequence spreads over the GPU and short ones share a warp; a warp runs through its
// range alone, with its own ring of stages (cp.async, 16 bytes a lane: in an earlier form
// of the stage 565 instructions, with the records' bulk copies 581) and its own online
// softmax.  Units cut between warps are joined once, at the CTA's end, and between
// CTAs by the last of them to arrive, in a fixed order.  (Ranges for CTAs, whose
// warps take turns at a unit's stages and join at its end: 48.9 instead of 43.7 us
// for the grouped-query batch, 8.7 instead of 3.8 for four short sequences.)
//
// Bound, head_dim 128 and block_size 16, one launch after another: eight sequences of
// 32K-128K tokens (713 MB) 141 to 151 us from GPU to GPU, 72 to 77 % of the measured
// copy rate; 128 sequences of ~1100 tokens, 8 query heads on each of 8 KV heads (160 MB)
// 46 us, 64 sequences with 32 heads (323 MB) 74 us; one of 8001 15.3, four of at most 50
// 5.6.  A stage takes 465 instructions (set-up and join included), half of them on the
// pipe of the ANDs: 55 % of the issue slots, 57 % of that pipe and 32 % of the tensor
// cores' cycles in the long case.  An SM is active for 91 % of that launch and 85 % of the
// grouped-query one; the rest is the spread of the last warps and the join.
// Included once, by pagedkv.cu.
#pragma once

#include "common.cuh"
#include "row_ops.cuh"

namespace pakv {

constexpr int kI4Warps = 4;
constexpr int kI4Tokens = 32;        // tokens of one stage
constexpr int kI4MaxCtas = 592;      // CTAs with partial results: 148 SMs x 4
constexpr int kI4HeaderBytes = 4096; // workspace: arrival counters of the CTAs

struct Int4DecodeParams {
    __nv_bfloat16 *out;                 // [B, Hq, D]
    const __nv_bfloat16 *query;         // [B, Hq, D]
    const uint8_t *key_cache, *value_cache;
    const int32_t *block_tables;        // [B, max_blocks]
    const int32_t *seq_lens;            // [B]
    int *counters;                      // [CTAs], zero between calls
    float2 *part_ml;                    // [2 CTAs][16] (m, l)
    float4 *part_o;                     // [2 CTAs][NG * D/16 chunks][32 lanes]
    float scale_log2;                   // scale * log2(e)
    int num_seqs, num_heads, num_kv_heads, group, max_blocks, num_blocks, min_stages;
};

template <int D, int BS, int NG>
struct Int4Lay {
    static constexpr int kRecs = kI4Tokens / BS;               // records of a stage, per cache
    static constexpr int kRec = BS * (D / 2 + 4);
    static constexpr int kStage = 2 * kRecs * kRec;            // K records, then V records
    static constexpr int kSlots = D == 128 ? 2 : 4;            // stages a warp holds
    static constexpr int kRing = kSlots * kStage;
    static constexpr int kChunks = D / 16;                     // float4s a lane holds of 8 heads
    static constexpr int kPart = NG * kChunks * 512;           // bytes of a warp's result
    // resident CTAs per SM: what registers and shared memory hold (64 sequences with 16 heads on each of 8 KV heads:
    // 50 us with two, 79 with registers for a third that does not fit)
    static constexpr int kCtas = NG == 1 ? 4 : D == 64 ? 3 : 2;
    static constexpr int kQf = kI4Warps * kRing;               // each warp's queries as operands
    static constexpr int kQfBytes = NG * (D / 32) * 512;
    static constexpr int kHead = kQf + kI4Warps * kQfBytes;    // results of the first units of warps 1, 2, 3
    static constexpr int kBytes = kHead + (kI4Warps - 1) * kPart;
    static_assert(kRing >= kPart, "a warp's last result stays in its ring");
    static_assert(kRing >= kI4Warps * 32 * 16 + 8 * (kI4Warps * 32 / (D / 4)), "and so does a join of shared parts");
    static_assert(kRec % 16 == 0 && kStage % 16 == 0, "copies are 16 bytes wide");
};

// A unit (sequence, KV head) of nt stages weighs nt + kI4UnitCost stages when the
// work is cut into ranges: what its queries' set-up and its result take.  2, 4 and 6 take
// 45.2, 45.9 and 47.4 us for the grouped-query batch, 72.1, 73.4 and 75.7 for 32 heads on
// 32, but 17.3, 15.4 and 15.2 for one 8K sequence, 56.8, 54.1 and 54.8 for 64 sequences
// with 16 heads a KV head and 58.3, 49.2 and 49.7 for four long ones with 12 (head_dim 64:
// within 2 %).
constexpr int kI4UnitCost = 4;

// A run of stages [t0, t1) of one unit in a worker's range.
struct Int4Seg {
    int s, h, len, nt, t0, t1, left;  // left: weight of the range behind this unit (negative: it ends in here)
};

// A unit that a worker holds a part of, as the join needs it.
template <int NG>
struct Int4Cut {
    int64_t unit;         // where it starts in the weight (its part: [NG][chunk][lane] float4, at the kept place)
    int s, h, nt;
    int from, to;         // it began in an earlier worker / goes on in the next; both 0: no such part
    float m[8 * NG], l[8 * NG];  // maximum in units of log2, sum of the weights
};

__device__ __forceinline__ int int4_len(const Int4DecodeParams &p, int s, int block_size)
{
    return min(max(p.seq_lens[s], 0), p.max_blocks * block_size);
}

__device__ __forceinline__ int int4_stages(int len) { return (int)(((unsigned)len + kI4Tokens - 1) / kI4Tokens); }

__device__ __forceinline__ int int4_weight(int len) { return len > 0 ? int4_stages(len) + kI4UnitCost : 0; }

// Moves to the next unit of the range; false at its end.
__device__ __forceinline__ bool int4_next(Int4Seg &g, const Int4DecodeParams &p, int block_size)
{
    if (g.left <= kI4UnitCost) return false;
    if (++g.h == p.num_kv_heads) {
        g.h = 0;
        do {
            if (++g.s >= p.num_seqs) return false;
            g.len = int4_len(p, g.s, block_size);
        } while (g.len == 0);
        g.nt = int4_stages(g.len);
    }
    g.t0 = 0;
    g.t1 = min(g.nt, g.left - kI4UnitCost);
    g.left -= g.nt + kI4UnitCost;
    return true;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 16 bytes global -> shared memory, asynchronous, past the L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// mma_f16_16816 without `volatile`: the compiler may interleave independent ones.
__device__ __forceinline__ void mma_codes(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Larger magnitude of two pairs of fp16 values, a NaN giving way.
__device__ __forceinline__ uint32_t max_abs_f16x2(uint32_t a, uint32_t b)
{
    const __half2 d = __hmax2(__habs2(*reinterpret_cast<__half2 *>(&a)), __habs2(*reinterpret_cast<__half2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// ev of vmul = 2^(10 - ev)
__device__ __forceinline__ int int4_scale_exp(float vmul) { return 137 - (int)(__float_as_uint(vmul) >> 23); }

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// How the weight is cut into the workers' (warps') ranges: equal, the first `rest` of
// them one longer.  (Shares that fall with a CTA's place on its SM, as the schedulers
// prefer older warps, even out one launch but not launches in a row, where a CTA takes
// the place that falls free: eight long sequences 142 instead of 134 us.)
struct Int4Split {
    int64_t each, rest;
    float cta;  // a CTA's share, about
};

__device__ __forceinline__ int64_t int4_begin(const Int4Split &x, int worker)
{
    return worker * x.each + min((int64_t)worker, x.rest);
}

// The CTA that holds position x: a guess in floating point, then the exact one.
__device__ __forceinline__ int int4_cta_of(const Int4Split &s, int64_t x)
{
    int cta = min((int)((float)x / s.cta), (int)gridDim.x - 1);
    while (int4_begin(s, cta * kI4Warps) > x) --cta;
    while (cta + 1 < (int)gridDim.x && int4_begin(s, (cta + 1) * kI4Warps) <= x) ++cta;
    return cta;
}

template <int D, int BS, int NG>
__global__ void __launch_bounds__(kI4Warps * 32, Int4Lay<D, BS, NG>::kCtas)
    decode_int4_kernel(const Int4DecodeParams p)
{
    using Lay = Int4Lay<D, BS, NG>;
    constexpr int W = kI4Warps, NS = Lay::kSlots, RECS = Lay::kRecs, REC = Lay::kRec;
    constexpr int KW = D / 32;    // words of a key row per lane (4 lanes a row)
    constexpr int VW = D / 64;    // words of a value row per lane (8 lanes a row)
    constexpr int MT = 4 * VW;    // 16-dim tiles of the output: a lane's 2 dims each
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Int4Seg s_ns[W], s_seg[W];
    __shared__ int64_t s_unit[W];
    __shared__ Int4Split s_split;
    __shared__ Int4Cut<NG> s_cut[W][2];   // of each warp: its first unit (if that ends in it), its last
    __shared__ int64_t s_sum[W], s_start[W];
    __shared__ int s_seq[W], s_first[2], s_end[2], s_last[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    uint8_t *const ring = smem + warp * Lay::kRing;
    uint8_t *const qop = smem + Lay::kQf + warp * Lay::kQfBytes;
    if (tid < W) s_seq[tid] = -1;
    if (lane < 2) s_cut[warp][lane].from = s_cut[warp][lane].to = 0;

    // ---- this worker's (warp's) range of the weight, in (sequence, KV head, position) order
    const int per = (p.num_seqs + W * 32 - 1) / (W * 32);
    const int s_lo = min(tid * per, p.num_seqs), s_hi = min(s_lo + per, p.num_seqs);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += int4_weight(int4_len(p, s, BS));
    int64_t scan = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(FULL, scan, off);
        if (lane >= off) scan += v;
    }
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    int64_t total = 0, before = scan - mine;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    before *= p.num_kv_heads;
    total *= p.num_kv_heads;
    Int4Split split;
    int workers = gridDim.x * W;
    if (total < (1ll << 31)) {
        workers = max(1, min((int)total / p.min_stages, workers));
        split.each = (int)total / workers;
    } else {
        workers = (int)min(total / p.min_stages, (int64_t)workers);
        split.each = total / workers;
    }
    split.rest = total - split.each * workers;
    split.cta = (float)total / (float)workers * W;
    for (int w = 0; w < W; ++w) {  // whose sequence is in here?
        const int id = blockIdx.x * W + w;
        const int64_t lo = int4_begin(split, id);
        if (id >= workers || lo < before || lo >= before + mine * p.num_kv_heads) continue;
        int64_t at = before;
        for (int s = s_lo; s < s_hi; ++s) {
            const int64_t n = (int64_t)int4_weight(int4_len(p, s, BS)) * p.num_kv_heads;
            if (lo < at + n) {
                s_seq[w] = s;
                s_start[w] = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    const int64_t lo = int4_begin(split, blockIdx.x * W + warp);
    const int range = (int)(int4_begin(split, blockIdx.x * W + warp + 1) - lo);
    if (tid == 0) s_split = split;
    Int4Seg seg = {};
    seg.s = s_seq[warp];
    bool more = seg.s >= 0;
    if (more) {
        seg.len = int4_len(p, seg.s, BS);
        seg.nt = int4_stages(seg.len);
        const int weight = seg.nt + kI4UnitCost;
        seg.h = (int)((lo - s_start[warp]) / weight);
        const int64_t unit = s_start[warp] + (int64_t)seg.h * weight;
        const int off = (int)(lo - unit);
        seg.t0 = max(0, off - kI4UnitCost);
        seg.t1 = min(seg.nt, off + range - kI4UnitCost);
        seg.left = range - (weight - off);
        more = seg.t0 < seg.t1;
        if (lane == 0) s_unit[warp] = unit;  // where the current unit starts in the weight
    }

    // ---- the copies.  A lane holds one table entry of the batch of stages being copied (32 entries:
    // 32 / RECS stages of one unit) and one of the batch after it.
    constexpr int CPR = BS * D / 32;  // 16-byte chunks of a record's codes
    constexpr int PPR = BS / 4;       // and of its pairs
    const uint32_t ring32 = smem_u32(ring);
    const uint32_t stride = (uint32_t)p.num_kv_heads * REC;
    const uint8_t *pk = nullptr, *pv = nullptr;  // this lane's chunk of block 0's records
    int pt = 0, pend = 0, pidx = 0, ent = 0, nent = 0, nstage = -1;  // nstage: the next batch's first (-1: none)
    unsigned badmask = 0, badbatch = 0;
    auto fetch = [&](Int4Seg &ns) {  // the next batch's unit, and its entries
        if (nstage >= ns.t1) {
            nstage = -1;
            if (int4_next(ns, p, BS)) {
                nstage = ns.t0;
                // its queries will be wanted soon
                const __nv_bfloat16 *q = p.query + ((int64_t)ns.s * p.num_heads + ns.h * p.group) * D;
                for (int i = lane * 64; i < p.group * D; i += 32 * 64)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
            }
        }
        if (nstage >= 0) {  // past the end the last entry again: a stage is always copied whole
            const int i = min(nstage * RECS + lane, (ns.len - 1) / BS);
            nent = p.block_tables[(int64_t)ns.s * p.max_blocks + i];
        }
        __syncwarp();
        if (lane == 0) s_ns[warp] = ns;
        __syncwarp();
    };
    auto take = [&] {
        Int4Seg ns = s_ns[warp];
        ent = nent;
        pt = nstage;
        pend = min(ns.t1, nstage + 32 / RECS);
        pidx = 0;
        const bool bad = (uint32_t)ent >= (uint32_t)p.num_blocks;
        badbatch = __any_sync(FULL, bad);
        if (bad) {
            record_status(kStatusBadBlock);
            ent = 0;  // block 0 stands in; the unit's result becomes NaN
        }
        const int64_t at = (int64_t)ns.h * REC + (CPR < 32 ? lane & (CPR - 1) : lane) * 16;
        pk = p.key_cache + at;
        pv = p.value_cache + at;
        nstage += 32 / RECS;
        fetch(ns);
    };
    // One stage into a slot, 16 bytes a lane and copy: the codes of both caches, then the pairs.
    auto issue = [&](int slot) {
        if (pt < pend) {
            badmask = (badmask & ~(1u << slot)) | (badbatch << slot);
            const int chunk = CPR < 32 ? lane & (CPR - 1) : lane;
            const uint32_t dst = ring32 + slot * Lay::kStage;
            // value rows are swizzled: chunk q of row r at q ^ r / 2 (r / 4)
            const int vchunk = D == 128 ? chunk ^ ((chunk >> 3) & 3) : chunk ^ ((chunk >> 3) & 1);
#pragma unroll
            for (int i = 0; i < (CPR < 32 ? RECS * CPR / 32 : RECS); ++i) {
                const int r = CPR < 32 ? i * (32 / CPR) + lane / CPR : i;
                const uint64_t off = (uint64_t)(uint32_t)__shfl_sync(FULL, ent, pidx + r) * stride;
                const uint8_t *k = pk + off, *v = pv + off;
                const uint32_t dk = dst + r * REC, dv = dk + RECS * REC;
#pragma unroll
                for (int x = 0; x < (CPR + 31) / 32; ++x) {
                    cp_async16(dk + chunk * 16 + x * 512, k + x * 512);
                    cp_async16(dv + vchunk * 16 + x * 512, v + x * 512);
                }
                if (chunk < PPR) {
                    cp_async16(dk + BS * (D / 2) + chunk * 16, k + BS * (D / 2));
                    cp_async16(dv + BS * (D / 2) + chunk * 16, v + BS * (D / 2));
                }
            }
            ++pt;
            pidx += RECS;
            if (pt >= pend && nstage >= 0) take();
        }
        cp_async_commit();  // an empty group keeps the count where nothing is left
    };
    if (more) {
        nstage = seg.t0;
        Int4Seg ns = seg;
        fetch(ns);
    }
    // Its result may be the query or the new rows that a kernel after it reads before its
    // own griddepcontrol.wait: that one never starts early (started early, one launch after
    // another: four short sequences 4.1 instead of 6.2 us, eight long ones 1 % less).
    pdl_wait();
    if (nstage >= 0) take();
    for (int i = 0; i < NS; ++i) issue(i);

    // rows of sequences without a token
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
        if (p.seq_lens[s] <= 0) {
            uint4 *row = reinterpret_cast<uint4 *>(p.out + (int64_t)s * p.num_heads * D);
            for (int i = tid; i < p.num_heads * D / 8; i += W * 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }

    constexpr int RB = D / 2;  // bytes of a row
    // offset of token `row` (0..7) of 8-token group q (0..3) of a stage
    auto row_at = [&](int q, int row) { return BS == 8 ? q * REC + row * RB
                                             : BS == 16 ? (q >> 1) * REC + ((q & 1) * 8 + row) * RB
                                                        : (q * 8 + row) * RB; };
    auto pair_at = [&](int q, int row) { return BS == 8 ? q * REC + BS * RB + row * 4
                                              : BS == 16 ? (q >> 1) * REC + BS * RB + ((q & 1) * 8 + row) * 4
                                                         : BS * RB + (q * 8 + row) * 4; };

    // this lane's row of the value tile's matrices: matrix lane / 8 is chunk 2 x2 + lane / 16, half
    // (lane / 8) % 2; 16-byte chunk q of row r lies at q ^ r / 2 (D 128) or q ^ r / 4 (D 64), so that
    // the 8 rows of a matrix fall in different banks
    int vlane[VW];
#pragma unroll
    for (int x2 = 0; x2 < VW; ++x2) {
        const int r = lane & 7, q = 2 * x2 + (lane >> 4);
        vlane[x2] = row_at((lane >> 3) & 1, r) + (D == 128 ? q ^ (r >> 1) : q ^ (r >> 2)) * 16;
    }

    int slot = 0;
    while (more) {
        // ---- the unit's queries as fp16, each head scaled by a power of two: its largest magnitude into
        // [2^14, 2^15), and 2^-4 of that for the odd dims, whose codes come as 16 c: exact for entries down to
        // 2^-27 of the largest.  A word's operands lie together.  (A product of a subnormal code is cut 2^-25
        // below its nominal exponent: at 2^-15 of the largest entry of its 16 dims, for products of up to 15
        // times an entry.)
        uint64_t qa[NG];  // a lane's two heads
        float qb[NG][2];
        const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int head = n * 8 + g;
            uint4 raw[KW];
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                raw[j] = make_uint4(0u, 0u, 0u, 0u);  // columns past the group are zero
                if (head < p.group)
                    raw[j] = *reinterpret_cast<const uint4 *>(
                        p.query + ((int64_t)seg.s * p.num_heads + seg.h * p.group + head) * D + c * (D / 4) + 8 * j);
            }
            uint32_t top2 = 0;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) top2 = max_nan_bf16x2(top2, u4_word(raw[j], i) & 0x7FFF7FFFu);
            top2 = max_nan_bf16x2(top2, __shfl_xor_sync(FULL, top2, 1));
            top2 = max_nan_bf16x2(top2, __shfl_xor_sync(FULL, top2, 2));
            const uint32_t top = max_nan_bf16x2(top2, prmt(top2, top2, 0x1032u)) & 0x7FFFu;
            const int e = max((int)(top >> 7) - 127, -100);
            const float even = pow2i(14 - e) * sign, odd = pow2i(10 - e) * sign;
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                float x[8];
                unpack8(raw[j], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[i];
                *reinterpret_cast<uint4 *>(qop + ((n * KW + j) * 32 + lane) * 16) =
                    make_uint4(pack_f16x2(x[0] * even, x[4] * even), pack_f16x2(x[1] * odd, x[5] * odd),
                               pack_f16x2(x[2] * even, x[6] * even), pack_f16x2(x[3] * odd, x[7] * odd));
            }
            sum += __shfl_xor_sync(FULL, sum, 1);
            sum += __shfl_xor_sync(FULL, sum, 2);
            // log2-logit = qa (s S + z qb): S = +-(q . codes) 2^-10 2^-e, below 4; an infinity or a NaN in the
            // query makes it NaN.  qa > 0, so the largest product is the largest logit.
            const float a = fminf(fmaxf(fabsf(p.scale_log2) * 1024.f * pow2i(min(e, 127)), 1.17549435e-38f), 3.4e38f);
            const float b = top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                                           : sum * (sign * 9.765625e-4f) * pow2i(-(e >> 1)) * pow2i((e >> 1) - e);
#pragma unroll
            for (int i = 0; i < 2; ++i) qb[n][i] = __shfl_sync(FULL, b, (2 * c + i) * 4);
            qa[n] = f32x2(__shfl_sync(FULL, a, 2 * c * 4), __shfl_sync(FULL, a, (2 * c + 1) * 4));
        }

        // m: minus the running maximum, in units of log2; mlim: the logit / qa from which it moves; vmul =
        // 2^(10 - ev): weights times value scales, in units of 2^m, were below 2^(ev + 1) when it was set
        float o[NG][MT][4], o1[NG][4], m[NG][2], mlim[NG][2], vmul[NG][2], zs[NG][2];
        uint64_t l[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = INFINITY;
                mlim[n][i] = -INFINITY;
                vmul[n][i] = pow2i(126);
                o1[n][i] = o1[n][2 + i] = zs[n][i] = 0.f;
            }
            l[n] = f32x2(0.f, 0.f);
        }
        // what the stages do not need waits in shared memory
        const int t1 = seg.t1, len = seg.len;
        int t = seg.t0;
        if (lane == 0) s_seg[warp] = seg;
        unsigned poison = 0;
        __syncwarp();

        for (; t < t1; ++t) {
            cp_async_wait<NS - 1>();
            __syncwarp();
            poison |= (badmask >> slot) & 1u;
            const uint8_t *kb = ring + slot * Lay::kStage, *vb = kb + RECS * REC;
            const uint32_t vb32 = smem_u32(vb);

            // ---- S = codes . q: 16 tokens x 8 heads x 16 dims a step, the stage's two token tiles in turn
            float sc[2][NG][4];
            uint32_t kw[2][2][KW];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint8_t *a = kb + row_at(2 * mt + hf, g) + c * (D / 8);
                    if constexpr (KW == 4) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(a);
                        kw[mt][hf][0] = u.x, kw[mt][hf][1] = u.y, kw[mt][hf][2] = u.z, kw[mt][hf][3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2 *>(a);
                        kw[mt][hf][0] = u.x, kw[mt][hf][1] = u.y;
                    }
                }
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const uint4 qf = *reinterpret_cast<const uint4 *>(qop + ((n * KW + j) * 32 + lane) * 16);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t x = kw[mt][0][j], y = kw[mt][1][j], x8 = x >> 8, y8 = y >> 8;
                        if (j == 0) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.f;
                        mma_codes(sc[mt][n], x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u, qf.x, qf.y);
                        mma_codes(sc[mt][n], x8 & 0x000F000Fu, y8 & 0x000F000Fu, x8 & 0x00F000F0u, y8 & 0x00F000F0u, qf.z,
                                  qf.w);
                    }
                }

            // ---- logits / qa and the rows' pairs; row g + 8 half of tile mt is token 8 (2 mt + half) + g
            float2 vp[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 kp = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(kb + pair_at(q, g)));
                vp[q] = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(vb + pair_at(q, g)));
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &y = sc[q >> 1][n][(q & 1) * 2 + i];
                        y = fmaf(kp.x, y, kp.y * qb[n][i]);
                    }
            }
            if (len - t * kI4Tokens < kI4Tokens) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (t * kI4Tokens + q * 8 + g >= len) {
                        vp[q] = make_float2(0.f, 0.f);
#pragma unroll
                        for (int n = 0; n < NG; ++n) sc[q >> 1][n][(q & 1) * 2] = sc[q >> 1][n][(q & 1) * 2 + 1] = -INFINITY;
                    }
            }

            // ---- weights: fp32 into l and the zeros' sum; times the value scale and rounded
            // to fp16 (2^-11 relative) for the tensor cores, one 8x8 transpose each.  Codes count from
            // 7.5: w c = w (c - 7.5) + 7.5 w, and what 7.5 times the rounded weights adds is taken out by
            // their sum (o1, a row of 2^-10: a normal number, whose products are not cut, see the queries),
            // while 7.5 times the unrounded ones goes into the zeros' sum.
            // Counted from 0, the codes' mean would cancel against the zeros and leave 2.9 times the
            // rounding.  The second tile takes 15 - c with negative weights: both its and the first
            // tile's accumulators stay near zero, where the tensor cores' truncation of long sums is small
            // (results of eight long sequences against the fp32 form's: 0.0025 off before, 0.0009 now).
            //
            // The maximum moves only when a logit passes it by more than 4, so a weight stays below 2^4.
            // vmul, which brings a head's weights w = p s' into the fp16 range, is set where the maximum
            // moves and where a scaled weight reaches 2^15, from the largest weight so far, not from the
            // largest scale: a row far above the others counts only with its weight.  Both are rare: the
            // stage's weights are made first and then, if they have to be, once more.
            float top[NG][2];
            bool move = false;
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[n][i] = fmaxf(fmaxf(sc[0][n][i], sc[0][n][2 + i]), fmaxf(sc[1][n][i], sc[1][n][2 + i]));
                    move |= top[n][i] > mlim[n][i];
                }
            uint32_t pf[NG][4];
            uint64_t ls[NG];
            float zz[NG][2];
            for (bool again = true;;) {
                uint32_t big = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float vs = q < 2 ? vp[q].x : -vp[q].x, z = fmaf(7.5f, vp[q].x, vp[q].y);
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        const float *y = &sc[q >> 1][n][(q & 1) * 2];
                        const float2 x = f32x2_split(fma_f32x2(qa[n], f32x2(y[0], y[1]), f32x2(m[n][0], m[n][1])));
                        const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                        const uint64_t pr = f32x2(p0, p1);
                        ls[n] = q ? add_f32x2(ls[n], pr) : pr;
                        zz[n][0] = q ? fmaf(p0, z, zz[n][0]) : p0 * z;
                        zz[n][1] = q ? fmaf(p1, z, zz[n][1]) : p1 * z;
                        // p s' first: it is finite, and 0 where p is, whatever vmul still is
                        const float2 w = f32x2_split(mul_f32x2(mul_f32x2(pr, f32x2(vs, vs)), f32x2(vmul[n][0], vmul[n][1])));
                        pf[n][q] = pack_f16x2(w.x, w.y);
                        big = max_abs_f16x2(big, pf[n][q]);
                    }
                }
                move |= ((big + 0x08000800u) & 0x80008000u) != 0u;  // 2^15 or more, in either half
                if (!__any_sync(FULL, move) || !again) break;
                again = false;
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const float2 qf = f32x2_split(qa[n]);
                    float corr[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = i ? qf.y : qf.x;
                        float to = top[n][i], wtop = 0.f;
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) to = fmaxf(to, __shfl_xor_sync(FULL, to, off));
                        const float mn = fminf(m[n][i], -(a * to));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            wtop = fmaxf(wtop, fast_exp2(fmaf(a, sc[q >> 1][n][(q & 1) * 2 + i], mn)) * fabsf(vp[q].x));
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) wtop = fmaxf(wtop, __shfl_xor_sync(FULL, wtop, off));
                        // what was summed so far falls by 2^-by; it and this stage set the new power of two
                        const float by = m[n][i] == INFINITY ? 400.f : fminf(m[n][i] - mn, 400.f);
                        const int ev = int4_scale_exp(vmul[n][i]);
                        const int en = min(max(max((int)(__float_as_uint(wtop) >> 23) - 127, ev - (int)by), -116), 127);
                        m[n][i] = mn;
                        mlim[n][i] = (4.f - mn) / a;
                        vmul[n][i] = pow2i(10 - en);
                        corr[i] = exp2f(-by);
                        zs[n][i] *= corr[i];  // a NaN stays one
                        const float oc = exp2f((float)(ev - en) - by);
                        o1[n][i] *= oc;
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            o[n][k][i] *= oc;
                            o[n][k][2 + i] *= oc;
                        }
                    }
                    l[n] = mul_f32x2(l[n], f32x2(corr[0], corr[1]));
                }
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                l[n] = add_f32x2(l[n], ls[n]);
                const float2 z = f32x2_split(add_f32x2(f32x2(zs[n][0], zs[n][1]), f32x2(zz[n][0], zz[n][1])));
                zs[n][0] = z.x, zs[n][1] = z.y;
#pragma unroll
                for (int q = 0; q < 4; ++q) pf[n][q] = movmatrix_trans(pf[n][q]);
            }

            // ---- O += codes' . w: 16 dims x 8 heads x 16 tokens a step
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    mma_codes(o1[n], 0x14001400u, 0u, 0x14001400u, 0u, pf[n][2 * mt], pf[n][2 * mt + 1]);
#pragma unroll
                for (int x2 = 0; x2 < VW; ++x2) {
                    // [chunk][half] of 8 tokens x 8 half words: a lane gets half word g of tokens 2c, 2c + 1
                    uint32_t v[2][2];
                    ldsm_x4_trans(vb32 + row_at(2 * mt, 0) + vlane[x2], v[0][0], v[0][1], v[1][0], v[1][1]);
#pragma unroll
                    for (int hw = 0; hw < 2; ++hw) {
                        const uint32_t flip = mt ? ~0u : 0u;  // 15 - c
                        const uint32_t x = v[hw][0] ^ flip, y = v[hw][1] ^ flip, x8 = (v[hw][0] >> 8) ^ flip,
                                       y8 = (v[hw][1] >> 8) ^ flip;
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            mma_codes(o[n][4 * x2 + 2 * hw], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu,
                                      y & 0x00F000F0u, pf[n][2 * mt], pf[n][2 * mt + 1]);
                            mma_codes(o[n][4 * x2 + 2 * hw + 1], x8 & 0x000F000Fu, x8 & 0x00F000F0u, y8 & 0x000F000Fu,
                                      y8 & 0x00F000F0u, pf[n][2 * mt], pf[n][2 * mt + 1]);
                        }
                    }
                }
            }

            // ---- hand the slot back
            __syncwarp();
            issue(slot);
            if (++slot == NS) slot = 0;
        }

        // ---- the unit's end: whole, it goes out; cut, it waits for the join
        const Int4Seg was = s_seg[warp];
        const int64_t here = s_unit[warp];
        seg = was;
        __syncwarp();
        if (lane == 0) s_unit[warp] = here + was.nt + kI4UnitCost;
        more = int4_next(seg, p, BS);
        const bool whole = was.t0 == 0 && was.t1 == was.nt;
        Int4Cut<NG> &cut = s_cut[warp][more ? 0 : 1];
        uint8_t *data = nullptr;
        float4 *part = nullptr;  // the first warp's first unit goes to the workspace at once
        if (!whole) {
            if (!more) {
                cp_async_wait<0>();  // nothing is left to come: the ring is free
                __syncwarp();
                data = ring;
            } else if (warp > 0) {
                data = smem + Lay::kHead + (warp - 1) * Lay::kPart;
            } else {
                part = p.part_o + (int64_t)2 * blockIdx.x * (NG * Lay::kChunks * 32);
            }
            if (lane == 0) {
                cut.unit = here;
                cut.s = was.s;
                cut.h = was.h;
                cut.nt = was.nt;
                cut.from = was.t0 > 0;
                cut.to = was.t1 < was.nt;
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int hd = n * 8 + 2 * c + i;
                const float2 lf = f32x2_split(l[n]);
                float lt = i ? lf.y : lf.x, zt = zs[n][i];
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) {
                    lt += __shfl_xor_sync(FULL, lt, off);
                    zt += __shfl_xor_sync(FULL, zt, off);
                }
                const float f = pow2i(int4_scale_exp(vmul[n][i]));  // out of the accumulators: 2^24 2^(ev - 10)
                zt = fmaf(o1[n][i] * -7.5f, f, zt);
                if (poison) lt = __uint_as_float(0x7FC00000u);
                const float inv = 1.f / lt;
                if (!whole && g == 0) {
                    cut.m[hd] = -m[n][i];
                    cut.l[hd] = lt;
                    if (part && hd < p.group) p.part_ml[2 * blockIdx.x * 16 + hd] = make_float2(-m[n][i], lt);
                }
#pragma unroll
                for (int k = 0; k < MT / 2; ++k) {  // dims 32 k + 4 g ..
                    const float4 r = make_float4(
                        fmaf(o[n][2 * k][i] * 16384.f, f, zt), fmaf(o[n][2 * k][2 + i] * 1024.f, f, zt),
                        fmaf(o[n][2 * k + 1][i] * 16384.f, f, zt),
                        fmaf(o[n][2 * k + 1][2 + i] * 1024.f, f, zt));
                    const int cell = (n * Lay::kChunks + i * (MT / 2) + k) * 32 + lane;
                    if (hd >= p.group) continue;
                    if (whole)
                        *reinterpret_cast<uint2 *>(
                            p.out + ((int64_t)was.s * p.num_heads + was.h * p.group + hd) * D + 32 * k + 4 * g) =
                            make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
                    else if (part)
                        part[cell] = r;
                    else
                        *reinterpret_cast<float4 *>(data + cell * 16) = r;
                }
            }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- the join.  Parts of one unit lie in neighbouring warps: a run of them is joined here, and
    // what is still only a part of its unit goes to the workspace (slot 0: began before this CTA,
    // 1: begins in it).  Part 2 w + k is warp w's first (0) or last (1) unit.
    const Int4Cut<NG> &mine_cut = s_cut[(lane >> 1) % W][lane & 1];
    const unsigned from = __ballot_sync(FULL, lane < 2 * W && mine_cut.from);
    const unsigned to = __ballot_sync(FULL, lane < 2 * W && mine_cut.to);
    const unsigned have = from | to;
    if (!have) return;
    // Part 0 is in the workspace already.  The others' runs begin where no earlier part belongs to the unit.
    const unsigned parts = have & ~1u, begins = parts & (~from | (parts & -parts));
    float *const wf = reinterpret_cast<float *>(smem + Lay::kQf);  // [part][head]: the queries are done with
    constexpr int H = 8 * NG;
    auto run_of = [&](int e) {  // the parts of e's run
        const int b = 31 - __clz(begins & ((2u << e) - 1));
        const unsigned after = begins & ~((2u << e) - 1);
        return parts & ~((1u << b) - 1) & (after ? (after & -after) - 1 : ~0u);
    };
    if (tid < 2 * W * H && ((parts >> (tid / H)) & 1u)) {
        const int e = tid / H, hd = tid % H;
        const unsigned run = run_of(e);
        float M = -INFINITY, L = 0.f;
        for (unsigned b = run; b; b &= b - 1) {
            const int x = __ffs(b) - 1;
            M = fmaxf(M, s_cut[x >> 1][x & 1].m[hd]);
        }
        for (unsigned b = run; b; b &= b - 1) {
            const int x = __ffs(b) - 1;
            const Int4Cut<NG> &u = s_cut[x >> 1][x & 1];
            const float f = fast_exp2(u.m[hd] - M);
            L = fmaf(f, u.l[hd], L);
            if (x == e) wf[tid] = f;
        }
        wf[2 * W * H + tid] = L;
        wf[4 * W * H + tid] = M;
    }
    __syncthreads();
    // A part of the unit shared with earlier / later CTAs, or -1: the first run's, the last one's.
    const int first_part = __ffs(parts) - 1, last_part = 31 - __clz(parts);  // -1: none
    const int left = (have & 1u) ? 0 : first_part >= 0 && ((from >> first_part) & 1u) ? first_part : -1;
    int right = last_part >= 0 && ((to >> last_part) & 1u) ? 31 - __clz(begins) : -1;
    for (int cell = tid; cell < NG * Lay::kChunks * 32; cell += W * 32) {
        const int k = (cell >> 5) % Lay::kChunks, hd = (cell >> 5) / Lay::kChunks * 8 + 2 * c + k / (MT / 2);
        if (hd >= p.group) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (unsigned b = parts; b;) {
            const int e = __ffs(b) - 1;
            b &= b - 1;
            const float4 v = *reinterpret_cast<const float4 *>(
                smem + (e & 1 ? (e >> 1) * Lay::kRing : Lay::kHead + ((e >> 1) - 1) * Lay::kPart) + cell * 16);
            const float f = wf[e * H + hd];
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
            const bool ends = !b || ((begins >> (__ffs(b) - 1)) & 1u);
            if (!ends) continue;
            // the run's last part: out it goes
            const float L = wf[2 * W * H + e * H + hd];
            const int b0 = 31 - __clz(begins & ((2u << e) - 1));
            if (b0 != left && b0 != right) {
                const Int4Cut<NG> &u = s_cut[e >> 1][e & 1];
                const float inv = 1.f / L;
                *reinterpret_cast<uint2 *>(p.out + ((int64_t)u.s * p.num_heads + u.h * p.group + hd) * D +
                                           32 * (k % (MT / 2)) + 4 * g) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            } else {
                const int64_t part = 2 * blockIdx.x + (b0 == left ? 0 : 1);
                p.part_o[part * (NG * Lay::kChunks * 32) + cell] = acc;
                if (g == 0 && k % (MT / 2) == 0) p.part_ml[part * 16 + hd] = make_float2(wf[4 * W * H + e * H + hd], L);
            }
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (left < 0 && right < 0) return;

    // ---- a unit cut between CTAs: the last one to arrive joins its parts, in order
    if (left == right) right = -1;
    __syncthreads();
    if (lane == 0 && warp < 2) {
        const int e = warp ? right : left;
        if (e >= 0) {
            const Int4Cut<NG> &u = s_cut[e >> 1][e & 1];
            const int first = ((from >> e) & 1u) ? int4_cta_of(s_split, u.unit + kI4UnitCost) : blockIdx.x;
            const int last = int4_cta_of(s_split, u.unit + kI4UnitCost + u.nt - 1);
            const int n = last - first;  // arrivals before the last one
            __threadfence();  // the CTA's part, behind the barrier above
            const int old = atomicAdd(p.counters + first, 1);
            __threadfence();  // the others' parts, ahead of the barrier below
            s_last[warp] = old == n;
            if (old == n) p.counters[first] = 0;
            s_first[warp] = first;
            s_end[warp] = last;
        }
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const int e = side ? right : left;
        if (e < 0 || !s_last[side]) continue;
        const Int4Cut<NG> *u = &s_cut[e >> 1][e & 1];
        const int first = s_first[side], last = s_end[side];
        const int items = p.group * (D / 4);
        // 4 dims of a head a thread and item; where those are fewer than the threads, `ways` of
        // them share the parts.  U parts of every item are in flight at a time.
        constexpr int U = 4, ITS = NG * D / 64;
        const int ways = items < W * 32 ? W * 32 / items : 1;
        const int way = tid / items;  // from `ways` on: nothing to do
        const int it0 = tid - way * items;
        uint8_t *const join = smem + side * Lay::kRing;  // rings are free
        float M[ITS], L[ITS];
        float4 sums[ITS];
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
            M[i] = -INFINITY;
            L[i] = 0.f;
            sums[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int w = way < ways ? first + way : last + 1; w <= last; w += ways * U) {
            float2 ml[ITS][U];
            float4 r[ITS][U];
#pragma unroll
            for (int i = 0; i < ITS; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int it = it0 + i * W * 32, hd = it / (D / 4), d4 = it % (D / 4);
                    const int x = w + u * ways;
                    const int64_t q = 2 * x + (x == first ? 1 : 0);
                    ml[i][u] = make_float2(-INFINITY, 0.f);
                    r[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (x <= last && it < items) {
                        ml[i][u] = __ldcg(&p.part_ml[q * 16 + hd]);
                        r[i][u] = __ldcg(&p.part_o[q * (NG * Lay::kChunks * 32) + ((hd >> 3) * Lay::kChunks +
                                                   (hd & 1) * (D / 32) + d4 / 8) * 32 + d4 % 8 * 4 + ((hd & 7) >> 1)]);
                    }
                }
#pragma unroll
            for (int i = 0; i < ITS; ++i) {
                const int it = it0 + i * W * 32;
                if (it >= items) break;
                float to = M[i];
#pragma unroll
                for (int u = 0; u < U; ++u) to = fmaxf(to, ml[i][u].x);
                const float corr = M[i] == -INFINITY ? 0.f : fast_exp2(M[i] - to);
                float4 &acc = sums[i];
                M[i] = to;
                L[i] *= corr;
                acc.x *= corr, acc.y *= corr, acc.z *= corr, acc.w *= corr;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float f = fast_exp2(ml[i][u].x - to);
                    L[i] = fmaf(f, ml[i][u].y, L[i]);
                    acc.x = fmaf(f, r[i][u].x, acc.x);
                    acc.y = fmaf(f, r[i][u].y, acc.y);
                    acc.z = fmaf(f, r[i][u].z, acc.z);
                    acc.w = fmaf(f, r[i][u].w, acc.w);
                }
            }
        }
        if (ways > 1) {
            if (way < ways) {
                *reinterpret_cast<float4 *>(join + tid * 16) = sums[0];
                if (tid % (D / 4) == 0)
                    *reinterpret_cast<float2 *>(join + W * 32 * 16 + tid / (D / 4) * 8) = make_float2(M[0], L[0]);
            }
        } else if (way == 0) {
#pragma unroll
            for (int i = 0; i < ITS; ++i) {
                const int it = it0 + i * W * 32;
                if (it >= items) break;
                const float inv = 1.f / L[i];
                *reinterpret_cast<uint2 *>(p.out + ((int64_t)u->s * p.num_heads + u->h * p.group) * D + 4 * it) =
                    make_uint2(pack_bf16x2(sums[i].x * inv, sums[i].y * inv), pack_bf16x2(sums[i].z * inv, sums[i].w * inv));
            }
        }
        if (ways > 1) {
            __syncthreads();
            if (tid < items) {
                const int hd = tid / (D / 4);
                const float2 *ml = reinterpret_cast<const float2 *>(join + W * 32 * 16);
                float M = -INFINITY, L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int y = 0; y < ways; ++y) M = fmaxf(M, ml[y * p.group + hd].x);
                for (int y = 0; y < ways; ++y) {
                    const float2 v = ml[y * p.group + hd];
                    const float4 r = *reinterpret_cast<const float4 *>(join + (y * items + tid) * 16);
                    const float f = fast_exp2(v.x - M);
                    L = fmaf(f, v.y, L);
                    acc.x = fmaf(f, r.x, acc.x);
                    acc.y = fmaf(f, r.y, acc.y);
                    acc.z = fmaf(f, r.z, acc.z);
                    acc.w = fmaf(f, r.w, acc.w);
                }
                const float inv = 1.f / L;
                *reinterpret_cast<uint2 *>(p.out + ((int64_t)u->s * p.num_heads + u->h * p.group) * D + 4 * tid) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            }
            __syncthreads();
        }
    }
}

}  // namespace pakv
