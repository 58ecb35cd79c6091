// kv8_attention.cuh - attention of a verify window over the 8-bit cache.
//
// Mathematics. The rows of a key/value head are its queries (token t, head h of its group): R = T *
// n_heads / n_kv_heads of them share every key and value. For a row, in base 2 (log2 e is in the
// row's factor), s_j = f * (q . (c_j - 128)) with f = |scale| * log2 e * k_scale * (the query's own
// power of two). A block's v_scale is r * 2^e, 1 <= r < 2. Kept running, block by block:
//   p_j = 2^(s_j - m),  l = sum p_j,  o = sum p_j 2^(e + d) r (c_j - 128),  out = o 2^-d / l,
// with d = m - n + 10, m at most 4 below the largest s_j and n at most 4 below the largest s_j + e, both
// whole numbers (so that their differences are exact): what is held in fp16, p_j 2^(e + d) r < 2^15, is
// large where a token's share of the output is, whatever its block's scale. o and l are rescaled only
// when m or n moves, which after the first blocks is rare. Where e + d is above kAttnFar (a value scale far
// above those that the output came from so far, with scores as far below), p_j is held times a power of two, so that
// neither it nor 2^(e + d) leaves fp32's range. fp16's range below 2^10, down to 2^-24, keeps a
// long tail of small weights. Codes and, after a shift by a power of two, 16-bit queries are exact in
// fp16; an fp32 query and its weights are two fp16 parts each. Sums are fp32; the matrix instructions
// truncate theirs, which shortens an output by up to 6e-6 of itself where a warp sums over some hundred blocks (in fp32; 16-bit
// outputs round by far more). For 16-bit queries the key
// codes enter as fp16 subnormals (two byte permutes per four codes) and the score starts at -128 * sum q,
// which is of the scores' own size: what that costs in rounding is far below theirs. For fp32 ones, and
// the value codes always (the sum of weights would be far above the result), they are centred, with two
// subtractions more.
//
// Layout. A matrix instruction (m16n8k16) takes 16 rows; its other operand is the record itself: a
// lane's eight bytes of a 256-byte tile are its part of two instructions' keys (eight dims of one
// token) or values (eight tokens of one dim), and the tokens whose scores a lane receives are the
// ones whose weights it must supply, so neither scores nor weights leave the registers.
// The row count is small and the cache is read once, so the work is a stream of records through
// registers, not a tile product: the matrix instructions that take register operands fit it, while
// operands staged for tcgen05 would have to be widened to fp16 in shared memory first (twice the
// bytes written and read there again).
//
// Split. The call's blocks, over all sequences, heads and groups of rows, are one list. Few segments
// (sequence, head, group) are cut into even parts, a CTA each; many into equal ranges of the list, in
// which a segment starts with kAttnSegCost units for its fixed work and a short one is left whole. A
// CTA's four warps take its blocks in turn, each with its own ring of shared-memory stages that bulk
// copies fill (one copy a block: keys, values and scales are one record). A CTA joins its warps'
// results in warp order. Ranges that end inside a sequence leave a part (rows, m, l) in the workspace,
// and a second kernel joins the parts in list order: the result does not depend on timing.
//
// What bounds it (GB300; the rate is of the records alone, of 6787 GB/s that a copy reaches):
//   1 sequence of 1,048,579 tokens, one head of 256 dims, 16 rows, bf16: 91 us, 5.9 TB/s: memory, and
//     ~9 us of launches, queries, first copies and joining;
//   64 sequences of 0 to 16k tokens, 8 heads of 128, 4 rows, bf16: 47.9 us, 5.1 TB/s: the same;
//   1 of 131,077 tokens, 4 heads of 128, 16 rows, fp32: 38.5 us, 3.5 TB/s: issue and latency of the two
//     parts' products at eight warps an SM, and the same fixed part;
//   32 windows of 4 over 8k to 33k tokens, 8 heads of 128, 32 rows, fp16: 244 us, 4.8 TB/s: the matrix
//     instructions and the widening of codes, at eight warps an SM (pipe 48 %, issue 40 %);
//   one token at 777 positions: 9.9 us, all latency.
// Heads of 160 to 256 dims spill 36 to 164 bytes in the forms of two parts (fp32, fp16 weights); no other
// form spills. The sums of 32 rows at 128 dims leave the compiler three registers: small changes of the masks cost up to 4 % there.
#pragma once

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"
#include "kv8_api.h"

namespace moe {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
// fp16 parts: one of a query and of a weight; of a weight two, for fp16 outputs, whose error one part's rounding
// would raise by 1.4 (but see kAttnShort); of both two, for fp32.
constexpr int kAttnPlain = 0, kAttnWeights = 1, kAttnSplit = 2;
constexpr int kAttnStages = 24;          // ring stages of a CTA, at most
constexpr int kAttnMaxCtas = 456;        // parts are kept for at most so many CTAs
// A row's references m and n move to their maxima only once those are kAttnSlack (in powers of two)
// above; the weights of the values are held times 2^kAttnShift.
constexpr float kAttnShift = 10.0f, kAttnSlack = 4.0f;
// The largest power of two by which a weight is multiplied on its way into a value's weight. (Above it the weight
// itself may be below fp32's range, and the factor above it: blocks whose value scales lie that far apart.)
constexpr float kAttnFar = 100.0f;
constexpr int kAttnWhole = 48;           // blocks of a segment that is left whole
constexpr int kAttnSegCost = 16;         // blocks that a segment's fixed work (queries, joining) costs
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.4426950408889634f;

// Row tiles of a pass over the blocks: MT tiles of 16 rows per warp; two warps share a ring where there are
// more rows. Further rows are further passes, which find the blocks in L2: four warps on a ring left one
// CTA with 128 rows of queries to convert, 20 us for a short sequence.
struct AttnGeom {
    int MT, RTW, RP, RB;  // RP = 16 MT RTW rows a pass, RB passes
};
inline AttnGeom attn_geom(int R, bool two) {
    AttnGeom g;
    g.MT = two ? 2 : 1;
    g.RTW = R > 16 * g.MT ? 2 : 1;
    g.RP = 16 * g.MT * g.RTW;
    g.RB = (R + g.RP - 1) / g.RP;
    return g;
}
// Two tiles a warp widen a block's codes once for 32 rows, and leave registers for eight warps an SM instead of
// twelve: better where the work is long (32 windows of 4 over 8k to 32k tokens: 252 against 285 us), not where it
// is short (4 over 3k: 22.1 both), about even at kAttnLong blocks of the page table. Not for fp32
// (two fp16 parts: 64 rows of 16k tokens 138 against 114 us) or wide heads, whose sums fill the registers.
constexpr int64_t kAttnLong = 24576;
// With more than 16 fp16 rows, weights of two parts take as much again as one part where the products bound the
// kernel: up to so many blocks latency does.
constexpr int64_t kAttnShort = 4096;

// workspace: int32 plan[n_seqs + 2] (what comes before each sequence in the list; the chunk, 0: a CTA
// per part), then two parts per CTA
inline __host__ __device__ int64_t attn_plan_bytes(int n_seqs) { return (static_cast<int64_t>(n_seqs) + 2 + 3) / 4 * 16; }
inline __host__ __device__ int64_t attn_part_floats(int RP, int D) { return static_cast<int64_t>(RP) * (D + 2); }

struct AttnPlan {
    AttnArgs a;
    AttnGeom g;
    int R, segs;     // rows of a key/value head; segments (head, pass) of a sequence
    int out_type, prec;
    int stages;      // ring stages per group of RTW warps
    int smem;
    int* plan;
    float* parts;
};

cudaError_t launch_attn_f32(const AttnPlan& p, cudaStream_t st);
cudaError_t launch_attn_f16(const AttnPlan& p, cudaStream_t st);
cudaError_t launch_attn_bf16(const AttnPlan& p, cudaStream_t st);
cudaError_t launch_attn_combine(const AttnPlan& p, cudaStream_t st);

// Blocks that a sequence's queries can see: n blocks from `first`.
__device__ __forceinline__ void attn_seq(const AttnArgs& a, int b, int& len, int& first, int& n, bool report) {
    len = gload(a.lens + b);
    const int64_t cap = static_cast<int64_t>(a.c.max_pages) * a.c.page_blocks * kKvBlock;
    if (len < 0) {
        if (report) set_err(a.err, MOE_ERR_LEN);
        len = 0;
    }
    if (len > cap) {
        if (report) set_err(a.err, MOE_ERR_PAGE);
        len = static_cast<int>(cap);
    }
    first = 0;
    if (a.window > 0) {
        const int64_t lo = static_cast<int64_t>(len) - a.T - a.window + 1;  // the first query's first position
        if (lo > 0) first = static_cast<int>(lo >> 5);
    }
    n = len > 0 ? ((len - 1) >> 5) + 1 - first : 0;
}

// The depth of window token t of the sequence whose tokens are bt ..: at most its index.
__device__ __forceinline__ int attn_depth(const AttnArgs& a, int64_t bt, int t) { return min(max(gload(a.depth + bt + t), 0), t); }

// How the list is cut. By parts (tb > 0): a segment of n blocks takes ceil(n / tb) CTAs, which share it
// evenly. By cost: a segment counts for kAttnSegCost + n, and the CTAs take equal ranges.
struct AttnCut {
    int tb, chunk;  // of the list per CTA; 1 by parts
    __host__ __device__ __forceinline__ int cost(int n) const { return !n ? 0 : tb ? (n + tb - 1) / tb : n + kAttnSegCost; }
};
// blocks: of all segments; segs: segments that have any; longest: blocks of the longest.
// (The host keeps the whole list, at its longest, below 2^31.)
__device__ __forceinline__ AttnCut attn_cut(int blocks, int segs, int longest, int ctas) {
    AttnCut c;
    c.tb = 0;
    c.chunk = (blocks + segs * kAttnSegCost + ctas - 1) / ctas;
    if (segs < ctas) {
        // a part has a block for each warp at least, or two where there are more parts than the joining reads at once
        const int least = min(max(longest / 32, kAttnWarps), 2 * kAttnWarps);
        const int tb = max((blocks + (ctas - segs) - 1) / (ctas - segs), least);  // then the parts are at most `ctas`
        if (tb <= c.chunk || tb <= least) c.tb = tb;
        // short segments are not worth cutting: a part costs as much as so many blocks
        else if (longest <= kAttnWhole) c.tb = longest;
        if (c.tb) c.chunk = 1;
    }
    return c;
}

#ifdef __CUDACC__

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d = a b + c, a: the four words that a lane holds of 16 rows by 16
__device__ __forceinline__ void mma_16816(float (&d)[4], uint4 a, uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint4 a, uint32_t b0, uint32_t b1) { mma_16816(d, a, b0, b1, d); }

// four codes -> two half2 of code * 2^-24 (fp16's subnormals; exact)
__device__ __forceinline__ void codes_sub(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = prmt(w, 0u, 0x4140u);
    hi = prmt(w, 0u, 0x4342u);
}

// four codes -> two half2 of code - 128 (exact)
__device__ __forceinline__ void codes_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = prmt(w, 0x64646464u, 0x4140u), b = prmt(w, 0x64646464u, 0x4342u);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint32_t pack_h2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

__device__ __forceinline__ uint32_t& word(uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A run of blocks [blk, end) of one segment within the CTA's range.
struct AttnPiece {
    int b, seg, len, first, n, blk, end;
    int left;  // of the CTA's range after this piece, in units of cost
};

// The rest of the CTA's range starts `off` into the current segment's kAttnSegCost + n units: its
// blocks, and what is left after them. (A range that ends within the fixed part has no blocks here.)
__device__ __forceinline__ void attn_take(AttnPiece& x, int off, int rest) {
    const int u = off > kAttnSegCost ? off - kAttnSegCost : 0, end = off + rest - kAttnSegCost;
    x.blk = x.first + u;
    x.end = x.first + (end < u ? u : end < x.n ? end : x.n);
    x.left = rest - (kAttnSegCost + x.n - off);
}
__device__ __forceinline__ bool attn_next(const AttnPlan& p, AttnPiece& x) {
    if (x.left <= kAttnSegCost) return false;  // no block of the next segment
    if (++x.seg == p.segs) {
        x.seg = 0;
        do {
            if (++x.b >= p.a.c.n_seqs) return false;
            attn_seq(p.a, x.b, x.len, x.first, x.n, false);
        } while (x.n == 0);
    }
    attn_take(x, 0, x.left);
    return true;
}

template <int D, int MT, int PREC>
struct AttnSmem {
    static constexpr bool SPLIT = PREC == kAttnSplit;
    static constexpr int kRec = kv8_record_bytes(D);
    static constexpr int kTileQ = D * 32 * (SPLIT ? 2 : 1);  // fragments of 16 rows
    static constexpr int kRowO = D + 8;                      // floats of a row in the joining buffer
    static __host__ __device__ int buf_bytes(int RTW) {
        const int q = kTileQ * MT * RTW, o = 16 * MT * RTW * kRowO * 4;
        return q > o ? q : o;
    }
    // buffer (queries, then the joined rows), the warps' m and l, row factors and offsets, output rows, the
    // warps' pieces, barriers and flags, ring
    static constexpr int kStats = kAttnWarps * 16 * MT * 20 + 2 * kAttnWarps * static_cast<int>(sizeof(AttnPiece));
    static __host__ __device__ int fixed(int RTW) { return (buf_bytes(RTW) + kStats + kAttnStages * 20 + 16 + 15) / 16 * 16; }
};

// Registers of a thread: for three CTAs an SM, or two; with 192 the joining kernel's CTAs find room beside two
// (100k tokens, 16 rows of 64 dims, fp16: 17.5 us, with 195 registers 21.3). Given as a limit, not as CTAs an SM: the compiler then
// keeps wide heads' loop as fast as at two CTAs (256 dims, fp16: 34 us, else 39).
constexpr int attn_regs(int D, int MT, int PREC) {
    return MT == 1 && D <= 128 && PREC == kAttnPlain ? 168 : D == 64 && PREC == kAttnWeights ? 192 : 255;
}

template <int D, int MT, int PREC>
__global__ void __maxnreg__(attn_regs(D, MT, PREC)) kv8_attention_kernel(const AttnPlan p) {
    using L = AttnSmem<D, MT, PREC>;
    constexpr bool SPLIT = PREC == kAttnSplit, W2 = PREC != kAttnPlain;  // two parts of a query; of a weight
    constexpr int kNB = D / 32, kND = D / 8;
    extern __shared__ __align__(128) uint8_t sm[];
    const AttnArgs& a = p.a;
    const int RTW = p.g.RTW, NG = kAttnWarps / RTW, RP = p.g.RP, S = p.stages;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int grp = wid / RTW, rt = wid - grp * RTW;
    uint4* qs = reinterpret_cast<uint4*>(sm);
    float* buf = reinterpret_cast<float*>(sm);
    float2* stat = reinterpret_cast<float2*>(sm + L::buf_bytes(RTW));        // [warps][16 MT]: m, l
    float2* qf = stat + kAttnWarps * 16 * MT;                                // [RP]: a row's factor and offset
    int* orow = reinterpret_cast<int*>(qf + 16 * MT * kAttnWarps);           // [RP]: a row's (token, head) in out, -1: none
    AttnPiece* pieces = reinterpret_cast<AttnPiece*>(orow + 16 * MT * kAttnWarps) + 2 * wid;  // computed, issued
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<AttnPiece*>(orow + 16 * MT * kAttnWarps) + 2 * kAttnWarps);  // [NG * S]
    uint64_t* empty = full + kAttnStages;
    int* flag = reinterpret_cast<int*>(empty + kAttnStages);                          // [NG * S]: the stage holds a record
    volatile int* dead = flag + kAttnStages;                                 // a wait gave up
    uint8_t* ring = sm + L::fixed(RTW) + static_cast<int64_t>(grp) * S * L::kRec;
    full += grp * S;
    empty += grp * S;
    flag += grp * S;

    if (rt == 0) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                mbar_init(full + i, 1 + a.test_expire);
                mbar_init(empty + i, RTW);
            }
            if (wid == 0) *dead = 0;
            fence_barrier_init();
        }
        __syncwarp();
    }
    pdl_wait();
    pdl_trigger();  // (the joining kernel waits for this one's end in turn)
    // ---- the list and this CTA's range: each warp sums the sequences for itself, a lane a run of them
    const int B = a.c.n_seqs, span = (B + 31) / 32, b0 = min(B, lane * span), b1 = min(B, b0 + span);
    AttnPiece x;
    int blocks = 0, some = 0, longest = 0;
    x.n = 0;
    for (int b = b0; b < b1; ++b) {
        attn_seq(a, b, x.len, x.first, x.n, blockIdx.x == 0 && wid == 0);
        blocks += x.n;
        some += x.n > 0;
        longest = max(longest, x.n);
    }
    const AttnCut cut = attn_cut(static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(blocks))) * p.segs,
                                 static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(some))) * p.segs,
                                 __reduce_max_sync(0xffffffffu, longest), gridDim.x);
    int mine = 0;
    if (span == 1) {  // the lane's one sequence is in x
        mine = cut.cost(x.n);
    } else {
        for (int b = b0; b < b1; ++b) {
            attn_seq(a, b, x.len, x.first, x.n, false);
            mine += cut.cost(x.n);
        }
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    const int U = __shfl_sync(0xffffffffu, before, 31) * p.segs;
    before -= mine;
    if (blockIdx.x == 0 && wid == 0) {  // the plan that the joining kernel reads
        int sum = before;
        for (int b = b0; b < b1; ++b) {
            int len, first, n;
            attn_seq(a, b, len, first, n, false);
            p.plan[b] = sum;
            sum += cut.cost(n);
        }
        if (lane == 0) {
            p.plan[B] = U / p.segs;
            p.plan[B + 1] = cut.tb ? 0 : cut.chunk;
        }
    }
    const int64_t from = static_cast<int64_t>(blockIdx.x) * cut.chunk;
    if (from >= U) return;
    const int u0 = static_cast<int>(from), u1 = u0 < U - cut.chunk ? u0 + cut.chunk : U;
    {
        const int who = __ffs(__ballot_sync(0xffffffffu, before * p.segs <= u0 && u0 < (before + mine) * p.segs)) - 1;
        int sum = __shfl_sync(0xffffffffu, before, who);
        x.b = who * span;
        if (span == 1) {
            x.len = __shfl_sync(0xffffffffu, x.len, who);
            x.first = __shfl_sync(0xffffffffu, x.first, who);
            x.n = __shfl_sync(0xffffffffu, x.n, who);
        } else {
            for (;; ++x.b) {
                attn_seq(a, x.b, x.len, x.first, x.n, false);
                if (u0 < (sum + cut.cost(x.n)) * p.segs) break;
                sum += cut.cost(x.n);
            }
        }
        const int off = u0 - sum * p.segs, k = cut.cost(x.n), seg = off / k, j = off - seg * k;
        x.seg = seg;
        if (cut.tb) {  // the first n % k parts have a block more
            const int each = x.n / k, more = x.n - each * k;
            x.blk = x.first + j * each + min(j, more);
            x.end = x.blk + each + (j < more);
            x.left = 0;
        } else {
            attn_take(x, j, u1 - u0);
            if (x.blk == x.end) return;  // the range ends within a segment's fixed part
        }
        if (lane == 0) pieces[0] = pieces[1] = x;
        __syncwarp();
    }

    // ---- queries of a piece: kAhead rows of a lane are loaded ahead, the others with the conversion
    constexpr int LPR = D <= 128 ? 16 : 32, RPW = 32 / LPR;  // lanes per row, rows of a warp at once
    constexpr int kStep = kAttnWarps * RPW;                   // rows of the CTA at once
    const int qr = wid * RPW + lane / LPR, pc = lane % LPR;   // the lane's first row; its eight dims: 8 pc ..
    using Q8 = Raw8<SPLIT ? MOE_F32 : MOE_BF16>;
    auto load_q = [&](Q8& v, int b, int seg, int rr) {
        const int kv = seg / p.g.RB, r = (seg - kv * p.g.RB) * RP + rr;
        v.clear();
        if (pc < kND && rr < RP && r < p.R) {
            const int t = r / a.G, h = kv * a.G + r - t * a.G;
            const int64_t at = b * a.qs + t * a.qt + h * a.qh + pc * 8;
            v.load(static_cast<const typename Elem<SPLIT ? MOE_F32 : MOE_BF16>::T*>(a.q) + at, a.qvec);
        }
    };
    constexpr int kAhead = 2;
    Q8 qa8[kAhead];
    auto load_qs = [&](int b, int seg, int r0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_q(qa8[i], b, seg, r0 + i * kStep);
    };
    load_qs(x.b, x.seg, qr);

    // ---- copies: the group's first warp issues its blocks S ahead of the arithmetic
    // (pieces[1].blk: the next block to look up)
    int is = 0, iph = 1, at = 0, ready = 0;  // stage, its phase before; blocks looked up
    const uint8_t* src = nullptr;            // records of up to 32 blocks, one a lane; nullptr: unreadable
    bool more = rt == 0;
    const uint64_t once = l2_evict_first();
    auto look_up = [&]() {
        AttnPiece t = pieces[1];
        while (t.blk + grp >= t.end) {
            more = attn_next(p, t);
            if (!more) return;
        }
        const int u = t.blk + grp + lane * NG;
        src = nullptr;
        if (u < t.end) {
            const int pi = u / a.c.page_blocks, page = gload(a.c.table + t.b * a.c.table_stride + pi);
            if (page >= 0 && page < a.c.n_pages)
                src = a.c.pool + ((static_cast<int64_t>(page) * a.c.n_kv + t.seg / p.g.RB) * a.c.page_blocks + u - pi * a.c.page_blocks) * L::kRec;
        }
        at = 0;
        ready = min(32, (t.end - t.blk - grp + NG - 1) / NG);
        t.blk += 32 * NG;
        __syncwarp();
        if (lane == 0) pieces[1] = t;
        __syncwarp();
    };
    auto issue = [&]() {
        if (at == ready) {
            if (more) look_up();
            if (!more) return;
        }
        if (RTW > 1 && !__all_sync(0xffffffffu, mbar_wait_bounded(empty + is, iph))) {
            if (lane == 0) set_err(a.err, MOE_ERR_TIMEOUT);
            *dead = 1;
            more = false;
            ready = at;
            return;
        }
        if (lane == at) {
            flag[is] = src != nullptr;
            mbar_arrive_expect_tx(full + is, src ? L::kRec : 0);
            // (read once, unless further passes over the rows follow: 94 instead of 98 us over a million tokens)
            if (src && p.g.RB == 1) bulk_g2s_hint(ring + is * L::kRec, src, L::kRec, full + is, once);
            else if (src) bulk_g2s(ring + is * L::kRec, src, L::kRec, full + is);
            else set_err(a.err, MOE_ERR_PAGE);
        }
        ++at;
        if (++is == S) {
            is = 0;
            iph ^= 1;
        }
    };
    for (int i = 0; i < S; ++i) issue();

    int cs = 0, cph = 0;  // the stage to consume and its phase
    bool lost = false;
    for (int piece = 0;; ++piece) {
        // ---- queries: shifted by a power of two into fp16's range, stored as the lanes take them
        {
        const int xb = pieces[0].b, xseg = pieces[0].seg, kv = xseg / p.g.RB, rb = xseg - kv * p.g.RB;
        const int rows = min(RP, p.R - rb * RP);
        for (int r0 = qr; r0 < RP; r0 += kAhead * kStep) {
            Q8 now[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) now[i] = qa8[i];
            if (r0 + kAhead * kStep < RP) load_qs(xb, xseg, r0 + kAhead * kStep);  // (the next rows are on their way)
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const Q8& v = now[i];
                const int rr = r0 + i * kStep;
                if (rr - lane / LPR >= rows) {  // none of the warp's rows has a query
                    if (rr < RP && pc < kND) {
                        const int tile = rr >> 4, row = rr & 15;
                        uint32_t* to = reinterpret_cast<uint32_t*>(qs + ((tile * kNB + (pc >> 2)) * 2) * 32 + (row & 7) * 4 + (pc & 3)) + (row >> 3);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            to[(e >> 1) * 128 + (e & 1) * 2] = 0;
                            if (SPLIT) to[(e >> 1) * 128 + (e & 1) * 2 + MT * RTW * D * 8] = 0;
                        }
                        if (pc == 0) qf[rr] = make_float2(0.0f, 0.0f);
                    }
                    continue;
                }
                float y[8], amax = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = SPLIT || p.out_type == MOE_BF16 ? v.get(e) : v.half(e);
                    const float z = fabsf(y[e]);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(z));
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) {
                    const float z = __shfl_xor_sync(0xffffffffu, amax, o);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(z));
                }
                // amax * 2^k in [2^13, 2^14); a negative scale turns the query's sign
                const bool fine = amax < INFINITY;
                int k = fine && amax > 0.0f ? 13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127) : 0;
                k = min(k, 120);
                const float up = __int_as_float((k + 127) << 23) * (a.scale < 0.0f ? -1.0f : 1.0f);
                float sum = 0.0f;
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y0 = fine ? y[2 * e] * up : 0.0f, y1 = fine ? y[2 * e + 1] * up : 0.0f;
                    hi[e] = pack_h2(y0, y1);
                    const float2 h2 = unpack_h2(hi[e]);
                    sum += h2.x + h2.y;
                    if (SPLIT) {
                        lo[e] = pack_h2(y0 - h2.x, y1 - h2.y);
                        const float2 l2 = unpack_h2(lo[e]);
                        sum += l2.x + l2.y;
                    }
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (rr < RP && pc < kND) {
                    // a lane's operand of a step: (row g, dims 0-1), (row g + 8, 0-1), (g, 2-3), (g + 8, 2-3) of its four
                    const int tile = rr >> 4, row = rr & 15;
                    uint32_t* at = reinterpret_cast<uint32_t*>(qs + ((tile * kNB + (pc >> 2)) * 2) * 32 + (row & 7) * 4 + (pc & 3)) + (row >> 3);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        at[(e >> 1) * 128 + (e & 1) * 2] = hi[e];
                        if (SPLIT) at[(e >> 1) * 128 + (e & 1) * 2 + MT * RTW * D * 8] = lo[e];
                    }
                    if (pc == 0) {
                        qf[rr] = make_float2(fine ? fabsf(a.scale) * kLog2e * __int_as_float((127 - k) << 23) * (SPLIT ? 1.0f : 16777216.0f)
                                                  : __int_as_float(0x7fffffff),
                                             SPLIT ? 0.0f : sum * (-128.0f / 16777216.0f));
                        const int r = rb * RP + rr, t = r / a.G;
                        orow[rr] = r < p.R ? t * a.n_heads + kv * a.G + r - t * a.G : -1;
                    }
                }
            }
        }
        }
        __syncthreads();

        float o[MT][kND][4], m[MT][2], dd[MT][2], fr[MT][2], off[MT][4];
        unsigned long long l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < kND; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.0f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                m[mt][q] = -INFINITY;
                dd[mt][q] = INFINITY;  // n = m - d + 10
                l[mt][q] = 0;
                const float2 f = qf[(rt * MT + mt) * 16 + q * 8 + g];
                fr[mt][q] = f.x;
                off[mt][2 * q] = off[mt][2 * q + 1] = f.y;
            }
        }
        const int xend = pieces[0].end, before_window = pieces[0].len - a.T;
        const int behind = a.window > 0 ? pieces[0].len - 1 - a.window : -1;  // the last query does not see this far back
        for (int u = pieces[0].blk + grp; u < xend; u += NG) {
            // (the lanes stay together; a wait that gives up ends the CTA's arithmetic)
            if (!lost && !__all_sync(0xffffffffu, mbar_try_wait(full + cs, cph)) &&
                (__any_sync(0xffffffffu, *dead) || !__all_sync(0xffffffffu, mbar_wait_retry(full + cs, cph)))) {
                if (lane == 0) set_err(a.err, MOE_ERR_TIMEOUT);
                *dead = 1;
                lost = true;
            }
            if (!lost && flag[cs]) {
                const uint8_t* rec = ring + cs * L::kRec;
                const float2 sc = *reinterpret_cast<const float2*>(rec);
                // v_scale = r * 2^e; a block of zeros (or below fp32's normal range) adds to l alone
                const bool some = sc.y >= 1.17549435e-38f && sc.y < INFINITY;
                const float e = some ? static_cast<float>(static_cast<int>(__float_as_uint(sc.y) >> 23) - 127) : -INFINITY;
                const float r = some ? __uint_as_float((__float_as_uint(sc.y) & 0x007fffffu) | 0x3f800000u) : sc.y < INFINITY ? 0.0f : NAN;
                const uint8_t* kp = rec + kKvHead + g * 32 + c * 8;
                // scores, in units of the row's factor times k_scale: where the codes enter as code * 2^-24, the
                // sum starts at -128 * 2^-24 times the query's sum
                float sa[MT][4][4];
#pragma unroll
                for (int i = 0; i < kNB; ++i) {
                    uint4 qa[MT], qb[MT], la[MT], lb[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint4* f = qs + (((rt * MT + mt) * kNB + i) * 2) * 32 + lane;
                        qa[mt] = f[0];
                        qb[mt] = f[32];
                        if (SPLIT) {
                            la[mt] = f[MT * RTW * D * 2];
                            lb[mt] = f[MT * RTW * D * 2 + 32];
                        }
                    }
                    uint32_t kk[4][4];
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        const uint2 w = *reinterpret_cast<const uint2*>(kp + (jj * kNB + i) * 256);
                        if (SPLIT) {
                            codes_h2(w.x, kk[jj][0], kk[jj][1]);
                            codes_h2(w.y, kk[jj][2], kk[jj][3]);
                        } else {
                            codes_sub(w.x, kk[jj][0], kk[jj][1]);
                            codes_sub(w.y, kk[jj][2], kk[jj][3]);
                        }
                    }
                    // sums of different tokens in turn, so that no product waits for the one before it
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            {
                                if (i == 0) mma_16816(sa[mt][jj], qa[mt], kk[jj][0], kk[jj][1], off[mt]);
                                else mma_16816(sa[mt][jj], qa[mt], kk[jj][0], kk[jj][1]);
                            }
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            mma_16816(sa[mt][jj], qb[mt], kk[jj][2], kk[jj][3]);
                    if (SPLIT) {
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma_16816(sa[mt][jj], la[mt], kk[jj][0], kk[jj][1]);
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma_16816(sa[mt][jj], lb[mt], kk[jj][2], kk[jj][3]);
                    }
                }
                // lane (g, c) holds rows g, g + 8 and tokens 8 c + 2 jj + e; an unseen one becomes -inf. (special: such tokens,
                // or a value scale far above those before it)
                const int t0 = u * kKvBlock;
                bool special = t0 > before_window - kKvBlock || t0 <= behind;  // (the last block ends at up to 2^31)
                if (special) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int row = pieces[0].seg % p.g.RB * RP + (rt * MT + mt) * 16 + q * 8 + g;
                            const int t = row / a.G, ps = row < p.R ? before_window + t : -1, j0 = t0 + 8 * c;
                            int from = a.window > 0 ? max(ps - a.window, -1) : -1;  // positions up to it are out of sight
                            uint32_t see;                                            // bit i: the query sees position j0 + i
                            if (a.tree && ps >= 0) {
                                const int64_t bt = static_cast<int64_t>(pieces[0].b) * a.T;
                                uint32_t bits = static_cast<uint32_t>(gload(a.tree + bt + t)) & (0xffffffffu >> (32 - a.T));
                                if (a.depth) {
                                    const int d = attn_depth(a, bt, t);
                                    from = max(before_window + d - a.window, -1);
#pragma unroll 1
                                    for (int w = 0; w < a.T; ++w)
                                        if (d - attn_depth(a, bt, w) >= a.window) bits &= ~(1u << w);
                                }
                                const int w = j0 - before_window;  // what lies before the window is seen
                                see = w >= 0 ? (w < 32 ? bits >> w : 0) : w > -8 ? (bits << -w) | ((1u << -w) - 1) : 0xffu;
                            } else {
                                see = ps >= j0 ? 0xffu >> max(7 - (ps - j0), 0) : 0;
                            }
                            see &= 0xffu << min(max(from + 1 - j0, 0), 8);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (!(see >> i & 1)) sa[mt][i >> 1][2 * q + (i & 1)] = -INFINITY;
                        }
                }
                // ---- running reference; o and l are rescaled only where one of the warp's rows outgrew it
                float f[MT][2], top[MT][2];
                bool grew = false;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float bm = fmaxf(sa[mt][0][2 * q], sa[mt][0][2 * q + 1]);
#pragma unroll
                        for (int jj = 1; jj < 4; ++jj) bm = fmaxf(bm, fmaxf(sa[mt][jj][2 * q], sa[mt][jj][2 * q + 1]));
                        f[mt][q] = fr[mt][q] * sc.x;
                        top[mt][q] = bm * f[mt][q];
                        const float room = fminf(kAttnSlack, kAttnSlack + kAttnShift - (e + dd[mt][q]));
                        grew |= top[mt][q] - m[mt][q] > room || room < kAttnSlack + kAttnShift - kAttnFar;
                    }
                if (__any_sync(0xffffffffu, grew)) {
                    bool far = false;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float bm = fmaxf(top[mt][q], __shfl_xor_sync(0xffffffffu, top[mt][q], 1));
                            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
                            bm = ceilf(bm);
                            const float m0 = m[mt][q], n0 = m0 - dd[mt][q] + kAttnShift, m1 = fmaxf(m0, bm), n1 = fmaxf(n0, bm + e);
                            const float al = m1 > m0 ? ex2(m0 - m1) : 1.0f, ol = n1 > n0 ? ex2(n0 - n1) : 1.0f;
                            m[mt][q] = m1;
                            if (n1 > -INFINITY) dd[mt][q] = m1 - n1 + kAttnShift;
                            l[mt][q] = mul2(l[mt][q], pk2(al, al));
#pragma unroll
                            for (int i = 0; i < kND; ++i) {
                                o[mt][i][2 * q] *= ol;
                                o[mt][i][2 * q + 1] *= ol;
                            }
                            far |= e + dd[mt][q] > kAttnFar;
                        }
                    special |= static_cast<bool>(__any_sync(0xffffffffu, far));
                }
                // ---- weights: the lane's tokens 8 c + 4 xx + 0..3 feed product step xx
                uint4 pa[MT][2], pl[MT][2];
                auto weights = [&](auto special) {  // masked tokens, or a block's scale far above the others'
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            // p is held times 2^lift
                            const float lift = decltype(special)::value ? fmaxf(e + dd[mt][q] - kAttnFar, 0.0f) : 0.0f;
                            const float fac = some ? r * ex2(decltype(special)::value ? fminf(e + dd[mt][q], kAttnFar) : e + dd[mt][q]) : r;
                            const float bias = decltype(special)::value ? lift - m[mt][q] : -m[mt][q], drop = ex2(-lift);
                            const unsigned long long ff = pk2(f[mt][q], f[mt][q]), bb = pk2(bias, bias);
#pragma unroll
                            for (int jj = 0; jj < 4; ++jj) {
                                const float s0 = sa[mt][jj][2 * q], s1 = sa[mt][jj][2 * q + 1];
                                float2 w = up2(fma2(pk2(s0, s1), ff, bb));
                                w.x = ex2(w.x);
                                w.y = ex2(w.y);
                                if (decltype(special)::value) {  // an unseen token adds nothing, whatever the scales are
                                    if (s0 == -INFINITY) w.x = 0.0f;
                                    if (s1 == -INFINITY) w.y = 0.0f;
                                    l[mt][q] = fma2(pk2(w.x, w.y), pk2(drop, drop), l[mt][q]);
                                } else {
                                    l[mt][q] = add2(l[mt][q], pk2(w.x, w.y));
                                }
                                w = up2(mul2(pk2(w.x, w.y), pk2(fac, fac)));
                                if (decltype(special)::value) {
                                    if (s0 == -INFINITY) w.x = 0.0f;
                                    if (s1 == -INFINITY) w.y = 0.0f;
                                }
                                const uint32_t h = pack_h2(w.x, w.y);
                                word(pa[mt][jj >> 1], (jj & 1) * 2 + q) = h;
                                if (W2) {
                                    const float2 h2 = unpack_h2(h);
                                    word(pl[mt][jj >> 1], (jj & 1) * 2 + q) = pack_h2(w.x - h2.x, w.y - h2.y);
                                }
                            }
                        }
                };
                if (special) weights(std::true_type{});
                else weights(std::false_type{});
                const uint8_t* vp = rec + kKvHead + kKvBlock * D + g * 32 + c * 8;
                constexpr int kRun = 4;  // dims' sums in turn, as above (kND is a multiple of 4)
#pragma unroll
                for (int i0 = 0; i0 < kND; i0 += kRun) {
                    uint32_t v[kRun][4];
#pragma unroll
                    for (int i = 0; i < kRun; ++i) {
                        const uint2 w = *reinterpret_cast<const uint2*>(vp + (i0 + i) * 256);
                        codes_h2(w.x, v[i][0], v[i][1]);
                        codes_h2(w.y, v[i][2], v[i][3]);
                    }
#pragma unroll
                    for (int xx = 0; xx < 2; ++xx)
#pragma unroll
                        for (int i = 0; i < kRun; ++i)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma_16816(o[mt][i0 + i], pa[mt][xx], v[i][2 * xx], v[i][2 * xx + 1]);
                    if (W2) {
#pragma unroll
                        for (int xx = 0; xx < 2; ++xx)
#pragma unroll
                            for (int i = 0; i < kRun; ++i)
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
                                    mma_16816(o[mt][i0 + i], pl[mt][xx], v[i][2 * xx], v[i][2 * xx + 1]);
                    }
                }
            }
            __syncwarp();  // the stage has been read
            if (RTW > 1 && lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(empty + cs)) : "memory");
            if (++cs == S) {
                cs = 0;
                cph ^= 1;
            }
            if (!lost) issue();
        }

        // ---- join the groups, in order, and write the piece's rows: to out, or as a part
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float2 l2 = up2(l[mt][q]);
                float ls = l2.x + l2.y;
                ls += __shfl_xor_sync(0xffffffffu, ls, 1);
                ls += __shfl_xor_sync(0xffffffffu, ls, 2);
                if (c == 0) stat[wid * 16 * MT + mt * 16 + q * 8 + g] = make_float2(m[mt][q], ls);
            }
        __syncthreads();
        float cf[MT][2], M[MT][2], Ls[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int at = mt * 16 + q * 8 + g;
                float mm = -INFINITY, ll = 0.0f;
                for (int k = 0; k < NG; ++k) mm = fmaxf(mm, stat[(k * RTW + rt) * 16 * MT + at].x);
                const float bs = mm == -INFINITY ? 0.0f : mm;
                for (int k = 0; k < NG; ++k) {
                    const float2 v = stat[(k * RTW + rt) * 16 * MT + at];
                    ll += v.y * ex2(v.x - bs);
                }
                M[mt][q] = mm;
                Ls[mt][q] = ll;
                cf[mt][q] = ll == 0.0f ? 0.0f : ex2(m[mt][q] - bs - dd[mt][q]) / ll;
            }
        const AttnPiece* xp = pieces;  // (read again: nothing of it is held during the loop)
        const int rows = min(RP, p.R - xp->seg % p.g.RB * RP);
        const bool whole = xp->blk == xp->first && xp->end == xp->first + xp->n;
        float* part = p.parts + (2LL * blockIdx.x + (piece ? 1 : 0)) * attn_part_floats(RP, D);
        const int64_t orow0 = static_cast<int64_t>(xp->b) * a.T * a.n_heads;
        // the next piece's first queries are on their way during the joining
        AttnPiece nx = pieces[0];
        const bool again = attn_next(p, nx);
        __syncwarp();
        if (lane == 0) pieces[0] = nx;
        __syncwarp();
        if (again) load_qs(nx.b, nx.seg, qr);
        if (grp == 0 && c == 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int rr = (rt * MT + mt) * 16 + q * 8 + g;
                    if (rr >= rows) continue;
                    if (!whole) {
                        part[static_cast<int64_t>(RP) * D + rr] = M[mt][q];
                        part[static_cast<int64_t>(RP) * D + RP + rr] = Ls[mt][q];
                    } else if (a.lse) {
                        a.lse[orow0 + orow[rr]] = Ls[mt][q] == 0.0f ? -INFINITY : M[mt][q] * kLn2 + logf(Ls[mt][q]);
                    }
                }
        }
        auto put = [&](int rr, int d, float4 v) {  // four neighbouring dims of a row
            if (!whole) {
                *reinterpret_cast<float4*>(part + static_cast<int64_t>(rr) * D + d) = v;
                return;
            }
            const int64_t at = (orow0 + orow[rr]) * D + d;
            if (SPLIT) {
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
            } else if (p.out_type == MOE_F16) {
                *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = make_uint2(pack_h2(v.x, v.y), pack_h2(v.z, v.w));
            } else {
                const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x, v.y), y1 = __floats2bfloat162_rn(v.z, v.w);
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
            }
        };
        {
            // after the CTA's last piece the ring is free: a buffer each, and one barrier instead of one a group
            // (of four; a million tokens 91.1 -> 90.2 us; two groups of wide heads 25.5 -> 26.2)
            float* others = reinterpret_cast<float*>(sm + L::fixed(RTW));
            const int each = RP * L::kRowO;
            const bool apart = !again && NG > 2 && (NG - 1) * each * 4 <= NG * S * L::kRec;
            float* to = apart && grp ? others + (grp - 1) * each : buf;
            for (int k = 0; k < NG; ++k) {
                if (apart || grp == k) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int r8 = (rt * MT + mt) * 16 + q * 8;
                            if (r8 >= rows) continue;
#pragma unroll
                            for (int i = 0; i < kND; ++i) {
                                float2* d = reinterpret_cast<float2*>(to + (r8 + g) * L::kRowO + i * 8 + 2 * c);
                                float2 v = make_float2(o[mt][i][2 * q] * cf[mt][q], o[mt][i][2 * q + 1] * cf[mt][q]);
                                if (k) {  // (not where they are apart)
                                    const float2 w = *d;
                                    v.x += w.x;
                                    v.y += w.y;
                                }
                                *d = v;
                            }
                        }
                }
                __syncthreads();
                if (apart) break;
            }
            for (int i = threadIdx.x; i < rows * (D / 4); i += kAttnThreads) {
                const int rr = i / (D / 4), d = (i - rr * (D / 4)) * 4;
                float4 v = *reinterpret_cast<const float4*>(buf + rr * L::kRowO + d);
                if (apart)
                    for (int k = 1; k < NG; ++k) {
                        const float4 w = *reinterpret_cast<const float4*>(others + (k - 1) * each + rr * L::kRowO + d);
                        v.x += w.x;
                        v.y += w.y;
                        v.z += w.z;
                        v.w += w.w;
                    }
                put(rr, d, v);
            }
            __syncthreads();
        }
        if (!again) break;
    }
    if (*dead && rt == 0)  // leave no copy of this CTA's in flight: a stage's last one is of this round or the one before
        for (int k = 0; k < S; ++k) mbar_wait_bounded(full + k, k < is ? iph ^ 1 : iph);
}

template <int D, int MT, int PREC>
cudaError_t launch_attn(AttnPlan p, cudaStream_t st) {
    using L = AttnSmem<D, MT, PREC>;
    auto kern = kv8_attention_kernel<D, MT, PREC>;
    constexpr int kMaxDev = 64;
    static std::atomic<int> sms[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    constexpr int kSmMax = 227 * 1024;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmMax);
        // (as the joining kernel: an SM that has to change its split waits until it is empty)
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    // CTAs per SM that the registers allow, fewer where the row buffer leaves no room for the ring
    int occ = MT == 1 && D <= 128 && PREC == kAttnPlain ? 3 : 2;
    const int NG = kAttnWarps / p.g.RTW, fixed = L::fixed(p.g.RTW);
    int stages = 0;
    for (;; --occ) {
        stages = ((228 * 1024) / occ - 1024 - fixed) / L::kRec / NG;
        if (stages >= 2 || occ == 1) break;
    }
    if (stages < 1) return cudaErrorInvalidConfiguration;
    if (stages * NG > kAttnStages) stages = kAttnStages / NG;
    p.stages = stages;
    p.smem = fixed + stages * NG * L::kRec;
    int grid = n * occ;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    e = launch_kernel(kern, dim3(grid), dim3(kAttnThreads), p.smem, st, true, p);
    return e;
}

#endif  // __CUDACC__

}  // namespace moe
