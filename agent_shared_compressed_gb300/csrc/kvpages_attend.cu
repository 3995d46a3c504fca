// kvpages_attend.cu -- attention of each sequence's newest tokens over its
// pages, joined with attention over other tokens (the shared pool's).
//
// For sequence b, query token i, query head j (KV head h = j / (nq / H)):
//   s_t = scale q . k_t,  t < len_b - (m - 1 - i)
//   out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
// joined: L = log(e^lse + e^base_lse), out = e^(lse-L) out + e^(base_lse-L) base.
// Exponentials are base 2 throughout.
//
// Bound: every cached byte is read once (4 query rows per KV head, say, do 16
// multiply-adds per byte of 8-bit cache: far below what the tensor cores can
// take), so the work is keeping enough bytes in flight on every SM and spending
// few instructions on each.
//
// Work split.  The unit is one or two 16-token blocks (8- and 4-bit pages: two)
// of one (sequence, KV head, tile of query rows).  All units of all sequences, in
// that order, are one list, cut into equal runs, one per warp: no warp has more to
// do than another, however ragged the lengths, and the cut follows from the
// lengths on the device, so a captured graph stays right as sequences grow.  A row
// tile counts PAT_ITEM blocks more than it has, for its start and end.  A warp that
// holds all of a row tile writes its result; otherwise it leaves a partial result
// (running maximum, sum and weighted values) and pages_join merges them in list
// order, so results do not depend on timing.  Where the tables are short, a team of
// a thread block's warps takes each row tile instead and merges it in shared
// memory, in one launch (team_blocks says when).
//
// A warp's units arrive by bulk copies, one per unit (the blocks of a head's tokens
// in a page are one run of bytes), in the warp's own ring in shared memory, on the
// warp's own barriers: warps do not wait for each other between start and merge.
//
// Products, with tokens or dims as the 16 rows and the query rows as the 8
// columns, so that a tile of up to 8 query rows wastes nothing:
//   S^T = K Q^T    C: tokens g, g + 8 x queries 2 tig, 2 tig + 1
//   O^T = V^T P^T  C: dims x queries 2 tig, 2 tig + 1
// P^T comes from S^T's fragment by two 8 x 8 transposes.  The codes are in
// fragment order already (kvp_pages.cuh): a lane takes 16 bytes of a key row or
// of a value token and expands them in registers, keys to fp16 and values to
// bf16, exactly (|code| <= 128).  What bounds 8- and 4-bit pages beside memory is
// that expansion, most of it on the integer pipe, which takes a warp's
// instruction every other cycle: two to four instructions per pair of codes.
//
// Key scales apply to the fp32 sums of their 32 dims.  Value scales go into the
// weights, one product operand per 32 dims, as a sum of two bf16: 2^-17 of the
// weight, and fp32's range, so that a token of large weight and tiny values (an
// attention sink) takes nothing from the others.  (One fp16 per weight is fewer
// instructions, but loses weights 2^-25 below the largest where that one's value is
// zero.)  4-bit values q s + z enter as (q - c) s + (z + c s) with c the integer of
// [0, 15] nearest to -z / s, formed once per token and group: then |z + c s| is at
// most s / 2 (or of the code term's sign, where zero is outside the group's range),
// and the two sums, of the code terms in the product and of the rest in fp32 once
// per 32 dims, do not cancel.  16-bit pages are multiplied as they are.
//
// Measured (of the 6789 GB/s that a copy reaches): four 32K caches of 8 bits, 4
// query rows a KV head, 56.7 us, 5.0 TB/s; 15 4K caches of 16 bits 45.4 us, 5.5 TB/s;
// one 128K with 4-bit values 50.7 us, 4.5 TB/s.
#include <algorithm>
#include <cmath>

#include "kvp_async.cuh"
#include "kvp_pages.cuh"

namespace kvp {

constexpr int PAT_MOST_WARPS = 16;             // of a block
// Blocks that a row tile counts beside its own (us with 2, 4, 8 of them: 64 ragged
// sequences of one row a head 56.8, 54.4, 57.8; 40 ragged ones of 64 rows, 8 bits,
// 166, 157, 161; four 32K caches 56.5, 55.5, 56.4).
constexpr uint32_t PAT_ITEM = 4;
constexpr uint32_t PAT_WAIT_LIMIT = 1u << 22;  // polls, about half a second
constexpr uint32_t PAT_BAR_BYTES = 1024;       // barriers, before the rings
constexpr int PAT_OWN_PLAN = 128;              // sequences that pages_join sums by itself
// The weights' reference is raised only when a score passes it by this much
// (base 2), so that the accumulators are rarely rescaled.
constexpr float PAT_SLACK = 8.0f;

struct PagesAttendArgs {
    PagesView pv;
    const uint16_t *q;
    const int32_t *table, *lens;
    const float *base_out, *base_lse;
    uint16_t *out;
    float *lse;
    float *part;     // [warps][2][rows][D] partial sums
    float2 *stats;   // [warps][2][rows] (reference, sum), base 2
    uint32_t *plan;  // [nseq + 1] units before each sequence, per row tile
    float scale2;    // scale * log2(e)
    int nseq, m, nq, G, R, RT, max_pages;
    int unit;  // tokens of a unit
    uint32_t nwarps;
    uint32_t polls, poll_lanes;  // polls of a copy by these lanes of a warp (the others': PAT_WAIT_LIMIT)
    int team;       // warps of a row tile where it is not cut from the list
    int join_rows;  // rows of a block of pages_join
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}
template <int N>
__device__ __forceinline__ void lds_floats(uint32_t at, float (&f)[N]) {
    if constexpr (N == 4) {
        const uint4 v = lds128(at);
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    } else {
        const uint2 v = lds64(at);
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    }
}
__device__ __forceinline__ float2 half2_f32(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
// N fp16 values as fp32.
template <int N>
__device__ __forceinline__ void lds_halfs(uint32_t at, float (&f)[N]) {
    uint32_t w[2] = {0u, 0u};
    if constexpr (N == 4) {
        const uint2 v = lds64(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = lds32(at);
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 v = half2_f32(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ void sts32(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t at, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}
__device__ __forceinline__ void sts128_zero(uint32_t at) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0u) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two bytes u as fp16 u - 128: 1024 + u by byte placement, less 1152 (exact).
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t sel) {
    const uint32_t x = __byte_perm(w, 0x64646464u, sel), bias = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// The bytes u of each 16-bit half (whatever their upper bytes hold) as bf16
// u - 128: 128 + (u mod 128), less 256 or, with u's top bit, 128 (exact).
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
    const uint32_t x = (w & 0x007F007Fu) | 0x43004300u, y = (w & 0x00800080u) ^ 0xC380C380u;
    const __nv_bfloat162 r =
        __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&x), *reinterpret_cast<const __nv_bfloat162 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// The low nibble q of each 16-bit half as bf16 q - c: 128 + q, plus the halves of
// y, -(128 + c) (exact).
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t w, uint32_t y) {
    const uint32_t x = (w & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 r =
        __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&x), *reinterpret_cast<const __nv_bfloat162 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// The transpose of an 8 x 8 matrix of 16-bit values, in fragment layout.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // results under 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The weights (w0, w1) of a token and two queries as value-product operands: a
// sum of two bf16, one operand each.
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t &hi, uint32_t &lo) {
    const uint32_t h = pack_bf16x2(w0, w1);
    const float2 d =
        __ffma2_rn(make_float2(bf16_lo(h), bf16_hi(h)), make_float2(-1.0f, -1.0f), make_float2(w0, w1));
    hi = transpose8(h), lo = transpose8(pack_bf16x2(d.x, d.y));
}
// The weights of two tokens and one query: the two bf16 of each in one operand's
// neighbouring columns.
__device__ __forceinline__ void twin_weights(float w0, float w1, uint32_t &b0, uint32_t &b1) {
    const uint32_t h = pack_bf16x2(w0, w1);
    b0 = transpose8(pack_bf16x2(w0, w0 - bf16_lo(h)));
    b1 = transpose8(pack_bf16x2(w1, w1 - bf16_hi(h)));
}
// The factor of a weighted sum x when it is scaled by f > 0: f, but 1 where f has
// underflowed to 0 and x is Inf or NaN (16-bit values may be), which it has to stay.
__device__ __forceinline__ float factor(float f, float x) { return f == 0.0f && !(fabsf(x) < INFINITY) ? 1.0f : f; }
// sq + w^2 and w f of a pair of bf16, and whether one of a pair is Inf or NaN.
__device__ __forceinline__ __nv_bfloat162 square_sum(uint32_t w, __nv_bfloat162 sq) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&w);
    return __hfma2(v, v, sq);
}
__device__ __forceinline__ uint32_t times(uint32_t w, __nv_bfloat162 f) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), f);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }
__device__ __forceinline__ bool not_finite(__nv_bfloat162 v) {
    const __nv_bfloat162 z = __hmul2(v, __float2bfloat162_rn(0.0f));  // 0 or -0, else NaN
    return (*reinterpret_cast<const uint32_t *>(&z) & 0x7FFF7FFFu) != 0u;
}
// Over the eight lanes of a quad position (the rows of a C fragment).
__device__ __forceinline__ float rows_add(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ float rows_top(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// The length that a sequence's table row can hold.  EARLY: read before the kernel's
// own wait (the kernel before it has passed its own).
template <bool EARLY = false>
__device__ __forceinline__ int seq_len(const PagesAttendArgs &a, int b, bool flag) {
    const int len = max(int(EARLY ? ld_l2_u32(a.lens + b) : ld_plain_u32(a.lens + b)), 0);
    const int64_t cap = int64_t(a.max_pages) << a.pv.logP;
    if (int64_t(len) <= cap) return len;
    if (flag) pages_flag(a.pv, FLAG_PAGE);
    return int(cap);
}

// Units of a sequence's row tile (both kernels).
__device__ __forceinline__ uint32_t tile_units(int len, int unit) {
    return len ? uint32_t((int64_t(len) + unit - 1 + int64_t(PAT_ITEM) * PAGES_BLOCK) / unit) : 0u;
}
// Units of a warp's run (both kernels).
__device__ __forceinline__ uint64_t run_length(uint64_t units, uint32_t nwarps) {
    return units ? (units + nwarps - 1) / nwarps : 1u;
}

// The shape of a block.  8- and 4-bit pages at head_dim 128: 12 warps (168
// registers) with units of two blocks measured 55.7 us on four 32K caches of 8 bits
// and 50.4 on one of 128K with 4-bit values; 16 warps, at 128 registers and with
// units of one block, 56.5 and 55.5; 14 warps, which spill, 63.9 on the latter.
// 16-row tiles take 250 registers, hence 8 warps, as do 16-bit pages, whose blocks
// are 8 KB each.  At head_dim 64 16 warps (20: 53.9 against 54.4 us on 64 ragged
// sequences, for a quarter more partial results), 12 for 16-row tiles (35.8 against
// 37.0 us with 16, which spill, on 30 4K caches with 16 rows).
template <int D, int FMT, int RC>
struct PatShape {
    static constexpr int WARPS = D == 128 ? (FMT == KVP_PAGES_BF16 || RC == 16 ? 8 : 12) : (RC == 16 ? 12 : 16);
    static constexpr int UB = FMT != KVP_PAGES_BF16 && RC <= 8 ? 2 : 1;  // blocks of a unit
    static constexpr uint32_t ITEM = PAT_ITEM / UB;  // units that a row tile counts beside its own
    static constexpr uint32_t SLOT = (UB * Block<D, FMT>::BYTES + 127u) / 128u * 128u;
    static constexpr uint32_t RING = 180224u / WARPS / SLOT;  // of about 176 KB
    static constexpr uint32_t LEAST = UB == 2 ? 2u : 3u;
    static constexpr uint32_t STAGES = RING < LEAST ? LEAST : (RING > 8u ? 8u : RING);
    // 4-bit values: a warp's scales, remainders (fp32 [16][NG]) and -(128 + c) (bf16 pairs)
    static constexpr uint32_t NE = 16u * Block<D, FMT>::NG;
    static constexpr uint32_t PREP = Block<D, FMT>::V4 ? NE * 10u * UB : 0u;
    static constexpr uint32_t OFF_PREP = PAT_BAR_BYTES + WARPS * STAGES * SLOT;
    static constexpr uint32_t OFF_PLAN = OFF_PREP + WARPS * PREP;
    static_assert(WARPS * STAGES * 8 <= PAT_BAR_BYTES, "a barrier per slot");
    // with the static part, within the 227 KB of a block
    static_assert(OFF_PLAN + 4u * (KVP_PAGES_MAX_SEQS + 1u) + 1024u <= 232448u, "shared memory of a block");
    static uint32_t bytes(int nseq) { return OFF_PLAN + 4u * uint32_t(nseq + 1); }
};

// Units before each sequence (of one row tile), in shared memory and, for pages_join,
// in the plan; returns their sum.  Up to 32 sequences, every warp finds them by itself
// (all write the same values).
__device__ __forceinline__ uint32_t make_plan(const PagesAttendArgs &a, uint32_t *pre, uint32_t *wsum, int unit, int threads) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = threads / 32;
    uint32_t carry = 0;
    if (a.nseq <= 32) {
        uint32_t n = lane < a.nseq ? tile_units(seq_len(a, lane, blockIdx.x == 0 && warp == 0), unit) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += y;
        }
        carry = __shfl_sync(0xffffffffu, n, 31);
        if (lane < a.nseq) {
            pre[lane + 1] = n;
            if (blockIdx.x == 0 && warp == 0) a.plan[lane + 1] = n;
        }
        if (lane == 0) {
            pre[0] = 0u;
            if (blockIdx.x == 0 && warp == 0) a.plan[0] = 0u;
        }
        __syncwarp();
    }
    for (int b0 = 0; a.nseq > 32 && b0 < a.nseq; b0 += threads) {
        const int b = b0 + tid;
        uint32_t n = b < a.nseq ? tile_units(seq_len(a, b, blockIdx.x == 0), unit) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += y;
        }
        if (lane == 31) wsum[warp] = n;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < warps; ++w) {
            const uint32_t s = wsum[w];
            before += w < warp ? s : 0u;
            carry += s;
        }
        if (b < a.nseq) {
            pre[b + 1] = before + n;
            if (blockIdx.x == 0) a.plan[b + 1] = before + n;
        }
        __syncthreads();
    }
    if (a.nseq > 32) {
        if (tid == 0) {
            pre[0] = 0u;
            if (blockIdx.x == 0) a.plan[0] = 0u;
        }
        __syncthreads();
    }
    return carry;
}

// What one row of a tile ends with: the base joined in and lse written (by `first`).
// `bl` is base_lse[row], which may be lse[row]: whoever calls this has read it before
// any thread gets here.
__device__ __forceinline__ float2 join_base(const PagesAttendArgs &a, uint64_t row, float lse, float bl, bool first) {
    // weights of (this, base); an empty row without a base has none
    float wa = 1.0f, wb = 0.0f;
    if (a.base_lse) {
        if (!(lse == -INFINITY && bl == -INFINITY)) {
            const float top = fmaxf(lse, bl);  // of a NaN and a number: the number
            const float ea = expf(lse - top), eb = expf(bl - top), tot = ea + eb;
            wa = ea / tot, wb = eb / tot;
            lse = top + logf(tot);
        }
    }
    if (first && a.lse) a.lse[row] = lse;
    return make_float2(wa, wb);
}

// RC: query rows of a tile (4, 8 or 16).  A tile of 4 has row i in the columns 2 i
// and 2 i + 1: the weights' first bf16 in the former, the second in the latter, so
// that one value product does for both, and a lane has the scores of one row.
//
// SOLO: a group of a.team warps takes one row tile, each an equal part of the
// tile's units, merged in shared memory: no list, no partial results, no join.
template <int D, int FMT, int RC, bool SOLO>
__global__ void __launch_bounds__(PatShape<D, FMT, RC>::WARPS * 32, 1)
    pages_attend(const __grid_constant__ PagesAttendArgs a) {
    using B = Block<D, FMT>;
    using SM = PatShape<D, FMT, RC>;
    constexpr int R8 = RC == 16 ? 2 : 1;  // groups of 8 columns
    constexpr bool TWICE = RC == 4;
    constexpr int CQ = TWICE ? 1 : 2;  // queries of a lane and group
    constexpr int NG = B::NG, MT = D / 16, RTILE = RC, WARPS = SM::WARPS, THREADS = WARPS * 32;
    constexpr int UB = SM::UB, GU = 32 / UB;  // units whose addresses the lanes hold
    constexpr uint32_t STAGES = SM::STAGES;
    constexpr bool Q8 = B::Q8, V4 = B::V4;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint32_t *pre = reinterpret_cast<uint32_t *>(sm + SM::OFF_PLAN);
    __shared__ uint32_t wsum[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const uint32_t bar = smem_addr(sm) + uint32_t(warp) * STAGES * 8u;
    const uint32_t ring = smem_addr(sm) + PAT_BAR_BYTES + uint32_t(warp) * STAGES * SM::SLOT;
    if (lane == 0) {
        for (uint32_t s = 0; s < STAGES; ++s) mbar_init1(bar + 8u * s);
        mbar_init_fence();
    }
    // the kernel before this one has completed past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool match = pages_match(a.pv);
    const uint32_t HRT = uint32_t(a.pv.H) * uint32_t(a.RT);
    // SOLO: the warp's place in its team, the team's sequence and row tile (the
    // tiles go round the blocks, so that all have as many), and the tile's units
    const int team = SOLO ? a.team : 1, place_in = warp % team;
    const uint32_t stask = SOLO ? uint32_t(warp / team) * gridDim.x + blockIdx.x : 0u;
    const bool sreal = stask < uint32_t(a.nseq) * HRT;
    const int sb = SOLO && sreal ? int(stask / HRT) : 0;
    const uint32_t stile = SOLO && sreal ? stask % HRT : 0u;
    uint32_t solo_units = 0, carry = 0;
    if constexpr (SOLO) {
        const uint32_t n = sreal ? tile_units(seq_len(a, sb, stile == 0), 16 * UB) : 0u;
        solo_units = n ? n - SM::ITEM : 0u;
    } else {
        carry = make_plan(a, pre, wsum, 16 * UB, THREADS);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!match) {
        if (tid == 0) pages_flag(a.pv, FLAG_HEADER);
        return;
    }
    const uint64_t units = SOLO ? solo_units : uint64_t(carry) * HRT;
    const uint64_t per = run_length(units, SOLO ? uint32_t(team) : a.nwarps);
    const uint32_t gw = blockIdx.x * WARPS + uint32_t(warp);
    const uint64_t f0 = (SOLO ? uint32_t(place_in) : gw) * per;
    const uint32_t cnt = f0 >= units ? 0u : uint32_t(f0 + per < units ? per : units - f0);
    if (cnt == 0u && !SOLO) return;

    // unit f: its sequence, row tile and place in the tile (ITEM empty places, then the blocks)
    auto locate = [&](uint64_t f, int &b, uint32_t &tile, uint32_t &at) {
        if constexpr (SOLO) {
            b = sb, tile = stile, at = uint32_t(f) + SM::ITEM;
            return;
        }
        const uint32_t p = (f >> 32) == 0 ? uint32_t(f) / HRT : uint32_t(f / HRT);
        int lo = 0, hi = a.nseq - 1;  // the last b with pre[b] <= p
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= p)
                lo = mid;
            else
                hi = mid - 1;
        }
        const uint32_t n = pre[lo + 1] - pre[lo];
        const uint64_t r = f - uint64_t(pre[lo]) * HRT;
        b = lo;
        if ((r >> 32) == 0) {
            tile = uint32_t(r) / n;
            at = uint32_t(r) - tile * n;
        } else {
            tile = uint32_t(r / n);
            at = uint32_t(r - uint64_t(tile) * n);
        }
    };
    // the lane's block of the GU units that start at `first` of the run: its address, or
    // 0 past the run or the sequence, in a tile's empty places and for a bad page id
    auto address = [&](uint32_t first, int &b, uint32_t &tile, uint32_t &at) -> uint64_t {
        const uint32_t u = first + uint32_t(lane / UB);
        if (u >= cnt) return 0;
        locate(f0 + u, b, tile, at);
        if (at < SM::ITEM) return 0;
        const uint32_t t0 = ((at - SM::ITEM) * UB + uint32_t(lane % UB)) * PAGES_BLOCK;
        if (UB > 1 && t0 >= uint32_t(seq_len(a, b, false))) return 0;
        const int page = int(ld_plain_u32(a.table + uint64_t(b) * uint32_t(a.max_pages) + (t0 >> a.pv.logP)));
        if (page < 0 || page >= a.pv.n_pages) {
            pages_flag(a.pv, FLAG_PAGE);
            return 0;
        }
        return reinterpret_cast<uint64_t>(a.pv.layer) + uint64_t(page) * a.pv.page_bytes +
               uint64_t(tile / uint32_t(a.RT)) * a.pv.tile_bytes +
               uint64_t((t0 & uint32_t(a.pv.P - 1)) / PAGES_BLOCK) * B::BYTES;
    };
    // the copies of unit n into slot s, by the lanes that hold its blocks (nothing to
    // copy: the phase still completes); two blocks of one page are one run of bytes
    auto issue = [&](uint32_t n, uint64_t src, uint32_t good, uint32_t s) {
        if (lane / UB != int(n % GU)) return;
        const uint32_t to = ring + s * SM::SLOT, at = bar + 8u * s;
        const uint32_t mine = (good >> (lane / UB * UB)) & (UB == 2 ? 3u : 1u);
        const bool lead = lane % UB == 0;
        if (lead) mbar_expect_tx(at, (UB == 2 ? uint32_t(__popc(mine)) : mine) * B::BYTES);
        fence_proxy_async();  // the warp's reads of the slot come first
        if (UB == 2 && mine == 3u && a.pv.P > PAGES_BLOCK) {
            if (lead) bulk_g2s(to, reinterpret_cast<const void *>(src), 2u * B::BYTES, at);
        } else if (src) {
            bulk_g2s(to + uint32_t(lane % UB) * B::BYTES, reinterpret_cast<const void *>(src), B::BYTES, at);
        }
    };

    int b = 0, len = 0;
    uint32_t tile = 0, place = 0, nplace = 0, seg0 = 0;
    uint64_t cur = address(0, b, tile, place), nxt = 0;
    uint32_t good = __ballot_sync(0xffffffffu, cur != 0), good_nxt = 0;
#pragma unroll
    for (uint32_t s = 0; s < STAGES; ++s)
        if (s < cnt) issue(s, cur, good, s);
    b = __shfl_sync(0xffffffffu, b, 0), tile = __shfl_sync(0xffffffffu, tile, 0), place = __shfl_sync(0xffffffffu, place, 0);
    if (cnt > uint32_t(GU)) {
        int lb;
        uint32_t lt, lp;
        nxt = address(GU, lb, lt, lp);
        good_nxt = __ballot_sync(0xffffffffu, nxt != 0);
    }
    bool fresh = true;             // the next unit starts a segment
    uint32_t slot = 0, phase = 0;  // ring position of the next unit

    // where the lane's bytes are in a slot
    const uint32_t k_off = Q8 ? B::key(uint32_t(g), uint32_t(tig) * (D / 4))
                              : B::key(uint32_t(lane & 15), uint32_t(lane >> 4) * 16u);
    const uint32_t v_off = Q8 ? B::value(uint32_t(2 * tig), uint32_t(g) * (B::VROW / 8))
                              : B::value(uint32_t((lane & 7) + ((lane >> 4) << 3)), uint32_t((lane >> 3) & 1) * 16u);
    const uint32_t v_odd = Q8 ? B::value(uint32_t(2 * tig + 1), uint32_t(g) * (B::VROW / 8)) : 0u;
    const uint32_t prep = smem_addr(sm) + SM::OFF_PREP + uint32_t(warp) * SM::PREP;
    const uint32_t polls = (a.poll_lanes >> lane) & 1u ? a.polls : PAT_WAIT_LIMIT;

    // The segment's state.  Query 8 t + 2 tig + c of the tile is column (t, c); of a
    // tile of 4, query tig.
    uint32_t qf[D / 16][R8][2];  // query fragments by k-step
    float qs[R8][CQ];            // factor of the scores (base 2)
    int lim[R8][CQ];             // tokens that the query sees
    float ref[R8][CQ];           // running maximum score, raised lazily
    float bar2[R8][CQ], off[R8][CQ];  // where it is raised; what weights are relative to
    int up = 0;                  // 16-bit pages: values, and acc, are taken times 2^-up
    float sum[R8][CQ];           // the lane's part of the sum of weights
    float acc[MT][R8][4];
    float zsum[V4 ? NG : 1][R8][CQ];

    // The queries of (b, tile): raw bf16 (Q8), or fragments as they are.
    uint4 qraw[Q8 ? NG : 1][R8];
    auto load_queries = [&](int sb, uint32_t st) {
        const int h = int(st) / a.RT, r0 = int(st) % a.RT * RTILE;
#pragma unroll
        for (int t = 0; t < R8; ++t) {
            const int r = r0 + 8 * t + (TWICE ? g >> 1 : g);
            const bool real = r < a.R;
            const int i = real ? r / a.G : 0, j = h * a.G + (real ? r - i * a.G : 0);
            const uint16_t *qrow = a.q + ((uint64_t(sb) * uint32_t(a.m) + uint32_t(i)) * uint32_t(a.nq) + uint32_t(j)) * D;
            if constexpr (Q8) {
#pragma unroll
                for (int k = 0; k < NG; ++k)
                    qraw[k][t] = real ? ld_once_v4(qrow + 32 * k + 8 * tig) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qf[k][t][e] = real ? ld_plain_u32(qrow + 16 * k + 8 * e + 2 * tig) : 0u;
            }
        }
    };
    if (cnt) load_queries(b, tile);

    for (uint32_t n = 0; n < cnt; ++n) {
        if (fresh) {
            fresh = false;
            seg0 = place;
            up = 0;
            nplace = SOLO ? solo_units + SM::ITEM : pre[b + 1] - pre[b];
            len = seq_len(a, b, false);
            const int r0 = int(tile) % a.RT * RTILE;
#pragma unroll
            for (int t = 0; t < R8; ++t) {
                int up = 0;
                if constexpr (Q8) {
                    // rows enter as fp16 times a power of two that brings their
                    // largest element to [2^14, 2^15): exact but for elements
                    // under 2^-28 of it
                    float top = 0.0f;
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        const uint32_t w[4] = {qraw[k][t].x, qraw[k][t].y, qraw[k][t].z, qraw[k][t].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int ex = int(__float_as_uint(top) >> 23);  // biased exponent
                    up = ex == 255 ? 0 : min(141 - ex, 126);
                    const float f = __uint_as_float(uint32_t(127 + up) << 23);
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        const uint32_t w[4] = {qraw[k][t].x, qraw[k][t].y, qraw[k][t].z, qraw[k][t].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            qf[2 * k + (e >> 1)][t][e & 1] = pack_f16x2(bf16_lo(w[e]) * f, bf16_hi(w[e]) * f);
                    }
                }
#pragma unroll
                for (int c = 0; c < CQ; ++c) {
                    const int rc = r0 + 8 * t + (TWICE ? tig : 2 * tig + c);
                    lim[t][c] = rc < a.R ? len - (a.m - 1 - rc / a.G) : 0;
                    const int u = __shfl_sync(0xffffffffu, up, (2 * tig + c) * 4);
                    qs[t][c] = Q8 ? a.scale2 * __uint_as_float(uint32_t(127 - u) << 23) : a.scale2;
                    ref[t][c] = -INFINITY, bar2[t][c] = -INFINITY, off[t][c] = 0.0f;
                    sum[t][c] = 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int t = 0; t < R8; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[k][t][e] = 0.0f;
            if constexpr (V4) {
#pragma unroll
                for (int k = 0; k < NG; ++k)
#pragma unroll
                    for (int t = 0; t < R8; ++t)
#pragma unroll
                        for (int c = 0; c < CQ; ++c) zsum[k][t][c] = 0.0f;
            }
        }
        // Every lane polls (and so sees the copied bytes), but whether the copy came
        // in time is the warp's decision: a lane that gave up by itself would be
        // missing from the votes, shuffles and products that the others go on to.
        if (!__all_sync(0xffffffffu, mbar_wait(bar + 8u * slot, phase, polls))) {
            // a copy did not arrive in time: report it, let the copies in flight
            // land (with the normal limit), and give the run up
            if (lane == 0) {
                pages_flag(a.pv, FLAG_TIMEOUT);
                uint32_t s = slot, p = phase;
                for (uint32_t k = n; k < cnt && k < n + STAGES; ++k) {
                    mbar_wait(bar + 8u * s, p, PAT_WAIT_LIMIT);
                    if (++s == STAGES) s = 0, p ^= 1u;
                }
            }
            break;
        }
        const uint32_t here = (good >> (n % GU * UB)) & (UB == 2 ? 3u : 1u);
        if (here) {
            const uint32_t at0 = ring + slot * SM::SLOT;
            const int t0 = int(place - SM::ITEM) * (PAGES_BLOCK * UB);
            // some query does not see all of the unit's tokens
            const bool tail = t0 + PAGES_BLOCK * UB > len - (a.m - 1) || (UB == 2 && here != 3u);
            if (Q8 && tail) {
                // tokens never written: their value scales (and zero points) may be anything
                const int nv = len - t0;
                if (lane < PAGES_BLOCK * UB && (lane >= nv || !((here >> (lane / PAGES_BLOCK)) & 1u))) {
                    const uint32_t sa = at0 + uint32_t(lane / PAGES_BLOCK) * B::BYTES + B::OFF_VS +
                                        uint32_t(lane % PAGES_BLOCK) * B::VSROW;
#pragma unroll
                    for (uint32_t k = 0; k < B::VSROW; k += 4) sts32(sa + k, 0.0f);
                }
                fence_proxy_async();  // before a later copy into the slot
                __syncwarp();
            }
            if constexpr (V4) {
#pragma unroll
                for (int u = 0; u < NG / 2 * UB; ++u) {
                    const int e = 32 * u + lane, t = e / NG, gr = e % NG;  // token of the unit, group
                    const float2 sz = half2_f32(lds32(at0 + uint32_t(u / (NG / 2)) * (B::BYTES - 64u * NG) + B::OFF_VS + 4u * uint32_t(e)));
                    float c;
                    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(sz.x));
                    // any integer will do; NaN (0 / 0) becomes 0
                    c = fminf(fmaxf(rintf(-sz.y * c), 0.0f), 15.0f);
                    sts32(prep + 4u * uint32_t(e), sz.x);
                    sts32(prep + 4u * (UB * SM::NE + uint32_t(e)), fmaf(c, sz.x, sz.y));
                    const uint32_t ca = prep + 8u * UB * SM::NE + 2u * uint32_t((t >> 1) * 2 * NG + gr * 2 + (t & 1));
                    sts16(ca, __bfloat16_as_ushort(__float2bfloat16_rn(-128.0f - c)));
                }
                __syncwarp();
            }
            // 16-bit pages: whether the lane's 1/32 of the block's values has one that is Inf,
            // NaN or of 2^64 or more: the sum of their squares is then beyond bf16.  Read
            // ahead of the scores, in four short chains (15 4K caches of 64 rows a head:
            // 123 us, 121 without the test, 133 from the product's own operands).
            bool odd_values = false;
            if constexpr (!Q8) {
                __nv_bfloat162 sq[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) sq[e] = __float2bfloat162_rn(0.0f);
#pragma unroll
                for (uint32_t k = 0; k < B::VROW / 32; ++k) {
                    const uint4 v = lds128(at0 + B::OFF_V + 512u * k + 16u * uint32_t(lane));
                    sq[0] = square_sum(v.x, sq[0]), sq[1] = square_sum(v.y, sq[1]);
                    sq[2] = square_sum(v.z, sq[2]), sq[3] = square_sum(v.w, sq[3]);
                }
                odd_values = not_finite(__hadd2(__hadd2(sq[0], sq[1]), __hadd2(sq[2], sq[3])));
            }
            // scores: x[u][t][c] token 16 u + g, [CQ + c] token 16 u + g + 8
            float x[UB][R8][2 * CQ];
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                const uint32_t at = at0 + uint32_t(u) * B::BYTES;
#pragma unroll
                for (int t = 0; t < R8; ++t)
#pragma unroll
                    for (int e = 0; e < 2 * CQ; ++e) x[u][t][e] = 0.0f;
                if constexpr (Q8) {
                    uint32_t w[2][NG][2];
                    float ks[2][NG];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t ka = at + k_off + uint32_t(hf) * 8u * B::KROW;
                        const uint4 v = lds128(ka);
                        w[hf][0][0] = v.x, w[hf][0][1] = v.y, w[hf][1][0] = v.z, w[hf][1][1] = v.w;
                        if constexpr (D == 128) {
                            const uint4 v2 = lds128(ka ^ 16u);
                            w[hf][2][0] = v2.x, w[hf][2][1] = v2.y, w[hf][3][0] = v2.z, w[hf][3][1] = v2.w;
                        }
                        lds_halfs<NG>(at + B::OFF_KS + uint32_t(8 * hf + g) * B::SROW, ks[hf]);
                    }
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        float c[R8][4];
#pragma unroll
                        for (int t = 0; t < R8; ++t) c[t][0] = c[t][1] = c[t][2] = c[t][3] = 0.0f;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t a0 = codes_f16(w[0][k][e], 0x4140u), a1 = codes_f16(w[1][k][e], 0x4140u);
                            const uint32_t a2 = codes_f16(w[0][k][e], 0x4342u), a3 = codes_f16(w[1][k][e], 0x4342u);
#pragma unroll
                            for (int t = 0; t < R8; ++t)
                                mma_f16(c[t], a0, a1, a2, a3, qf[2 * k + e][t][0], qf[2 * k + e][t][1]);
                        }
#pragma unroll
                        for (int t = 0; t < R8; ++t)
#pragma unroll
                            for (int e = 0; e < 2 * CQ; ++e)
                                x[u][t][e] = fmaf(c[t][e / CQ * 2 + e % CQ], ks[e / CQ][k], x[u][t][e]);
                    }
                } else {
                    float c[R8][4];
#pragma unroll
                    for (int t = 0; t < R8; ++t) c[t][0] = c[t][1] = c[t][2] = c[t][3] = 0.0f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t w[4];
                        ldsm4(w, (at + k_off) ^ (32u * uint32_t(k)));
#pragma unroll
                        for (int t = 0; t < R8; ++t) mma_bf16(c[t], w[0], w[1], w[2], w[3], qf[k][t][0], qf[k][t][1]);
                    }
#pragma unroll
                    for (int t = 0; t < R8; ++t)
#pragma unroll
                        for (int e = 0; e < 2 * CQ; ++e) x[u][t][e] = c[t][e / CQ * 2 + e % CQ];
                }
#pragma unroll
                for (int t = 0; t < R8; ++t)
#pragma unroll
                    for (int e = 0; e < 2 * CQ; ++e) x[u][t][e] *= qs[t][e % CQ];
            }
            if (tail) {
#pragma unroll
                for (int u = 0; u < UB; ++u)
#pragma unroll
                    for (int t = 0; t < R8; ++t)
#pragma unroll
                        for (int e = 0; e < 2 * CQ; ++e)
                            if (t0 + 16 * u + g + 8 * (e / CQ) >= lim[t][e % CQ] || !((here >> u) & 1u)) x[u][t][e] = -INFINITY;
            }
            bool raise = false;
            float top[R8][CQ];
#pragma unroll
            for (int t = 0; t < R8; ++t)
#pragma unroll
                for (int c = 0; c < CQ; ++c) {
                    top[t][c] = fmaxf(x[0][t][c], x[0][t][CQ + c]);
                    if constexpr (UB == 2) top[t][c] = fmaxf(top[t][c], fmaxf(x[UB - 1][t][c], x[UB - 1][t][CQ + c]));
                    raise |= top[t][c] > bar2[t][c];
                }
            if (__any_sync(0xffffffffu, raise)) {
                float f[R8][CQ];
                bool lost = false;  // a factor has underflowed
#pragma unroll
                for (int t = 0; t < R8; ++t)
#pragma unroll
                    for (int c = 0; c < CQ; ++c) {
                        const float nr = fmaxf(ref[t][c], rows_top(top[t][c]));
                        f[t][c] = ref[t][c] == -INFINITY ? 1.0f : exp2f(ref[t][c] - nr);
                        lost |= f[t][c] == 0.0f;
                        ref[t][c] = nr, bar2[t][c] = nr + PAT_SLACK;
                        off[t][c] = nr == -INFINITY ? 0.0f : nr;
                        sum[t][c] *= f[t][c];
                        if constexpr (V4) {
#pragma unroll
                            for (int k = 0; k < NG; ++k) zsum[k][t][c] *= f[t][c];
                        }
                    }
                if (!Q8 && __any_sync(0xffffffffu, lost)) {
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int t = 0; t < R8; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[k][t][e] *= factor(f[t][e % CQ], acc[k][t][e]);
                } else {
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int t = 0; t < R8; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[k][t][e] *= f[t][e % CQ];
                }
            }
            float p[UB][R8][2 * CQ];
#pragma unroll
            for (int u = 0; u < UB; ++u)
#pragma unroll
                for (int t = 0; t < R8; ++t)
#pragma unroll
                    for (int c = 0; c < CQ; ++c) {
                        p[u][t][c] = exp2_fast(x[u][t][c] - off[t][c]);
                        p[u][t][CQ + c] = exp2_fast(x[u][t][CQ + c] - off[t][c]);
                        sum[t][c] += p[u][t][c] + p[u][t][CQ + c];
                    }
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                const uint32_t at = at0 + uint32_t(u) * B::BYTES;
                if constexpr (Q8) {
                    float sv[2][NG], zv[2][V4 ? NG : 1];  // value scales of tokens g and g + 8
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        if constexpr (V4) {
                            const uint32_t pa = prep + 4u * NG * uint32_t(16 * u + 8 * hf + g);
                            lds_floats<NG>(pa, sv[hf]);
                            lds_floats<NG>(pa + 4u * UB * SM::NE, zv[hf]);
                        } else {
                            lds_halfs<NG>(at + B::OFF_VS + uint32_t(8 * hf + g) * B::VSROW, sv[hf]);
                        }
                    }
                    uint32_t vw[2][2][V4 ? NG / 2 : NG];  // [token half][odd token]: the lane's granule
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t va = at + (k ? v_odd : v_off) + uint32_t(hf) * 8u * B::VROW;
                            if constexpr (B::VROW == 128) {
                                const uint4 v = lds128(va);
                                vw[hf][k][0] = v.x, vw[hf][k][1] = v.y, vw[hf][k][NG - 2] = v.z, vw[hf][k][NG - 1] = v.w;
                            } else if constexpr (B::VROW == 64) {
                                const uint2 v = lds64(va);
                                vw[hf][k][0] = v.x, vw[hf][k][1] = v.y;
                            } else {
                                vw[hf][k][0] = lds32(va);
                            }
                        }
                    uint32_t cv[2][V4 ? NG : 1];  // [token half]
                    if constexpr (V4) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t ca = prep + 8u * UB * SM::NE + 4u * NG * uint32_t(8 * u + 4 * hf + tig);
                            if constexpr (NG == 4) {
                                const uint4 v = lds128(ca);
                                cv[hf][0] = v.x, cv[hf][1] = v.y, cv[hf][NG - 2] = v.z, cv[hf][NG - 1] = v.w;
                            } else {
                                const uint2 v = lds64(ca);
                                cv[hf][0] = v.x, cv[hf][1] = v.y;
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < NG; ++e) {
                        uint32_t hi[R8][2], lo[R8][2];
#pragma unroll
                        for (int t = 0; t < R8; ++t) {
                            if constexpr (TWICE) {
                                twin_weights(p[u][t][0] * sv[0][e], p[u][t][1] * sv[1][e], hi[t][0], hi[t][1]);
                            } else {
#pragma unroll
                                for (int hf = 0; hf < 2; ++hf)
                                    split_weights(p[u][t][2 * hf] * sv[hf][e], p[u][t][2 * hf + 1] * sv[hf][e], hi[t][hf],
                                                  lo[t][hf]);
                            }
                        }
                        uint32_t v[2][4];  // [token half][dim of the granule's word]
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if constexpr (!V4) {
                                // byte j of both tokens' words to the halves' low bytes
                                v[hf][0] = codes_bf16(__byte_perm(vw[hf][0][e], vw[hf][1][e], 0x5410u));
                                v[hf][1] = codes_bf16(__byte_perm(vw[hf][0][e], vw[hf][1][e], 0x5511u));
                                v[hf][2] = codes_bf16(__byte_perm(vw[hf][0][e], vw[hf][1][e], 0x6622u));
                                v[hf][3] = codes_bf16(__byte_perm(vw[hf][0][e], vw[hf][1][e], 0x7733u));
                            } else {
                                const uint32_t w = __byte_perm(vw[hf][0][e / 2], vw[hf][1][e / 2], e & 1 ? 0x7632u : 0x5410u);
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[hf][j] = nibbles_bf16(w >> (4 * j), cv[hf][e]);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < R8; ++t)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t a0 = v[0][2 * k], a1 = v[0][2 * k + 1], a2 = v[1][2 * k], a3 = v[1][2 * k + 1];
                                mma_bf16(acc[2 * e + k][t], a0, a1, a2, a3, hi[t][0], hi[t][1]);
                                if constexpr (!TWICE) mma_bf16(acc[2 * e + k][t], a0, a1, a2, a3, lo[t][0], lo[t][1]);
                            }
                        if constexpr (V4) {
#pragma unroll
                            for (int t = 0; t < R8; ++t)
#pragma unroll
                                for (int c = 0; c < 2 * CQ; ++c)
                                    zsum[e][t][c % CQ] = fmaf(p[u][t][c], zv[c / CQ][e], zsum[e][t][c % CQ]);
                        }
                    }
                } else {
                    if (__any_sync(0xffffffffu, odd_values) || up) {
                        // Weights go up to 2^PAT_SLACK and are divided by their sum at the
                        // end.  Values of 2^64 or more (below it, 2^31 of them do not pass
                        // fp32's range), and all after the first of them, are taken times a
                        // power of two that leaves all of the sequence's weights, times the
                        // largest bf16, within half of that range.
                        // Tokens that hold Inf or NaN are added one by one, in fp32, to the
                        // queries that see them, and are zeros to the product, whose operands
                        // may not meet them: 0 * Inf would reach queries that do not see the
                        // token, and of a weight's two bf16 the second is often 0 or negative.
                        // So are tokens that were never written, whatever they hold.  Two
                        // lanes look at a token, each at half of its row, every lane from
                        // another 16 bytes on, for the banks.
                        constexpr uint32_t CHUNKS = B::VROW / 32;
                        const int nv = len - t0, tl = lane >> 1;
                        const uint32_t half = at + B::OFF_V + uint32_t(tl) * B::VROW + uint32_t(lane & 1) * (B::VROW / 2);
                        __nv_bfloat162 odd = __float2bfloat162_rn(0.0f), sq = odd;  // odd: NaN once a value is Inf or NaN
                        if (tl < nv) {
#pragma unroll
                            for (uint32_t k = 0; k < CHUNKS; ++k) {
                                const uint4 v = lds128(half + 16u * ((k + uint32_t(lane)) % CHUNKS));
                                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    odd = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w4[e]), __float2bfloat162_rn(0.0f), odd);
                                    sq = square_sum(w4[e], sq);
                                }
                            }
                        }
                        if (up == 0 && __any_sync(0xffffffffu, not_finite(sq))) {
                            up = int(PAT_SLACK) + 1 + 32 - __clz(len);
#pragma unroll
                            for (int k = 0; k < MT; ++k)
#pragma unroll
                                for (int r = 0; r < R8; ++r)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) acc[k][r][e] *= power2(-up);
                        }
                        uint32_t bits = __ballot_sync(0xffffffffu, not_finite(odd));
                        bits = (bits | bits >> 1) & 0x55555555u;  // bit 2 t: token t
                        for (uint32_t left = bits; left; left &= left - 1u) {
                            const int t = (__ffs(int(left)) - 1) >> 1;
#pragma unroll
                            for (int r = 0; r < R8; ++r)
#pragma unroll
                                for (int c = 0; c < CQ; ++c) {
                                    // the token's weight and score are with lane row t % 8
                                    const int from = ((t & 7) << 2) | tig;
                                    const float pw = __shfl_sync(0xffffffffu, t < 8 ? p[u][r][c] : p[u][r][CQ + c], from);
                                    const float ps = __shfl_sync(0xffffffffu, t < 8 ? x[u][r][c] : x[u][r][CQ + c], from);
                                    if (t0 + t >= lim[r][c]) continue;
#pragma unroll
                                    for (int k = 0; k < MT; ++k)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {  // dims 16 k + 8 h + g
                                            const uint32_t d2 = uint32_t(k) * 32u + uint32_t(h) * 16u + uint32_t(g >> 1) * 4u;
                                            const uint32_t y2 = lds32(at + B::value(uint32_t(t), d2));
                                            const float y = (g & 1 ? bf16_hi(y2) : bf16_lo(y2)) * power2(-up);
                                            acc[k][r][2 * h + c] =
                                                fmaf(ps > -INFINITY ? factor(pw, y) : pw, y, acc[k][r][2 * h + c]);
                                        }
                                }
                        }
                        __syncwarp();
                        if (tl >= nv || ((bits >> (lane & 30)) & 1u)) {
#pragma unroll
                            for (uint32_t k = 0; k < CHUNKS; ++k) sts128_zero(half + 16u * ((k + uint32_t(lane)) % CHUNKS));
                        } else if (up) {
                            const __nv_bfloat162 f = __float2bfloat162_rn(power2(-up));
#pragma unroll
                            for (uint32_t k = 0; k < CHUNKS; ++k) {
                                const uint32_t to = half + 16u * ((k + uint32_t(lane)) % CHUNKS);
                                const uint4 v = lds128(to);
                                sts128(to, make_uint4(times(v.x, f), times(v.y, f), times(v.z, f), times(v.w, f)));
                            }
                        }
                        fence_proxy_async();  // before a later copy into the slot
                        __syncwarp();
                    }
                    uint32_t hi[R8][2], lo[R8][2];
#pragma unroll
                    for (int t = 0; t < R8; ++t) {
                        if constexpr (TWICE) {
                            twin_weights(p[u][t][0], p[u][t][1], hi[t][0], hi[t][1]);
                        } else {
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
                                split_weights(p[u][t][2 * hf], p[u][t][2 * hf + 1], hi[t][hf], lo[t][hf]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < MT; ++k) {
                        uint32_t w[4];
                        ldsm4_t(w, (at + v_off) ^ (32u * uint32_t(k)));
#pragma unroll
                        for (int t = 0; t < R8; ++t) {
                            mma_bf16(acc[k][t], w[0], w[1], w[2], w[3], hi[t][0], hi[t][1]);
                            if constexpr (!TWICE) mma_bf16(acc[k][t], w[0], w[1], w[2], w[3], lo[t][0], lo[t][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();  // every lane is done with the slot
        if (n + STAGES < cnt) {
            const bool far = n % GU + STAGES >= uint32_t(GU);
            issue(n + STAGES, far ? nxt : cur, far ? good_nxt : good, slot);
        }
        if (++slot == STAGES) slot = 0, phase ^= 1u;
        if (n % GU == uint32_t(GU) - 1u) {
            cur = nxt, good = good_nxt;
            int lb;
            uint32_t lt, lp;
            nxt = address(n + 1u + uint32_t(GU), lb, lt, lp);
            good_nxt = __ballot_sync(0xffffffffu, nxt != 0);
        }
        ++place;
        if (place < nplace && n + 1 < cnt) continue;
        // the segment's end; the next one's queries are requested first
        int nb = b;
        uint32_t ntile = tile;
        if (!SOLO && place == nplace && ++ntile == HRT) {
            ntile = 0;
            do ++nb;
            while (nb < a.nseq && pre[nb + 1] == pre[nb]);
        }
        if (n + 1 < cnt) load_queries(nb, ntile);
        const int h = int(tile) / a.RT, r0 = int(tile) % a.RT * RTILE;
        const bool whole = SOLO ? cnt == solo_units : seg0 == 0 && place == nplace;
        // slot 0: the segment that the run starts with; 1: its last
        const uint64_t ps = (uint64_t(gw) * 2u + (n + 1 == place - seg0 ? 0u : 1u)) * RTILE;
#pragma unroll
        for (int t = 0; t < R8; ++t)
#pragma unroll
            for (int c = 0; c < CQ; ++c) {
                const int rr = TWICE ? tig : 8 * t + 2 * tig + c, r = r0 + rr;
                const float l0 = rows_add(sum[t][c]);
                // acc's unit: a row's result is acc / l, and a part's weight goes by l and base2
                const float l = Q8 ? l0 : l0 * power2(-up), base2 = Q8 ? ref[t][c] : ref[t][c] + float(up);
                if constexpr (TWICE) {
#pragma unroll
                    for (int k = 0; k < MT; ++k) acc[k][t][0] += acc[k][t][1], acc[k][t][2] += acc[k][t][3];
                }
                if constexpr (V4) {
#pragma unroll
                    for (int e = 0; e < NG; ++e) {
                        const float z = rows_add(zsum[e][t][c]);
                        acc[2 * e][t][c] += z, acc[2 * e][t][2 + c] += z;
                        acc[2 * e + 1][t][c] += z, acc[2 * e + 1][t][2 + c] += z;
                    }
                }
                if (r >= a.R) continue;
                if (whole) {
                    const int i = r / a.G, j = h * a.G + r - i * a.G;
                    const uint64_t row = (uint64_t(b) * uint32_t(a.m) + uint32_t(i)) * uint32_t(a.nq) + uint32_t(j);
                    const float bl = a.base_lse ? a.base_lse[row] : -INFINITY;
                    __syncwarp(0x11111111u << tig);  // the row's lanes have it before one writes lse
                    const float lse = l0 > 0.0f ? (ref[t][c] + log2f(l0)) * 0.69314718055994531f : (l0 == 0.0f ? -INFINITY : l0);
                    const float2 w = join_base(a, row, lse, bl, g == 0);
                    const float inv = l > 0.0f ? w.x / l : (l == 0.0f ? 0.0f : l);
                    uint16_t *o = a.out + row * D;
                    const float *bo = a.base_out && w.y != 0.0f ? a.base_out + row * D : nullptr;
                    if constexpr (Q8) {
#pragma unroll
                        for (int e = 0; e < NG; ++e) {
                            float y[4] = {acc[2 * e][t][c] * inv, acc[2 * e][t][2 + c] * inv, acc[2 * e + 1][t][c] * inv,
                                          acc[2 * e + 1][t][2 + c] * inv};
                            if (bo) {
                                const float4 v = *reinterpret_cast<const float4 *>(bo + 32 * e + 4 * g);
                                y[0] = fmaf(w.y, v.x, y[0]), y[1] = fmaf(w.y, v.y, y[1]);
                                y[2] = fmaf(w.y, v.z, y[2]), y[3] = fmaf(w.y, v.w, y[3]);
                            }
                            *reinterpret_cast<uint2 *>(o + 32 * e + 4 * g) =
                                make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < MT; ++k)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int d = 16 * k + 8 * u + g;
                                float y = acc[k][t][2 * u + c] * factor(inv, acc[k][t][2 * u + c]);
                                if (bo) y = fmaf(w.y, bo[d], y);
                                reinterpret_cast<__nv_bfloat16 *>(o)[d] = __float2bfloat16_rn(y);
                            }
                    }
                } else {
                    // SOLO: in the warp's own ring, whose copies have all been used
                    float *mine = reinterpret_cast<float *>(sm + PAT_BAR_BYTES + uint32_t(warp) * STAGES * SM::SLOT);
                    float *o = SOLO ? mine + rr * D : a.part + (ps + uint32_t(rr)) * D;
                    if constexpr (Q8) {
#pragma unroll
                        for (int e = 0; e < NG; ++e)
                            *reinterpret_cast<float4 *>(o + 32 * e + 4 * g) =
                                make_float4(acc[2 * e][t][c], acc[2 * e][t][2 + c], acc[2 * e + 1][t][c], acc[2 * e + 1][t][2 + c]);
                    } else {
#pragma unroll
                        for (int k = 0; k < MT; ++k)
#pragma unroll
                            for (int u = 0; u < 2; ++u) o[16 * k + 8 * u + g] = acc[k][t][2 * u + c];
                    }
                    if (g == 0) {
                        float2 *st = SOLO ? reinterpret_cast<float2 *>(mine + RTILE * D) + rr : a.stats + ps + uint32_t(rr);
                        *st = make_float2(base2, l);
                    }
                }
            }
        fresh = true;
        if (place == nplace) place = 0;
        b = nb, tile = ntile;
    }
    if constexpr (!SOLO) return;

    // The tile's rows, a warp of the team at a time: its warps' parts, in order
    static_assert(RTILE * (D * 4 + 8) <= STAGES * SM::SLOT, "a warp's part fits its ring");
    __syncthreads();
    const uint32_t parts = uint32_t((units + per - 1) / per);
    if (!sreal || parts == 1u) return;  // written by the warp that had it all
    const int h = int(stile) / a.RT, r0 = int(stile) % a.RT * RTILE;
    const uint8_t *part = sm + PAT_BAR_BYTES + uint32_t(warp - place_in) * STAGES * SM::SLOT;
    for (int rr = place_in; rr < min(RTILE, a.R - r0); rr += team) {
        constexpr int VPL = D / 32;
        float y[VPL], M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int k = 0; k < VPL; ++k) y[k] = 0.0f;
        for (uint32_t w = 0; w < parts; ++w)
            M = fmaxf(M, reinterpret_cast<const float2 *>(part + w * STAGES * SM::SLOT + RTILE * D * 4)[rr].x);
        for (uint32_t w = 0; w < parts; ++w) {
            const float *src = reinterpret_cast<const float *>(part + w * STAGES * SM::SLOT);
            const float2 st = reinterpret_cast<const float2 *>(src + RTILE * D)[rr];
            const float f = st.x == -INFINITY ? 0.0f : exp2f(st.x - M);
            L = fmaf(f, st.y, L);
#pragma unroll
            for (int k = 0; k < VPL; ++k) {
                const float v = src[rr * D + lane * VPL + k];
                y[k] = fmaf(Q8 ? f : factor(f, v), v, y[k]);
            }
        }
        const int r = r0 + rr, i = r / a.G, j = h * a.G + r - i * a.G;
        const uint64_t row = (uint64_t(sb) * uint32_t(a.m) + uint32_t(i)) * uint32_t(a.nq) + uint32_t(j);
        const float lse = L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : (L == 0.0f ? -INFINITY : L);
        const float bl = a.base_lse ? a.base_lse[row] : -INFINITY;
        __syncwarp();  // every lane has it before one writes lse
        const float2 w = join_base(a, row, lse, bl, lane == 0);
        const float inv = L > 0.0f ? w.x / L : (L == 0.0f ? 0.0f : L);
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            y[k] *= Q8 ? inv : factor(inv, y[k]);
            if (a.base_out && w.y != 0.0f) y[k] = fmaf(w.y, a.base_out[row * D + lane * VPL + k], y[k]);
        }
#pragma unroll
        for (int k = 0; k < VPL; k += 2)
            *reinterpret_cast<uint32_t *>(a.out + row * D + lane * VPL + k) = pack_bf16x2(y[k], y[k + 1]);
    }
}

// Merges the partial results of the rows whose blocks several warps had, and
// writes the rows of empty sequences.  A block takes a.join_rows rows of a row
// tile, one after the other; its WARPS warps take every WARPS-th partial, eight of
// them in flight at a time.  A block finds
// out what it has to merge before pages_attend has ended (up to PAT_OWN_PLAN
// sequences; beyond, from the plan that pages_attend leaves), and all but block 0
// leave at once if that is nothing: block 0 stays for pages_attend's end, so that
// this grid's end means the other's.
// ODD: values may be Inf or NaN (16-bit pages).
template <int D, int RTILE, int WARPS, bool ODD>
__global__ void __launch_bounds__(32 * WARPS) pages_join(const __grid_constant__ PagesAttendArgs a) {
    constexpr int VPL = D / 32, DEEP = 8;  // values of a lane
    __shared__ float macc[WARPS][D], mst[WARPS][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t HRT = uint32_t(a.pv.H) * uint32_t(a.RT);
    const uint32_t splits = uint32_t(min(RTILE, a.R) + a.join_rows - 1) / uint32_t(a.join_rows);  // blocks of a row tile
    const uint32_t task = blockIdx.x / splits, b = task / HRT;
    const int h = int(task % HRT) / a.RT, rt = int(task % HRT) % a.RT;
    const int r0 = rt * RTILE + int(blockIdx.x % splits) * a.join_rows;
    // the next attention's blocks may be placed; they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t before = 0, n = 0, all = 0;
    if (a.nseq <= PAT_OWN_PLAN) {
        // pages_attend has passed its own wait, so the lengths are final
        for (int k = lane; k < a.nseq; k += 32) {
            const uint32_t u = tile_units(seq_len<true>(a, k, false), a.unit);
            all += u;
            before += k < int(b) ? u : 0u;
            n += k == int(b) ? u : 0u;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        before = __reduce_add_sync(0xffffffffu, before);
        n = __reduce_add_sync(0xffffffffu, n);
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        before = ld_l2_u32(a.plan + b), n = ld_l2_u32(a.plan + b + 1) - before, all = ld_l2_u32(a.plan + a.nseq);
    }
    const uint64_t per = run_length(uint64_t(all) * HRT, a.nwarps);
    const uint64_t first = uint64_t(before) * HRT + uint64_t(h * a.RT + rt) * n;
    const uint64_t w0 = first / per, w1 = n ? (first + n - 1) / per : w0;
    const bool whole = n && w0 == w1;  // one warp had it all
    if (whole && blockIdx.x) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (whole || !pages_match(a.pv)) return;
    const uint32_t parts = n ? uint32_t(w1 - w0 + 1) : 0u;
    for (int r = r0; r < min(min(r0 + a.join_rows, rt * RTILE + RTILE), a.R); ++r) {
        float acc[VPL], M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int k = 0; k < VPL; ++k) acc[k] = 0.0f;
        for (uint32_t c0 = uint32_t(warp); c0 < parts; c0 += DEEP * WARPS) {
            float2 st[DEEP];
            float v[DEEP][VPL];
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                const uint32_t c = c0 + uint32_t(k * WARPS);
                st[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int u = 0; u < VPL; ++u) v[k][u] = 0.0f;
                if (c < parts) {
                    const uint64_t w = w0 + c;
                    const uint64_t ps = (w * 2u + (first > w * per ? 1u : 0u)) * RTILE + uint32_t(r % RTILE);
                    const uint2 s = ld_once_v2(a.stats + ps);
                    st[k] = make_float2(__uint_as_float(s.x), __uint_as_float(s.y));
                    const float *src = a.part + ps * D + lane * VPL;
                    if constexpr (VPL == 4) {
                        const uint4 x = ld_once_v4(src);
                        v[k][0] = __uint_as_float(x.x), v[k][1] = __uint_as_float(x.y);
                        v[k][VPL - 2] = __uint_as_float(x.z), v[k][VPL - 1] = __uint_as_float(x.w);
                    } else {
                        const uint2 x = ld_once_v2(src);
                        v[k][0] = __uint_as_float(x.x), v[k][1] = __uint_as_float(x.y);
                    }
                }
            }
            float nm = M;
#pragma unroll
            for (int k = 0; k < DEEP; ++k) nm = fmaxf(nm, st[k].x);
            const float f0 = nm == -INFINITY ? 1.0f : exp2f(M - nm);
            M = nm, L *= f0;
#pragma unroll
            for (int u = 0; u < VPL; ++u) acc[u] *= ODD ? factor(f0, acc[u]) : f0;
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                if (st[k].x == -INFINITY) continue;  // an empty part
                const float f = exp2f(st[k].x - nm);
                L = fmaf(f, st[k].y, L);
#pragma unroll
                for (int u = 0; u < VPL; ++u) acc[u] = fmaf(ODD ? factor(f, v[k][u]) : f, v[k][u], acc[u]);
            }
        }
#pragma unroll
        for (int k = 0; k < VPL; ++k) macc[warp][lane * VPL + k] = acc[k];
        if (lane == 0) mst[warp][0] = M, mst[warp][1] = L;
        const int i = r / a.G, j = h * a.G + r - i * a.G;
        const uint64_t row = (uint64_t(b) * uint32_t(a.m) + uint32_t(i)) * uint32_t(a.nq) + uint32_t(j);
        const float bl = a.base_lse ? a.base_lse[row] : -INFINITY;  // before thread 0 writes lse
        __syncthreads();
        if (threadIdx.x < D) {
            float top = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) top = fmaxf(top, mst[k][0]);
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                const float f = mst[k][0] == -INFINITY ? 0.0f : exp2f(mst[k][0] - top);
                l = fmaf(f, mst[k][1], l);
                const float v = macc[k][threadIdx.x];
                o = fmaf(ODD ? factor(f, v) : f, v, o);
            }
            const float lse = l > 0.0f ? (top + log2f(l)) * 0.69314718055994531f : (l == 0.0f ? -INFINITY : l);
            const float2 w = join_base(a, row, lse, bl, threadIdx.x == 0);
            const float inv = l > 0.0f ? w.x / l : (l == 0.0f ? 0.0f : l);
            o *= ODD ? factor(inv, o) : inv;
            if (a.base_out && w.y != 0.0f) o = fmaf(w.y, a.base_out[row * D + threadIdx.x], o);
            reinterpret_cast<__nv_bfloat16 *>(a.out)[row * D + threadIdx.x] = __float2bfloat16_rn(o);
        }
        __syncthreads();  // the next row writes macc again
    }
}

static thread_local uint32_t g_next_polls = 0, g_next_lanes = 0;
static thread_local bool g_limit_next = false;

static unsigned attend_grid() { return unsigned(sm_count()); }
// Rows of a tile.  us of tiles of 8 and of 16 rows on 15 4K caches, 8 KV heads:
//   rows       12      16      20      24      28      32      40      52      64
//   k8v8, 128  62  51  64  53  82  87  82  89 111  90 111  90 130 130 178 167 207 171
//   k8v4, 128  58  53  60  55  78  91  78  92 105  93 105  94 124 135 169 173 196 177
//   k8v8, 64   36  34  36  35  50  56  51  57  62  58  63  59  79  76 102 101 113 102
//   k8v4, 64   36  37  36  38  52  59  52  59  64  61  65  62  81  81 104 106 116 108
//   bf16, 128  52  53  54  55 125  62 126  64  99  65 100  66 117 137 269 118 210 123
//   bf16, 64   32  27  33  28  65  50  66  51  54  53  55  55  66  59  94  91  99  92
// An odd number of groups of 8 rows goes in tiles of 8 with 8- and 4-bit pages, where
// it wins at three groups and is about even beyond; with 16-bit pages more than 8 rows
// go in tiles of 16 (40 rows at head_dim 128 lose by that).  Up to 4 rows a tile of 4
// forms no exponential or split twice: one 128K sequence with 4-bit values 50.6 us,
// 55.9 in a tile of 8.
static int tile_rows(int rows, int format) {
    if (rows <= 4) return 4;
    const int eights = (rows + 7) / 8;
    return eights == 1 || (format != KVP_PAGES_BF16 && eights % 2 == 1) ? 8 : 16;
}

// Blocks of a team's warp up to which a team per row tile beats equal runs of the
// list.  It has one launch and nothing cut, but waits for the longest sequence, so
// that the limits are below where ragged lengths lose.  us, teams against runs, 8 KV
// heads of 4 rows.  Where teams employ half of the GPU's warps or more, 64 sequences:
//   tokens      700      1-700    1000     1-1000   1500     1-1500
//   k8v8, 128   25  32   23  25   33  38   28  29   44  48   39  33
//   k8v4, 128   24  31   22  24   31  37   27  28   41  45   37  32
//   bf16, 128   34  42   23  28   46  54   30  35   66  73   41  44
//   k8v8, 64    17  22   13  16   20  26   17  19   26  31   22  23
//   k8v4, 64    17  22   13  16   20  26   16  18   26  31   22  23
//   bf16, 64    19  26   14  20   25  32   17  23   35  41   23  27
// (at head_dim 128 15, 21 and 31 blocks a warp, 22, 31 and 47 with 16 bits; at 64 11,
// 16 and 24).  With more row tiles than the GPU has warps, in several waves: 64 x 200
// of 64 rows (13, k8v8 at 128) 51 and 92, 512 x 200 of 4 rows 62 and 66 (bf16 75 and 93,
// at 64 40 and 60; k8v4 at 64 33 and 47).  Where they employ fewer, one sequence:
//   tokens      400          700          1000         1500
//   k8v8, 128   7.4   8.8    9.0   8.9    11.1  9.1    13.5  9.3    (4 blocks: 768)
//   k8v4, 128   7.5   8.7    8.8   9.0    10.7  9.1    13.0  9.2
//   bf16, 128   6.8   7.5    8.1   7.7     9.7  7.9    12.4  8.2    (512)
//   k8v8, 64    6.0   8.0    6.9   8.2     7.7  8.4     9.3  8.4    (1024)
//   k8v4, 64    6.1   8.0    6.9   8.2     7.7  8.4     9.1  8.4
//   bf16, 64    5.7   7.3    6.7   7.6     7.5  7.8     8.8  8.0
template <int D, int FMT>
static int team_blocks(bool half) {
    return half ? (FMT != KVP_PAGES_BF16 && D == 128 ? 16 : 24) : 4;
}

template <int D, int FMT, int RC, bool SOLO>
static int launch_tiles(cudaLaunchConfig_t &cfg, const PagesAttendArgs &a, unsigned grid) {
    using SM = PatShape<D, FMT, RC>;
    // the opt-in to more than 48 KB, once per device (to the most that any call needs)
    static bool ready[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVP_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        if (cudaFuncSetAttribute(pages_attend<D, FMT, RC, SOLO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(SM::bytes(KVP_PAGES_MAX_SEQS))) != cudaSuccess)
            return KVP_ERR_CUDA;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(SM::WARPS * 32);
    cfg.dynamicSmemBytes = SM::bytes(SOLO ? 0 : a.nseq);
    if (cudaLaunchKernelEx(&cfg, pages_attend<D, FMT, RC, SOLO>, a) != cudaSuccess) return KVP_ERR_CUDA;
    count_launch();
    return KVP_OK;
}

template <int D, int FMT, int RC>
static int launch_attend(PagesAttendArgs &a, cudaStream_t st) {
    using SM = PatShape<D, FMT, RC>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    a.nwarps = attend_grid() * SM::WARPS;
    a.unit = PAGES_BLOCK * SM::UB;
    const unsigned tiles = unsigned(a.nseq) * unsigned(a.pv.H) * unsigned(a.RT);
    // the largest team of warps for which one wave of blocks holds all tiles, or one
    // warp and several waves
    a.team = SM::WARPS;
    while (a.team > 1 && (SM::WARPS % a.team || uint64_t(attend_grid()) * unsigned(SM::WARPS / a.team) < tiles)) --a.team;
    const int64_t most = (int64_t(a.max_pages) << a.pv.logP) / PAGES_BLOCK;  // blocks that a table may hold
    if (most <= int64_t(team_blocks<D, FMT>(2 * uint64_t(tiles) * a.team >= a.nwarps)) * a.team) {
        const unsigned per_block = unsigned(SM::WARPS / a.team);
        const int rc = launch_tiles<D, FMT, RC, true>(cfg, a, (tiles + per_block - 1) / per_block);
        return rc == KVP_OK ? launch_status() : rc;
    }
    const int rc = launch_tiles<D, FMT, RC, false>(cfg, a, attend_grid());
    if (rc != KVP_OK) return rc;
    // Rows of a row tile to a block, so that about a wave of blocks does (one row a
    // block: 64 x 200 tokens of 64 rows 131 us, 90 so, 15 x 4096 177 and 171; of 4
    // rows 19.9 and 19.0; with 16 instead of 12 blocks an SM 19.9, with 8 as with 12).
    const unsigned rows = unsigned(std::min(RC, a.R));
    const uint64_t wave = uint64_t(attend_grid()) * 12u;
    const unsigned most_rows = unsigned(std::min<uint64_t>(rows, (uint64_t(tiles) * rows + wave - 1) / wave));
    const unsigned splits = (rows + most_rows - 1) / most_rows;
    a.join_rows = int((rows + splits - 1) / splits);
    cfg.gridDim = dim3(tiles * splits);
    cfg.dynamicSmemBytes = 0;
    // Warps for a row's partials, of which it has about nwarps / (row tiles): 16
    // where there are 64 or more of them, 8 a warp in flight (one 128K sequence, 300
    // partials a row: 71 against 76 us with 4 warps); 4 warps where there are fewer
    // (a step of 15 agents, 16 partials: 20.0 against 23.8 us with 16).
    const bool many = a.nwarps / tiles >= 64u;
    cfg.blockDim = dim3(many ? 512 : 128);
    constexpr bool ODD = FMT == KVP_PAGES_BF16;
    if (cudaLaunchKernelEx(&cfg, many ? pages_join<D, RC, 16, ODD> : pages_join<D, RC, 4, ODD>, a) != cudaSuccess)
        return KVP_ERR_CUDA;
    count_launch();
    return launch_status();
}

template <int D, int FMT>
static int launch_attend(PagesAttendArgs &a, int rows, cudaStream_t st) {
    return rows == 4 ? launch_attend<D, FMT, 4>(a, st)
                     : (rows == 8 ? launch_attend<D, FMT, 8>(a, st) : launch_attend<D, FMT, 16>(a, st));
}

static int attend_counts_ok(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (n_seqs < 0 || n_q_tokens <= 0 || n_q_heads <= 0 || n_q_heads % cfg->n_kv_heads != 0) return KVP_ERR_ARG;
    if (n_seqs > KVP_PAGES_MAX_SEQS || n_q_tokens > 64 || n_q_heads > 65536) return KVP_ERR_SIZE;
    if (int64_t(n_seqs) * n_q_tokens * n_q_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    return KVP_OK;
}

// Workspace: the plan, the partial rows' statistics, the partial rows.
struct AttendWs {
    uint64_t stats, part, total;
};
static AttendWs attend_ws(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    const uint64_t rows =
        uint64_t(attend_grid()) * PAT_MOST_WARPS * 2u * uint64_t(tile_rows(n_q_tokens * (n_q_heads / cfg->n_kv_heads), cfg->format));
    AttendWs w;
    w.stats = align256(4ull * uint64_t(n_seqs + 1));
    w.part = w.stats + align256(rows * 8ull);
    w.total = w.part + rows * uint64_t(cfg->head_dim) * 4ull;
    return w;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvpages_attend_workspace_bytes(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    if (attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads) != KVP_OK) return 0;
    return size_t(attend_ws(cfg, n_seqs, n_q_tokens, n_q_heads).total);
}

int kvp_test_limit_next_pages_attend_lanes(uint32_t polls, uint32_t lanes) {
    g_next_polls = polls, g_next_lanes = lanes;
    g_limit_next = true;
    return KVP_OK;
}

int kvp_test_limit_next_pages_attend(uint32_t polls) {
    return kvp_test_limit_next_pages_attend_lanes(polls, 0xFFFFFFFFu);
}

int kvpages_attend(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, int n_q_tokens,
                   int n_q_heads, const void *q, float scale, const int32_t *table, int max_pages,
                   const int32_t *lens, const float *base_out, const float *base_lse, void *out, float *lse, void *ws,
                   size_t ws_bytes, void *stream) {
    const int rc = attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads);
    if (rc != KVP_OK) return rc;
    if (!pages || layer < 0 || layer >= cfg->n_layers || max_pages <= 0) return KVP_ERR_ARG;
    if (!q || !table || !lens || !out || !ws || (base_out == nullptr) != (base_lse == nullptr)) return KVP_ERR_ARG;
    if (!std::isfinite(scale)) return KVP_ERR_ARG;
    if (!aligned(pages, 256) || !aligned(q, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(base_out, 16) ||
        !aligned(base_lse, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16))
        return KVP_ERR_ALIGN;
    const AttendWs w = attend_ws(cfg, n_seqs, n_q_tokens, n_q_heads);
    if (ws_bytes < w.total) return KVP_ERR_SIZE;
    // unit counts are 32-bit
    const unsigned __int128 blocks = (unsigned __int128)uint32_t(max_pages) * uint32_t(cfg->page_tokens / 16) * uint32_t(n_seqs);
    if (blocks >> 31) return KVP_ERR_SIZE;
    if (n_seqs == 0) return KVP_OK;
    PagesAttendArgs a;
    a.pv = pages_view(const_cast<void *>(pages), *cfg, layer);
    a.q = static_cast<const uint16_t *>(q);
    a.table = table, a.lens = lens, a.base_out = base_out, a.base_lse = base_lse;
    a.out = static_cast<uint16_t *>(out), a.lse = lse;
    a.plan = static_cast<uint32_t *>(ws);
    a.stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + w.stats);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.part);
    a.scale2 = scale * 1.4426950408889634f;
    a.nseq = n_seqs, a.m = n_q_tokens, a.nq = n_q_heads, a.G = n_q_heads / cfg->n_kv_heads;
    a.R = n_q_tokens * a.G;
    const int rows = tile_rows(a.R, cfg->format);
    a.RT = (a.R + rows - 1) / rows;
    a.max_pages = max_pages;
    a.polls = g_limit_next ? g_next_polls : PAT_WAIT_LIMIT;
    a.poll_lanes = g_limit_next ? g_next_lanes : 0xFFFFFFFFu;
    g_limit_next = false;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool d128 = cfg->head_dim == 128;
    switch (cfg->format) {
        case KVP_PAGES_BF16:
            return d128 ? launch_attend<128, KVP_PAGES_BF16>(a, rows, st) : launch_attend<64, KVP_PAGES_BF16>(a, rows, st);
        case KVP_PAGES_K8V8:
            return d128 ? launch_attend<128, KVP_PAGES_K8V8>(a, rows, st) : launch_attend<64, KVP_PAGES_K8V8>(a, rows, st);
        default:
            return d128 ? launch_attend<128, KVP_PAGES_K8V4>(a, rows, st) : launch_attend<64, KVP_PAGES_K8V4>(a, rows, st);
    }
}

}  // extern "C"
