// kvprompt.cu -- attention of whole prompts: every token of several sequences' new
// tokens over its own sequence's keys and values, causal, with a window and first
// tokens that stay visible, joined with attention over other tokens.
//
// For sequence b with n_b new tokens and T_b keys, new token i is at place
// p = T_b - n_b + i and sees t <= p, with a window w only t > p - w or t < z:
//   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
// joined: L = log(e^lse + e^base_lse), out = e^(lse-L) out + e^(base_lse-L) base.
// Exponentials are base 2 throughout.
//
// Bound: the tensor cores, 4 d multiply-adds for a query row and a key that it sees.
//
// A block takes 256 query rows of one KV head as two halves of 128: the heads of a
// group side by side (row = token * G + head), so that grouped heads share every
// key and value that is brought in, and goes through the keys that any of its rows
// sees, 128 at a time: first the first tokens, then the window's.  Products on
// tcgen05, 128 x 128 (x d) tiles, everything but keys and values staying on the SM:
//   S = Q K^T   operands in shared memory, S in TMEM (128 columns a half)
//   O += P V    P as bf16 in TMEM over the first half of S's columns, O in TMEM
// Warps 0-3 and 4-7 do the softmax of a half each, a thread a row (no shuffles), and
// write its result; warp 8 issues the products; warp 9 finds the work and brings
// queries, keys and values (TMA, 128-byte swizzle, a ring of tiles); warp 10 looks after
// the values.  While one half's softmax runs the tensor core has the other's products.
// A half's tile is a chain: scores, softmax (some 1200 cycles, its exponentials 512 of
// them), values, next scores (1030 cycles of products, of 2060 for both halves); with
// the handovers 2630 cycles measured a tile, 78 % of the products' rate.
//
// A row's reference (its largest score so far) is raised only when a score passes it
// by 2^8, so that O is hardly ever rescaled; weights are taken relative to 2^40 times
// the reference, so that sums of up to 2^30 values up to bf16's largest stay finite.
// A weight's exponent is one multiply-add of a product x = q . k, scale x - (reference + 40).
// The reference is a rounded product there, the multiply-add's own is not, and the sum with
// 40 is rounded: from scores of some 2^31 on either is off by as much as exponents reach.  So
// rows keep their largest x, and from references of 2^12 on (whose last bit is 2^-11) it is
// subtracted first: scale (x - x_largest) - 40.
// Weights are rounded to bf16 for the value product (2^-8 at most, of either sign; the
// sum takes them before that): a second product for the rest of them would cost
// a quarter of the tensor time for no more than the result's own rounding to bf16.
//
// Values that some of the rows do not see must not meet them in the product, not even
// with weight 0, if they are Inf or NaN.  Rows of a tile that nobody sees are zeroed in
// shared memory.  Tiles that only some of the rows see whole are looked over (a block has a
// few of them, however long the sequence): Inf and NaN there are zeros to the product, and
// are added to the results of the rows that do see them.
//
// Measured (32 query over 8 KV heads of 128; cuBLAS reaches 1895 TFLOP/s): 16384 tokens
// 1.25 ms, 1760 TFLOP/s, at first (1.34 ms in a graph that runs for a tenth of a second, where the
// power limit lowers the clock); 8192 tokens with a window of 1024 and 4 first tokens 120 us, 1080
// TFLOP/s of what is seen: products of 9.25 tiles where a row sees 8, and a block's start and end, as
// long as 4; 509 tokens over 32768 in two parts 189 us (209 under the power limit).  32 heads of 64,
// window 256, 17 first tokens, 7 ragged prompts of 37 to 1851: 68 us.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda.h>

#include "kvp_async.cuh"
#include "kvp_internal.cuh"

namespace kvp {

constexpr int PT_KEYS = 128;                  // keys of a tile
// Three warpgroups: 384 threads start with 168 registers each (64512 of the SM's), the third
// gives 80 of its back and each of the others takes 40 more: 2 * 128 * 208 + 128 * 88 = 64512.
constexpr int PT_THREADS = 384, PT_MORE = 208, PT_LESS = 88;
// First tokens that a narrow tile holds.  Without it, 4 of them cost a window of 1024 a fifteenth (8192
// tokens: 120 us, 128).
constexpr int PT_FEW = 32;
constexpr int PT_MOST = 1 << 30;              // rows: sums and differences of places fit 32 bits
constexpr uint32_t PT_WAIT_LIMIT = WAIT_POLLS;
// Block numbers without work, one after the other, after which the other warps are given an empty
// piece of work, so that their waits begin anew (a number takes 1.2 us).
constexpr uint32_t PT_IDLE = 4096;
// (Rows with references beyond PT_FAR take longer: 16384 tokens 1.55 ms, 1.31.)
constexpr float PT_SLACK = 8.0f, PT_BIAS = 40.0f, PT_FAR = 4096.0f;

struct PromptArgs {
    CUtensorMap q_map, k_map, v_map;
    const uint16_t *v;
    int64_t v_ts, v_hs;  // strides in elements
    const int32_t *q_first, *k_first, *k_lens;
    const float *base_out, *base_lse;
    uint16_t *out;
    float *lse;
    uint32_t *error;
    float *part;    // [splits][n nq][d] sums of weighted values
    float2 *stats;  // [splits][n nq] (reference, sum)
    float scale2;   // |scale| * log2(e); 1 for a scale of 0, whose scores are set to 0
    int nseq, n, nk, nq, H, G, window, sinks;
    int half_tokens;  // tokens of a half: 128 / G
    int tiles, splits;
    uint32_t negative, flat;  // the scale's sign; whether it is 0
    uint32_t sectors;         // whether out and the workspace lie on 32-byte boundaries
    uint32_t polls;           // of a copy, by the warp that issues products
};

__device__ __forceinline__ void prompt_flag(const PromptArgs &a, uint32_t f) {
    if (a.error) atomicOr(a.error, f);
}

// A sequence's new tokens and keys; n = 0 where its numbers lie outside the tensors.
struct PromptSeq {
    int first, n, k_first, T;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs &a, int b, bool flag) {
    PromptSeq s;
    s.first = int(ld_plain_u32(a.q_first + b));
    const int end = int(ld_plain_u32(a.q_first + b + 1));
    s.k_first = int(ld_plain_u32(a.k_first + b)), s.T = int(ld_plain_u32(a.k_lens + b));
    s.n = int(uint32_t(end) - uint32_t(s.first));
    if (s.first < 0 || end < s.first || end > a.n || s.k_first < 0 || s.T < 0 || int64_t(s.k_first) + s.T > a.nk) {
        if (flag) prompt_flag(a, FLAG_PAGE);
        s.n = 0;
    }
    return s;
}

// The log of a row's sum of exponentials, from its sum in units of 2^(ref + PT_BIAS).
__device__ __forceinline__ float row_lse(float ref, float sum) {
    return sum > 0.0f ? (ref + log2f(sum * 0x1p40f)) * 0.69314718055994531f : (sum == 0.0f ? -INFINITY : sum);
}

// N runs of 32 bytes to one place after the other; `whole`: it lies on a sector's boundary.
template <int N>
__device__ __forceinline__ void st_sectors(void *to, const uint32_t *v, uint32_t whole) {
    uint8_t *p = static_cast<uint8_t *>(to);
    if (whole) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                         ::"l"(p + 32 * k), "r"(v[8 * k]), "r"(v[8 * k + 1]), "r"(v[8 * k + 2]), "r"(v[8 * k + 3]), "r"(v[8 * k + 4]),
                           "r"(v[8 * k + 5]), "r"(v[8 * k + 6]), "r"(v[8 * k + 7]) : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 2 * N; ++k)
            *reinterpret_cast<uint4 *>(p + 16 * k) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
}

// A finite mean of bf16 values is not beyond bf16's largest (the rounded weights' sum
// may be, by 2^-8).
__device__ __forceinline__ float within_bf16(float y) {
    constexpr float MOST = 3.3895313892515355e38f;
    return fabsf(y) < INFINITY ? fminf(fmaxf(y, -MOST), MOST) : y;
}

// What a row ends with: the weights of its own result (already divided by its sum)
// and of the base, and its lse (written by one of those who call this).  bl: base_lse[row],
// which may be lse[row] and has been read by all of them.
__device__ __forceinline__ float2 prompt_join(const PromptArgs &a, uint64_t row, float lse, float bl, bool writes) {
    float wa = 1.0f, wb = 0.0f;
    if (a.base_lse) {
        if (!(lse == -INFINITY && bl == -INFINITY)) {
            const float top = fmaxf(lse, bl);
            const float ea = expf(lse - top), eb = expf(bl - top), tot = ea + eb;
            wa = ea / tot, wb = eb / tot;
            lse = top + logf(tot);
        }
    }
    if (writes && a.lse) a.lse[row] = lse;
    return make_float2(wa, wb);
}

// A row's end by a warp: lane l has dims l d/32 ...; acc and sum are in units of
// 2^(ref + PT_BIAS).
template <int D>
__device__ __forceinline__ void prompt_write(const PromptArgs &a, uint64_t row, float ref, float sum, const float (&acc)[D / 32], int lane) {
    constexpr int VPL = D / 32;
    const float bl = a.base_lse ? a.base_lse[row] : -INFINITY;
    __syncwarp();  // every lane has it before one writes lse
    const float2 f = prompt_join(a, row, row_lse(ref, sum), bl, lane == 0);
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float y = within_bf16(acc[i] * inv) * f.x;
        if (a.base_out && f.y != 0.0f) y = fmaf(f.y, a.base_out[row * D + lane * VPL + i], y);
        reinterpret_cast<__nv_bfloat16 *>(a.out)[row * D + lane * VPL + i] = __float2bfloat16_rn(y);
    }
}

// ---------------------------------------------------------------------------
// tcgen05 and TMA.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_g2s(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
#define KVP_R8(x, i) "=r"((x)[(i)]), "=r"((x)[(i) + 1]), "=r"((x)[(i) + 2]), "=r"((x)[(i) + 3]), "=r"((x)[(i) + 4]), \
                     "=r"((x)[(i) + 5]), "=r"((x)[(i) + 6]), "=r"((x)[(i) + 7])
#define KVP_I8(x, i) "r"((x)[(i)]), "r"((x)[(i) + 1]), "r"((x)[(i) + 2]), "r"((x)[(i) + 3]), "r"((x)[(i) + 4]), \
                     "r"((x)[(i) + 5]), "r"((x)[(i) + 6]), "r"((x)[(i) + 7])
// 32 columns of the thread's TMEM lane.
__device__ __forceinline__ void tc_ld32(uint32_t at, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : KVP_R8(x, 0), KVP_R8(x, 8), KVP_R8(x, 16), KVP_R8(x, 24) : "r"(at));
}
__device__ __forceinline__ void tc_st32(uint32_t at, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::KVP_I8(x, 0), KVP_I8(x, 8), KVP_I8(x, 16), KVP_I8(x, 24), "r"(at) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t *x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 ::KVP_I8(x, 0), KVP_I8(x, 8), "r"(at) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// (the registers of a load are its results only once it has been waited for)
__device__ __forceinline__ void tc_landed(uint32_t *x) {
    asm volatile("" : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                      "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])
                 :: "memory");
}
__device__ __forceinline__ float pt_exp2(float x) {  // results under 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One lane of a whole warp.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0u;
}

// Two bf16, with zeros for Inf and NaN.
__device__ __forceinline__ uint32_t finite_halves(uint32_t v) {
    const uint32_t lo = (v & 0x7F80u) == 0x7F80u ? 0u : v & 0xFFFFu, hi = (v & 0x7F800000u) == 0x7F800000u ? 0u : v & 0xFFFF0000u;
    return lo | hi;
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
    uint32_t r;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// A shared-memory operand in rows of 128 bytes under the 128-byte swizzle: groups of 8
// rows are 1024 bytes apart (lbo: from one 64-element column of rows to the next, for
// the operand whose rows run along the sum).
__device__ __forceinline__ uint64_t tc_operand(uint32_t at, uint32_t lbo) {
    return uint64_t((at & 0x3FFFFu) >> 4) | uint64_t(lbo >> 4) << 16 | uint64_t(1024u >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// bf16 x bf16 -> fp32, 128 x n.
__device__ __forceinline__ constexpr uint32_t tc_kind(uint32_t n) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (n >> 3) << 17 | (128u >> 4) << 24;
}
constexpr uint32_t TC_NEGATE_A = 1u << 13, TC_B_BY_ROWS = 1u << 16;

template <int D>
struct PromptTile {
    static constexpr uint32_t BYTES = 128u * D * 2u;   // of 128 rows of queries, keys or values
    static constexpr uint32_t CHUNK = 128u * 128u;     // 64 dims of them
    static constexpr uint32_t SLOTS = D == 128 ? 4 : 6;
    static constexpr uint32_t OFF_Q = 1024, OFF_RING = OFF_Q + 2 * BYTES;
    static constexpr uint32_t SMEM = OFF_RING + SLOTS * BYTES + 1024;  // and the base's alignment
    static_assert(SMEM <= 232448, "shared memory of a block");
    // barriers, 8 bytes each, and what else lies before the queries
    static constexpr uint32_t FULL = 0, FREE = 64, Q = 128, QFREE = 136, S = 144, P = 160, O = 176, DONE = 192, WORK = 200,
                              READ = 216, NEXT = 232, TMEM = 240, DEAD = 244, ANSWER = 256, ODD = 272,
                              ITEM = 320;
};

// A piece of work: 256 rows (or fewer) of one sequence and KV head, and the keys that some
// of them see: [0, a_end) and [b0, b_end), in tiles, of which tiles j0 .. j0 + nt - 1.
struct alignas(16) PromptWork {
    int valid, split, h;
    int row, count;      // first row of q, tokens
    int k_first;         // first row of k and v
    int p_first;         // place of the first token (below 0: before the first key)
    int a_end, b0, b_end, na, j0, nt;
    int unused[3];

    __device__ __forceinline__ int p_last() const { return p_first + count - 1; }
    // Whether the first tile holds a few first tokens only: PT_FEW columns of it do then.  (They
    // lie before every row's window, so that all rows see them.)
    __device__ __forceinline__ bool few() const { return na == 1 && a_end <= PT_FEW && j0 == 0 && nt > 0; }
    __device__ __forceinline__ void tile(int j, int &t0, int &end) const {
        j += j0;
        if (j < na)
            t0 = j * PT_KEYS, end = min(t0 + PT_KEYS, a_end);
        else
            t0 = b0 + (j - na) * PT_KEYS, end = min(t0 + PT_KEYS, b_end);
    }
    // Whether some row does not see all of the tile's tokens.
    __device__ __forceinline__ bool part_seen(const PromptArgs &a, int t0, int end) const {
        return end - 1 > p_first || (a.window && t0 <= p_last() - a.window && end > a.sinks);
    }
};
static_assert(sizeof(PromptWork) == 64, "four 16-byte loads");

// The work of a block number; false if it has none.  Sequence b has its tiles from number
// q_first[b] / tokens + b on: more numbers than tiles, but found without a sum.  (By a warp.)
__device__ __forceinline__ bool prompt_work(const PromptArgs &a, uint32_t block, PromptWork &w) {
    const int lane = threadIdx.x & 31, tokens = 2 * a.half_tokens;
    w.split = int(block % uint32_t(a.splits));
    w.h = int(block / uint32_t(a.splits) % uint32_t(a.H));
    const int slot = a.tiles - 1 - int(block / uint32_t(a.splits) / uint32_t(a.H));  // the last tokens first: of one prompt they see the most
    int lo = 0, hi = a.nseq - 1;  // the last b with its first tile at or before this one, 32 places at a time
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = min(lo + (lane + 1) * step, hi);
        const bool before = max(int(ld_plain_u32(a.q_first + at)), 0) / tokens + at <= slot;
        const int n = __popc(__ballot_sync(0xffffffffu, before));  // (a run of ones)
        const int nlo = n ? min(lo + n * step, hi) : lo, nhi = n < 32 ? min(lo + (n + 1) * step, hi) - 1 : hi;
        lo = nlo, hi = max(nlo, nhi);
    }
    const PromptSeq s = prompt_seq(a, lo, false);  // (prompt_report says what is wrong)
    const int64_t i0 = int64_t(slot - lo - max(s.first, 0) / tokens) * tokens;
    if (i0 < 0 || i0 >= s.n) return false;
    w.valid = 1;
    w.row = s.first + int(i0), w.count = min(tokens, s.n - int(i0));
    w.k_first = s.k_first;
    w.p_first = s.T - s.n + int(i0);
    auto tiles_of = [](int n) { return (n + PT_KEYS - 1) / PT_KEYS; };
    w.b_end = max(w.p_last() + 1, 0), w.b0 = a.window ? max(w.p_first - a.window + 1, 0) : 0;
    w.a_end = min(a.sinks, w.b0);
    // no more (whole) tiles without the gap: without it
    const int apart = tiles_of(w.b_end - w.b0) + (w.a_end > PT_FEW ? tiles_of(w.a_end) : 0);
    if (tiles_of(w.b_end) <= apart) w.a_end = 0, w.b0 = 0;
    w.na = tiles_of(w.a_end);
    const int all = w.na + tiles_of(w.b_end - w.b0);
    w.j0 = int(int64_t(all) * w.split / a.splits), w.nt = int(int64_t(all) * (w.split + 1) / a.splits) - w.j0;
    return true;
}

// Reports a sequence with numbers outside the tensors, or that decrease: block numbers are at least
// as many as sequences, and some of them have one each to look at (the search above need not meet
// a sequence whose numbers are out of order).
__device__ __forceinline__ void prompt_report(const PromptArgs &a, uint32_t block) {
    const uint32_t each = uint32_t(a.splits) * uint32_t(a.H);
    const int b = a.tiles - 1 - int(block / each);
    if (block % each == 0u && b < a.nseq) prompt_seq(a, b, true);
}

// Waits until the barrier's phase is over; gives up when the limit or another warp's
// wait has run out.
__device__ __forceinline__ bool pt_wait(const PromptArgs &a, uint32_t bar, uint32_t parity, uint32_t dead, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try(bar, parity)) return true;
        if (i >= 4096 && i % 64 == 0) {
            uint32_t d;
            asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(d) : "r"(dead) : "memory");
            if (d) return false;
            __nanosleep(64);
        }
    }
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(dead), "r"(1u) : "memory");
    prompt_flag(a, FLAG_TIMEOUT);
    return false;
}

// The same for a whole warp (one decision for all lanes).
__device__ __forceinline__ bool warp_wait(const PromptArgs &a, uint32_t bar, uint32_t parity, uint32_t dead) {
    return __all_sync(0xffffffffu, pt_wait(a, bar, parity, dead, PT_WAIT_LIMIT));
}

// The place of the n-th of a running number of tiles in a ring, and the parity of its round.
struct RingPlace {
    uint32_t at, parity;
};
template <uint32_t SLOTS>
__device__ __forceinline__ RingPlace ring_place(uint32_t n) {
    return {n % SLOTS, (n / SLOTS) & 1u};
}

template <int D>
__global__ void __launch_bounds__(PT_THREADS, 1) prompt_attend(const __grid_constant__ PromptArgs a) {
    using T = PromptTile<D>;
    extern __shared__ uint8_t sm_raw[];
    const uint32_t sm = (smem_addr(sm_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 3) {
        const CUtensorMap *map = tid == 0 ? &a.q_map : (tid == 1 ? &a.k_map : &a.v_map);
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }

    const uint32_t dead = sm + T::DEAD;
    if (warp == 9 && lane == 0) {
        for (uint32_t i = 0; i < T::SLOTS; ++i) mbar_init_n(sm + T::FULL + 8 * i, 1), mbar_init_n(sm + T::FREE + 8 * i, 1);
        mbar_init_n(sm + T::Q, 1), mbar_init_n(sm + T::QFREE, 1), mbar_init_n(sm + T::DONE, 1), mbar_init_n(sm + T::NEXT, 1);
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init_n(sm + T::S + 8 * i, 1), mbar_init_n(sm + T::O + 8 * i, 1);
            // an arrival a warp, and in the first half the one of those who see to the copies
            mbar_init_n(sm + T::P + 8 * i, i ? 4 : 5);
            mbar_init_n(sm + T::WORK + 8 * i, 1), mbar_init_n(sm + T::READ + 8 * i, 10);  // by warps 0-8 and 10
        }
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(dead), "r"(0u) : "memory");
        mbar_init_fence();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm + T::TMEM), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_before();
    }
    __syncthreads();
    tc_after();
    // what the kernel before this one writes is there from here on; the next one may be placed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // The k-th piece of this block's work, once it is there; false if there is none, or a wait
    // ran out.  (By a warp.)
    auto next_work = [&](uint32_t k, PromptWork &w) {
        const uint32_t at = k & 1u;
        // (a half that has no rows waits while the other works: 64 polls for each of its tiles)
        const uint32_t limit = PT_WAIT_LIMIT + (k ? 64u * uint32_t(w.nt) : 0u);
        if (!__all_sync(0xffffffffu, pt_wait(a, sm + T::WORK + 8 * at, (k >> 1) & 1u, dead, limit))) return false;
        uint32_t *to = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(to[4 * i]), "=r"(to[4 * i + 1]), "=r"(to[4 * i + 2]), "=r"(to[4 * i + 3])
                         : "r"(sm + T::ITEM + 64 * at + 16 * i) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(sm + T::READ + 8 * at);
        return w.valid != 0;
    };
    // (A block has all 512 columns of TMEM: they start at 0.  S, and over it P, at 128 half, O at
    // 256 + D half.  At head_dim 64 P has room beside S, and the next scores need then not wait for
    // its product; measured slower, 351 against 306 us on 8192 tokens: the softmax has one more
    // barrier, and it is what bounds that.)

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PT_LESS));
        if (warp == 9) {
            // --- work and copies.  A block's own number is its first work; then it takes over numbers
            // of blocks that have not begun (cluster launch control), one at a time, when the copies
            // of what it has are all under way: that leaves the others their share, and the next
            // queries, keys and values come while the last tiles and results are worked on.
            uint32_t block = blockIdx.x, k = 0, n = 0, queries = 0, asked = 0, idle = 0;
            bool ok = true, more = true;
            while (ok) {
                PromptWork w = {};
                if (more && !prompt_work(a, block, w)) w.valid = ++idle % PT_IDLE == 0u;
                if (w.valid || !more) {
                    const uint32_t at = k & 1u;
                    if (k >= 2 && !(ok = warp_wait(a, sm + T::READ + 8 * at, ((k >> 1) - 1u) & 1u, dead))) break;
                    if (lane == 0) {
                        const uint32_t *from = reinterpret_cast<const uint32_t *>(&w);
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                         ::"r"(sm + T::ITEM + 64 * at + 16 * i), "r"(from[4 * i]), "r"(from[4 * i + 1]),
                                           "r"(from[4 * i + 2]), "r"(from[4 * i + 3]) : "memory");
                        mbar_arrive(sm + T::WORK + 8 * at);
                    }
                    __syncwarp();
                    ++k;
                    if (!more) break;
                }
                if (w.valid && w.nt > 0) {
                    const int halves = w.count > a.half_tokens ? 2 : 1;
                    if (queries > 0 && !(ok = warp_wait(a, sm + T::QFREE, (queries - 1u) & 1u, dead))) break;
                    if (lane == 0) {
                        mbar_expect_tx(sm + T::Q, uint32_t(halves) * uint32_t(a.half_tokens) * uint32_t(a.G) * D * 2u);
                        for (int half = 0; half < halves; ++half)
                            for (int c = 0; c < D / 64; ++c)
                                tma_g2s(sm + T::OFF_Q + uint32_t(half) * T::BYTES + uint32_t(c) * T::CHUNK, &a.q_map, 64 * c,
                                        w.h * a.G, w.row + half * a.half_tokens, sm + T::Q);
                    }
                    ++queries;
                    for (int c = 0; c < 2 * w.nt; ++c, ++n) {  // K_0 V_0 K_1 V_1 ... round the ring
                        const RingPlace to = ring_place<T::SLOTS>(n);
                        if (n >= T::SLOTS && !(ok = warp_wait(a, sm + T::FREE + 8 * to.at, to.parity ^ 1u, dead))) break;
                        if (lane == 0) {
                            int t0, end;
                            w.tile(c / 2, t0, end);
                            mbar_expect_tx(sm + T::FULL + 8 * to.at, T::BYTES);
                            for (int e = 0; e < D / 64; ++e)
                                tma_g2s(sm + T::OFF_RING + to.at * T::BYTES + uint32_t(e) * T::CHUNK, c & 1 ? &a.v_map : &a.k_map,
                                        64 * e, w.h, w.k_first + t0, sm + T::FULL + 8 * to.at);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                // the next number
                if (lane == 0) {
                    mbar_expect_tx(sm + T::NEXT, 16);
                    fence_proxy_async();  // the former answer has been read
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                 ::"r"(sm + T::ANSWER), "r"(sm + T::NEXT) : "memory");
                    prompt_report(a, block);
                }
                __syncwarp();
                ++asked;
                if (!(ok = warp_wait(a, sm + T::NEXT, (asked - 1u) & 1u, dead))) break;
                uint32_t got;
                asm volatile(
                    "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
                    "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                    "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                    "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
                    : "=r"(got), "=r"(block) : "r"(sm + T::ANSWER) : "memory");
                __syncwarp();
                more = got != 0u;
            }
            // whoever gave up: what is in flight lands before the block ends
            if (lane == 0) {
                for (uint32_t i = n > T::SLOTS ? n - T::SLOTS : 0; i < n; ++i)
                    mbar_wait(sm + T::FULL + 8 * (i % T::SLOTS), (i / T::SLOTS) & 1u, PT_WAIT_LIMIT);
                if (queries) mbar_wait(sm + T::Q, (queries - 1u) & 1u, PT_WAIT_LIMIT);
                if (asked) mbar_wait(sm + T::NEXT, (asked - 1u) & 1u, PT_WAIT_LIMIT);
            }
            __syncwarp();
        } else if (warp == 8) {
            // --- products.  The whole warp goes through the loop, with numbers that are the same
            // in all lanes as far as the compiler can see, and one lane issues: the operands' descriptors
            // are then formed in uniform registers.  (In a branch of one lane each product costs 130
            // cycles instead of 65.)
            const uint32_t kind_s = tc_kind(128) | (a.negative ? TC_NEGATE_A : 0u), kind_o = tc_kind(D) | TC_B_BY_ROWS;
            const uint32_t kind_few = tc_kind(PT_FEW) | (a.negative ? TC_NEGATE_A : 0u);
            auto scores = [&](uint32_t half, uint32_t at, uint32_t kind) {  // S = Q K^T
                const uint64_t qd = tc_operand(sm + T::OFF_Q + half * T::BYTES, 16);
                const uint64_t kd = tc_operand(sm + T::OFF_RING + at * T::BYTES, 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = uint64_t((uint32_t(k / 4) * T::CHUNK + uint32_t(k % 4) * 32u) >> 4);
                    tc_mma_ss(half * 128u, qd + off, kd + off, kind, k > 0);
                }
                tc_commit(sm + T::S + 8 * half);
            };
            auto values = [&](uint32_t half, uint32_t at, bool add, bool few) {  // O += P V
                const uint64_t vd = tc_operand(sm + T::OFF_RING + at * T::BYTES, T::CHUNK);
#pragma unroll
                for (int k = 0; k < PT_KEYS / 16; ++k)
                    if (k < PT_FEW / 16 || !few) tc_mma_ts(256u + half * D, half * 128u + 8u * uint32_t(k), vd + uint64_t(k * 2048 >> 4), kind_o, add || k > 0);
            };
            auto wait = [&](uint32_t bar, uint32_t parity, uint32_t limit) {
                const bool ok = __all_sync(0xffffffffu, pt_wait(a, sm + bar, parity, dead, limit));
                tc_after();
                return ok;
            };
            bool ok = true;
            uint32_t at = 0, round = 0;                           // the next tile's place in the ring, its round's parity
            uint32_t queries = 0, done0 = 0, done1 = 0;           // parities of the queries and of the halves' tiles
            auto forward = [&]() {
                if (++at == T::SLOTS) at = 0, round ^= 1u;
            };
            PromptWork w;
            for (uint32_t k = 0; next_work(k, w); ++k) {
                const int tiles = __shfl_sync(0xffffffffu, w.nt, 0);
                const bool two = __shfl_sync(0xffffffffu, w.count, 0) > a.half_tokens;
                const bool few = __shfl_sync(0xffffffffu, int(w.few()), 0) != 0;
                if (tiles == 0) continue;
                if (!(ok = wait(T::Q, queries, PT_WAIT_LIMIT) && wait(T::FULL + 8 * at, round, a.polls))) break;
                queries ^= 1u;
                if (elect()) {
                    scores(0, at, few ? kind_few : kind_s);
                    if (two) scores(1, at, few ? kind_few : kind_s);
                    tc_commit(sm + T::FREE + 8 * at);
                    if (tiles == 1) tc_commit(sm + T::QFREE);
                }
                __syncwarp();
                forward();
                for (int j = 0; j < tiles; ++j) {
                    const bool more = j + 1 < tiles, last_scores = j + 2 == tiles;
                    const uint32_t v_at = at;
                    forward();
                    const uint32_t k_at = at;  // (of the next tile, if there is one)
                    if (!(ok = wait(T::P, done0, PT_WAIT_LIMIT))) break;
                    if (elect()) {
                        values(0, v_at, j > 0, few && j == 0);
                        if (!two) tc_commit(sm + T::FREE + 8 * v_at);
                        if (more) {
                            scores(0, k_at, kind_s);
                            if (!two) {
                                tc_commit(sm + T::FREE + 8 * k_at);
                                if (last_scores) tc_commit(sm + T::QFREE);
                            }
                        } else {
                            tc_commit(sm + T::O);
                        }
                    }
                    __syncwarp();
                    done0 ^= 1u;
                    if (two) {
                        if (!(ok = wait(T::P + 8, done1, PT_WAIT_LIMIT))) break;
                        if (elect()) {
                            values(1, v_at, j > 0, few && j == 0);
                            tc_commit(sm + T::FREE + 8 * v_at);
                            if (more) {
                                scores(1, k_at, kind_s);
                                tc_commit(sm + T::FREE + 8 * k_at);
                                if (last_scores) tc_commit(sm + T::QFREE);
                            } else {
                                tc_commit(sm + T::O + 8);
                            }
                        }
                        __syncwarp();
                        done1 ^= 1u;
                    }
                    if (more) forward();
                }
                if (!ok) break;
            }
            // (a block that gave up: nothing may be in flight when TMEM is given back)
            if (elect()) tc_commit(sm + T::DONE);
            __syncwarp();
            mbar_wait(sm + T::DONE, 0, PT_WAIT_LIMIT);
            __syncwarp();
        } else if (warp == 10) {
            // --- what the products wait for beside the softmax, as one more arrival at the first
            // half's barrier: the copies of V_j and K_{j+1} (a wait costs the others some 100 cycles
            // even if there is nothing to wait for), and V_j in a state that no row can come to harm
            // by: rows of a tile that nobody sees are zeroed, and where some rows see a part only it
            // is looked over for Inf and NaN, whose product with a weight of 0 is NaN.
            uint32_t n = 0, done = 0;
            auto there = [&](uint32_t i) {
                const RingPlace of = ring_place<T::SLOTS>(i);
                return __all_sync(0xffffffffu, pt_wait(a, sm + T::FULL + 8 * of.at, of.parity, dead, a.polls));
            };
            PromptWork w;
            bool ok = true;
            for (uint32_t k = 0; ok && next_work(k, w); ++k) {
                // (the flag of four pieces of work before: the slowest reader is at most two behind)
                const uint32_t odd_at = sm + T::ODD + 4u * (k & 3u);
                if (lane == 0) asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(odd_at), "r"(0u) : "memory");
                for (int j = 0; j < w.nt; ++j, n += 2) {
                    const bool more = j + 1 < w.nt;
                    if (!(ok = there(n + 1))) break;
                    int t0, end;
                    w.tile(j, t0, end);
                    const int rows = end - t0;
                    const uint32_t tile = sm + T::OFF_RING + ring_place<T::SLOTS>(n + 1).at * T::BYTES;
                    constexpr int PER = D / 8, STEP = 32 / PER;  // 16-byte pieces of a row, rows of a pass
                    const int c = lane % PER;
                    const uint32_t mine = tile + uint32_t(c / 8) * T::CHUNK + uint32_t(c % 8) * 16u;  // (in whatever place of the row)
                    if (w.part_seen(a, t0, end)) {
                        __nv_bfloat162 odd[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) odd[e] = __float2bfloat162_rn(0.0f);
#pragma unroll 8
                        for (int row = lane / PER; row < PT_KEYS; row += STEP) {
                            uint32_t v[4] = {0u, 0u, 0u, 0u};
                            if (row < rows)
                                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(mine + uint32_t(row) * 128u) : "memory");
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                odd[e] = __hfma2(*reinterpret_cast<__nv_bfloat162 *>(&v[e]), __float2bfloat162_rn(0.0f), odd[e]);
                        }
                        odd[0] = __hadd2(__hadd2(odd[0], odd[1]), __hadd2(odd[2], odd[3]));
                        const bool bad = (*reinterpret_cast<uint32_t *>(&odd[0]) & 0x7FFF7FFFu) != 0u;
                        if (__any_sync(0xffffffffu, bad)) {
                            if (bad) {
                                asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(odd_at), "r"(1u) : "memory");
                                for (int row = lane / PER; row < rows; row += STEP)
#pragma unroll
                                    for (uint32_t e = 0; e < 4; ++e) {
                                        const uint32_t at = mine + uint32_t(row) * 128u + 4u * e;
                                        uint32_t v;
                                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(finite_halves(v)) : "memory");
                                    }
                            }
                            fence_proxy_async();
                        }
                    }
                    const int used = w.few() && j == 0 ? PT_FEW : PT_KEYS;  // rows that enter the product
                    if (rows < used) {
                        for (int row = rows + lane / PER; row < used; row += STEP)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(mine + uint32_t(row) * 128u), "r"(0u) : "memory");
                        fence_proxy_async();
                    }
                    if (more && !(ok = there(n + 2))) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sm + T::P);
                    if (!(ok = warp_wait(a, sm + T::P, done, dead))) break;
                    done ^= 1u;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PT_MORE));
        // --- softmax: a thread a row
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // the warp's 32 lanes of TMEM
        const uint32_t s_at = uint32_t(half) * 128u + lanes, o_at = 256u + uint32_t(half) * D + lanes;
        const int tl = r / a.G, i = half * a.half_tokens + tl;  // the row's token
        bool ok = true;
        uint32_t done = 0, ended = 0;  // parities of the half's tiles and results
        PromptWork w;
        // Whether any thread of the half says so.  What ends a half's work is decided by all of its
        // warps: one that gave up by itself would be missing from the others' barriers.
        auto any_of_half = [&](bool says) {
            uint32_t any;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n}"
                         : "=r"(any) : "r"(uint32_t(says)), "r"(1 + half) : "memory");
            return any != 0u;
        };
        for (uint32_t k = 0; !any_of_half(!ok || !next_work(k, w)); ++k) {
            if (half == 1 && w.count <= a.half_tokens) continue;
            const bool real = tl < a.half_tokens && i < w.count;
            const int p = w.p_first + (real ? i : w.count - 1);
            float raw = -INFINITY, sum = 0.0f;  // the reference, over the scale
            // What is added to a score for a weight's exponent; whether the reference is far from 0.
            auto offset = [&]() { return -(raw == -INFINITY ? 0.0f : raw * a.scale2) - PT_BIAS; };
            auto is_far = [&]() { return real && raw > -INFINITY && fabsf(raw * a.scale2) >= PT_FAR; };
            // Tiles [in0, in1) are seen whole by all rows: nothing to hide.
            const int in0 = w.na - w.j0 + (a.window ? (max(w.p_last() - a.window + 1 - w.b0, 0) + PT_KEYS - 1) / PT_KEYS : 0);
            const int in1 = w.na - w.j0 + max(w.p_first + 1 - w.b0, 0) / PT_KEYS;
            int j = 0;
            float bar = -INFINITY;  // passed by a score that needs a look at the reference (by all, of a far one)
            if (w.few()) {
                if ((ok = warp_wait(a, sm + T::S + 8 * uint32_t(half), done, dead))) {
                    tc_after();
                    uint32_t x[32];
                    float *xf = reinterpret_cast<float *>(x);
                    tc_ld32(s_at, x);
                    tc_wait_ld();
                    tc_landed(x), tc_landed(x + 16);
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        xf[c] = c < w.a_end ? (a.flat ? 0.0f : xf[c]) : -INFINITY;
                        top = fmaxf(top, xf[c]);
                    }
                    raw = top;
                    float off = offset();
                    bar = is_far() ? -INFINITY : raw * a.scale2 + PT_SLACK;
                    if (__any_sync(0xffffffffu, is_far())) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) xf[c] -= raw == -INFINITY ? 0.0f : raw;
                        off = -PT_BIAS;
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float y0 = pt_exp2(fmaf(xf[2 * c], a.scale2, off)), y1 = pt_exp2(fmaf(xf[2 * c + 1], a.scale2, off));
                        sum += y0 + y1;
                        x[c] = pack_bf16x2(y0, y1);
                    }
                    tc_st16(s_at, x);
                    tc_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sm + T::P + 8 * uint32_t(half));
                    done ^= 1u;
                }
                j = 1;
            }
            for (; ok && j < w.nt; ++j) {
                const bool inner = j >= in0 && j < in1 && !a.flat;
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // the columns that the row sees, as bits
                if (!inner) {
                    int t0, end;
                    w.tile(j, t0, end);
                    const int last = min(end - 1, p) - t0, from = a.window ? p - a.window + 1 - t0 : 0, first = a.sinks - t0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) see[c] = bits_below(last + 1 - 32 * c) & (~bits_below(from - 32 * c) | bits_below(first - 32 * c));
                }
                if (!warp_wait(a, sm + T::S + 8 * uint32_t(half), done, dead)) {
                    ok = false;
                    break;
                }
                tc_after();
                uint32_t x[128];
                float *xf = reinterpret_cast<float *>(x);
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(s_at + 32u * uint32_t(c), x + 32 * c);
                float off = offset();
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) tc_landed(x + 16 * c);
                if (!inner) {
                    if (a.flat) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) xf[c] = 0.0f;
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        if (__all_sync(0xffffffffu, see[w] == 0xFFFFFFFFu)) continue;
#pragma unroll
                        for (int c = 32 * w; c < 32 * w + 32; ++c) xf[c] = see[w] & (1u << (c & 31)) ? xf[c] : -INFINITY;
                    }
                }
                float m[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) m[c] = fmaxf(xf[2 * c], xf[2 * c + 1]);
#pragma unroll
                for (int c = 4; c < 64; ++c) m[c & 3] = max3(m[c & 3], xf[2 * c], xf[2 * c + 1]);
                const float most = fmaxf(max3(m[0], m[1], m[2]), m[3]), top = most * a.scale2;
                if (__any_sync(0xffffffffu, top > bar)) {
                    const bool raise = top > bar && (most - raw) * a.scale2 > PT_SLACK;
                    const float f = raise ? pt_exp2((raw - most) * a.scale2) : 1.0f;
                    if (raise) raw = most;
                    off = offset();
                    bar = is_far() ? -INFINITY : raw * a.scale2 + PT_SLACK;
                    sum *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tc_ld32(o_at + uint32_t(c), o);
                            tc_wait_ld();
                            tc_landed(o), tc_landed(o + 16);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st32(o_at + uint32_t(c), o);
                        }
                    }
                    if (__any_sync(0xffffffffu, is_far())) {
                        const float less = raw == -INFINITY ? 0.0f : -raw;
#pragma unroll
                        for (int c = 0; c < 128; c += 2) {
                            const float2 y = __fadd2_rn(make_float2(xf[c], xf[c + 1]), make_float2(less, less));
                            xf[c] = y.x, xf[c + 1] = y.y;
                        }
                        off = -PT_BIAS;
                    }
                }
                float2 t0 = make_float2(sum, 0.0f), t1 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int c = 32 * u; c < 32 * u + 32; ++c) {
                        const float2 e = __ffma2_rn(make_float2(xf[2 * c], xf[2 * c + 1]), make_float2(a.scale2, a.scale2),
                                                    make_float2(off, off));
                        const float2 y = make_float2(pt_exp2(e.x), pt_exp2(e.y));
                        (c & 1 ? t1 : t0) = __fadd2_rn(c & 1 ? t1 : t0, y);
                        x[c] = pack_bf16x2(y.x, y.y);
                    }
                    tc_st32(s_at + 32u * uint32_t(u), x + 32 * u);
                }
                tc_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm + T::P + 8 * uint32_t(half));
                sum = (t0.x + t0.y) + (t1.x + t1.y);
                done ^= 1u;
            }
            if (ok && w.nt > 0) {
                ok = warp_wait(a, sm + T::O + 8 * uint32_t(half), ended, dead);
                ended ^= 1u;
                tc_after();
            }
            uint32_t odd;  // whether there are Inf or NaN among values that some row does not see
            asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(odd) : "r"(sm + T::ODD + 4u * (k & 3u)) : "memory");
            if (ok && odd && w.nt > 0) {  // they were zeros to the product: to O of the rows that see them
                const uint16_t *vr = a.v + w.k_first * a.v_ts + w.h * a.v_hs;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc_ld32(o_at + uint32_t(c), o);
                    tc_wait_ld();
                    tc_landed(o), tc_landed(o + 16);
#pragma unroll 1
                    for (int j = 0; j < w.nt; ++j) {
                        if (j >= in0 && j < in1) {
                            j = in1 - 1;
                            continue;
                        }
                        int t0, end;
                        w.tile(j, t0, end);
                        if (!w.part_seen(a, t0, end)) continue;
#pragma unroll 1
                        for (int t = t0; t < end; ++t) {
                            const uint16_t *from = vr + t * a.v_ts + c;  // (the same of all lanes)
                            uint32_t v[16];
                            bool any = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint4 four = ld_l2_v4(from + 8 * e);
                                v[4 * e] = four.x, v[4 * e + 1] = four.y, v[4 * e + 2] = four.z, v[4 * e + 3] = four.w;
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) any |= finite_halves(v[e]) != v[e];
                            if (!any || t > p || (a.window && t <= p - a.window && t >= a.sinks)) continue;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint32_t x = v[e] - finite_halves(v[e]);  // Inf and NaN alone
                                o[2 * e] = __float_as_uint(__uint_as_float(o[2 * e]) + bf16_lo(x));
                                o[2 * e + 1] = __float_as_uint(__uint_as_float(o[2 * e + 1]) + bf16_hi(x));
                            }
                        }
                    }
                    __syncwarp();
                    tc_st32(o_at + uint32_t(c), o);
                }
                tc_wait_st();
            }
            if (ok) {
                const float ref = raw * a.scale2;
                const uint64_t row = uint64_t(w.row + i) * uint32_t(a.nq) + uint32_t(w.h * a.G + r - tl * a.G);
                // Each thread stores its own row, 32 bytes (a sector) at a time.  The code is short, as it
                // is met with once a block and has to be fetched for that.
                auto load = [&](int c, uint32_t *o) {
                    if (w.nt > 0) {
                        tc_ld32(o_at + uint32_t(c), o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                };
                if (a.splits == 1) {
                    float2 f = make_float2(1.0f, 0.0f);
                    uint32_t o[32];
                    load(0, o);
                    if (real) f = prompt_join(a, row, row_lse(ref, sum), a.base_lse ? a.base_lse[row] : -INFINITY, true);
                    const float inv = sum > 0.0f ? __frcp_rn(sum) : (sum == 0.0f ? 0.0f : sum);
                    const float *bo = real && a.base_out && f.y != 0.0f ? a.base_out + row * D : nullptr;
                    uint16_t *to = a.out + row * D;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float of[32];
                        tc_wait_ld();
                        tc_landed(o), tc_landed(o + 16);
                        float most = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            of[e] = __uint_as_float(o[e]) * inv, of[e + 1] = __uint_as_float(o[e + 1]) * inv;
                            most = max3(most, fabsf(of[e]), fabsf(of[e + 1]));
                        }
                        if (c + 32 < D) load(c + 32, o);
                        if (most > 3.3e38f) {  // near the end of bf16's range
#pragma unroll
                            for (int e = 0; e < 32; ++e) of[e] = within_bf16(of[e]);
                        }
                        if (bo) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 b4 = *reinterpret_cast<const float4 *>(bo + c + e);
                                of[e] = fmaf(f.y, b4.x, of[e] * f.x), of[e + 1] = fmaf(f.y, b4.y, of[e + 1] * f.x);
                                of[e + 2] = fmaf(f.y, b4.z, of[e + 2] * f.x), of[e + 3] = fmaf(f.y, b4.w, of[e + 3] * f.x);
                            }
                        }
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(of[2 * e], of[2 * e + 1]);
                        if (real) st_sectors<2>(to + c, v, a.sectors);
                        __syncwarp();
                    }
                } else {
                    const uint64_t at = uint64_t(w.split) * uint32_t(a.n) * uint32_t(a.nq) + row;
                    if (real) a.stats[at] = make_float2(ref, sum);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        load(c, o);
                        tc_wait_ld();
                        tc_landed(o), tc_landed(o + 16);
                        if (real) st_sectors<4>(a.part + at * D + c, o, a.sectors);
                        __syncwarp();
                    }
                }
            }
            __syncwarp();
        }
        tc_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(0u), "r"(512u));
    }
}

// The parts of rows whose keys several blocks had, a warp a row.
template <int D>
__global__ void __launch_bounds__(256) prompt_join_parts(const __grid_constant__ PromptArgs a) {
    constexpr int VPL = D / 32;
    const int lane = threadIdx.x & 31;
    const uint64_t rows = uint64_t(a.n) * uint32_t(a.nq);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint64_t row = uint64_t(blockIdx.x) * 8u + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int tok = int(row / uint32_t(a.nq));
    // rows of no sequence, or of one that was skipped, have no parts
    int lo = 0, hi = a.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (int(ld_plain_u32(a.q_first + mid)) <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    const PromptSeq s = prompt_seq(a, lo, false);
    if (tok < s.first || tok >= s.first + s.n) return;
    float M = -INFINITY, L = 0.0f, acc[VPL];
#pragma unroll
    for (int e = 0; e < VPL; ++e) acc[e] = 0.0f;
    for (int c = 0; c < a.splits; ++c) M = fmaxf(M, __uint_as_float(ld_plain_u32(&a.stats[c * rows + row].x)));
    for (int c = 0; c < a.splits; ++c) {
        const float2 st = a.stats[c * rows + row];
        if (st.x == -INFINITY && st.y == 0.0f) continue;  // an empty part
        const float f = exp2f(st.x - M);
        L = fmaf(f, st.y, L);
#pragma unroll
        for (int e = 0; e < VPL; ++e) acc[e] = fmaf(f, a.part[(c * rows + row) * D + lane * VPL + e], acc[e]);
    }
    prompt_write<D>(a, row, M, L, acc, lane);
}

static int prompt_ok(const kvp_prompt_shape *s) {
    if (!s) return KVP_ERR_ARG;
    if (s->n_seqs < 0 || s->n_q_tokens < 0 || s->n_k_tokens < 0 || s->n_q_heads <= 0 || s->n_kv_heads <= 0 ||
        s->n_q_heads % s->n_kv_heads != 0)
        return KVP_ERR_ARG;
    if (s->head_dim != 64 && s->head_dim != 128) return KVP_ERR_UNSUPPORTED_D;
    if (s->n_seqs > KVP_PROMPT_MAX_SEQS || s->n_q_heads > 65536 || s->n_q_heads / s->n_kv_heads > 128) return KVP_ERR_SIZE;
    if (int64_t(s->n_q_tokens) * s->n_q_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    if (s->n_q_tokens > PT_MOST || s->n_k_tokens > PT_MOST) return KVP_ERR_SIZE;
    return KVP_OK;
}

// Blocks: tiles of 256 rows (tokens times the heads of a group) for every KV head.
static int prompt_tokens(const kvp_prompt_shape *s) { return 2 * (128 / (s->n_q_heads / s->n_kv_heads)); }
static int64_t prompt_tiles(const kvp_prompt_shape *s) { return int64_t(s->n_q_tokens / prompt_tokens(s)) + s->n_seqs; }

// Where the blocks would leave SMs idle, the keys of each are cut into `splits` parts, joined by a
// second kernel.  The number is the one that is expected to take least, in tiles: rounds of the SMs,
// each a part's tiles and PT_START for its start and end, PT_MOVE for the way of a block's 256 rows of
// sums to memory and back; it has to gain a twentieth, and to do with PT_PARTS bytes.  A turn of 509
// tokens over 32768 (64 blocks): 195 us in 2 parts, 200 in 7 (three full rounds).
constexpr int PT_START = 5, PT_MOVE = 6, PT_MOST_SPLITS = 32;
constexpr uint64_t PT_PARTS = 256u << 20;
static int prompt_splits(const kvp_prompt_shape *s, int window, int sinks) {
    const int64_t blocks = prompt_tiles(s) * s->n_kv_heads, sms = sm_count();
    int64_t keys = s->n_k_tokens / std::max(1, s->n_seqs);
    if (window > 0) keys = std::min<int64_t>(keys, int64_t(window) + prompt_tokens(s) + std::min(sinks, PT_KEYS));
    const int64_t tiles = keys / PT_KEYS + 1;
    const uint64_t a_part_bytes = uint64_t(s->n_q_tokens) * uint64_t(s->n_q_heads) * uint64_t(s->head_dim * 4 + 8);
    int best = 1;
    int64_t least = 0;
    for (int n = 1; n <= PT_MOST_SPLITS && n <= tiles && (n == 1 || a_part_bytes * n <= PT_PARTS); ++n) {
        const int64_t rounds = (blocks * n + sms - 1) / sms, a_part = (tiles + n - 1) / n;
        const int64_t takes = rounds * (a_part + PT_START + (n > 1 ? PT_MOVE : 0));
        if (n == 1 || takes * (best == 1 ? 21 : 20) < least * 20) best = n, least = takes;
    }
    return best;
}
// Workspace: the parts' statistics and sums.
struct PromptSplit {
    uint64_t part, total;
};
static PromptSplit prompt_split(const kvp_prompt_shape *s, int splits) {
    PromptSplit w;
    const uint64_t rows = uint64_t(s->n_q_tokens) * uint64_t(s->n_q_heads) * uint64_t(splits > 1 ? splits : 0);
    w.part = align256(rows * 8u);
    w.total = std::max<uint64_t>(256, w.part + rows * uint64_t(s->head_dim) * 4u);
    return w;
}

// cuTensorMapEncodeTiled, from the driver that the runtime has loaded.
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
    static std::atomic<void *> found{nullptr};
    void *f = found.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// A rows tensor as a tensor map: boxes of 64 dims x `heads` x `tokens`.
static int rows_map(CUtensorMap *map, const kvp_rows *r, int tokens, int heads, int d, int box_heads, int box_tokens) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return KVP_ERR_CUDA;
    const cuuint64_t size[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(tokens)};
    // the stride of a single head or token says nothing
    const cuuint64_t stride[2] = {heads > 1 ? cuuint64_t(r->head_stride) * 2 : cuuint64_t(d) * 2,
                                  tokens > 1 ? cuuint64_t(r->token_stride) * 2 : cuuint64_t(d) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(r->ptr), size, stride, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? KVP_OK
               : KVP_ERR_ARG;
}

static thread_local uint32_t g_next_polls = 0;
static thread_local bool g_limit_next = false;

template <int D>
static int launch_prompt(const PromptArgs &a, unsigned grid, cudaStream_t st) {
    static bool ready[64] = {false};  // the opt-in to more than 48 KB, once per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVP_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        if (cudaFuncSetAttribute(prompt_attend<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(PromptTile<D>::SMEM)) !=
            cudaSuccess)
            return KVP_ERR_CUDA;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(PT_THREADS);
    cfg.dynamicSmemBytes = PromptTile<D>::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, prompt_attend<D>, a) != cudaSuccess) return KVP_ERR_CUDA;
    count_launch();
    if (a.splits > 1) {
        cfg.gridDim = dim3(unsigned((uint64_t(a.n) * uint64_t(a.nq) + 7) / 8));
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, prompt_join_parts<D>, a) != cudaSuccess) return KVP_ERR_CUDA;
        count_launch();
    }
    return launch_status();
}

static int rows_ok(const kvp_rows *r, int tokens, int heads) {
    if (!r || (!r->ptr && tokens > 0)) return KVP_ERR_ARG;
    if (!aligned(r->ptr, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return KVP_ERR_ALIGN;
    constexpr int64_t MOST = int64_t(1) << 38;  // elements: a copy's stride is below 2^40 bytes
    if ((tokens > 1 && (r->token_stride <= 0 || r->token_stride >= MOST)) ||
        (heads > 1 && (r->head_stride <= 0 || r->head_stride >= MOST)))
        return KVP_ERR_ARG;
    return KVP_OK;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvprompt_workspace_bytes(const kvp_prompt_shape *shape) {
    if (prompt_ok(shape) != KVP_OK) return 0;
    return size_t(prompt_split(shape, prompt_splits(shape, 0, 0)).total);
}

int kvprompt_attend(const kvp_prompt_shape *shape, const kvp_rows *q, const kvp_rows *k, const kvp_rows *v,
                    const int32_t *q_first, const int32_t *k_first, const int32_t *k_lens, float scale, int window,
                    int sinks, const float *base_out, const float *base_lse, void *out, float *lse, uint32_t *error,
                    void *ws, size_t ws_bytes, void *stream) {
    int rc = prompt_ok(shape);
    if (rc != KVP_OK) return rc;
    if (window < 0 || sinks < 0 || !std::isfinite(scale)) return KVP_ERR_ARG;
    if (!q_first || !k_first || !k_lens || !out || !ws || (base_out == nullptr) != (base_lse == nullptr)) return KVP_ERR_ARG;
    if ((rc = rows_ok(q, shape->n_q_tokens, shape->n_q_heads)) != KVP_OK) return rc;
    if ((rc = rows_ok(k, shape->n_k_tokens, shape->n_kv_heads)) != KVP_OK) return rc;
    if ((rc = rows_ok(v, shape->n_k_tokens, shape->n_kv_heads)) != KVP_OK) return rc;
    if (!aligned(q_first, 4) || !aligned(k_first, 4) || !aligned(k_lens, 4) || !aligned(base_out, 16) ||
        !aligned(base_lse, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(error, 4) || !aligned(ws, 16))
        return KVP_ERR_ALIGN;
    if (ws_bytes < kvprompt_workspace_bytes(shape)) return KVP_ERR_SIZE;
    if (shape->n_seqs == 0 || shape->n_q_tokens == 0) return KVP_OK;
    PromptArgs a;
    a.v = static_cast<const uint16_t *>(v->ptr), a.v_ts = v->token_stride, a.v_hs = v->head_stride;
    a.q_first = q_first, a.k_first = k_first, a.k_lens = k_lens;
    a.base_out = base_out, a.base_lse = base_lse;
    a.out = static_cast<uint16_t *>(out), a.lse = lse, a.error = error;
    a.negative = scale < 0.0f, a.flat = scale == 0.0f;
    a.scale2 = a.flat ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
    a.nseq = shape->n_seqs, a.n = shape->n_q_tokens, a.nk = shape->n_k_tokens;
    a.nq = shape->n_q_heads, a.H = shape->n_kv_heads, a.G = a.nq / a.H;
    a.window = std::min(window, PT_MOST), a.sinks = std::min(sinks, PT_MOST);  // (no more keys than that)
    a.half_tokens = 128 / a.G;
    a.splits = std::min(prompt_splits(shape, a.window, a.sinks), prompt_splits(shape, 0, 0));
    const PromptSplit w = prompt_split(shape, a.splits);
    a.stats = static_cast<float2 *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.part);
    const int64_t tiles = prompt_tiles(shape), grid = tiles * a.H * a.splits;
    if (grid >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    a.tiles = int(tiles);
    // (with no keys at all nothing is copied: the maps are those of the queries)
    const bool some = shape->n_k_tokens > 0;
    const int keys = some ? a.nk : a.n, heads = some ? a.H : a.nq;
    if ((rc = rows_map(&a.q_map, q, a.n, a.nq, shape->head_dim, a.G, a.half_tokens)) != KVP_OK) return rc;
    if ((rc = rows_map(&a.k_map, some ? k : q, keys, heads, shape->head_dim, 1, PT_KEYS)) != KVP_OK) return rc;
    if ((rc = rows_map(&a.v_map, some ? v : q, keys, heads, shape->head_dim, 1, PT_KEYS)) != KVP_OK) return rc;
    a.sectors = aligned(out, 32) && aligned(ws, 32);
    a.polls = g_limit_next ? g_next_polls : PT_WAIT_LIMIT;
    g_limit_next = false;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return shape->head_dim == 128 ? launch_prompt<128>(a, unsigned(grid), st) : launch_prompt<64>(a, unsigned(grid), st);
}

int kvp_test_limit_next_prompt(uint32_t polls) {
    g_next_polls = polls;
    g_limit_next = true;
    return KVP_OK;
}

int kvprompt_status(const uint32_t *error, void *stream) {
    if (!error) return KVP_ERR_ARG;
    if (!aligned(error, 4)) return KVP_ERR_ALIGN;
    uint32_t f = 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&f, error, sizeof f, cudaMemcpyDeviceToHost, st) != cudaSuccess) return KVP_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return KVP_ERR_CUDA;
    return flags_to_status(f);
}

}  // extern "C"
