// kvpages_append.cu -- writing new tokens into the page container, and reading
// a container's tokens back.
//
// kvpages_append, per new token and head, in one pass over the projection's
// output:
//   y = x rsqrt(mean(x^2) + eps) w             (queries and keys, if asked)
//   (y_i, y_{i + r/2}) turned by position * w_i  (i < r/2)
//   q_out = bf16(y);  the key's and the value's codes into their page;
//   k_out, v_out = bf16(the value that the page now holds).
// A lane quad holds one row of one token (see kvp_pages.cuh): both halves of
// every rotated pair and all of a scale group are within the quad, so the norm
// is two shuffles and a group's extremes two more.  A warp holds the same head
// of eight tokens, so that every branch on the kind of row is uniform and the
// (cos, sin) of its tokens, formed once per block, serve all heads.
//
// Angles.  position * w_i is only needed modulo a turn, and w_i / 2 pi modulo 1
// is a 64-bit fraction W_i, formed on the host from the fp32 frequency and 128
// bits of 1 / 2 pi.  position * W_i in 64-bit integers wraps at exactly one
// turn, so the reduced angle is off by less than |position| * 2^-64 turns (W_i is cut
// off, not rounded) at any position, for frequencies below 2^60; sincospif finishes in
// fp32.  (The same reduction in fp64 costs some hundred
// fp64 instructions an angle, and this GPU's fp64 rate is low.)
#include <algorithm>
#include <cmath>

#include "kvp_pages.cuh"

namespace kvp {

constexpr int APP_THREADS = 256;
constexpr int APP_WARPS = APP_THREADS / 32;
// Blocks of an SM: what 128 (head_dim 128), 80 and 64 registers a thread allow.  With three of
// head_dim 128, at 80 registers, which spill, 8192 tokens took 62 us where two took 47, with
// blocks of 10 warps 47.4 against 46.8.  Of head_dim 64 four spill where there are codes to form
// (8192 tokens of 32 heads in 4 bits 38.0 us, 26.4 with three) and gain where there are none (three
// ragged prompts of 32 heads in 16 bits 23.6 us, 26.4 with three, 31.9 with five).
constexpr int app_blocks(int d, int format) { return d == 128 ? 2 : (format == KVP_PAGES_BF16 ? 4 : 3); }
constexpr int APP_TOKENS = 8;  // tokens of a block: one per lane quad of a warp

struct AppendArgs {
    PagesView pv;
    const uint16_t *q, *k, *v;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // strides in elements
    const int64_t *slots, *positions;
    const uint16_t *q_norm, *k_norm;
    uint16_t *q_out, *k_out, *v_out;
    float eps;
    int n, nq, rot;
    int group_steps, run;  // steps of a token group, of a block
    int64_t steps;
    uint64_t turn[64];  // w_i / 2 pi mod 1, in units of 2^-64
    uint8_t axis[64];   // which of the positions pair i turns by
};

// The kernels here are placed while the one before them in the stream still runs
// (a programmatic dependent launch): they read and write nothing before its end.
// Then the next one may be placed.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// fp16 of a scale or zero point, kept finite; an overflow sets `bad`.
__device__ __forceinline__ uint32_t half_bits(float x, uint32_t &bad) {
    uint32_t h = __half_as_ushort(__float2half_rn(x));
    if ((h & 0x7C00u) == 0x7C00u) {
        bad |= FLAG_RANGE;
        h = (h & 0x8000u) | 0x7BFFu;
    }
    return h;
}
__device__ __forceinline__ float half_value(uint32_t h) { return __half2float(__ushort_as_half(uint16_t(h))); }

// 1 / s for an fp16 scale s (0 for 0), within 2^-22.
__device__ __forceinline__ float rcp_scale(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.0f ? r : 0.0f;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float most2(float m, float2 a) { return fmaxf(m, fmaxf(fabsf(a.x), fabsf(a.y))); }

// A row's elements that are Inf or NaN set to zero; whether there were any.
template <int NB>
__device__ __forceinline__ bool drop_nonfinite(float2 (&x)[NB][4]) {
    float2 odd = both(0.0f);  // NaN once an element is Inf or NaN
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) odd = fma2(x[b][j], both(0.0f), odd);
    if (odd.x + odd.y == 0.0f) return false;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[b][j] = make_float2(finite(x[b][j].x) ? x[b][j].x : 0.0f, finite(x[b][j].y) ? x[b][j].y : 0.0f);
    return true;
}

// Two quotients (t + e) / s decided exactly, t being the sum's rounding and y within 2^-10 of
// the quotients: k is the whole number below one (or, next to a whole number, either), held in
// [least, most - 1], and the sign of (t + e) - (k + 1/2) s says on which side of k + 1/2 it lies.
// (k + 1/2) s has at most 19 bits; where the quotient is near k + 1/2, t is within a factor of
// two of it, so that both differences are exact, and elsewhere they are far from 0.  The result
// rounds to nearest even to the code.  (No choice by element, two at a time: bf16 rows have ties in
// every 50th group of 4-bit codes, so that half of a warp's rows come here.)
__device__ __forceinline__ float2 decide2(float2 t, float2 e, float s, float2 y, float least, float most) {
    constexpr float WHOLE = 12582912.0f;
    float2 k = add2(add2(add2(y, both(-0.5f)), both(WHOLE)), both(-WHOLE));
    k = make_float2(fminf(fmaxf(k.x, least), most - 1.0f), fminf(fmaxf(k.y, least), most - 1.0f));
    const float2 mid = add2(k, both(0.5f)), d = add2(fma2(mid, both(-s), t), e);
    const bool some = s > 0.0f;  // (a scale of 0: codes 0)
    return add2(mid, make_float2(some && d.x != 0.0f ? copysignf(0.25f, d.x) : 0.0f, some && d.y != 0.0f ? copysignf(0.25f, d.y) : 0.0f));
}

// Codes of a row at 8 bits: s = fp16(max|x| fl(1/127)), code = x / s rounded to
// nearest (ties to even).  x * rcp(s) is within 2^-14 of the quotient, so only
// a product that near a half-integer is decided exactly.  x becomes the values
// held.
template <int D>
__device__ __forceinline__ void encode8(float2 (&x)[D / 32][4], Lane8<D> &c, uint32_t (&sb)[D / 32], uint32_t &bad) {
    constexpr int NB = D / 32;
    constexpr float MAGIC = 12582912.0f + 128.0f;  // 1.5 * 2^23 + the codes' bias
    if (drop_nonfinite<NB>(x)) bad |= FLAG_NONFINITE;
    float m[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        m[b] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) m[b] = most2(m[b], x[b][j]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) m[b] = quad_max(m[b]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        sb[b] = half_bits(m[b] * (1.0f / 127.0f), bad);
        const float s = half_value(sb[b]), rs = rcp_scale(s);
        float2 r[4];
        float near = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = fma2(x[b][j], both(rs), both(MAGIC));
            const float2 whole = add2(r[j], both(-MAGIC));
            near = most2(near, fma2(x[b][j], both(rs), make_float2(-whole.x, -whole.y)));
        }
        if (near > 0.5f - 0x1p-14f || s < 0x1p-14f || m[b] > 8320000.0f) {
            // near a border; or the scale is an fp16 subnormal or saturated, where codes can pass 127
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = add2(decide2(x[b][j], both(0.0f), s, mul2(x[b][j], both(rs)), -127.0f, 127.0f), both(MAGIC));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t lo = __byte_perm(__float_as_uint(r[2 * e].x), __float_as_uint(r[2 * e].y), 0x0040u);
            const uint32_t hi = __byte_perm(__float_as_uint(r[2 * e + 1].x), __float_as_uint(r[2 * e + 1].y), 0x0040u);
            c.w[b][e] = __byte_perm(lo, hi, 0x5410u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[b][j] = mul2(add2(r[j], both(-MAGIC)), both(s));
    }
}

// Codes of a value or key row at 4 bits: s = fp16(fl(max - min) fl(1/15)), z =
// fp16(min), code = (x - z) / s rounded to nearest even, in [0, 15], decided as
// above with x - z carried exactly.  x becomes the values held.
template <int D>
__device__ __forceinline__ void encode4(float2 (&x)[D / 32][4], Lane4<D> &c, uint32_t (&szb)[D / 32], uint32_t &bad) {
    constexpr int NB = D / 32;
    constexpr float MAGIC = 12582912.0f;
    if (drop_nonfinite<NB>(x)) bad |= FLAG_NONFINITE;
    float hi[NB], lo[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        hi[b] = fmaxf(x[b][0].x, x[b][0].y), lo[b] = fminf(x[b][0].x, x[b][0].y);
#pragma unroll
        for (int j = 1; j < 4; ++j) {
            hi[b] = fmaxf(hi[b], fmaxf(x[b][j].x, x[b][j].y));
            lo[b] = fminf(lo[b], fminf(x[b][j].x, x[b][j].y));
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) hi[b] = quad_max(hi[b]), lo[b] = -quad_max(-lo[b]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t sh = half_bits((hi[b] - lo[b]) * (1.0f / 15.0f), bad), zh = half_bits(lo[b], bad);
        szb[b] = sh | zh << 16;
        const float s = half_value(sh), z = half_value(zh), rs = rcp_scale(s);
        float2 r[4];
        float near = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 y = mul2(add2(x[b][j], both(-z)), both(rs));
            y = make_float2(fminf(fmaxf(y.x, 0.0f), 15.0f), fminf(fmaxf(y.y, 0.0f), 15.0f));
            r[j] = add2(y, both(MAGIC));
            const float2 whole = add2(r[j], both(-MAGIC));
            near = most2(near, add2(y, make_float2(-whole.x, -whole.y)));
        }
        if (near > 0.5f - 0x1p-14f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // x - z = t + e exactly
                const float2 t = add2(x[b][j], both(-z)), xx = add2(t, both(z)), u = add2(xx, make_float2(-t.x, -t.y));
                const float2 e = add2(add2(x[b][j], make_float2(-xx.x, -xx.y)), add2(u, both(-z)));
                r[j] = add2(decide2(t, e, s, mul2(t, both(rs)), 0.0f, 15.0f), both(MAGIC));
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // the low bits of 2^23 1.5 + code are the code: place four nibbles by sums of shifts
            const uint32_t lo2 = (__float_as_uint(r[2 * e].x) & 15u) | (__float_as_uint(r[2 * e].y) & 15u) << 4;
            const uint32_t hi2 = (__float_as_uint(r[2 * e + 1].x) & 15u) | (__float_as_uint(r[2 * e + 1].y) & 15u) << 4;
            c.h[b][e] = lo2 | hi2 << 8;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[b][j] = fma2(add2(r[j], both(-MAGIC)), both(s), both(z));
    }
}

// The codes in the order of 4-bit keys: a word's even nibbles below its odd ones.
template <int D>
__device__ __forceinline__ Lane4K<D> key_order(const Lane4<D> &c) {
    Lane4K<D> k;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        uint32_t w = c.h[b][0] | c.h[b][1] << 16;
        uint32_t x = (w ^ w >> 4) & 0x00F000F0u;
        w ^= x ^ x << 4;
        x = (w ^ w >> 8) & 0x0000FF00u;
        k.w[b] = w ^ x ^ x << 8;
    }
    return k;
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ void unpack8(uint4 v, float2 (&x)[4]) {
    x[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x)), x[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    x[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z)), x[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}

// Eight pairs turned by their cosines and sines.
__device__ __forceinline__ void turn(float2 (&lo)[4], float2 (&hi)[4], const float *cosines, const float *sines) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const float4 c = *reinterpret_cast<const float4 *>(cosines + 2 * j);
        const float4 s = *reinterpret_cast<const float4 *>(sines + 2 * j);
        const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
        const float2 ss[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 l = lo[j + k], h = hi[j + k];
            lo[j + k] = fma2(l, cc[k], mul2(h, make_float2(-ss[k].x, -ss[k].y)));
            hi[j + k] = fma2(h, cc[k], mul2(l, ss[k]));
        }
    }
}

// The lane's share of a contiguous bf16 row.
template <int D>
__device__ __forceinline__ void store_row(uint16_t *row, int tig, const float2 (&x)[D / 32][4]) {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) *reinterpret_cast<uint4 *>(row + 32 * b + 8 * tig) = pack8(x[b]);
}

// The work is a list of steps: a group of APP_TOKENS tokens has one for every
// APP_WARPS of its nq query, H key and H value rows (a warp takes a row of all of
// the group's tokens).  A block takes an equal run of the list, as many blocks as
// the GPU holds at once: there is no last, half-empty wave (8192 tokens: 47.5
// against 51.2 us with a block per group).  A row's loads are issued while the row
// before it is worked on.
template <int D, int FMT>
__global__ void __launch_bounds__(APP_THREADS, app_blocks(D, FMT)) pages_append(const __grid_constant__ AppendArgs a) {
    using B = Block<D, FMT>;
    constexpr int NB = D / 32;
    // rows padded to start on other banks; read as float4
    __shared__ __align__(16) float cosines[APP_TOKENS][D / 2 + 4], sines[APP_TOKENS][D / 2 + 4], norm[2][D];
    // what pair i turns by, and where its positions begin: a warp's lanes want 32 of them
    // at once, which the parameters' constant memory gives one by one
    __shared__ uint64_t turns[D / 2];
    __shared__ const int64_t *from[D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tq = lane >> 2, tig = lane & 3;
    const int H = a.pv.H, rows = a.nq + 2 * H;
    const int64_t first = int64_t(blockIdx.x) * a.run;
    int left = int(min(int64_t(a.run), a.steps - first));  // steps of this block
    int64_t grp = first / a.group_steps;
    int st = int(first % a.group_steps);
    auto load = [&](int64_t g, int s, uint4 (&v)[NB]) {
        const int64_t tok = g * APP_TOKENS + tq;
        const int row = s * APP_WARPS + warp;
        const bool is_q = row < a.nq, is_v = row >= a.nq + H;
        const uint16_t *src = is_q ? a.q + tok * a.q_ts + row * a.q_hs
                                   : (is_v ? a.v + tok * a.v_ts + (row - a.nq - H) * a.v_hs
                                           : a.k + tok * a.k_ts + (row - a.nq) * a.k_hs);
        const bool real = row < rows && tok < a.n;
        // (by way of L2: 8192 tokens 45.8 us, 47.6 with ld_once_v4; pages_read the other
        // way round, 62.4 and 61.5)
#pragma unroll
        for (int b = 0; b < NB; ++b) v[b] = real ? ld_l2_v4(src + 32 * b + 8 * tig) : make_uint4(0, 0, 0, 0);
    };
    if (threadIdx.x < D / 2) {
        turns[threadIdx.x] = a.turn[threadIdx.x];
        from[threadIdx.x] = a.positions + int64_t(a.axis[threadIdx.x]) * a.n;
    }
    const int log_half = a.rot == 128 ? 6 : 5;
    wait_for_previous();
    uint4 in[NB];
    load(grp, st, in);
    const bool match = pages_match(a.pv);
    for (int i = threadIdx.x; i < 2 * D; i += APP_THREADS) {
        const uint16_t *w = i < D ? a.q_norm : a.k_norm;
        norm[i / D][i % D] = w ? __uint_as_float(uint32_t(w[i % D]) << 16) : 1.0f;
    }
    int64_t tok = 0;
    bool real = false, fresh = true;
    uint8_t *blk = nullptr;  // the token's block of head 0
    uint32_t row16 = 0, bad = match ? 0u : FLAG_HEADER;
    for (; left > 0; --left) {
        if (fresh) {  // a new group: its angles, and the places of its tokens
            fresh = false;
            __syncthreads();
            tok = grp * APP_TOKENS + tq;
            real = tok < a.n;
            const int64_t slot = real ? a.slots[tok] : -1;
            if (a.rot > 0) {
                for (int i = threadIdx.x; i < APP_TOKENS << log_half; i += APP_THREADS) {
                    const int t = i >> log_half, p = i & ((1 << log_half) - 1);
                    const int64_t at = grp * APP_TOKENS + t;
                    float s = 0.0f, c = 1.0f;
                    if (at < a.n) {
                        const int64_t part = int64_t(uint64_t(from[p][at]) * turns[p]);  // mod one turn
                        sincospif(2.0f * (float(part) * 0x1p-64f), &s, &c);
                    }
                    cosines[t][p] = c, sines[t][p] = s;
                }
            }
            blk = nullptr;
            if (slot >= (int64_t(a.pv.n_pages) << a.pv.logP)) {
                bad |= FLAG_PAGE;
            } else if (match && slot >= 0) {
                const int64_t page = slot >> a.pv.logP;
                const uint32_t at = uint32_t(slot) & uint32_t(a.pv.P - 1);
                blk = a.pv.layer + uint64_t(page) * a.pv.page_bytes + uint64_t(at / PAGES_BLOCK) * B::BYTES;
                row16 = at % PAGES_BLOCK;
            }
            __syncthreads();
        }
        const int r = st * APP_WARPS + warp;
        if (++st == a.group_steps) st = 0, ++grp, fresh = true;
        float2 x[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) unpack8(in[b], x[b]);
        if (left > 1) load(grp, st, in);
        if (r >= rows) continue;
        const bool is_q = r < a.nq, is_v = r >= a.nq + H;
        const int h = is_q ? r : (is_v ? r - a.nq - H : r - a.nq);
        uint8_t *hb = blk ? blk + uint64_t(h) * a.pv.tile_bytes : nullptr;
        if (!is_v) {
            if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
                float2 ss = both(0.0f);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = fma2(x[b][j], x[b][j], ss);
                const float inv = rsqrtf(quad_sum(ss.x + ss.y) * (1.0f / D) + a.eps);
                const float *w = norm[is_q ? 0 : 1] + 8 * tig;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float4 v = *reinterpret_cast<const float4 *>(w + 32 * b + 2 * j);
                        x[b][j] = mul2(mul2(x[b][j], both(inv)), make_float2(v.x, v.y));
                        x[b][j + 1] = mul2(mul2(x[b][j + 1], both(inv)), make_float2(v.z, v.w));
                    }
            }
            if (a.rot > 0) {
                const float *c = cosines[tq] + 8 * tig, *s = sines[tq] + 8 * tig;
                if (NB == 4 && a.rot == 128) {
                    turn(x[0], x[NB - 2], c, s);
                    turn(x[1], x[NB - 1], c + 32, s + 32);
                } else {
                    turn(x[0], x[1], c, s);
                }
            }
            if (is_q) {
                if (real) store_row<D>(a.q_out + (tok * a.nq + h) * D, tig, x);
                continue;
            }
        }
        if constexpr (!B::Q8) {
            if (hb) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t at = (4 * b + tig) * 16;
                    *reinterpret_cast<uint4 *>(hb + (is_v ? B::value(row16, at) : B::key(row16, at))) = pack8(x[b]);
                }
            }
        } else if constexpr (B::K4) {
            // Keys and values share the encoder: with one each, fetching instructions is what a step waits
            // for most (8192 tokens into 4-bit pages, nothing returned: 17.5 us; before halves were decided two
            // at a time 20.8, and 24.4 with one each; 8-bit pages gain nothing).
            Lane4<D> c;
            uint32_t szb[NB];
            encode4<D>(x, c, szb, bad);
            if (hb && is_v) {
                store_value4<D, FMT>(hb, row16, tig, c);
                if (tig == 0) {
                    uint32_t *s = reinterpret_cast<uint32_t *>(hb + B::OFF_VS + row16 * B::VSROW);
#pragma unroll
                    for (int i = 0; i < NB; ++i) s[i] = szb[i];
                }
            } else if (hb) {
                store_key4<D, FMT>(hb, row16, tig, key_order<D>(c));
                if (tig == 0) {  // the scales, then the zero points
                    uint32_t *s = reinterpret_cast<uint32_t *>(hb + B::OFF_KS + row16 * B::SROW);
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) {
                        s[i] = __byte_perm(szb[2 * i], szb[2 * i + 1], 0x5410u);
                        s[NB / 2 + i] = __byte_perm(szb[2 * i], szb[2 * i + 1], 0x7632u);
                    }
                }
            }
        } else if (!is_v) {
            Lane8<D> c;
            uint32_t sb[NB];
            encode8<D>(x, c, sb, bad);
            if (hb) {
                store_key8<D, FMT>(hb, row16, tig, c);
                if (tig == 0) {
                    uint32_t *s = reinterpret_cast<uint32_t *>(hb + B::OFF_KS + row16 * B::SROW);
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) s[i] = sb[2 * i] | sb[2 * i + 1] << 16;
                }
            }
        } else if constexpr (!B::V4) {
            Lane8<D> c;
            uint32_t sb[NB];
            encode8<D>(x, c, sb, bad);
            if (hb) {
                store_value8<D, FMT>(hb, row16, tig, c);
                if (tig == 0) {
                    uint32_t *s = reinterpret_cast<uint32_t *>(hb + B::OFF_VS + row16 * B::VSROW);
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) s[i] = sb[2 * i] | sb[2 * i + 1] << 16;
                }
            }
        } else {
            Lane4<D> c;
            uint32_t szb[NB];
            encode4<D>(x, c, szb, bad);
            if (hb) {
                store_value4<D, FMT>(hb, row16, tig, c);
                if (tig == 0) {
                    uint32_t *s = reinterpret_cast<uint32_t *>(hb + B::OFF_VS + row16 * B::VSROW);
#pragma unroll
                    for (int i = 0; i < NB; ++i) s[i] = szb[i];
                }
            }
        }
        uint16_t *back = is_v ? a.v_out : a.k_out;
        if (back && real) store_row<D>(back + (tok * H + h) * D, tig, x);
    }
    if (bad) pages_flag(a.pv, bad);
}

// ---------------------------------------------------------------------------
// Reading back.  A warp takes a 16-token block of one sequence and head; a
// quad takes a row.  Output rows past the sequence's length are zeros.
// ---------------------------------------------------------------------------
struct ReadArgs {
    PagesView pv;
    const int32_t *table, *lens;
    uint16_t *k, *v;  // [B][H][Tmax][d]
    int max_pages, tmax, nblk;
    uint64_t tasks;
};

template <int D, int FMT>
__global__ void __launch_bounds__(256) pages_read(const __grid_constant__ ReadArgs a) {
    using B = Block<D, FMT>;
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 31, tq = lane >> 2, tig = lane & 3;
    wait_for_previous();
    if (!pages_match(a.pv)) {
        if (threadIdx.x == 0) pages_flag(a.pv, FLAG_HEADER);
        return;
    }
    const uint64_t nwarps = uint64_t(gridDim.x) * (blockDim.x / 32);
    for (uint64_t w = uint64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); w < a.tasks; w += nwarps) {
        const uint32_t blk16 = uint32_t(w % uint32_t(a.nblk));
        const uint32_t bh = uint32_t(w / uint32_t(a.nblk));
        const uint32_t h = bh % uint32_t(a.pv.H), b = bh / uint32_t(a.pv.H);
        const int t0 = int(blk16) * PAGES_BLOCK;
        int len = min(max(a.lens[b], 0), a.tmax);
        if (len > 0 && int64_t(len) > int64_t(a.max_pages) << a.pv.logP) {  // the table is shorter than the sequence
            if (lane == 0) pages_flag(a.pv, FLAG_PAGE);
            len = int(int64_t(a.max_pages) << a.pv.logP);
        }
        const uint8_t *src = nullptr;
        if (t0 < len) {
            const int page = a.table[uint64_t(b) * uint32_t(a.max_pages) + uint32_t(t0 >> a.pv.logP)];
            if (page >= 0 && page < a.pv.n_pages)
                src = a.pv.layer + uint64_t(page) * a.pv.page_bytes + uint64_t(h) * a.pv.tile_bytes +
                      uint64_t((uint32_t(t0) & uint32_t(a.pv.P - 1)) / PAGES_BLOCK) * B::BYTES;
            else if (lane == 0)
                pages_flag(a.pv, FLAG_PAGE);
        }
        const uint64_t out = (uint64_t(bh) * uint32_t(a.tmax) + uint32_t(t0)) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 8 * i + tq;
            if (t0 + t >= a.tmax) continue;
            float x[NB][8];
            const bool there = src && t0 + t < len;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (there) {
                    if (kv == 0)
                        load_key_row<D, FMT>(src, t, tig, x);
                    else
                        load_value_row<D, FMT>(src, t, tig, x);
                } else {
#pragma unroll
                    for (int g = 0; g < NB; ++g)
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[g][j] = 0.0f;
                }
                uint16_t *row = (kv == 0 ? a.k : a.v) + out + uint64_t(t) * D;
#pragma unroll
                for (int g = 0; g < NB; ++g)
                    st_stream_v4(row + 32 * g + 8 * tig, make_uint4(pack_bf16x2(x[g][0], x[g][1]), pack_bf16x2(x[g][2], x[g][3]),
                                                                    pack_bf16x2(x[g][4], x[g][5]), pack_bf16x2(x[g][6], x[g][7])));
            }
        }
    }
}

__global__ void pages_init(uint32_t *h, const __grid_constant__ kvp_pages_config c, uint64_t layer_stride,
                           uint64_t total) {
    const int i = threadIdx.x;  // 64 words
    uint32_t w = 0u;
    switch (i) {
        case 0: w = PAGES_MAGIC; break;
        case 1: w = PAGES_VERSION; break;
        case 2: w = uint32_t(c.n_layers); break;
        case 3: w = uint32_t(c.n_kv_heads); break;
        case 4: w = uint32_t(c.head_dim); break;
        case 5: w = uint32_t(c.page_tokens); break;
        case 7: w = uint32_t(c.format); break;
        case 8: w = uint32_t(c.n_pages); break;
        case 10: w = uint32_t(layer_stride); break;
        case 11: w = uint32_t(layer_stride >> 32); break;
        case 12: w = uint32_t(total); break;
        case 13: w = uint32_t(total >> 32); break;
        default: break;
    }
    h[i] = w;
}

template <typename Args>
static int launch(void (*kernel)(Args), const Args &a, unsigned grid, unsigned threads, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return KVP_ERR_CUDA;
    count_launch();
    return launch_status();
}
template <int D, int FMT>
static int launch_append(const AppendArgs &a, unsigned grid, cudaStream_t st) {
    return launch(pages_append<D, FMT>, a, grid, APP_THREADS, st);
}
template <int D, int FMT>
static int launch_read(const ReadArgs &a, unsigned grid, cudaStream_t st) {
    return launch(pages_read<D, FMT>, a, grid, 256, st);
}

static bool rows_aligned(const kvp_rows *r) {
    return aligned(r->ptr, 16) && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

int kvpages_init(const kvp_pages_config *cfg, void *pages, size_t pages_bytes, void *stream) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (!pages) return KVP_ERR_ARG;
    if (!aligned(pages, 256)) return KVP_ERR_ALIGN;
    const PagesGeom g = pages_geom(*cfg);
    if (pages_bytes < g.total) return KVP_ERR_SIZE;
    pages_init<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint32_t *>(pages), *cfg, g.layer_stride,
                                                                g.total);
    count_launch();
    return launch_status();
}

int kvpages_append(void *pages, const kvp_pages_config *cfg, int layer, int n_tokens, int n_q_heads, const kvp_rows *q,
                   const kvp_rows *k, const kvp_rows *v, const int64_t *slots, const int64_t *positions,
                   const void *q_norm, const void *k_norm, float eps, int rot_dim, const float *inv_freq, void *q_out,
                   void *k_out, void *v_out, void *stream) {
    static const uint8_t one_axis[64] = {0};
    return kvpages_append_axes(pages, cfg, layer, n_tokens, n_q_heads, q, k, v, slots, positions, 1, one_axis, q_norm, k_norm,
                               eps, rot_dim, inv_freq, q_out, k_out, v_out, stream);
}

int kvpages_append_axes(void *pages, const kvp_pages_config *cfg, int layer, int n_tokens, int n_q_heads,
                        const kvp_rows *q, const kvp_rows *k, const kvp_rows *v, const int64_t *slots,
                        const int64_t *positions, int n_axes, const uint8_t *axes, const void *q_norm,
                        const void *k_norm, float eps, int rot_dim, const float *inv_freq, void *q_out, void *k_out,
                        void *v_out, void *stream) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (!pages || layer < 0 || layer >= cfg->n_layers || n_tokens < 0 || n_q_heads < 0) return KVP_ERR_ARG;
    if (n_q_heads > 65536) return KVP_ERR_SIZE;
    if (!k || !v || !k->ptr || !v->ptr || !slots) return KVP_ERR_ARG;
    if (n_q_heads > 0 && (!q || !q->ptr || !q_out)) return KVP_ERR_ARG;
    if (rot_dim != 0 && rot_dim != 64 && !(rot_dim == 128 && cfg->head_dim == 128)) return KVP_ERR_ARG;
    if (n_axes < 1 || n_axes > KVP_MAX_AXES) return KVP_ERR_ARG;
    if (rot_dim > 0 && (!positions || !inv_freq || !axes)) return KVP_ERR_ARG;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i]) || axes[i] >= n_axes) return KVP_ERR_ARG;
    if ((q_norm || k_norm) && !(std::isfinite(eps) && eps >= 0.0f)) return KVP_ERR_ARG;
    if (!aligned(pages, 256) || !rows_aligned(k) || !rows_aligned(v) || (n_q_heads > 0 && !rows_aligned(q)) ||
        !aligned(slots, 8) || !aligned(positions, 8) || !aligned(q_norm, 16) || !aligned(k_norm, 16) ||
        !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return KVP_ERR_ALIGN;
    if (n_tokens == 0) return KVP_OK;
    AppendArgs a;
    a.pv = pages_view(pages, *cfg, layer);
    a.q = n_q_heads > 0 ? static_cast<const uint16_t *>(q->ptr) : nullptr;
    a.q_ts = n_q_heads > 0 ? q->token_stride : 0;
    a.q_hs = n_q_heads > 0 ? q->head_stride : 0;
    a.k = static_cast<const uint16_t *>(k->ptr), a.k_ts = k->token_stride, a.k_hs = k->head_stride;
    a.v = static_cast<const uint16_t *>(v->ptr), a.v_ts = v->token_stride, a.v_hs = v->head_stride;
    a.slots = slots, a.positions = positions;
    a.q_norm = static_cast<const uint16_t *>(q_norm), a.k_norm = static_cast<const uint16_t *>(k_norm);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out), a.v_out = static_cast<uint16_t *>(v_out);
    a.eps = eps, a.n = n_tokens, a.nq = n_q_heads, a.rot = rot_dim;
    for (int i = 0; i < 64; ++i) {
        a.turn[i] = i < rot_dim / 2 ? turn_fraction(inv_freq[i]) : 0;
        a.axis[i] = i < rot_dim / 2 ? axes[i] : 0;
    }
    const int rows = n_q_heads + 2 * cfg->n_kv_heads;
    a.group_steps = (rows + APP_WARPS - 1) / APP_WARPS;
    a.steps = (int64_t(n_tokens) + APP_TOKENS - 1) / APP_TOKENS * a.group_steps;
    const int64_t blocks = std::min<int64_t>(a.steps, int64_t(sm_count()) * app_blocks(cfg->head_dim, cfg->format));
    a.run = int((a.steps + blocks - 1) / blocks);
    const unsigned grid = unsigned((a.steps + a.run - 1) / a.run);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool d128 = cfg->head_dim == 128;
    switch (cfg->format) {
        case KVP_PAGES_BF16:
            return d128 ? launch_append<128, KVP_PAGES_BF16>(a, grid, st) : launch_append<64, KVP_PAGES_BF16>(a, grid, st);
        case KVP_PAGES_K8V8:
            return d128 ? launch_append<128, KVP_PAGES_K8V8>(a, grid, st) : launch_append<64, KVP_PAGES_K8V8>(a, grid, st);
        case KVP_PAGES_K8V4:
            return d128 ? launch_append<128, KVP_PAGES_K8V4>(a, grid, st) : launch_append<64, KVP_PAGES_K8V4>(a, grid, st);
        default:
            return d128 ? launch_append<128, KVP_PAGES_K4V4>(a, grid, st) : launch_append<64, KVP_PAGES_K4V4>(a, grid, st);
    }
}

int kvpages_read(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, const int32_t *table,
                 int max_pages, const int32_t *lens, int max_tokens, void *k_dst, void *v_dst, void *stream) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (!pages || layer < 0 || layer >= cfg->n_layers || n_seqs < 0 || max_pages <= 0 || max_tokens <= 0)
        return KVP_ERR_ARG;
    if (!table || !lens || !k_dst || !v_dst) return KVP_ERR_ARG;
    if (!aligned(pages, 256) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(k_dst, 16) || !aligned(v_dst, 16))
        return KVP_ERR_ALIGN;
    if (int64_t(n_seqs) * cfg->n_kv_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    if (n_seqs == 0) return KVP_OK;
    ReadArgs a;
    a.pv = pages_view(const_cast<void *>(pages), *cfg, layer);
    a.table = table, a.lens = lens;
    a.k = static_cast<uint16_t *>(k_dst), a.v = static_cast<uint16_t *>(v_dst);
    a.max_pages = max_pages, a.tmax = max_tokens;
    a.nblk = int((int64_t(max_tokens) + PAGES_BLOCK - 1) / PAGES_BLOCK);
    a.tasks = uint64_t(n_seqs) * uint64_t(cfg->n_kv_heads) * uint64_t(a.nblk);
    // two to three waves of blocks: 15 4K caches 61.3 us, 64.5 with 8 blocks an SM (about
    // one wave); 7 ragged ones 23.7 us, 24.8 with 32
    const unsigned grid = unsigned(std::min<uint64_t>((a.tasks + 7) / 8, uint64_t(sm_count()) * 16));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool d128 = cfg->head_dim == 128;
    switch (cfg->format) {
        case KVP_PAGES_BF16:
            return d128 ? launch_read<128, KVP_PAGES_BF16>(a, grid, st) : launch_read<64, KVP_PAGES_BF16>(a, grid, st);
        case KVP_PAGES_K8V8:
            return d128 ? launch_read<128, KVP_PAGES_K8V8>(a, grid, st) : launch_read<64, KVP_PAGES_K8V8>(a, grid, st);
        case KVP_PAGES_K8V4:
            return d128 ? launch_read<128, KVP_PAGES_K8V4>(a, grid, st) : launch_read<64, KVP_PAGES_K8V4>(a, grid, st);
        default:
            return d128 ? launch_read<128, KVP_PAGES_K4V4>(a, grid, st) : launch_read<64, KVP_PAGES_K4V4>(a, grid, st);
    }
}

}  // extern "C"
