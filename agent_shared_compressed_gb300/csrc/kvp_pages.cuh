// kvp_pages.cuh -- the page container's byte format and its device codec.
//
// A container holds n_layers x n_pages pages; a page holds page_tokens tokens
// of every KV head.  Within a page, head h's tokens are page_tokens / 16
// blocks of 16 tokens, each one contiguous run of bytes (keys, values, key
// scales, value scales), so that one bulk copy brings everything attention
// needs of 16 tokens of a head into shared memory.  The order of the codes
// inside a block is the one that the tensor-core fragments of attention want,
// so the copied bytes are operands as they stand: no transposition, no second
// staging, and no two lanes of a shared-memory load on one bank.
//
// Dims of a row by lane quad (tig = 0..3): the lane owns dims 32 b + 8 tig + j
// (b < d/32, j < 8), that is 8 dims of every 32-dim scale group, in all formats
// and for keys and values alike; a quad holds one row.
#pragma once

#include <cstring>

#include "kvp_internal.cuh"

namespace kvp {

constexpr uint32_t PAGES_MAGIC = 0x4750564Bu;  // "KVPG"
constexpr uint32_t PAGES_VERSION = 1u;
constexpr uint64_t PAGES_HEADER_BYTES = 256;
constexpr int PAGES_ERR_WORD = 6;
constexpr int PAGES_BLOCK = 16;  // tokens of a block

// Header words: magic, version, L, H, d, page_tokens, error, format, n_pages.

struct PagesGeom {
    uint64_t block;         // bytes of a 16-token block of one head
    uint64_t tile;          // bytes of one head's tokens in a page
    uint64_t page;          // bytes of a page (all heads)
    uint64_t layer_stride;  // 256-byte aligned
    uint64_t total;
};

__host__ __device__ inline uint32_t pages_block_bytes(int d, int format) {
    const uint32_t row = uint32_t(d), ng = uint32_t(d / 32);
    if (format == KVP_PAGES_BF16) return 16u * 4u * row;
    if (format == KVP_PAGES_K8V8) return 16u * (2u * row + 4u * ng);
    return 16u * (row + row / 2u + 6u * ng);
}

inline PagesGeom pages_geom(const kvp_pages_config &c) {
    PagesGeom g;
    g.block = pages_block_bytes(c.head_dim, c.format);
    g.tile = g.block * uint64_t(c.page_tokens / PAGES_BLOCK);
    g.page = g.tile * uint64_t(c.n_kv_heads);
    g.layer_stride = align256(g.page * uint64_t(c.n_pages));
    g.total = PAGES_HEADER_BYTES + uint64_t(c.n_layers) * g.layer_stride;
    return g;
}

int pages_ok(const kvp_pages_config *c);  // KVP_OK or an error code (kvp_host.cu)

// What a kernel needs of the container and one of its layers.
struct PagesView {
    uint8_t *base;   // the container (header)
    uint8_t *layer;  // page 0 of the layer
    uint64_t page_bytes, tile_bytes;
    int L, H, d, P, logP, n_pages, format;
};

inline PagesView pages_view(void *pages, const kvp_pages_config &c, int layer) {
    const PagesGeom g = pages_geom(c);
    PagesView v;
    v.base = static_cast<uint8_t *>(pages);
    v.layer = v.base + PAGES_HEADER_BYTES + uint64_t(layer) * g.layer_stride;
    v.page_bytes = g.page;
    v.tile_bytes = g.tile;
    v.L = c.n_layers;
    v.H = c.n_kv_heads;
    v.d = c.head_dim;
    v.P = c.page_tokens;
    v.logP = 0;
    while ((1 << v.logP) < c.page_tokens) ++v.logP;
    v.n_pages = c.n_pages;
    v.format = c.format;
    return v;
}

// w / 2 pi mod 1 in units of 2^-64, cut off towards 0, for an fp32 w: its 24-bit integer
// times the first 128 bits of 1 / 2 pi's binary fraction, shifted by its exponent.
inline uint64_t turn_fraction(float w) {
    constexpr uint64_t HI = 0x28be60db9391054aull, LO = 0x7f09d5f47d4d3770ull;  // 1 / 2 pi * 2^128
    uint32_t bits;
    std::memcpy(&bits, &w, 4);
    const int ex = int(bits >> 23 & 255u);
    const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);  // |w| = m 2^(max(ex, 1) - 150)
    // m / 2 pi = p 2^-128 with p of 152 bits, as three 64-bit words
    const unsigned __int128 p0 = (unsigned __int128)m * LO, p1 = (unsigned __int128)m * HI + (p0 >> 64);
    const uint64_t word[3] = {uint64_t(p0), uint64_t(p1), uint64_t(p1 >> 64)};
    // the turn's 64-bit fraction: bits [s, s + 64) of p, s = 64 - (max(ex, 1) - 150)
    const int s = 214 - (ex ? ex : 1);
    uint64_t r = 0;
    for (int i = 0; i < 3; ++i) {
        const int at = 64 * i - s;  // where the word's bit 0 lands
        if (at >= 0 && at < 64) r |= word[i] << at;
        if (at < 0 && at > -64) r |= word[i] >> -at;
    }
    return bits >> 31 ? 0u - r : r;
}

// Whether the container's header is the one the caller described.
__device__ __forceinline__ bool pages_match(const PagesView &v) {
    const uint4 a = *reinterpret_cast<const uint4 *>(v.base);
    const uint4 b = *reinterpret_cast<const uint4 *>(v.base + 16);
    const uint32_t n = *reinterpret_cast<const uint32_t *>(v.base + 32);
    return a.x == PAGES_MAGIC && a.y == PAGES_VERSION && a.z == uint32_t(v.L) && a.w == uint32_t(v.H) &&
           b.x == uint32_t(v.d) && b.y == uint32_t(v.P) && b.w == uint32_t(v.format) && n == uint32_t(v.n_pages);
}

__device__ __forceinline__ void pages_flag(const PagesView &v, uint32_t f) {
    atomicOr(reinterpret_cast<uint32_t *>(v.base) + PAGES_ERR_WORD, f);
}

// ---------------------------------------------------------------------------
// A block's sections and the place of a row's bytes in them.  `t` is the
// token within the block (0..15).  The XORs put the lanes of one shared-memory
// load of attention on distinct banks; they move whole 16-byte chunks within
// 128-byte lines, so a global access keeps its sectors.
// ---------------------------------------------------------------------------
template <int D, int FMT>
struct Block {
    static constexpr bool Q8 = FMT != KVP_PAGES_BF16;
    static constexpr bool V4 = FMT == KVP_PAGES_K8V4;
    static constexpr int NG = D / 32;                               // scale groups of a row
    static constexpr uint32_t KROW = Q8 ? D : 2 * D;                // bytes of a key row
    static constexpr uint32_t VROW = V4 ? D / 2 : KROW;             // bytes of a value row
    static constexpr uint32_t SROW = 2 * NG;                        // key scales of a token (fp16)
    static constexpr uint32_t VSROW = V4 ? 4 * NG : 2 * NG;         // value scales (fp16), V4: (scale, zero) pairs
    static constexpr uint32_t OFF_V = 16 * KROW;
    static constexpr uint32_t OFF_KS = OFF_V + 16 * VROW;
    static constexpr uint32_t OFF_VS = OFF_KS + (Q8 ? 16 * SROW : 0);
    static constexpr uint32_t BYTES = OFF_VS + (Q8 ? 16 * VSROW : 0);

    // byte `x` of key row t
    static __host__ __device__ __forceinline__ uint32_t key(uint32_t t, uint32_t x) {
        const uint32_t at = t * KROW + x;
        if (!Q8) return at ^ ((t & 7u) << 4);
        return D == 128 ? at ^ ((t & 1u) << 4) : at;
    }
    // byte `x` of value row t
    static __host__ __device__ __forceinline__ uint32_t value(uint32_t t, uint32_t x) {
        const uint32_t at = t * VROW + x;
        if (!Q8) return OFF_V + (at ^ ((t & 7u) << 4));
        if (VROW == 32) return OFF_V + (at ^ (((t >> 2) & 1u) << 5));
        return OFF_V + (at ^ (((t >> 1) & 3u) << 5));
    }
};

// Bytes of a row by lane quad:
//  bf16 : chunk 4 b + tig (16 bytes) holds dims 32 b + 8 tig + 0..7
//  8-bit keys: the lane's d/4 bytes are contiguous, 32-bit word 2 b + e holds
//         dims 32 b + 8 tig + 4 e + 0..3 (code + 128): the key operand of two
//         k-steps of 16 dims per group
//  8-bit values: two granules of d/8 bytes, granule e's word b holds dims
//         32 b + 8 tig + 4 e + 0..3 (code + 128): granule g = 2 tig + e is what
//         lane g of a value fragment reads
//  4-bit values: two granules of d/16 bytes; nibble 4 b + j of granule e
//         is dim 32 b + 8 tig + 4 e + j

// The lane's share of a row of 8-bit codes as it goes into the cache.
template <int D>
struct Lane8 {
    uint32_t w[D / 32][2];  // [group][e]: four codes + 128
};

template <int D, int FMT>
__device__ __forceinline__ void store_key8(uint8_t *blk, uint32_t t, int tig, const Lane8<D> &c) {
    using B = Block<D, FMT>;
    *reinterpret_cast<uint4 *>(blk + B::key(t, tig * (D / 4))) = make_uint4(c.w[0][0], c.w[0][1], c.w[1][0], c.w[1][1]);
    if constexpr (D == 128)
        *reinterpret_cast<uint4 *>(blk + B::key(t, tig * 32 + 16)) =
            make_uint4(c.w[2][0], c.w[2][1], c.w[3][0], c.w[3][1]);
}
template <int D, int FMT>
__device__ __forceinline__ void load_key8(const uint8_t *blk, uint32_t t, int tig, Lane8<D> &c) {
    using B = Block<D, FMT>;
    const uint4 a = ld_once_v4(blk + B::key(t, tig * (D / 4)));
    c.w[0][0] = a.x, c.w[0][1] = a.y, c.w[1][0] = a.z, c.w[1][1] = a.w;
    if constexpr (D == 128) {
        const uint4 b = ld_once_v4(blk + B::key(t, tig * 32 + 16));
        c.w[2][0] = b.x, c.w[2][1] = b.y, c.w[3][0] = b.z, c.w[3][1] = b.w;
    }
}
template <int D, int FMT>
__device__ __forceinline__ void store_value8(uint8_t *blk, uint32_t t, int tig, const Lane8<D> &c) {
    using B = Block<D, FMT>;
    if constexpr (D == 128) {
        *reinterpret_cast<uint4 *>(blk + B::value(t, tig * 32)) = make_uint4(c.w[0][0], c.w[1][0], c.w[2][0], c.w[3][0]);
        *reinterpret_cast<uint4 *>(blk + B::value(t, tig * 32 + 16)) =
            make_uint4(c.w[0][1], c.w[1][1], c.w[2][1], c.w[3][1]);
    } else {
        *reinterpret_cast<uint4 *>(blk + B::value(t, tig * 16)) = make_uint4(c.w[0][0], c.w[1][0], c.w[0][1], c.w[1][1]);
    }
}
template <int D, int FMT>
__device__ __forceinline__ void load_value8(const uint8_t *blk, uint32_t t, int tig, Lane8<D> &c) {
    using B = Block<D, FMT>;
    if constexpr (D == 128) {
        const uint4 a = ld_once_v4(blk + B::value(t, tig * 32)), b = ld_once_v4(blk + B::value(t, tig * 32 + 16));
        c.w[0][0] = a.x, c.w[1][0] = a.y, c.w[2][0] = a.z, c.w[3][0] = a.w;
        c.w[0][1] = b.x, c.w[1][1] = b.y, c.w[2][1] = b.z, c.w[3][1] = b.w;
    } else {
        const uint4 a = ld_once_v4(blk + B::value(t, tig * 16));
        c.w[0][0] = a.x, c.w[1][0] = a.y, c.w[0][1] = a.z, c.w[1][1] = a.w;
    }
}

// 4-bit values: h[b][e] holds the four nibbles of group b, granule e (16 bits).
template <int D>
struct Lane4 {
    uint32_t h[D / 32][2];
};
template <int D, int FMT>
__device__ __forceinline__ void store_value4(uint8_t *blk, uint32_t t, int tig, const Lane4<D> &c) {
    using B = Block<D, FMT>;
    if constexpr (D == 128)
        *reinterpret_cast<uint4 *>(blk + B::value(t, tig * 16)) =
            make_uint4(c.h[0][0] | c.h[1][0] << 16, c.h[2][0] | c.h[3][0] << 16, c.h[0][1] | c.h[1][1] << 16,
                       c.h[2][1] | c.h[3][1] << 16);
    else
        *reinterpret_cast<uint2 *>(blk + B::value(t, tig * 8)) =
            make_uint2(c.h[0][0] | c.h[1][0] << 16, c.h[0][1] | c.h[1][1] << 16);
}
template <int D, int FMT>
__device__ __forceinline__ void load_value4(const uint8_t *blk, uint32_t t, int tig, Lane4<D> &c) {
    using B = Block<D, FMT>;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (D == 128) {
        const uint4 a = ld_once_v4(blk + B::value(t, tig * 16));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
        const uint2 a = ld_once_v2(blk + B::value(t, tig * 8));
        w[0] = a.x, w[1] = a.y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int b = 0; b < D / 32; ++b) c.h[b][e] = (w[e * (D / 64) + b / 2] >> (16 * (b & 1))) & 0xFFFFu;
}

// Four codes + 128 of a word as fp32 codes: 2^23 + u, less 2^23 + 128 (exact).
__device__ __forceinline__ void codes8(uint32_t w, float (&x)[4]) {
    x[0] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650u)) - 8388736.0f;
    x[1] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7651u)) - 8388736.0f;
    x[2] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7652u)) - 8388736.0f;
    x[3] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7653u)) - 8388736.0f;
}

// The fp16 scales of a row's groups.
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t *p, float (&s)[NG]) {
    uint32_t w[2] = {0u, 0u};
    if constexpr (NG == 4) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x, w[1] = a.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
        s[i] = __half2float(__ushort_as_half(uint16_t(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu)));
}
// ... and (scale, zero point) pairs.
template <int NG>
__device__ __forceinline__ void load_scale_zero(const uint8_t *p, float (&s)[NG], float (&z)[NG]) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (NG == 4) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x, w[1] = a.y;
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        s[i] = __half2float(__ushort_as_half(uint16_t(w[i] & 0xFFFFu)));
        z[i] = __half2float(__ushort_as_half(uint16_t(w[i] >> 16)));
    }
}

// The lane's values of one key / value row, in fp32: x[b][j] is dim 32 b + 8 tig + j.
template <int D, int FMT>
__device__ __forceinline__ void load_key_row(const uint8_t *blk, uint32_t t, int tig, float (&x)[D / 32][8]) {
    using B = Block<D, FMT>;
    if constexpr (!B::Q8) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const uint4 v = ld_once_v4(blk + B::key(t, (4 * b + tig) * 16));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[b][2 * i] = bf16_lo(w[i]), x[b][2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        Lane8<D> c;
        float s[B::NG];
        load_key8<D, FMT>(blk, t, tig, c);
        load_scales<B::NG>(blk + B::OFF_KS + t * B::SROW, s);
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y[4];
                codes8(c.w[b][e], y);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[b][4 * e + j] = y[j] * s[b];
            }
    }
}
template <int D, int FMT>
__device__ __forceinline__ void load_value_row(const uint8_t *blk, uint32_t t, int tig, float (&x)[D / 32][8]) {
    using B = Block<D, FMT>;
    if constexpr (!B::Q8) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const uint4 v = ld_once_v4(blk + B::value(t, (4 * b + tig) * 16));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[b][2 * i] = bf16_lo(w[i]), x[b][2 * i + 1] = bf16_hi(w[i]);
        }
    } else if constexpr (!B::V4) {
        Lane8<D> c;
        float s[B::NG];
        load_value8<D, FMT>(blk, t, tig, c);
        load_scales<B::NG>(blk + B::OFF_VS + t * B::VSROW, s);
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y[4];
                codes8(c.w[b][e], y);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[b][4 * e + j] = y[j] * s[b];
            }
    } else {
        Lane4<D> c;
        float s[B::NG], z[B::NG];
        load_value4<D, FMT>(blk, t, tig, c);
        load_scale_zero<B::NG>(blk + B::OFF_VS + t * B::VSROW, s, z);
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[b][4 * e + j] = fmaf(float((c.h[b][e] >> (4 * j)) & 15u), s[b], z[b]);
    }
}

}  // namespace kvp
