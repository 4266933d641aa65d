// Writing 16-bit keys and values into the 4-bit cache, and reading them back.
// Blocks of 64 dims: code = sign and the E2M1 magnitude nearest to
// fl32(|x| * fl32(6 * fl32(1 / A))), A the block's absmax, and x' = fl32(E2M1 value *
// fl32(A / 6)).  A is the absmax of 16-bit numbers and so one of them: the cache keeps
// it in that type, 2 bytes a block, unrounded.
//
// One lane has 8 dims of four neighbouring tokens, of K and of V: eight 16-byte loads
// (or stores) under way, and where the four slots are one aligned group, as a prompt's
// are, its V pieces are whole 8-byte words of the cache.  The magnitudes' maximum is taken
// on the bits (8 lanes share a block: three DPP steps), and the hardware's conversions
// round to codes and widen them, in place of seven comparisons a value.
//
// Both are bound by HBM where tokens are many: 16381 tokens of 32 heads of 128 are written
// in 62 us (5.5 TB/s) and read in 53 (6.4 TB/s); with a lane for 8 dims of one token and
// V in 2-byte accesses both took 251 us.  A few tokens are a launch: 3.7 us.
#include "kvcache.h"
#include "launch_limit.h"
#include "quant_util.h"

namespace i8mp {

namespace {

constexpr int kThreads = 256;
constexpr int kQuad = 4;   // tokens of a lane
constexpr int kSpan = 32;  // tokens whose quads are aligned together

// Calls that move more than the last-level cache holds (values and cache together) pass
// it by with the 16-bit values (non-temporal).  32 heads of 128, us, passing by / not:
// 16381 tokens (255 MiB of values) written 63 / 68, read 54 / 73; 32768 written 122 /
// 139, read 105 / 138, read and summed 291 / 300.  Below that a neighbour finds the
// values in the cache: 8000 tokens (125 MiB) read and summed 82 / 70, written 33 / 30.
constexpr int64_t kLastLevel = 256 << 20;

template <bool kBf16>
__device__ inline float wide(uint32_t h) {
    return kBf16 ? __uint_as_float(h << 16) : h2f((half_bits)h);
}

// E2M1 magnitude code of a non-negative fp32 value, ties to the even code; a NaN gives 0
__device__ inline uint32_t mag_code(float v) {
    return (uint32_t)(v > 0.25f) + (uint32_t)(v >= 0.75f) + (uint32_t)(v > 1.25f) + (uint32_t)(v >= 1.75f) +
           (uint32_t)(v > 2.5f) + (uint32_t)(v >= 3.5f) + (uint32_t)(v > 5.0f);
}

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// largest value of the 8 lanes that share a block
__device__ inline uint32_t block_max(uint32_t v) {
    const auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = up(v, (uint32_t)dpp_i32<kDppQuadSwap1>((int32_t)v));
    v = up(v, (uint32_t)dpp_i32<kDppQuadSwap2>((int32_t)v));
    return up(v, (uint32_t)dpp_i32<kDppHalfMirror>((int32_t)v));
}

// the chunk's largest magnitude, as the type's bits
__device__ inline uint32_t chunk_top(const uint4& x) {
    const uint32_t mag = 0x7fff7fffu;
    us2 m = __builtin_elementwise_max(__builtin_bit_cast(us2, x.x & mag), __builtin_bit_cast(us2, x.y & mag));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, x.z & mag));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, x.w & mag));
    return m.x > m.y ? m.x : m.y;
}

// what a block's values are multiplied by, from its A; IEEE reciprocal
__device__ inline float factor(float a) { return a > 0.0f ? 6.0f * (1.0f / a) : 0.0f; }

// The 8 codes of a lane's chunk and the bits of its block's A.  All lanes of a block call.
template <bool kBf16>
__device__ inline uint32_t quantize8(const uint4& x, uint32_t& a_bits) {
    constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = block_max(chunk_top(x));
    uint32_t packed = 0;
    const float inv = factor(wide<kBf16>(top));
    // 6 / A passes the largest fp32 number where A < 1.76e-38 (bfloat16 only)
    if (top < kInf && (!kBf16 || inv < INFINITY)) {
        // an element's magnitude is at most A, so products are within 6 and an ulp
#define I8MP_PAIR(i)                                                                                            \
    packed = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(packed, wide<kBf16>(w[i] & 0xffffu) * inv,                \
                                                      wide<kBf16>(w[i] >> 16) * inv, 1.0f, i)
        I8MP_PAIR(0);
        I8MP_PAIR(1);
        I8MP_PAIR(2);
        I8MP_PAIR(3);
#undef I8MP_PAIR
    } else {  // an infinity, a NaN (left out of A) or such an A: products that are NaN count as zeros
        float f[8], mx = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = fabsf(wide<kBf16>((w[e >> 1] >> (16 * (e & 1))) & 0xffffu));
            mx = fmaxf(mx, f[e]);
        }
        top = block_max(__float_as_uint(mx));
        mx = __uint_as_float(top);
        const float by = factor(mx);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t sign = (w[e >> 1] >> (16 * (e & 1) + 15)) & 1u;
            packed |= (mag_code(f[e] * by) | (sign << 3)) << (4 * e);
        }
        top = kBf16 ? top >> 16 : (uint32_t)f2h(mx);
    }
    a_bits = top;
    return packed;
}

// x' of 8 codes under A's bits
template <bool kBf16>
__device__ inline void values8(uint32_t codes, uint32_t a_bits, float (&x)[8]) {
    const float d = wide<kBf16>(a_bits) / 6.0f;  // IEEE division
#define I8MP_PAIR(i)                                                              \
    do {                                                                          \
        const f2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, i);    \
        x[2 * i] = v.x * d;                                                       \
        x[2 * i + 1] = v.y * d;                                                   \
    } while (0)
    I8MP_PAIR(0);
    I8MP_PAIR(1);
    I8MP_PAIR(2);
    I8MP_PAIR(3);
#undef I8MP_PAIR
}

// Which tokens and dims a lane has: 8 NB lanes a head, heads side by side, four tokens.
// Tokens come in spans of 32, whose quads start where the span's first slot puts a
// group's edge (a span has up to nine then): a prompt that starts inside a group still
// has its tokens in whole groups.
template <int NB>
struct Lane {
    int64_t tok0;     // first token of the quad: may lie before the span
    int64_t from, to; // the span's tokens
    int h, b, part;   // head, block, dims 8 part .. + 7 of it
    bool live;
};

template <int NB>
__device__ inline Lane<NB> lane_of(const KvMoveArgs& a) {
    Lane<NB> l;
    const uint32_t per = (uint32_t)a.c.heads * 8 * NB;  // lanes of a quad
    uint32_t i, quad;
    if (per >= kThreads) {  // several workgroups a quad of tokens
        const uint32_t groups = (per + kThreads - 1) / kThreads;
        quad = blockIdx.x / groups;
        i = (blockIdx.x - quad * groups) * kThreads + threadIdx.x;
        l.live = i < per;
    } else {                // several quads a workgroup
        const uint32_t quads = kThreads / per, q = threadIdx.x / per;
        quad = blockIdx.x * quads + q;
        i = threadIdx.x - q * per;
        l.live = q < quads;
    }
    const uint32_t span = quad / (kSpan / kQuad + 1);
    l.from = (int64_t)span * kSpan;
    l.to = l.from + kSpan < a.tokens ? l.from + kSpan : a.tokens;
    if (l.from < a.tokens) {
        l.tok0 = l.from - (int64_t)(a.slots[l.from] & 3) + (quad - span * (kSpan / kQuad + 1)) * kQuad;
        l.live = l.live && l.tok0 < l.to;
    } else {
        l.live = false;
    }
    l.part = (int)(i & 7);
    l.b = (int)(i >> 3) & (NB - 1);
    l.h = (int)(i / (8 * NB));
    return l;
}

// A slot's place: first byte of its slab's row of K codes, of V codes, of K scales.
struct Spot {
    uint8_t* k;
    uint8_t* v;
    uint8_t* s;
};

template <int NB>
__device__ inline Spot spot_of(const KvCache& c, int64_t slot, const Lane<NB>& l) {
    const int P = c.page_size, t = (int)(slot & (P - 1));
    uint8_t* slab = c.data + ((slot >> c.page_shift) * c.heads + l.h) * ((int64_t)P * 68 * NB);
    Spot s;
    s.k = slab + t * 32 * NB + (l.part >> 1) * 8 * NB + l.b * 8 + (l.part & 1) * 4;
    // dims 8 part + 0..3 and + 4..7 are V groups m = 2 part and 2 part + 1
    s.v = slab + P * 32 * NB + (t >> 2) * 128 * NB + l.part * 16 * NB + l.b * 8 + ((t & 1) * 2 + ((t >> 1) & 1)) * 2;
    s.s = slab + P * 64 * NB + (t * NB + l.b) * 2;
    return s;
}

__device__ inline bool in_cache(const KvCache& c, int64_t slot) { return slot >= 0 && slot < (c.pages << c.page_shift); }

// the four slots of a lane's tokens, -1 for none; true if they are one group of the cache
template <int NB>
__device__ inline bool slots_of(const KvMoveArgs& a, const Lane<NB>& l, int64_t (&slot)[kQuad]) {
    bool whole = true;
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        const int64_t t = l.tok0 + i;
        slot[i] = t >= l.from && t < l.to ? a.slots[t] : -1;
        if (!in_cache(a.c, slot[i])) slot[i] = -1;
        whole &= slot[i] == slot[0] + i;
    }
    return whole & (slot[0] >= 0) & ((slot[0] & 3) == 0);
}

// 4 x 16 bits of two tokens' halves -> the words (token 0, token 2) and (token 1, token 3)
__device__ inline uint2 v_words(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3, bool high) {
    const uint32_t sel = high ? 0x07060302u : 0x05040100u;  // halves of (b, a): a low, b high
    return make_uint2(__builtin_amdgcn_perm(t2, t0, sel), __builtin_amdgcn_perm(t3, t1, sel));
}

template <bool kPast>
__device__ inline uint4 load16(const half_bits* p) {
    if constexpr (kPast) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u4*>(p)));
    return *reinterpret_cast<const uint4*>(p);
}

template <bool kPast>
__device__ inline void store16(void* p, const u4& x) {
    if constexpr (kPast) __builtin_nontemporal_store(x, static_cast<u4*>(p));
    else *static_cast<u4*>(p) = x;
}

// quantizes and stores a lane's share of four tokens
template <bool kBf16, int NB>
__device__ inline void store_quad(const KvCache& c, const Lane<NB>& l, const int64_t (&slot)[kQuad], bool whole,
                                  const uint4 (&k)[kQuad], const uint4 (&v)[kQuad]) {
    uint32_t kc[kQuad], vc[kQuad], ka[kQuad], va[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        kc[i] = quantize8<kBf16>(k[i], ka[i]);
        vc[i] = quantize8<kBf16>(v[i], va[i]);
    }
    const int v_scales = c.page_size * 2 * NB;  // behind the K scales
    if (whole) {
        const Spot s = spot_of<NB>(c, slot[0], l);
#pragma unroll
        for (int i = 0; i < kQuad; ++i) *reinterpret_cast<uint32_t*>(s.k + i * 32 * NB) = kc[i];
        *reinterpret_cast<uint2*>(s.v) = v_words(vc[0], vc[1], vc[2], vc[3], false);
        *reinterpret_cast<uint2*>(s.v + 8 * NB) = v_words(vc[0], vc[1], vc[2], vc[3], true);
        if (l.part < kQuad) {  // lane `part` of the block stores token part's scales
            const uint32_t kk = l.part < 2 ? (l.part ? ka[1] : ka[0]) : (l.part == 2 ? ka[2] : ka[3]);
            const uint32_t vv = l.part < 2 ? (l.part ? va[1] : va[0]) : (l.part == 2 ? va[2] : va[3]);
            uint8_t* dst = s.s + l.part * 2 * NB;
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)kk;
            *reinterpret_cast<uint16_t*>(dst + v_scales) = (uint16_t)vv;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        if (slot[i] < 0) continue;
        const Spot s = spot_of<NB>(c, slot[i], l);
        *reinterpret_cast<uint32_t*>(s.k) = kc[i];
        *reinterpret_cast<uint16_t*>(s.v) = (uint16_t)vc[i];
        *reinterpret_cast<uint16_t*>(s.v + 8 * NB) = (uint16_t)(vc[i] >> 16);
        if (l.part == 0) {
            *reinterpret_cast<uint16_t*>(s.s) = (uint16_t)ka[i];
            *reinterpret_cast<uint16_t*>(s.s + v_scales) = (uint16_t)va[i];
        }
    }
}

template <bool kBf16, int NB, bool kPast>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvMoveArgs a) {
    const Lane<NB> l = lane_of<NB>(a);
    if (!l.live) return;  // the 8 lanes of a block leave together
    int64_t slot[kQuad];
    const bool whole = slots_of(a, l, slot);
    const int dim = l.b * 64 + l.part * 8;
    const half_bits* ks = static_cast<const half_bits*>(a.k) + l.tok0 * a.ldk + l.h * a.hsk + dim;
    const half_bits* vs = static_cast<const half_bits*>(a.v) + l.tok0 * a.ldv + l.h * a.hsv + dim;
    uint4 k[kQuad], v[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        const bool live = slot[i] >= 0;
        k[i] = live ? load16<kPast>(ks + i * a.ldk) : make_uint4(0, 0, 0, 0);
        v[i] = live ? load16<kPast>(vs + i * a.ldv) : make_uint4(0, 0, 0, 0);
    }
    store_quad<kBf16, NB>(a.c, l, slot, whole, k, v);
}

// ---- rotation by position -------------------------------------------------------
// Pair i of a head's first `rotary` dims turns by its token's angle i: (a cos - b sin,
// b cos + a sin), rounded to fp32 from the exact value, then to the 16-bit type.  The
// products of 11-bit and 24-bit numbers are exact in 64 bits and their sum rounds once
// at 2^-53, so the rounding to fp32 is that of the exact value but where it lies within
// 2^-29 of a border: the keys' codes, which a value next to a border of the 4-bit grid
// decides, do not depend on how the sum was formed.
typedef v4f v4f_any __attribute__((aligned(4)));

template <bool kBf16>
__device__ inline half_bits narrow(float x) {
    if constexpr (kBf16) return __builtin_bit_cast(half_bits, (__bf16)x);
    else return f2h(x);
}

// x cos + y sin
template <bool kBf16>
__device__ inline half_bits turn(uint32_t x, uint32_t y, float c, float s) {
    float r = (float)__builtin_fma((double)wide<kBf16>(x), (double)c, (double)wide<kBf16>(y) * (double)s);
    asm("" : "+v"(r));  // else the compiler makes one rounding of the two
    return narrow<kBf16>(r);
}

__device__ inline uint32_t half_of(const uint4& x, int e) {
    const uint32_t w = e < 4 ? (e < 2 ? x.x : x.y) : (e < 6 ? x.z : x.w);
    return (w >> (16 * (e & 1))) & 0xffffu;
}

__device__ inline void load8(const float* p, float (&x)[8]) {
    const v4f a = *reinterpret_cast<const v4f_any*>(p), b = *reinterpret_cast<const v4f_any*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
}

// 8 dims of a head whose pairs are the 8 of `other`; sign -1: these are the pairs' first
template <bool kBf16>
__device__ inline uint4 turn_halves(const uint4& own, const uint4& other, const float (&c)[8], const float (&s)[8], float sign) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = turn<kBf16>(half_of(own, 2 * i), half_of(other, 2 * i), c[2 * i], sign * s[2 * i]) |
               (uint32_t)turn<kBf16>(half_of(own, 2 * i + 1), half_of(other, 2 * i + 1), c[2 * i + 1], sign * s[2 * i + 1]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 dims that are four pairs
template <bool kBf16>
__device__ inline uint4 turn_pairs(const uint4& x, const v4f& c, const v4f& s) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = half_of(x, 2 * i), b = half_of(x, 2 * i + 1);
        w[i] = turn<kBf16>(a, b, c[i], -s[i]) | (uint32_t)turn<kBf16>(b, a, c[i], s[i]) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// the tables' row of a token
__device__ inline int64_t row_of(const KvAppendArgs& a, int64_t token) {
    const int64_t p = a.positions[token];
    return p < 0 ? 0 : p < a.table_rows ? p : a.table_rows - 1;
}

// Heads of q that a lane turns by one token's angles.  Four, with their conversions to 64 bits, take 140 registers and
// leave a SIMD three waves; with two, four fit: 16381 tokens of 32 / 32 heads of 128 appended in 141 us, with four in 150.
// (bfloat16 heads of 256 keep 12 bytes a lane in scratch for it.)
constexpr int kTurnHeads = 2;

// q: a lane has two 8-dim pieces of kTurnHeads heads of a token, those that turn into each other, so that q may
// be turned in place.  Pieces of a head, `half` = rotary / 16 pairs first: (u, u + half), then those that do not
// turn, two by two; where pairs are neighbours, (2 u, 2 u + 1).
template <bool kBf16, int NB, bool kPast>
__device__ inline void turn_queries(const KvAppendArgs& a, uint32_t block) {
    constexpr int kUnits = 4 * NB;
    const uint32_t groups = (uint32_t)(a.q_heads + kTurnHeads - 1) / kTurnHeads;  // heads g, g + groups, ...
    const uint32_t i = block * kThreads + threadIdx.x, u = i % kUnits, rest = i / kUnits;
    const uint32_t t = rest / groups, g = rest - t * groups;
    if (t >= a.m.tokens) return;
    const int half = a.rotary / 16;
    int p0 = (int)u, p1 = p0 + half;
    if (a.interleaved || p0 >= half) {
        p0 = a.interleaved ? 2 * (int)u : 2 * half + 2 * ((int)u - half);
        p1 = p0 + 1;
    }
    const int64_t row = row_of(a, t);
    const float *cos = a.cos + row * a.ldcos, *sin = a.sin + row * a.ldsin;
    const half_bits* from = a.q + (int64_t)t * a.ldq;
    half_bits* to = a.out + (int64_t)t * a.ldo;
    uint4 x[kTurnHeads][2];
#pragma unroll
    for (int j = 0; j < kTurnHeads; ++j) {
        const int64_t h = g + (int64_t)j * groups;
        if (h >= a.q_heads) break;
        x[j][0] = load16<kPast>(from + h * a.hsq + p0 * 8);
        x[j][1] = load16<kPast>(from + h * a.hsq + p1 * 8);
    }
    float c[8], s[8];
    if (p0 * 8 < a.rotary) {  // the angles of pairs 8 u .. 8 u + 7
        load8(cos + 8 * u, c);
        load8(sin + 8 * u, s);
    }
#pragma unroll
    for (int j = 0; j < kTurnHeads; ++j) {
        const int64_t h = g + (int64_t)j * groups;
        if (h >= a.q_heads) break;
        __builtin_amdgcn_sched_barrier(0);
        uint4 y0 = x[j][0], y1 = x[j][1];
        if (p0 * 8 < a.rotary) {
            if (a.interleaved) {  // rotary is a multiple of 16: both pieces turn
                y0 = turn_pairs<kBf16>(x[j][0], v4f{c[0], c[1], c[2], c[3]}, v4f{s[0], s[1], s[2], s[3]});
                y1 = turn_pairs<kBf16>(x[j][1], v4f{c[4], c[5], c[6], c[7]}, v4f{s[4], s[5], s[6], s[7]});
            } else {
                y0 = turn_halves<kBf16>(x[j][0], x[j][1], c, s, -1.0f);
                y1 = turn_halves<kBf16>(x[j][1], x[j][0], c, s, 1.0f);
            }
        }
        store16<kPast>(to + h * a.hso + p0 * 8, __builtin_bit_cast(u4, y0));
        store16<kPast>(to + h * a.hso + p1 * 8, __builtin_bit_cast(u4, y1));
    }
}

// k, v and q in one launch.  Reading a token's angles (64 bytes a lane, 16 of k) and turning k cost 34 us beside the 60 of
// a write of 16381 tokens of 32 heads of 128; q alone streams at 5.7 TB/s.
template <bool kBf16, int NB, bool kPast>
__global__ __launch_bounds__(kThreads, 4) void kv_append_kernel(KvAppendArgs a) {
    if (blockIdx.x >= a.kv_blocks) {
        turn_queries<kBf16, NB, kPast>(a, blockIdx.x - a.kv_blocks);
        return;
    }
    const Lane<NB> l = lane_of<NB>(a.m);
    if (!l.live) return;
    int64_t slot[kQuad];
    const bool whole = slots_of(a.m, l, slot);
    const int dim = l.b * 64 + l.part * 8;
    const half_bits* ks = static_cast<const half_bits*>(a.m.k) + l.tok0 * a.m.ldk + l.h * a.m.hsk;
    const half_bits* vs = static_cast<const half_bits*>(a.m.v) + l.tok0 * a.m.ldv + l.h * a.m.hsv + dim;
    const int half = a.rotary / 2;
    const bool turns = dim < a.rotary, halves = turns && !a.interleaved, first = dim < half;
    const int other = halves ? (first ? dim + half : dim - half) : dim;
    uint4 k[kQuad], v[kQuad], o[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        const bool live = slot[i] >= 0;
        k[i] = live ? load16<false>(ks + i * a.m.ldk + dim) : make_uint4(0, 0, 0, 0);
        o[i] = live && halves ? load16<false>(ks + i * a.m.ldk + other) : make_uint4(0, 0, 0, 0);
        v[i] = live ? load16<kPast>(vs + i * a.m.ldv) : make_uint4(0, 0, 0, 0);
    }
    if (turns) {
#pragma unroll
        for (int i = 0; i < kQuad; ++i) {
            // one token's angles in registers at a time; so a call of few tokens waits four times for a position and
            // then its angles (64 tokens: 6.6 us, the write without rotation 4)
            __builtin_amdgcn_sched_barrier(0);
            if (slot[i] < 0) continue;
            const int64_t row = row_of(a, l.tok0 + i);
            const float *cos = a.cos + row * a.ldcos, *sin = a.sin + row * a.ldsin;
            if (a.interleaved) {
                const v4f c = *reinterpret_cast<const v4f_any*>(cos + dim / 2), s = *reinterpret_cast<const v4f_any*>(sin + dim / 2);
                k[i] = turn_pairs<kBf16>(k[i], c, s);
            } else {
                float c[8], s[8];
                load8(cos + (first ? dim : dim - half), c);
                load8(sin + (first ? dim : dim - half), s);
                k[i] = turn_halves<kBf16>(k[i], o[i], c, s, first ? -1.0f : 1.0f);
            }
        }
    }
    store_quad<kBf16, NB>(a.m.c, l, slot, whole, k, v);
}

// one lane's 8 values of a token in the output's type
template <int kType, bool kPast>
__device__ inline void store8(void* base, int64_t at, const float (&x)[8]) {
    if constexpr (kType == I8MP_DTYPE_F32) {
        float* p = static_cast<float*>(base) + at;
        store16<kPast>(p, __builtin_bit_cast(u4, make_float4(x[0], x[1], x[2], x[3])));
        store16<kPast>(p + 4, __builtin_bit_cast(u4, make_float4(x[4], x[5], x[6], x[7])));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kType == I8MP_DTYPE_BF16) {
                typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                w[e] = __builtin_bit_cast(uint32_t, b2{(__bf16)x[2 * e], (__bf16)x[2 * e + 1]});
            } else {
                w[e] = __builtin_bit_cast(uint32_t, h2_t{(_Float16)x[2 * e], (_Float16)x[2 * e + 1]});
            }
        }
        store16<kPast>(static_cast<half_bits*>(base) + at, u4{w[0], w[1], w[2], w[3]});
    }
}

template <bool kBf16, int NB, int kType, bool kPast>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvMoveArgs a) {
    const Lane<NB> l = lane_of<NB>(a);
    if (!l.live) return;
    int64_t slot[kQuad];
    const bool whole = slots_of(a, l, slot);
    const int v_scales = a.c.page_size * 2 * NB;
    uint32_t kc[kQuad], vc[kQuad], ka[kQuad], va[kQuad];
    if (whole) {
        const Spot s = spot_of<NB>(a.c, slot[0], l);
        const uint2 lo = *reinterpret_cast<const uint2*>(s.v), hi = *reinterpret_cast<const uint2*>(s.v + 8 * NB);
#pragma unroll
        for (int i = 0; i < kQuad; ++i) {
            kc[i] = *reinterpret_cast<const uint32_t*>(s.k + i * 32 * NB);
            ka[i] = *reinterpret_cast<const uint16_t*>(s.s + i * 2 * NB);
            va[i] = *reinterpret_cast<const uint16_t*>(s.s + i * 2 * NB + v_scales);
            // words (token 0, token 2) and (token 1, token 3), dims 0..3 in lo and 4..7 in hi
            const uint32_t a0 = i & 1 ? lo.y : lo.x, a1 = i & 1 ? hi.y : hi.x;
            vc[i] = __builtin_amdgcn_perm(a1, a0, i >> 1 ? 0x07060302u : 0x05040100u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kQuad; ++i) {
            kc[i] = vc[i] = ka[i] = va[i] = 0;
            if (slot[i] < 0) continue;
            const Spot s = spot_of<NB>(a.c, slot[i], l);
            kc[i] = *reinterpret_cast<const uint32_t*>(s.k);
            vc[i] = *reinterpret_cast<const uint16_t*>(s.v) | ((uint32_t)*reinterpret_cast<const uint16_t*>(s.v + 8 * NB) << 16);
            ka[i] = *reinterpret_cast<const uint16_t*>(s.s);
            va[i] = *reinterpret_cast<const uint16_t*>(s.s + v_scales);
        }
    }
    const int dim = l.b * 64 + l.part * 8;
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        if (l.tok0 + i < l.from || l.tok0 + i >= l.to) continue;
        float x[8];
        values8<kBf16>(kc[i], ka[i], x);
        store8<kType, kPast>(a.k, (l.tok0 + i) * a.ldk + l.h * a.hsk + dim, x);
        values8<kBf16>(vc[i], va[i], x);
        store8<kType, kPast>(a.v, (l.tok0 + i) * a.ldv + l.h * a.hsv + dim, x);
    }
}

// workgroups for the tokens of one launch
int64_t move_blocks(const KvMoveArgs& a, int64_t tokens) {
    const int64_t per = (int64_t)a.c.heads * 8 * a.c.blocks, quads = ceil_div(tokens, kSpan) * (kSpan / kQuad + 1);
    return per >= kThreads ? quads * ceil_div(per, kThreads) : ceil_div(quads, kThreads / per);
}

// Tokens in launches of at most i8mp_launch_blocks workgroups, and as many more with `beside` lanes a token: whole spans.
template <typename F>
hipError_t in_pieces(const KvMoveArgs& args, int elem, int64_t beside, F launch) {
    const int64_t per = ceil_div((int64_t)args.c.heads * 8 * args.c.blocks, kThreads);
    const int64_t lanes = i8mp_launch_blocks * kThreads;
    int64_t most = i8mp_launch_blocks / per / (kSpan / kQuad + 1) * kSpan;
    if (most * beside > lanes) most = lanes / beside / kSpan * kSpan;
    if (most < kSpan) most = kSpan;
    for (int64_t t = 0; t < args.tokens; t += most) {
        KvMoveArgs a = args;
        a.tokens = args.tokens - t < most ? args.tokens - t : most;
        a.slots = args.slots + t;
        a.k = static_cast<uint8_t*>(args.k) + t * args.ldk * elem;
        a.v = static_cast<uint8_t*>(args.v) + t * args.ldv * elem;
        launch(a, dim3((unsigned)move_blocks(a, a.tokens)));
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

bool past_cache(const KvMoveArgs& a, int elem) {
    return a.tokens * a.c.heads * (2 * a.c.blocks * (64 * elem + 34)) > kLastLevel;
}

template <bool kBf16, int NB>
hipError_t write(const KvMoveArgs& args, hipStream_t stream) {
    const bool past = past_cache(args, 2);
    return in_pieces(args, 2, 0, [&](const KvMoveArgs& a, dim3 grid) {
        if (past) hipLaunchKernelGGL((kv_write_kernel<kBf16, NB, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((kv_write_kernel<kBf16, NB, false>), grid, dim3(kThreads), 0, stream, a);
    });
}

template <bool kBf16, int NB>
hipError_t append(const KvAppendArgs& args, hipStream_t stream) {
    const int64_t groups = args.q ? ceil_div(args.q_heads, kTurnHeads) : 0;
    const bool past = past_cache(args.m, 2);
    return in_pieces(args.m, 2, groups * 4 * NB, [&](const KvMoveArgs& m, dim3 grid) {
        KvAppendArgs a = args;
        const int64_t t = m.slots - args.m.slots;
        a.m = m;
        a.positions += t;
        if (a.q) a.q += t * a.ldq, a.out += t * a.ldo;
        a.kv_blocks = grid.x;
        grid.x += (unsigned)ceil_div(m.tokens * groups * 4 * NB, kThreads);
        if (past) hipLaunchKernelGGL((kv_append_kernel<kBf16, NB, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((kv_append_kernel<kBf16, NB, false>), grid, dim3(kThreads), 0, stream, a);
    });
}

template <bool kBf16, int NB, int kType>
hipError_t read_as(const KvMoveArgs& args, hipStream_t stream) {
    constexpr int kElem = kType == I8MP_DTYPE_F32 ? 4 : 2;
    const bool past = past_cache(args, kElem);
    return in_pieces(args, kElem, 0, [&](const KvMoveArgs& a, dim3 grid) {
        if (past) hipLaunchKernelGGL((kv_read_kernel<kBf16, NB, kType, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((kv_read_kernel<kBf16, NB, kType, false>), grid, dim3(kThreads), 0, stream, a);
    });
}

template <bool kBf16, int NB>
hipError_t read(const KvMoveArgs& a, hipStream_t stream) {
    return a.out_dtype == I8MP_DTYPE_F32   ? read_as<kBf16, NB, I8MP_DTYPE_F32>(a, stream)
           : a.out_dtype == I8MP_DTYPE_F16 ? read_as<kBf16, NB, I8MP_DTYPE_F16>(a, stream)
                                           : read_as<kBf16, NB, I8MP_DTYPE_BF16>(a, stream);
}

}  // namespace

hipError_t launch_kv_write(const KvMoveArgs& a, hipStream_t stream) {
    if (a.c.bf16)
        return a.c.blocks == 1 ? write<true, 1>(a, stream) : a.c.blocks == 2 ? write<true, 2>(a, stream) : write<true, 4>(a, stream);
    return a.c.blocks == 1 ? write<false, 1>(a, stream) : a.c.blocks == 2 ? write<false, 2>(a, stream) : write<false, 4>(a, stream);
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
    if (a.m.c.bf16)
        return a.m.c.blocks == 1 ? append<true, 1>(a, stream) : a.m.c.blocks == 2 ? append<true, 2>(a, stream) : append<true, 4>(a, stream);
    return a.m.c.blocks == 1 ? append<false, 1>(a, stream) : a.m.c.blocks == 2 ? append<false, 2>(a, stream) : append<false, 4>(a, stream);
}

hipError_t launch_kv_read(const KvMoveArgs& a, hipStream_t stream) {
    if (a.c.bf16)
        return a.c.blocks == 1 ? read<true, 1>(a, stream) : a.c.blocks == 2 ? read<true, 2>(a, stream) : read<true, 4>(a, stream);
    return a.c.blocks == 1 ? read<false, 1>(a, stream) : a.c.blocks == 2 ? read<false, 2>(a, stream) : read<false, 4>(a, stream);
}

}  // namespace i8mp
