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
    uint32_t kc[kQuad], vc[kQuad], ka[kQuad], va[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        kc[i] = quantize8<kBf16>(k[i], ka[i]);
        vc[i] = quantize8<kBf16>(v[i], va[i]);
    }
    const int v_scales = a.c.page_size * 2 * NB;  // behind the K scales
    if (whole) {
        const Spot s = spot_of<NB>(a.c, slot[0], l);
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
        const Spot s = spot_of<NB>(a.c, slot[i], l);
        *reinterpret_cast<uint32_t*>(s.k) = kc[i];
        *reinterpret_cast<uint16_t*>(s.v) = (uint16_t)vc[i];
        *reinterpret_cast<uint16_t*>(s.v + 8 * NB) = (uint16_t)(vc[i] >> 16);
        if (l.part == 0) {
            *reinterpret_cast<uint16_t*>(s.s) = (uint16_t)ka[i];
            *reinterpret_cast<uint16_t*>(s.s + v_scales) = (uint16_t)va[i];
        }
    }
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

// Tokens in launches of at most 2^22 workgroups (a grid holds fewer than 2^32 lanes).
template <typename F>
hipError_t in_pieces(const KvMoveArgs& args, int elem, F launch) {
    const int64_t per = ceil_div((int64_t)args.c.heads * 8 * args.c.blocks, kThreads);
    const int64_t most = ((int64_t)1 << 22) / per / (kSpan / kQuad + 1) * kSpan;
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
    return in_pieces(args, 2, [&](const KvMoveArgs& a, dim3 grid) {
        if (past) hipLaunchKernelGGL((kv_write_kernel<kBf16, NB, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((kv_write_kernel<kBf16, NB, false>), grid, dim3(kThreads), 0, stream, a);
    });
}

template <bool kBf16, int NB, int kType>
hipError_t read_as(const KvMoveArgs& args, hipStream_t stream) {
    constexpr int kElem = kType == I8MP_DTYPE_F32 ? 4 : 2;
    const bool past = past_cache(args, kElem);
    return in_pieces(args, kElem, [&](const KvMoveArgs& a, dim3 grid) {
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

hipError_t launch_kv_read(const KvMoveArgs& a, hipStream_t stream) {
    if (a.c.bf16)
        return a.c.blocks == 1 ? read<true, 1>(a, stream) : a.c.blocks == 2 ? read<true, 2>(a, stream) : read<true, 4>(a, stream);
    return a.c.blocks == 1 ? read<false, 1>(a, stream) : a.c.blocks == 2 ? read<false, 2>(a, stream) : read<false, 4>(a, stream);
}

}  // namespace i8mp
