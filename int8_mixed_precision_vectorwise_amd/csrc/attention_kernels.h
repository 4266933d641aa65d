// Attention over the 4-bit key/value cache: for a query row at position p of a
// sequence of length L (token j visible iff j < L and (j < prefix, or j <= p and
// p - j < window)),
//   s_j = scale q . k_j,  s_j <- cap tanh(s_j / cap),  s_j <- s_j - slope |p - j|,
//   out = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^s_j  over the visible j,
// in one pass over the cache with a running maximum.  k_j and v_j stay 4-bit up to
// the matrix instructions: an E2M1 value is exact in fp16 and in bfloat16, so the
// products run on the codes' values, and the block scales A / 6 enter in fp32: on
// the 64-deep partial sums of q . k, and on the weights e^s of v.
#pragma once

#include <type_traits>

#include "kvcache.h"

namespace i8mp {

namespace {

constexpr int kTile = 32;       // keys of a tile
constexpr int kCols = 16;       // query rows of an MFMA's columns; a row tile has T times as many
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// the 16-bit type's vectors, matrix instruction and conversions
template <bool kBf16>
struct Half {
    typedef _Float16 T;
    typedef T v2 __attribute__((ext_vector_type(2)));
    typedef T v8 __attribute__((ext_vector_type(8)));
    static __device__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    template <int kByte>
    static __device__ v2 codes(uint32_t w) {
        return __builtin_bit_cast(v2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, kByte));
    }
    static __device__ float wide(uint32_t h) { return h2f((half_bits)h); }
};
template <>
struct Half<true> {
    typedef __bf16 T;
    typedef T v2 __attribute__((ext_vector_type(2)));
    typedef T v8 __attribute__((ext_vector_type(8)));
    static __device__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    template <int kByte>
    static __device__ v2 codes(uint32_t w) {
        return __builtin_bit_cast(v2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, kByte));
    }
    static __device__ float wide(uint32_t h) { return __uint_as_float(h << 16); }
};

// 8 codes -> their exact 16-bit values, in order
template <bool kBf16>
__device__ inline typename Half<kBf16>::v8 codes8(uint32_t w) {
    typedef Half<kBf16> H;
    const typename H::v2 a = H::template codes<0>(w), b = H::template codes<1>(w), c = H::template codes<2>(w),
                         d = H::template codes<3>(w);
    return typename H::v8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// largest value of the four lanes l, l ^ 16, l ^ 32, l ^ 48 (lanes of one column)
__device__ inline float column_max(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float column_sum(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One sequence's rows and the key tiles that a row tile of it can see.  Device
// values (lengths, offsets, prefixes) are brought into range here, so that no
// later index can leave its buffer.
struct Seq {
    int64_t row0;   // first token row of q
    int q_len, length, past, prefix;
};

__device__ inline Seq sequence(const KvAttnArgs& a, int b) {
    Seq s;
    int64_t q0 = (int64_t)b * a.max_q, q1 = q0 + a.max_q;
    if (a.q_offsets) {
        q0 = a.q_offsets[b];
        q1 = a.q_offsets[b + 1];
    }
    q0 = q0 < 0 ? 0 : (q0 > a.tokens ? a.tokens : q0);
    q1 = q1 < q0 ? q0 : (q1 > a.tokens ? a.tokens : q1);
    s.row0 = q0;
    s.q_len = (int)(q1 - q0 > a.max_q ? a.max_q : q1 - q0);
    const int n = (int)(q1 - q0);
    const int64_t most = a.max_len;
    int64_t len = a.lengths[b];
    len = len < 0 ? 0 : (len > most ? most : len);
    s.length = (int)len;
    s.past = s.length - n;
    const int pre = a.prefix ? a.prefix[b] : 0;
    s.prefix = pre < 0 ? 0 : (pre > s.length ? s.length : pre);
    return s;
}

// Rows of q that are no sequence's queries get zeros and lse = -inf where the call asks for
// it (a.fill): those in front of the first offset and behind the last, shared out among
// the row tiles of all sequences, and a sequence's queries past max_q among its own.
__device__ inline void fill_rows(const KvAttnArgs& a, int64_t from, int64_t to, int64_t stripe, int64_t stripes, int h) {
    const int lanes = a.c.blocks * 8;  // 8 dims each
    for (int64_t r = from + stripe; r < to; r += stripes)
        for (int i = threadIdx.x; i < a.group * lanes; i += blockDim.x) {
            const int oh = h * a.group + i / lanes;
            *reinterpret_cast<uint4*>(a.out + r * a.ldo + oh * a.hso + i % lanes * 8) = make_uint4(0, 0, 0, 0);
            if (a.lse && i % lanes == 0) a.lse[r * a.q_heads + oh] = -INFINITY;
        }
}
__device__ inline void fill_rest(const KvAttnArgs& a, const Seq& s, int b, int rt, int h) {
    const auto row = [&](int i) {
        const int64_t r = a.q_offsets[i];
        return r < 0 ? 0 : (r > a.tokens ? a.tokens : r);
    };
    const int64_t stripe = (int64_t)b * a.row_tiles + rt, stripes = (int64_t)a.batch * a.row_tiles;
    fill_rows(a, 0, row(0), stripe, stripes, h);
    fill_rows(a, row(a.batch), a.tokens, stripe, stripes, h);
    fill_rows(a, s.row0 + s.q_len, s.row0 + (s.length - s.past), rt, a.row_tiles, h);
}

// Key tiles that the queries [i0, i1] can see: tiles [0, head) for the prefix, then
// [low, low + n - head): a run of n tiles, numbered 0 .. n - 1.
struct Span {
    int head, low, n;
};

__device__ inline Span span_of(const Seq& s, int i0, int i1, int window) {
    const int p1 = s.past + i1;                      // last position
    int p0 = s.past + i0;
    p0 = p0 < 0 ? 0 : p0;
    Span r{0, 0, 0};
    if (p1 < 0 || s.length == 0) return r;
    const int lo = window > 0 && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
    int hi = p1 + 1;                                 // first key past the causal ones
    if (s.prefix > hi) hi = s.prefix;
    r.low = lo / kTile;
    const int pre = (s.prefix + kTile - 1) / kTile;
    r.head = pre < r.low ? pre : r.low;
    r.n = r.head + (hi + kTile - 1) / kTile - r.low;
    return r;
}

// A segment, one kv head of one row tile with n key tiles, is cut into this many
// parts, nearly equal, each for one workgroup (at least one part: rows that see
// nothing still get their zeros).
__device__ inline int parts_of(const KvAttnArgs& a, int n) {
    int p = (n + a.chunk_tiles - 1) / a.chunk_tiles;
    p = p > a.chunks ? a.chunks : p;
    return p < 1 ? 1 : p;
}

// First token of tile n of a span.
__device__ inline int tile_token(const Span& span, int n) { return (n < span.head ? n : n - span.head + span.low) * kTile; }

// Where the two halves (16 keys each) of a tile lie.  kOne: pages hold at least a
// tile, so both are on one page, the second right behind the first.
template <bool kOne>
struct Place {
    const uint8_t* codes[kOne ? 1 : 2];   // slab + the keys' K codes
    const uint8_t* scales[kOne ? 1 : 2];  // slab + the keys' place among the scales
    bool live[kOne ? 1 : 2];              // the page id was in range
};

// The pages of up to 64 of a wave's tiles, n, n + W, ... (W waves): lane i loads those of
// the i-th, so that a tile's address later takes a lane read and no load.
template <bool kOne>
struct Pages {
    int32_t id[kOne ? 1 : 2];
};

template <bool kOne, int W>
__device__ inline Pages<kOne> load_pages(const KvAttnArgs& a, const int32_t* table, const Span& span, int n, int n1,
                                         int length, int lane) {
    Pages<kOne> p;
    const int nn = n + lane * W;
    const int t0 = tile_token(span, nn < n1 ? nn : n);
#pragma unroll
    for (int u = 0; u < (kOne ? 1 : 2); ++u) {
        const int t = t0 + 16 * u;
        p.id[u] = table[(t < length ? t : length - 1) >> a.c.page_shift];  // past the end: the last page, masked
        // waited for here: else the compiler, which sees a load on one path only, waits for
        // every DMA before each lane read
        asm volatile("" : "+v"(p.id[u]));
    }
    return p;
}

template <int NB, bool kOne>
__device__ inline Place<kOne> place_of(const KvAttnArgs& a, const Pages<kOne>& pages, int slot, int h, int t0) {
    Place<kOne> w;
    const uint32_t slab = (uint32_t)a.c.page_size * (68 * NB);
#pragma unroll
    for (int u = 0; u < (kOne ? 1 : 2); ++u) {
        const int32_t id = __builtin_amdgcn_readlane(pages.id[u], slot);
        w.live[u] = (uint32_t)id < (uint32_t)a.c.pages;
        const uint8_t* base = a.c.data + (uint64_t)((w.live[u] ? (uint32_t)id : 0u) * (uint64_t)a.c.heads + (uint32_t)h) * slab;
        const uint32_t at = (uint32_t)(t0 + 16 * u) & (uint32_t)(a.c.page_size - 1);
        w.codes[u] = base + at * 32 * NB;
        w.scales[u] = base + at * 2 * NB;
    }
    return w;
}

// A tile in LDS: K codes (1024 NB bytes, 32 NB a key), V codes (the same), then for
// each half the scales of K and of V (32 NB bytes each).  A DMA instruction moves 16
// bytes a lane (codes) or 4 (scales, and the codes of a half that has only 512 bytes).
template <int NB, bool kOne>
struct Stage {
    static constexpr int kScales = 2048 * NB;
    static constexpr int kBytes = kScales + (NB == 4 ? 512 : 256);
    static constexpr int kIns = (kOne || NB > 1 ? 2 * NB : 8) + (kOne ? (NB == 4 ? 2 : 1) : 2);
};

__device__ inline __amdgpu_buffer_rsrc_t slab_rsrc(const uint8_t* base) {  // every access is inside the slab
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, 0x7fffffff, 0x00020000);
}
__device__ inline void dma16(__amdgpu_buffer_rsrc_t src, uint8_t* lds, uint32_t lane_offset, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, (int)lane_offset, (int)offset, 0, 0);
}
__device__ inline void dma4(__amdgpu_buffer_rsrc_t src, uint8_t* lds, uint32_t lane_offset, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 4, (int)lane_offset, (int)offset, 0, 0);
}

// Requests a tile; lane i's bytes land at i times their size from the place given.  `v`
// is where the V codes are behind the K codes, `s` the lane's scale bytes behind theirs.
template <int NB, bool kOne>
__device__ inline void request(const Place<kOne>& w, uint8_t* lds, int lane, uint32_t v, const uint32_t (&s)[2]) {
#pragma unroll
    for (int u = 0; u < (kOne ? 1 : 2); ++u) {
        const __amdgpu_buffer_rsrc_t codes = slab_rsrc(w.codes[u]), scales = slab_rsrc(w.scales[u]);
        constexpr int kHalf = kOne ? 1024 * NB : 512 * NB;
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // K, V
            uint8_t* to = lds + x * 1024 * NB + u * kHalf;
            const uint32_t from = x ? v : 0;
            if constexpr (kHalf >= 1024) {
#pragma unroll
                for (int o = 0; o < kHalf; o += 1024) dma16(codes, to + o, lane * 16, from + o);
            } else {
#pragma unroll
                for (int o = 0; o < kHalf; o += 256) dma4(codes, to + o, lane * 4, from + o);
            }
        }
        if (kOne) {
            dma4(scales, lds + Stage<NB, kOne>::kScales, s[0], 0);
            if (NB == 4) dma4(scales, lds + Stage<NB, kOne>::kScales + 256, s[1], 0);
        } else if (lane < 16 * NB) {
            dma4(scales, lds + Stage<NB, kOne>::kScales + u * 64 * NB, s[0], 0);
        }
    }
}

template <int n>
__device__ inline void wait_loads() {  // all but the n newest
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(n) : "memory");
}

// A tile's share of one lane, codes and scales of its two halves, out of LDS: K codes
// at k, V codes at v, K scales at s and V scales 32 NB bytes behind, the second halves
// 512 NB (codes) and 64 NB bytes behind the first.  Instructions of their own, with
// their wait: for an LDS read of its own the compiler waits for every DMA under way.
typedef unsigned v2u __attribute__((ext_vector_type(2)));

__device__ inline void read_share(uint32_t (&kc)[2][2], uint32_t (&vc)[2][2], uint32_t (&ks)[2][2], uint32_t (&vs)[2][2],
                                  uint32_t k, uint32_t v, uint32_t s) {
    v2u r[8];
    asm volatile(
        "ds_read_b64 %0, %8\n ds_read_b64 %1, %8 offset:512\n"
        "ds_read_b64 %2, %9\n ds_read_b64 %3, %9 offset:512\n"
        "ds_read_b64 %4, %10\n ds_read_b64 %5, %10 offset:64\n"
        "ds_read_b64 %6, %10 offset:32\n ds_read_b64 %7, %10 offset:96\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
        : "v"(k), "v"(v), "v"(s)
        : "memory");
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kc[u][i] = r[u][i];
            vc[u][i] = r[2 + u][i];
            ks[u][i] = r[4 + u][i];
            vs[u][i] = r[6 + u][i];
        }
}

__device__ inline void read_share(uint32_t (&kc)[2][4], uint32_t (&vc)[2][4], uint32_t (&ks)[2][4], uint32_t (&vs)[2][4],
                                  uint32_t k, uint32_t v, uint32_t s) {
    v4u r[8];
    asm volatile(
        "ds_read_b128 %0, %8\n ds_read_b128 %1, %8 offset:1024\n"
        "ds_read_b128 %2, %9\n ds_read_b128 %3, %9 offset:1024\n"
        "ds_read_b128 %4, %10\n ds_read_b128 %5, %10 offset:128\n"
        "ds_read_b128 %6, %10 offset:64\n ds_read_b128 %7, %10 offset:192\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
        : "v"(k), "v"(v), "v"(s)
        : "memory");
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kc[u][i] = r[u][i];
            vc[u][i] = r[2 + u][i];
            ks[u][i] = r[4 + u][i];
            vs[u][i] = r[6 + u][i];
        }
}

__device__ inline void read_share(uint32_t (&kc)[2][8], uint32_t (&vc)[2][8], uint32_t (&ks)[2][8], uint32_t (&vs)[2][8],
                                  uint32_t k, uint32_t v, uint32_t s) {
    v4u r[16];
    asm volatile(
        "ds_read_b128 %0, %16\n ds_read_b128 %1, %16 offset:16\n"
        "ds_read_b128 %2, %16 offset:2048\n ds_read_b128 %3, %16 offset:2064\n"
        "ds_read_b128 %4, %17\n ds_read_b128 %5, %17 offset:16\n"
        "ds_read_b128 %6, %17 offset:2048\n ds_read_b128 %7, %17 offset:2064\n"
        "ds_read_b128 %8, %18\n ds_read_b128 %9, %18 offset:16\n"
        "ds_read_b128 %10, %18 offset:256\n ds_read_b128 %11, %18 offset:272\n"
        "ds_read_b128 %12, %18 offset:128\n ds_read_b128 %13, %18 offset:144\n"
        "ds_read_b128 %14, %18 offset:384\n ds_read_b128 %15, %18 offset:400\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7]),
          "=&v"(r[8]), "=&v"(r[9]), "=&v"(r[10]), "=&v"(r[11]), "=&v"(r[12]), "=&v"(r[13]), "=&v"(r[14]), "=&v"(r[15])
        : "v"(k), "v"(v), "v"(s)
        : "memory");
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            kc[u][i] = r[2 * u + i / 4][i % 4];
            vc[u][i] = r[4 + 2 * u + i / 4][i % 4];
            ks[u][i] = r[8 + 2 * u + i / 4][i % 4];
            vs[u][i] = r[12 + 2 * u + i / 4][i % 4];
        }
}

// The scale of block b of the i-th of a lane's four keys
template <bool kBf16, int NB>
__device__ inline float scale_at(const uint32_t (&w)[NB * 2], int i, int b) {
    const int j = i * NB + b;
    if (kBf16) return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
    return Half<false>::wide((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
}

// A row's end, from its reference m and the sum l of its weights: 0 for a row that sees
// nothing, and NaN, like the row's output, where a score was no number.
__device__ inline float norm_of(float l) { return l == 0.0f ? 0.0f : 1.0f / (6.0f * l); }
__device__ inline float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// How weights are kept in the 16-bit type's range.  A row's reference is a maximum that
// stays as it was until a score passes it by 2^kSlack, so that few tiles rescale (2048
// queries behind 2048 tokens, 64 / 8 heads of 128, bfloat16: 268 us, 312 with no slack).
// A weight that is far above a row's others is rounded less often the closer the reference
// is to it (an equal one is a power of two): with two roundings, in fp16, the output's
// error is 1.5 times that of its own rounding at a slack of 2^7, 1.3 at 2^2 and 1.25 at
// none, for a 4096-token prompt, at 0, 4 and 11 % of its time (355 us).
// In fp16 weights are 2^9 times e^(s - reference), at most 2^11 so, and the scales A
// that they meet are taken times 2^(4 - e), 2^e the first power above every finite A the
// wave has met (a larger one than before rescales the sums).  Products are then below
// 2^15, and a weight is rounded at 2^-34 of the reference's: enough as long as the key that
// draws the weight does not have values far below others that draw next to none.  So once
// the A's that a wave has met (of keys in sight or not) span more than 2^kSpan, it goes on
// with fp32 products, each as two bfloat16 numbers that hold it to 2^-18, in two matrix
// instructions.  A 4096-token prompt of 64 heads of 128 takes 372 us, 366 without the
// sizes, 560 in the wide form; 64 sequences of 8192, 64 / 8 heads, 93, 92 and 105.
template <bool kBf16>
constexpr float kSlack = kBf16 ? 8.0f : 2.0f;
template <bool kBf16>
constexpr float kShift = kBf16 ? 0.0f : 9.0f;
constexpr int kLeastLarge = -11;  // 2^(4 - e) is an fp16 number
constexpr int kSpan = 14;

// The sizes of A that a wave has met (fp16): all that are finite are below 2^large, and
// those that are not 0 have bits of at least `low`, a power of 2 or 0.  The guess that it
// starts with, 2^-5 .. 2^3, spares most waves the search in their first tile (decode of 64
// sequences in a window of 1024 tokens: 23.4 us without it, 22.6 with it); where that
// tile does not fit, its own sizes take the guess's place.
struct Sizes {
    int large = 3, low = 10 << 10;
    bool guess = true;
};

// The products P A of a lane's 8 weights with a block's scales, in the order of the
// keys.  bfloat16: fp32 products, rounded once, as the output is.  fp16: the weights are
// rounded to fp16 and multiplied there, two roundings, each of the output's size: packed
// products on scales that are paired once a tile take half the instructions (a
// 4096-token prompt of 64 heads of 128: 453 us, 486 with one rounding).
template <bool kBf16, int NB>
struct Weights {
    uint32_t a[2][2 * NB];
    __device__ void take(const uint32_t (&vs)[2][2 * NB], int) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) a[u][i] = vs[u][i];
    }
    __device__ typename Half<true>::v8 times(const float (&w)[2][4], int b) const {
        typename Half<true>::v8 r;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) r[4 * u + i] = (__bf16)(w[u][i] * scale_at<true, NB>(a[u], i, b));
        return r;
    }
};
template <int NB>
struct Weights<false, NB> {
    Half<false>::v2 a[2][2][NB];  // half, pair of keys, block
    __device__ void take(const uint32_t (&vs)[2][2 * NB], int e) {
        const _Float16 f = (_Float16)__builtin_amdgcn_exp2f((float)(4 - e));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int j = 2 * i * NB + b, k = j + NB;  // block b of keys 2 i and 2 i + 1
                    const uint32_t lo = (vs[u][j >> 1] >> (16 * (j & 1))) & 0xffffu, hi = vs[u][k >> 1] >> (16 * (k & 1));
                    a[u][i][b] = __builtin_bit_cast(Half<false>::v2, lo | hi << 16) * Half<false>::v2{f, f};
                }
    }
    __device__ Half<false>::v8 times(const float (&w)[2][4], int b) const {
        Half<false>::v2 r[4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                r[2 * u + i] = Half<false>::v2{(_Float16)w[u][2 * i], (_Float16)w[u][2 * i + 1]} * a[u][i][b];
        return Half<false>::v8{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
    }
};

// V^T for dims 64 b + 4 m + j of a block: a word holds two tokens' dims 0 .. 3; pairing the
// words' nibbles makes bytes (token 0, token 1) and (token 2, token 3) of one dim
struct Nibbles {
    uint32_t ev[2], od[2];  // dims 0 and 2, dims 1 and 3
};
__device__ inline Nibbles pair_nibbles(uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1) {
    Nibbles n;
    n.ev[0] = (a0 & 0x0f0f0f0fu) | ((b0 << 4) & 0xf0f0f0f0u);
    n.od[0] = ((a0 >> 4) & 0x0f0f0f0fu) | (b0 & 0xf0f0f0f0u);
    n.ev[1] = (a1 & 0x0f0f0f0fu) | ((b1 << 4) & 0xf0f0f0f0u);
    n.od[1] = ((a1 >> 4) & 0x0f0f0f0fu) | (b1 & 0xf0f0f0f0u);
    return n;
}
template <bool kBf16>
__device__ inline typename Half<kBf16>::v8 values_of(const Nibbles& n, int j) {
    typedef Half<kBf16> H;
    const uint32_t x0 = j & 1 ? n.od[0] : n.ev[0], x1 = j & 1 ? n.od[1] : n.ev[1];
    typename H::v2 e[4];
    e[0] = j < 2 ? H::template codes<0>(x0) : H::template codes<1>(x0);
    e[1] = j < 2 ? H::template codes<2>(x0) : H::template codes<3>(x0);
    e[2] = j < 2 ? H::template codes<0>(x1) : H::template codes<1>(x1);
    e[3] = j < 2 ? H::template codes<2>(x1) : H::template codes<3>(x1);
    return typename H::v8{e[0].x, e[0].y, e[1].x, e[1].y, e[2].x, e[2].y, e[3].x, e[3].y};
}

// What is done to the scores: a factor alone, which then rides on the exponential's
// argument; a cap or a distance term (or a factor of 0); a cap far above most scores.
//
// The cap is cap (1 - 2 / (1 + e^2y)), y = s / cap, which is off by up to 2^-23 of the cap:
// 1e-5 of a weight at a cap of 64.  A larger one, which has to leave the scores far below it
// as they are, takes cap (y + y z q(z)), z = y^2, at |y| <= 1/2, with q fitted to the least
// largest error of (tanh y / y - 1) / z on [0, 1/4]: within 2^-23.7 of tanh y with fp32's
// roundings; past 1/2 the other form is within 2^-20 of its value.  In kernels of their own,
// since as branches of one they cost ordinary caps 5 to 18 % (a 4096-token prompt of 64
// heads of 128, cap 50: 467 us, 488 to 500 so); cap 1000 takes 630.
enum Form { kFactor, kTerms, kFarCap };
constexpr float kFarFrom = 64.0f * kLog2e;  // in units of log2 e, as KvAttnArgs::cap
constexpr float kTanhSmall = 0.5f;
__device__ inline float tanh_small(float y) {
    const float z = y * y;
    const float q = fmaf(fmaf(fmaf(0.01725699193775654f, z, -0.05305295065045357f), z, 0.1332598775625229f), z, -0.33333149552345276f);
    return fmaf(y, z * q, y);
}

// What a page holds past a sequence's end may be anything: the scales of V are taken as 0
// there (the lane's i-th key of half u if 16 u + i >= left), and on no page.
template <int NB>
__device__ inline void mask_scales(uint32_t (&vs)[2][2 * NB], bool live0, bool live1, int left) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                const int w = i * NB + bb;
                const bool keep = (16 * u + i < left) & (u ? live1 : live0);
                vs[u][w >> 1] = keep ? vs[u][w >> 1] : vs[u][w >> 1] & (w & 1 ? 0xffffu : 0xffff0000u);
            }
}

// Takes a tile's scales of V into the sizes met, and the sums to a larger power of 2 if
// one is needed.  False, and nothing changed, if the sizes would span more than 2^kSpan.
template <int NB, int T>
__device__ inline __attribute__((always_inline)) bool meet(const uint32_t (&vs)[2][2 * NB], v4f (&acc)[T][NB][4], Sizes& sizes) {
    // none is negative, so the numbers are in the order of their bits (and take three a step)
    typedef Half<false>::v2 h2;
    h2 big = __builtin_bit_cast(h2, vs[0][0]), small = big;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
            big = __builtin_elementwise_maximum(big, __builtin_bit_cast(h2, vs[u][i]));
            small = __builtin_elementwise_minimum(small, __builtin_bit_cast(h2, vs[u][i]));
        }
    const us2 b = __builtin_bit_cast(us2, big), l = __builtin_bit_cast(us2, small);
    const int top_bits = b.x > b.y ? b.x : b.y, low_bits = l.x < l.y ? l.x : l.y;
    const bool above = top_bits >= (sizes.large + 15) << 10;
    if (__ballot(above | (low_bits < sizes.low))) {
        us2 least = {0xffff, 0xffff};  // less 1: a 0 is the largest
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) least = __builtin_elementwise_min(least, __builtin_bit_cast(us2, vs[u][i]) - us2{1, 1});
        const int not_0 = least.x < least.y ? least.x : least.y;
        if (__ballot(above | (not_0 + 1 < sizes.low))) {  // and not only blocks of zeros
            us2 finite = {0, 0};  // numbers moved up to 0x8400 and past it, the rest below
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i)
                    finite = __builtin_elementwise_max(finite, __builtin_bit_cast(us2, vs[u][i]) + us2{0x8400, 0x8400});
            const int top = finite.x > finite.y ? finite.x : finite.y;
            const Sizes met = sizes.guess ? Sizes{kLeastLarge, 0x7c00} : sizes;
            int large = (((int)column_max((float)top) - 0x8400) >> 10) - 14;
            large = __builtin_amdgcn_readfirstlane(large > met.large ? large : met.large);
            int low = (1 - (int)column_max((float)-not_0)) & 0x1fc00;
            low = __builtin_amdgcn_readfirstlane(low < met.low ? low : met.low);
            // subnormal numbers reach 2^10 below the first exponent
            if (large + 15 - (low ? low >> 10 : -10) > kSpan + 1) return false;
            const float drop = __builtin_amdgcn_exp2f((float)(sizes.large - large));
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][bb][j] *= drop;
            sizes = Sizes{large, low};
        }
    }
    sizes.guess = false;
    return true;
}

// One workgroup: one sequence, kv head, row tile of 16 T query rows (token-major,
// then the heads of the group) and a run of key tiles, which its waves take in turn.
// S^T = K Q^T leaves a lane with 4 keys of each half tile and one query row, which is the
// layout that P^T needs as the second operand of O^T = V^T P^T, so P never moves between
// lanes.  Tiles come through a ring of kRing stages of LDS for each wave, filled by DMA:
// a tile is read into registers whole and its stage requested anew before the products,
// and waves meet only at the end.
//
// What bounds it.  Few rows: HBM; 64 sequences of 8191 tokens, 64 / 8 heads of 128, are
// read at 4.9 TB/s, one of 131072 tokens at 4.6; short contexts, a prologue and
// epilogue of about 4 us.  Many rows: the VALU: converting 4-bit codes (shared by the row
// tile), exponentials and the scaling of weights take about 380 instructions for 48 rows
// of 32 keys beside 48 matrix instructions, which hold the SIMD for about 10 of their 16
// cycles each.  A 4096-token prompt of 64 heads of 128: 745 TFLOP/s.
//
// simd_waves(): those of a SIMD, by their registers (512 a lane for all of them).
// T = 3 takes 248 registers with head_dim 128; with 256 two sets of rows already spill.
// 2048 queries behind 2048 tokens, 64 / 8 heads of 128, bfloat16, in row tiles of 16, 32
// and 48: 351, 305 and 268 us.
constexpr int simd_waves(int NB, int T) { return NB == 4 ? 2 : T == 1 ? 4 : NB == 1 ? 3 : 2; }
template <int NB>
constexpr int kRing() { return NB == 1 ? 4 : 2; }

template <bool kBf16, int NB, int T, int W, bool kOne, Form kForm>
__global__ __launch_bounds__(64 * W, simd_waves(NB, T)) void kv_attention_kernel(KvAttnArgs a) {
    typedef Half<kBf16> H;
    typedef typename H::v8 v8;
    typedef Stage<NB, kOne> St;
    constexpr bool kScored = kForm != kFactor;
    constexpr int R = kRing<NB>();
    // V's scales are made ready before the scores or after them: before, with fp16 and
    // kScored (a 4096-token prompt of 64 heads of 128, cap 50, pages of 16 tokens: 478 us,
    // after 500; of 64: 466 and 473); else after (six pieces of prompts of up to 3701
    // tokens, 32 / 8 heads of 128: 202 us, before 207)
    constexpr bool kEarly = !kBf16 && kScored;
    // one LDS array: the waves' rings, later their sums [wave][row][64 NB + 4] and maxima
    // (a second object would make the compiler wait for every DMA before an LDS read)
    constexpr int kRows = kCols * T;
    constexpr int kPart = W * kCols * (64 * NB + 4) * 4, kRings = W * R * St::kBytes;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[(kPart > kRings ? kPart : kRings) + W * kCols * 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    // part-major: the later parts, which shorter sequences lack, come last
    uint32_t id = a.block0 + blockIdx.x;
    const uint32_t segments = (uint32_t)a.batch * (uint32_t)a.row_tiles * (uint32_t)a.c.heads;
    const int chunk = (int)(id / segments);
    id -= chunk * segments;
    const uint32_t segment = id;
    const int h = (int)(id % (uint32_t)a.c.heads);
    id /= (uint32_t)a.c.heads;
    // a prompt's last row tiles, which see most, come first
    const int rt = a.row_tiles - 1 - (int)(id % (uint32_t)a.row_tiles);
    const int b = (int)(id / (uint32_t)a.row_tiles);
    const Seq s = sequence(a, b);
    const int rows = s.q_len * a.group;
    const int r0 = rt * kRows;
    if (a.fill && chunk == 0) fill_rest(a, s, b, rt, h);
    if (r0 >= rows) return;
    const int r1 = r0 + kRows < rows ? r0 + kRows : rows;
    const int i0 = r0 / a.group, i1 = (r1 - 1) / a.group;
    const Span span = span_of(s, i0, i1, a.window);
    const int parts = parts_of(a, span.n);
    if (chunk >= parts) return;
    const int n0 = (int)((int64_t)span.n * chunk / parts), n1 = (int)((int64_t)span.n * (chunk + 1) / parts);

    int pos[T], head[T], qi[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int row = r0 + kCols * t + c;
        qi[t] = row < rows ? row / a.group : 0;
        head[t] = h * a.group + (row < rows ? row - qi[t] * a.group : 0);
        pos[t] = s.past + qi[t];
    }
    const int reach = a.window > 0 ? a.window : 0x7fffffff;
    const int pos0 = s.past + i0, pos1 = s.past + i1;

    const int32_t* table = a.table + (int64_t)b * a.ldt;
    const uint32_t P = (uint32_t)a.c.page_size;
    const uint32_t at_v = P * 32 * NB;                        // V codes behind the K codes
    uint32_t at_s[2];                                         // the lane's scale bytes behind their place
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = (lane + 64 * i) * 4 & (128 * NB - 1), half = o / (64 * NB), kv = o / (32 * NB) & 1;
        at_s[i] = P * 64 * NB + kv * P * 2 * NB + half * 32 * NB + (o & (32 * NB - 1));
    }
    uint8_t* ring = smem + wave * R * St::kBytes;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring;
    Pages<kOne> pages;
    uint32_t live = 0;                                        // bits 2 i, 2 i + 1: the halves of the i-th next tile are live
    int first = n0 + wave;
    // requests tile n into a stage, `place` tiles ahead of the one in use
    const auto ask = [&](int n, int stage, int place) {
        int slot = (n - first) / W;
        const Place<kOne> w = place_of<NB, kOne>(a, pages, slot, h, tile_token(span, n));
        live |= ((uint32_t)w.live[0] | (uint32_t)w.live[kOne ? 0 : 1] << 1) << (2 * place);
        request<NB, kOne>(w, ring + stage * St::kBytes, lane, at_v, at_s);
    };
    const int last = n0 + wave + (n1 - 1 - n0 - wave) / W * W;  // the wave's last tile, if it has any
    // requests the tiles from n on, with none under way
    const auto start = [&](int n) __attribute__((always_inline)) {
        first = n;
        pages = load_pages<kOne, W>(a, table, span, first, n1, s.length, lane);
        live = 0;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (first + i * W <= last) ask(first + i * W, i, i);
    };
    if (first < n1) start(first);

    // a factor below 0 is taken into q's sign
    const uint32_t flip = !kScored && a.scale < 0.0f ? 0x80008000u : 0u;
    v8 q[T][NB][2];
    float slope[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const half_bits* qrow = a.q + (s.row0 + qi[t]) * a.ldq + head[t] * a.hsq;
        const bool live_row = r0 + kCols * t + c < rows;
#pragma unroll
        for (int bb = 0; bb < NB; ++bb)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                uint4 x = live_row ? *reinterpret_cast<const uint4*>(qrow + 64 * bb + 16 * g + 8 * st) : make_uint4(0, 0, 0, 0);
                x = make_uint4(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
                q[t][bb][st] = __builtin_bit_cast(v8, x);
            }
        slope[t] = kScored && a.alibi ? a.alibi[head[t]] * kLog2e : 0.0f;
    }

    // a score is x * unit, in units of log2 e
    const float unit = kScored ? 1.0f : fabsf(a.to_s);
    // a row's reference, as what is added to a score to get its weight's exponent; the
    // exponent past which the reference moves (any, for a row that has seen no key yet);
    // the sum of this lane's weights
    float nb[T], thr[T], l[T];
    Sizes sizes;
    v4f acc[T][NB][4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        nb[t] = 0.0f;
        thr[t] = -INFINITY;
        l[t] = 0.0f;
#pragma unroll
        for (int bb = 0; bb < NB; ++bb)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][bb][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }

    int stage = 0, n = first;
    // The loop over the tiles, with V's scales in the 16-bit type until one does not fit in
    // (fp16: then the loop with kWide takes up that tile again)
    const auto run = [&](auto wide) __attribute__((always_inline)) {
        constexpr bool kWide = decltype(wide)::value;
        for (; n < n1; n += W) {
            const int t0 = tile_token(span, n);
            const bool live0 = live & 1, live1 = live & 2;
            uint32_t kc[2][NB * 2];  // keys 16 u + c: group g's dims, 8 bytes a block
            uint32_t ks[2][NB * 2];  // scales of keys 16 u + 4 g .. + 3
            uint32_t vc[2][NB * 2];  // values of keys 16 u + 4 g .. + 3: dims 64 b + 4 c .. + 3
            uint32_t vs[2][NB * 2];
            if (n + (R - 1) * W <= last)
                wait_loads<(R - 1) * St::kIns>();  // the tiles requested after it stay in flight
            else
                wait_loads<0>();
            const uint32_t st = ring_at + stage * St::kBytes;
            read_share(kc, vc, ks, vs, st + (c * 32 + g * 8) * NB, st + 1024 * NB + (g * 128 + c * 8) * NB,
                       st + St::kScales + g * 8 * NB);
            live >>= 2;
            const int nn = n + R * W;
            if (nn <= last) {
                if ((nn - first) / W >= 64) {
                    first = nn;
                    pages = load_pages<kOne, W>(a, table, span, first, n1, s.length, lane);
                }
                ask(nn, stage, R - 1);
            }
            stage = stage + 1 < R ? stage + 1 : 0;
            // every key of the tile visible to every row: no masks
            const bool whole = live0 & live1 & (pos0 >= 0) &
                               ((t0 + kTile <= s.prefix) |
                                ((t0 + kTile - 1 <= pos0) & ((a.window == 0) | (pos1 - t0 < a.window))));
            Weights<kBf16, NB> scales;  // not with kWide
            const auto take = [&]() __attribute__((always_inline)) {
                if (!whole) mask_scales<NB>(vs, live0, live1, s.length - t0 - 4 * g);
                if constexpr (!kBf16 && !kWide)
                    if (!meet<NB, T>(vs, acc, sizes)) return false;
                if constexpr (!kWide) scales.take(vs, sizes.large);
                return true;
            };
            if constexpr (kEarly)
                if (!take()) break;
            float x[T][2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v8 k[NB][2];
#pragma unroll
                for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                    for (int st = 0; st < 2; ++st) k[bb][st] = codes8<kBf16>(kc[u][2 * bb + st]);
                float sk[4][NB];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int bb = 0; bb < NB; ++bb) sk[i][bb] = scale_at<kBf16, NB>(ks[u], i, bb) * unit;
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    v4f p[NB];
#pragma unroll
                    for (int bb = 0; bb < NB; ++bb) {
                        p[bb] = H::mfma(k[bb][0], q[t][bb][0], v4f{0.0f, 0.0f, 0.0f, 0.0f});
                        p[bb] = H::mfma(k[bb][1], q[t][bb][1], p[bb]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[t][u][i] = kScored ? p[0][i] * sk[i][0] : fmaf(p[0][i], sk[i][0], nb[t]);
#pragma unroll
                        for (int bb = 1; bb < NB; ++bb) x[t][u][i] = fmaf(p[bb][i], sk[i][bb], x[t][u][i]);
                    }
                }
            }
            if (kScored) {
                if (a.softcap > 0.0f) {
                    // the scores that may be past the polynomial: of a near cap all, of a far one few tiles'
                    bool past = true;
                    if constexpr (kForm == kFarCap) {
                        float most = 0.0f;
#pragma unroll
                        for (int t = 0; t < T; ++t)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    x[t][u][i] *= a.to_y;
                                    most = fmaxf(most, fabsf(x[t][u][i]));
                                }
                        past = __ballot(most > kTanhSmall) != 0;
                    }
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        const float top = a.cap + nb[t];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float y = x[t][u][i];
                                if (past) {
                                    const float e = __builtin_amdgcn_exp2f(y * (kForm == kFarCap ? 2.0f * kLog2e : a.to_e));
                                    x[t][u][i] = fmaf(__builtin_amdgcn_rcpf(1.0f + e), -2.0f * a.cap, top);
                                }
                                if constexpr (kForm == kFarCap)
                                    x[t][u][i] = fabsf(y) > kTanhSmall ? x[t][u][i] : fmaf(tanh_small(y), a.cap, nb[t]);
                            }
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < T; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[t][u][i] = fmaf(x[t][u][i], a.to_s, nb[t]);
                }
                if (a.alibi) {
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        const float away = (float)(pos[t] - t0 - 4 * g);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[t][u][i] = fmaf(-slope[t], fabsf(away - (float)(16 * u + i)), x[t][u][i]);
                    }
                }
            }
            if (!whole) {
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = t0 + 16 * u + 4 * g + i;
                            // bitwise, so that this is compares and a select: short circuits became
                            // branches, and among them the compiler lost a copy of a score
                            const bool see = (((j < s.prefix) & (pos[t] >= 0)) | ((j <= pos[t]) & (pos[t] - j < reach))) &
                                             (u ? live1 : live0);
                            x[t][u][i] = see ? x[t][u][i] : -INFINITY;
                        }
            }
            if constexpr (!kEarly)
                if (!take()) break;
            typedef Half<kBf16 || kWide> V;
            typename V::v8 pa[T][NB], rest[kWide ? T : 1][NB];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float top = x[t][0][0];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, x[t][u][i]);
                if (__ballot(top > thr[t])) {  // some row's reference moves, or is its first
                    top = column_max(top);
                    const bool fresh = thr[t] == -INFINITY;
                    // (a fresh row with no key in sight stays as it is)
                    float by = top - kShift<kBf16>;
                    by = fresh ? (top == -INFINITY ? 0.0f : by) : fmaxf(by, 0.0f);
                    const float drop = fresh ? 0.0f : __builtin_amdgcn_exp2f(-by);
                    thr[t] = fresh & (top == -INFINITY) ? thr[t] : kShift<kBf16> + kSlack<kBf16>;
                    nb[t] -= by;
                    l[t] *= drop;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][u][i] -= by;
#pragma unroll
                    for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t][bb][j] *= drop;
                }
                float w[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[u][i] = __builtin_amdgcn_exp2f(x[t][u][i]);
                        l[t] += w[u][i];
                    }
                if constexpr (kWide) {
                    const float f = __builtin_amdgcn_exp2f((float)(4 - sizes.large));
#pragma unroll
                    for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const bool masked = !whole && x[t][u][i] == -INFINITY;
                                const float p = masked ? 0.0f : w[u][i] * f * scale_at<false, NB>(vs[u], i, bb);
                                pa[t][bb][4 * u + i] = (__bf16)p;
                                rest[t][bb][4 * u + i] = (__bf16)(p - (float)pa[t][bb][4 * u + i]);
                            }
                } else {
#pragma unroll
                    for (int bb = 0; bb < NB; ++bb) pa[t][bb] = scales.times(w, bb);
                    // a masked key's value may be no number: its product is 0
                    if (!whole) {
#pragma unroll
                        for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    pa[t][bb][4 * u + i] = x[t][u][i] == -INFINITY ? (typename H::T)0.0f : pa[t][bb][4 * u + i];
                    }
                }
            }
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                const Nibbles v = pair_nibbles(vc[0][2 * bb], vc[0][2 * bb + 1], vc[1][2 * bb], vc[1][2 * bb + 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const typename V::v8 va = values_of<kBf16 || kWide>(v, j);
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        acc[t][bb][j] = V::mfma(va, pa[t][bb], acc[t][bb][j]);
                        if constexpr (kWide) acc[t][bb][j] = V::mfma(va, rest[t][bb], acc[t][bb][j]);
                    }
                }
            }
        }
    };
    run(std::false_type{});
    if constexpr (!kBf16) {
        if (n < n1) {
            wait_loads<0>();
            start(n);
            stage = 0;
            run(std::true_type{});
        }
    }

    // join the waves, 16 rows at a time: O^T row 4 g + i of acc[bb][j] is dim 64 bb + 4 (4 g + i) + j
    float (*part)[kCols][64 * NB + 4] = reinterpret_cast<float (*)[kCols][64 * NB + 4]>(smem);
    float2 (*ml)[kCols] = reinterpret_cast<float2 (*)[kCols]>(smem + sizeof(smem) - W * kCols * 8);
    const int d0 = tid & 15;  // 16 lanes a row, 4 dims a step
    wait_loads<0>();  // this wave's DMA has landed; after the barrier every wave's
    const float grow = kBf16 ? 1.0f : __builtin_amdgcn_exp2f((float)(sizes.large - 4));
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const float ls = column_sum(l[t]);
        const float ms = thr[t] == -INFINITY ? -INFINITY : -nb[t];
        __syncthreads();  // the rings, or the rows before these, are out of use
#pragma unroll
        for (int bb = 0; bb < NB; ++bb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<v4f*>(&part[wave][c][64 * bb + 4 * (4 * g + i)]) =
                    v4f{acc[t][bb][0][i], acc[t][bb][1][i], acc[t][bb][2][i], acc[t][bb][3][i]} * grow;
        if (g == 0) ml[wave][c] = make_float2(ms, ls);
        __syncthreads();
        // fewer than 4 waves take the 16 rows in turns, more share the blocks of a row
#pragma unroll
        for (int cr = (tid >> 4) & 15; cr < kCols; cr += 4 * W) {
            const int orow = r0 + kCols * t + cr;
            if (orow < r1) {
                float mm = -INFINITY, ll = 0.0f, f[W];
#pragma unroll
                for (int w = 0; w < W; ++w) mm = fmaxf(mm, ml[w][cr].x);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    f[w] = ml[w][cr].x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[w][cr].x - mm);
                    ll = fmaf(ml[w][cr].y, f[w], ll);
                }
                const int oi = orow / a.group;
                const int64_t tok = s.row0 + oi;
                const int oh = h * a.group + orow - oi * a.group;
                const int64_t slot = ((int64_t)segment * a.chunks + chunk) * a.slot_rows + kCols * t + cr;
                const float norm = parts > 1 ? 1.0f : norm_of(ll);
#pragma unroll
                for (int bb = W <= 4 ? 0 : tid >> 8; bb < NB; bb += W <= 4 ? 1 : W / 4) {
                    v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const v4f y = *reinterpret_cast<const v4f*>(&part[w][cr][64 * bb + 4 * d0]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[j] = fmaf(y[j], f[w], o[j]);
                    }
                    if (parts > 1) {
                        *reinterpret_cast<v4f*>(a.part + slot * 64 * NB + 64 * bb + 4 * d0) = o;
                    } else {
                        typedef typename H::T t4 __attribute__((ext_vector_type(4)));
                        typename H::T* dst = reinterpret_cast<typename H::T*>(a.out) + tok * a.ldo + oh * a.hso + 64 * bb + 4 * d0;
                        *reinterpret_cast<t4*>(dst) = t4{(typename H::T)(o[0] * norm), (typename H::T)(o[1] * norm),
                                                         (typename H::T)(o[2] * norm), (typename H::T)(o[3] * norm)};
                    }
                }
                if (d0 == 0 && tid < 256) {
                    if (parts > 1)
                        reinterpret_cast<float2*>(a.part_ml)[slot] = make_float2(mm, ll);
                    else if (a.lse)
                        a.lse[tok * a.q_heads + oh] = lse_of(mm, ll);
                }
            }
        }
    }
}

// Joins the parts of a segment's rows, in the order of its keys.  A workgroup takes
// a.join_rows rows (1 to 16) of one segment: 16 lanes a row, 4 NB dims each, times
// 16 / join_rows sets of lanes that share the parts and meet in LDS.
template <bool kBf16, int NB>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttnArgs a) {
    typedef Half<kBf16> H;
    __shared__ float red[16][64 * NB + 4], red_l[16];
    const int tid = threadIdx.x;
    const uint32_t segment = blockIdx.x / (uint32_t)a.join_groups;
    const int e = (int)(segment / (uint32_t)a.c.heads), h = (int)(segment % (uint32_t)a.c.heads);
    const int b = e / a.row_tiles, rt = a.row_tiles - 1 - (e - b * a.row_tiles);
    const Seq s = sequence(a, b);
    const int rows = s.q_len * a.group;
    const int t0 = rt * a.tile_rows;
    if (t0 >= rows) return;
    const int t1 = t0 + a.tile_rows < rows ? t0 + a.tile_rows : rows;
    const int parts = parts_of(a, span_of(s, t0 / a.group, (t1 - 1) / a.group, a.window).n);
    if (parts < 2) return;  // written already
    const int set = tid >> 4, d0 = tid & 15;
    const int rr = set % a.join_rows, cl = set / a.join_rows, step = 16 / a.join_rows;
    const int cr = (int)(blockIdx.x % (uint32_t)a.join_groups) * a.join_rows + rr, row = t0 + cr;
    // rows past the last read the last row's parts
    const int64_t base0 = (int64_t)segment * a.chunks * a.slot_rows + (row < t1 ? cr : t1 - 1 - t0);
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    float m = -INFINITY, l = 0.0f;
    v4f o[NB];
#pragma unroll
    for (int bb = 0; bb < NB; ++bb) o[bb] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kAhead = NB == 4 ? 2 : 4;  // parts in flight
    for (int w = cl; w < parts; w += step * kAhead) {
        float2 p[kAhead];
        v4f x[kAhead][NB];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = base0 + (int64_t)(w + k * step < parts ? w + k * step : w) * a.slot_rows;
            p[k] = ml[at];
#pragma unroll
            for (int bb = 0; bb < NB; ++bb)
                x[k][bb] = *reinterpret_cast<const v4f*>(a.part + at * 64 * NB + 64 * bb + 4 * d0);
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            p[k] = w + k * step < parts ? p[k] : make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, p[k].x);
        }
        const float base = top == -INFINITY ? 0.0f : top;
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = top;
        l *= keep;
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) o[bb] *= keep;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float f = __builtin_amdgcn_exp2f(p[k].x - base);
            l = fmaf(p[k].y, f, l);
#pragma unroll
            for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[bb][j] = fmaf(x[k][bb][j], f, o[bb][j]);
        }
    }
    float top = m;
    if (step > 1) {  // the sets of a row meet: rr, rr + join_rows, ...
        if (d0 == 0) red_l[set] = m;
        __syncthreads();
        for (int k = 0; k < step; ++k) top = fmaxf(top, red_l[rr + k * a.join_rows]);
        __syncthreads();
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) *reinterpret_cast<v4f*>(&red[set][64 * bb + 4 * d0]) = o[bb] * f;
        if (d0 == 0) red_l[set] = l * f;
        __syncthreads();
        if (cl > 0) return;
        l = 0.0f;
        for (int k = 0; k < step; ++k) l += red_l[rr + k * a.join_rows];
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) {
            o[bb] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < step; ++k) o[bb] += *reinterpret_cast<const v4f*>(&red[rr + k * a.join_rows][64 * bb + 4 * d0]);
        }
    }
    if (row >= t1) return;
    const int qi = row / a.group;
    const int64_t tok = s.row0 + qi;
    const int oh = h * a.group + row - qi * a.group;
    const float norm = norm_of(l);
#pragma unroll
    for (int bb = 0; bb < NB; ++bb) {
        typedef typename H::T t4 __attribute__((ext_vector_type(4)));
        typename H::T* dst = reinterpret_cast<typename H::T*>(a.out) + tok * a.ldo + oh * a.hso + 64 * bb + 4 * d0;
        *reinterpret_cast<t4*>(dst) = t4{(typename H::T)(o[bb][0] * norm), (typename H::T)(o[bb][1] * norm),
                                         (typename H::T)(o[bb][2] * norm), (typename H::T)(o[bb][3] * norm)};
    }
    if (d0 == 0 && a.lse) a.lse[tok * a.q_heads + oh] = lse_of(top, l);
}

inline Form form_of(const KvAttnArgs& a) {
    if (a.softcap > 0.0f && a.cap > kFarFrom) return kFarCap;
    return a.softcap > 0.0f || a.alibi || fabsf(a.scale) < 1e-30f ? kTerms : kFactor;
}

template <bool kBf16, int NB, int T, int W, bool kOne>
void launch_main(const KvAttnArgs& a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.batch * a.row_tiles * a.c.heads * a.chunks, most = ((int64_t)1 << 25) / W;
    const dim3 block(64 * W);
    for (int64_t b0 = 0; b0 < blocks; b0 += most) {  // a grid holds fewer than 2^32 lanes
        KvAttnArgs x = a;
        x.block0 = (uint32_t)b0;
        const dim3 grid((unsigned)(blocks - b0 < most ? blocks - b0 : most));
        switch (form_of(a)) {
            case kFarCap: hipLaunchKernelGGL((kv_attention_kernel<kBf16, NB, T, W, kOne, kFarCap>), grid, block, 0, stream, x); break;
            case kTerms: hipLaunchKernelGGL((kv_attention_kernel<kBf16, NB, T, W, kOne, kTerms>), grid, block, 0, stream, x); break;
            default: hipLaunchKernelGGL((kv_attention_kernel<kBf16, NB, T, W, kOne, kFactor>), grid, block, 0, stream, x);
        }
    }
}

template <bool kBf16, int NB, int T, int W>
void launch_tiles(const KvAttnArgs& a, hipStream_t stream) {
    if (a.c.page_size >= kTile)
        launch_main<kBf16, NB, T, W, true>(a, stream);
    else
        launch_main<kBf16, NB, T, W, false>(a, stream);
}

template <bool kBf16, int NB>
hipError_t launch(const KvAttnArgs& a, hipStream_t stream) {
    if (a.tile_rows == kCols && a.waves == 4)
        launch_tiles<kBf16, NB, 1, 4>(a, stream);
    else if (a.tile_rows == kCols && a.waves == 8)
        launch_tiles<kBf16, NB, 1, 8>(a, stream);
    if constexpr (NB < 4) {
        if (a.tile_rows == 2 * kCols)
            launch_tiles<kBf16, NB, 2, 4>(a, stream);
        else if (a.tile_rows == 3 * kCols && a.waves == 4)
            launch_tiles<kBf16, NB, 3, 4>(a, stream);
    }
    if constexpr (NB == 2) {
        if (a.waves == 1) launch_tiles<kBf16, NB, 3, 1>(a, stream);
    }
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.chunks > 1) {
        const int64_t joins = (int64_t)a.batch * a.row_tiles * a.c.heads * a.join_groups;
        hipLaunchKernelGGL((kv_join_kernel<kBf16, NB>), dim3((unsigned)joins), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace i8mp
