// Attention over the 4-bit key/value cache: for a query row at position p of a
// sequence of length L (token j visible iff j < L and (j < prefix, or j <= p and
// p - j < window)),
//   s_j = scale q . k_j,  s_j <- cap tanh(s_j / cap),  s_j <- s_j - slope |p - j|,
//   out = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^s_j  over the visible j,
// in one pass over the cache with a running maximum.  k_j and v_j stay 4-bit up to
// the matrix instructions: an E2M1 value is exact in fp16 and in bfloat16, so the
// products run on the codes' values, and the block scales A / 6 enter in fp32: on
// the 64-deep partial sums of q . k, and on the weights e^s of v.
#include "kvcache.h"

namespace i8mp {

namespace {

constexpr int kWaves = 4;       // waves of a workgroup, each taking every kWaves-th key tile
constexpr int kTile = 32;       // keys of a tile
constexpr int kRows = 16;       // query rows of a row tile: the columns of an MFMA
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
    const int64_t most = a.max_len;
    int64_t len = a.lengths[b];
    len = len < 0 ? 0 : (len > most ? most : len);
    s.length = (int)len;
    s.past = s.length - s.q_len;
    const int pre = a.prefix ? a.prefix[b] : 0;
    s.prefix = pre < 0 ? 0 : (pre > s.length ? s.length : pre);
    return s;
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

// A tile's share of one lane (row r = lane % 16, group g = lane / 16), as loaded.
template <int NB>
struct KeyTile {
    uint32_t k[2][NB * 2];   // keys 16 u + r: group g's dims, 8 bytes a block
    uint32_t v[2][NB * 2];   // values of keys 16 u + 4 g .. + 3: dims 64 b + 4 r .. + 3
    uint32_t ks[2][NB * 2];  // scales of keys 16 u + 4 g .. + 3
    uint32_t vs[2][NB * 2];
    bool live[2];            // the page id was in range
};

template <int N>
__device__ inline void load_words(uint32_t (&d)[N], const uint8_t* p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = reinterpret_cast<const uint4*>(p)[i];
            d[4 * i] = x.x;
            d[4 * i + 1] = x.y;
            d[4 * i + 2] = x.z;
            d[4 * i + 3] = x.w;
        }
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        d[0] = x.x;
        d[1] = x.y;
    }
}

template <int NB>
__device__ inline void load_tile(const KvAttnArgs& a, const int32_t* table, int h, int t0, int length, int lane,
                                 KeyTile<NB>& kt) {
    const int r = lane & 15, g = lane >> 4;
    const int P = a.c.page_size;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        int t = t0 + 16 * u;
        t = t < length ? t : (length - 1) & ~15;        // past the end: the last page again, masked
        const int64_t id = table[t >> a.c.page_shift];
        kt.live[u] = id >= 0 && id < a.c.pages;
        const uint8_t* slab = a.c.data + ((kt.live[u] ? id : 0) * a.c.heads + h) * a.c.slab();
        const int at = t & (P - 1);
        load_words(kt.k[u], slab + (at + r) * 32 * NB + g * 8 * NB);
        load_words(kt.v[u], slab + P * 32 * NB + ((at >> 2) + g) * 128 * NB + r * 8 * NB);
        load_words(kt.ks[u], slab + P * 64 * NB + (at + 4 * g) * 2 * NB);
        load_words(kt.vs[u], slab + P * 66 * NB + (at + 4 * g) * 2 * NB);
    }
}

// 16-bit scale of block b of the i-th of a lane's four tokens
template <bool kBf16, int NB>
__device__ inline float scale_at(const uint32_t (&w)[NB * 2], int i, int b) {
    const int j = i * NB + b;
    return Half<kBf16>::wide((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
}

// One workgroup: one sequence, kv head, row tile of 16 query rows (token-major,
// then the heads of the group) and a run of key tiles.  S^T = K Q^T leaves a
// lane with 4 keys x 2 of one query column, which is the layout that P^T needs
// as the second operand of O^T = V^T P^T, so P never moves between lanes.
template <bool kBf16, int NB>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_attention_kernel(KvAttnArgs a) {
    typedef Half<kBf16> H;
    typedef typename H::v8 v8;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    int64_t id = blockIdx.x;
    const int chunk = (int)(id % a.chunks);
    id /= a.chunks;
    const int h = (int)(id % a.c.heads);
    id /= a.c.heads;
    const int rt = (int)(id % a.row_tiles);
    const int b = (int)(id / a.row_tiles);
    const Seq s = sequence(a, b);
    const int rows = s.q_len * a.group;
    const int r0 = rt * kRows;
    if (r0 >= rows) return;
    const int r1 = r0 + kRows < rows ? r0 + kRows : rows;
    const Span span = span_of(s, r0 / a.group, (r1 - 1) / a.group, a.window);
    const int n0 = chunk * a.chunk_tiles;
    if (chunk > 0 && n0 >= span.n) return;
    const int n1 = n0 + a.chunk_tiles < span.n ? n0 + a.chunk_tiles : span.n;

    const int row = r0 + c;
    const bool live_row = row < rows;
    const int qi = live_row ? row / a.group : 0;
    const int head = h * a.group + (live_row ? row % a.group : 0);
    const int pos = s.past + qi;
    // this row sees keys [0, see_pre) and [see_lo, pos]
    const int see_pre = pos >= 0 ? s.prefix : 0;
    const int see_lo = a.window > 0 ? pos - a.window + 1 : 0;
    const int pos0 = s.past + r0 / a.group, pos1 = s.past + (r1 - 1) / a.group;
    const float slope = a.alibi ? a.alibi[head] * kLog2e : 0.0f;
    const half_bits* qrow = a.q + (s.row0 + qi) * a.ldq + head * a.hsq;
    v8 q[NB][2];
#pragma unroll
    for (int bb = 0; bb < NB; ++bb)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const uint4 x = live_row ? *reinterpret_cast<const uint4*>(qrow + 64 * bb + 16 * g + 8 * st)
                                     : make_uint4(0, 0, 0, 0);
            q[bb][st] = __builtin_bit_cast(v8, x);
        }

    // s in units of log2 e: without a cap the factor goes onto the block scales
    const float pre = a.scale / 6.0f * (a.softcap > 0.0f ? 1.0f : kLog2e);
    const int32_t* table = a.table + (int64_t)b * a.ldt;
    float m = -INFINITY, l = 0.0f;
    v4f acc[NB][4];
#pragma unroll
    for (int bb = 0; bb < NB; ++bb)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[bb][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int n = n0 + wave; n < n1; n += kWaves) {
        const int t0 = (n < span.head ? n : n - span.head + span.low) * kTile;
        KeyTile<NB> kt;
        load_tile<NB>(a, table, h, t0, s.length, lane, kt);
        float sc[2][4];
        // every key of the tile visible to every row: no masks
        const bool whole = kt.live[0] & kt.live[1] & (pos0 >= 0) &
                           ((t0 + kTile <= s.prefix) |
                            ((t0 + kTile - 1 <= pos0) & ((a.window == 0) | (pos1 - t0 < a.window))));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            v4f p[NB];
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                p[bb] = H::mfma(codes8<kBf16>(kt.k[u][2 * bb]), q[bb][0], v4f{0.0f, 0.0f, 0.0f, 0.0f});
                p[bb] = H::mfma(codes8<kBf16>(kt.k[u][2 * bb + 1]), q[bb][1], p[bb]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = p[0][i] * (scale_at<kBf16, NB>(kt.ks[u], i, 0) * pre);
#pragma unroll
                for (int bb = 1; bb < NB; ++bb) x = fmaf(p[bb][i], scale_at<kBf16, NB>(kt.ks[u], i, bb) * pre, x);
                sc[u][i] = x;
            }
        }
        if (a.softcap > 0.0f) {
            const float inv = 2.0f * kLog2e / a.softcap, cap = a.softcap * kLog2e;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // tanh x = (1 - e^-2|x|) / (1 + e^-2|x|), with x's sign
                    const float e = __builtin_amdgcn_exp2f(-fabsf(sc[u][i]) * inv);
                    sc[u][i] = copysignf(cap * (1.0f - e) / (1.0f + e), sc[u][i]);
                }
        }
        if (a.alibi) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[u][i] = fmaf(-slope, fabsf((float)(pos - (t0 + 16 * u + 4 * g + i))), sc[u][i]);
        }
        if (!whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = t0 + 16 * u + 4 * g + i;
                    // bitwise, so that this is compares and a select: short circuits became
                    // branches, and among them the compiler lost a copy of a score
                    const bool see = ((j < see_pre) | ((j >= see_lo) & (j <= pos))) & kt.live[u];
                    sc[u][i] = see ? sc[u][i] : -INFINITY;
                }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[u][i]);
        top = column_max(top);
        if (__ballot(top > m)) {
            const float drop = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
            l *= drop;
#pragma unroll
            for (int bb = 0; bb < NB; ++bb)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[bb][j] *= drop;
            m = top;
        }
        const float base = m == -INFINITY ? 0.0f : m;  // nothing seen yet: e^-inf below stays 0
        float w[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[u][i] = __builtin_amdgcn_exp2f(sc[u][i] - base);
                l += w[u][i];
            }
        // P A, rounded to the 16-bit type: like the output, one rounding of it.  A
        // masked key's scale may be anything, so its product is replaced.
        v8 pa[NB];
#pragma unroll
        for (int bb = 0; bb < NB; ++bb)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = w[u][i] * scale_at<kBf16, NB>(kt.vs[u], i, bb);
                    pa[bb][4 * u + i] = (typename H::T)(whole || sc[u][i] != -INFINITY ? y : 0.0f);
                }
        // V^T: a word holds two tokens' dims 0 .. 3; pairing the words' nibbles makes
        // bytes (token 0, token 1) and (token 2, token 3) of one dim
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) {
            uint32_t ev[2], od[2];  // dims 0 and 2, dims 1 and 3
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t wa = kt.v[u][2 * bb], wb = kt.v[u][2 * bb + 1];
                ev[u] = (wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u);
                od[u] = ((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x0 = j & 1 ? od[0] : ev[0], x1 = j & 1 ? od[1] : ev[1];
                typename H::v2 e[4];
                e[0] = j < 2 ? H::template codes<0>(x0) : H::template codes<1>(x0);
                e[1] = j < 2 ? H::template codes<2>(x0) : H::template codes<3>(x0);
                e[2] = j < 2 ? H::template codes<0>(x1) : H::template codes<1>(x1);
                e[3] = j < 2 ? H::template codes<2>(x1) : H::template codes<3>(x1);
                const v8 va{e[0].x, e[0].y, e[1].x, e[1].y, e[2].x, e[2].y, e[3].x, e[3].y};
                acc[bb][j] = H::mfma(va, pa[bb], acc[bb][j]);
            }
        }
    }

    // join the waves: O^T row 4 g + i of acc[bb][j] is dim 64 bb + 4 (4 g + i) + j
    __shared__ float part[kWaves][kRows][64 * NB + 4];
    __shared__ float ml[kWaves][kRows][2];
    l = column_sum(l);
#pragma unroll
    for (int bb = 0; bb < NB; ++bb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave][c][64 * bb + 4 * (4 * g + i) + j] = acc[bb][j][i];
    if (g == 0) {
        ml[wave][c][0] = m;
        ml[wave][c][1] = l;
    }
    __syncthreads();
    const int cr = tid >> 4, d0 = tid & 15;  // 16 lanes a row, 4 dims a step
    const int orow = r0 + cr;
    if (orow >= r1) return;
    float mm = -INFINITY, ll = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, ml[w][cr][0]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        f[w] = ml[w][cr][0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[w][cr][0] - mm);
        ll = fmaf(ml[w][cr][1], f[w], ll);
    }
    const int64_t tok = s.row0 + orow / a.group;
    const int oh = h * a.group + orow % a.group;
    const int64_t flat = tok * a.q_heads + oh;
    const bool last = a.chunks == 1;
    const float norm = last ? (ll > 0.0f ? 1.0f / (6.0f * ll) : 0.0f) : 1.0f;
#pragma unroll
    for (int bb = 0; bb < NB; ++bb) {
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) x = fmaf(part[w][cr][64 * bb + 4 * d0 + j], f[w], x);
            o[j] = x * norm;
        }
        if (last) {
            typename H::T* dst = reinterpret_cast<typename H::T*>(a.out) + tok * a.ldo + oh * a.hso + 64 * bb + 4 * d0;
            typedef typename H::T t4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<t4*>(dst) = t4{(typename H::T)o[0], (typename H::T)o[1], (typename H::T)o[2], (typename H::T)o[3]};
        } else {
            *reinterpret_cast<float4*>(a.part + (flat * a.chunks + chunk) * 64 * NB + 64 * bb + 4 * d0) =
                make_float4(o[0], o[1], o[2], o[3]);
        }
    }
    if (d0 == 0) {
        if (!last) {
            float* dst = a.part_ml + (flat * a.chunks + chunk) * 2;
            dst[0] = mm;
            dst[1] = ll;
        } else if (a.lse) {
            a.lse[flat] = ll > 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
        }
    }
}

// Joins the chunks of a row in ascending order, one wave a row: so the result does
// not depend on which workgroup ended first.
template <bool kBf16, int NB>
__global__ __launch_bounds__(64) void kv_join_kernel(KvAttnArgs a) {
    typedef Half<kBf16> H;
    const int lane = threadIdx.x;
    const int64_t id = blockIdx.x;
    const int head = (int)(id % a.q_heads);
    const int64_t bi = id / a.q_heads;
    const int qi = (int)(bi % a.max_q);
    const Seq s = sequence(a, (int)(bi / a.max_q));
    if (qi >= s.q_len) return;
    const int row = qi * a.group + head % a.group;
    const int r0 = row / kRows * kRows, rows = s.q_len * a.group;
    const int r1 = r0 + kRows < rows ? r0 + kRows : rows;
    const Span span = span_of(s, r0 / a.group, (r1 - 1) / a.group, a.window);
    int n = (span.n + a.chunk_tiles - 1) / a.chunk_tiles;
    n = n < 1 ? 1 : n;
    const int64_t tok = s.row0 + qi;
    const int64_t flat = tok * a.q_heads + head;
    const float* ml = a.part_ml + flat * a.chunks * 2;
    const float* part = a.part + flat * a.chunks * 64 * NB;
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, ml[2 * i]);
    float l = 0.0f, o[NB];
#pragma unroll
    for (int bb = 0; bb < NB; ++bb) o[bb] = 0.0f;
    for (int i = 0; i < n; ++i) {
        const float f = ml[2 * i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[2 * i] - m);
        l = fmaf(ml[2 * i + 1], f, l);
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) o[bb] = fmaf(part[(int64_t)i * 64 * NB + 64 * bb + lane], f, o[bb]);
    }
    const float norm = l > 0.0f ? 1.0f / (6.0f * l) : 0.0f;
#pragma unroll
    for (int bb = 0; bb < NB; ++bb)
        reinterpret_cast<typename H::T*>(a.out)[tok * a.ldo + head * a.hso + 64 * bb + lane] = (typename H::T)(o[bb] * norm);
    if (lane == 0 && a.lse) a.lse[flat] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// How the keys are cut: enough workgroups to fill the chip, each with at least two
// tiles a wave.
void plan(KvAttnArgs& a) {
    a.row_tiles = (int32_t)ceil_div((int64_t)a.max_q * a.group, kRows);
    int64_t most = a.max_len;
    if (a.window > 0 && !a.prefix && a.window + (int64_t)a.max_q + 2 * kTile < most) most = a.window + (int64_t)a.max_q + 2 * kTile;
    const int64_t tiles = ceil_div(most, kTile);
    const int64_t groups = (int64_t)a.batch * a.c.heads * a.row_tiles;
    const int64_t want = 1024;
    int64_t per = ceil_div(tiles * groups, want);
    per = round_up(per < 2 * kWaves ? 2 * kWaves : per, kWaves);
    a.chunk_tiles = (int32_t)per;
    a.chunks = (int32_t)ceil_div(tiles > 0 ? tiles : 1, per);
}

template <bool kBf16, int NB>
hipError_t launch(const KvAttnArgs& a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.batch * a.row_tiles * a.c.heads * a.chunks;
    hipLaunchKernelGGL((kv_attention_kernel<kBf16, NB>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.chunks > 1) {
        const int64_t joins = (int64_t)a.batch * a.max_q * a.q_heads;
        hipLaunchKernelGGL((kv_join_kernel<kBf16, NB>), dim3((unsigned)joins), dim3(64), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvAttnArgs& args) {
    KvAttnArgs a = args;
    plan(a);
    if (a.chunks <= 1) return 0;
    return (size_t)a.tokens * a.q_heads * a.chunks * (64 * a.c.blocks + 2) * 4;
}

hipError_t launch_kv_attention(const KvAttnArgs& args, void* workspace, hipStream_t stream) {
    KvAttnArgs a = args;
    plan(a);
    a.part = static_cast<float*>(workspace);
    a.part_ml = a.part + (a.chunks > 1 ? a.tokens * a.q_heads * a.chunks * 64 * a.c.blocks : 0);
    if (a.c.bf16)
        return a.c.blocks == 1 ? launch<true, 1>(a, stream) : a.c.blocks == 2 ? launch<true, 2>(a, stream) : launch<true, 4>(a, stream);
    return a.c.blocks == 1 ? launch<false, 1>(a, stream) : a.c.blocks == 2 ? launch<false, 2>(a, stream) : launch<false, 4>(a, stream);
}

}  // namespace i8mp
