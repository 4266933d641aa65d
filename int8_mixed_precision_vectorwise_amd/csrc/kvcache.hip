// Writing 16-bit keys and values into the 4-bit cache, and reading them back.
// The format is that of the 4-bit weights: blocks of 64, code = sign and the
// E2M1 magnitude nearest to fl32(|x| * fl32(6 * fl32(1 / A))), A the block's absmax, and
// x' = fl32(E2M1 value * fl32(A / 6)).  A is the absmax of 16-bit numbers and so
// one of them: the cache keeps it in that type, 2 bytes a block, unrounded.
#include "kvcache.h"

namespace i8mp {

namespace {

constexpr int kThreads = 256;

// fp32 of a 16-bit float's bits
template <bool kBf16>
__device__ inline float wide(uint32_t h) {
    return kBf16 ? __uint_as_float(h << 16) : h2f((half_bits)h);
}

template <bool kBf16>
__device__ inline uint32_t narrow(float f) {  // round to nearest even
    return kBf16 ? (uint32_t)__builtin_bit_cast(half_bits, (__bf16)f) : (uint32_t)f2h(f);
}

// E2M1 magnitude code of a non-negative fp32 value, ties to the even code; a NaN gives 0
__device__ inline uint32_t mag_code(float v) {
    return (uint32_t)(v > 0.25f) + (uint32_t)(v >= 0.75f) + (uint32_t)(v > 1.25f) + (uint32_t)(v >= 1.75f) +
           (uint32_t)(v > 2.5f) + (uint32_t)(v >= 3.5f) + (uint32_t)(v > 5.0f);
}

__device__ inline float code_value(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const uint32_t mag = e ? (((e + 126u) << 23) | (m << 22)) : (m ? 0x3f000000u : 0u);
    return __uint_as_float(mag | ((c & 8u) << 28));
}

// slab byte of the V codes of dims 4 m .. 4 m + 3 of block b, token t
__device__ inline int v_byte(int t, int m, int b, int nb) {
    return (t >> 2) * 128 * nb + m * 8 * nb + b * 8 + ((t & 1) * 2 + ((t >> 1) & 1)) * 2;
}

// One lane per 8 dims of one token, head and block, of K or of V: 8 lanes share
// a block, so its absmax takes 3 shuffles.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvMoveArgs a) {
    const int nb = a.c.blocks;
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int part = (int)(t & 7);
    const int64_t blk = t >> 3;
    const int b = (int)(blk % nb);
    const int64_t th = blk / nb;
    const int h = (int)(th % a.c.heads);
    const int64_t tok = th / a.c.heads;
    if (tok >= a.tokens) return;  // 8 lanes of a block leave together
    const int64_t slot = a.slots[tok];
    if (slot < 0 || slot >= (a.c.pages << a.c.page_shift)) return;
    const bool is_v = blockIdx.y != 0;
    const half_bits* src = static_cast<const half_bits*>(is_v ? a.v : a.k) + tok * (is_v ? a.ldv : a.ldk) +
                           h * (is_v ? a.hsv : a.hsk) + b * 64 + part * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8], mx = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = fabsf(wide<kBf16>((w[e >> 1] >> (16 * (e & 1))) & 0xffffu));
        mx = fmaxf(mx, f[e]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 1, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 2, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 4, 64));
    const float inv = mx > 0.0f ? 6.0f * (1.0f / mx) : 0.0f;  // IEEE reciprocal
    uint32_t packed = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t sign = (w[e >> 1] >> (16 * (e & 1) + 15)) & 1u;
        packed |= (mag_code(f[e] * inv) | (sign << 3)) << (4 * e);
    }
    const int at = (int)(slot & (a.c.page_size - 1));
    const int P = a.c.page_size;
    uint8_t* slab = a.c.data + ((slot >> a.c.page_shift) * a.c.heads + h) * a.c.slab();
    if (is_v) {
        uint8_t* codes = slab + P * 32 * nb;
        *reinterpret_cast<uint16_t*>(codes + v_byte(at, part * 2, b, nb)) = (uint16_t)packed;
        *reinterpret_cast<uint16_t*>(codes + v_byte(at, part * 2 + 1, b, nb)) = (uint16_t)(packed >> 16);
    } else {
        *reinterpret_cast<uint32_t*>(slab + at * 32 * nb + (part >> 1) * 8 * nb + b * 8 + (part & 1) * 4) = packed;
    }
    if (part == 0)
        *reinterpret_cast<uint16_t*>(slab + P * (is_v ? 66 : 64) * nb + (at * nb + b) * 2) = (uint16_t)narrow<kBf16>(mx);
}

// One lane per 8 dims, as above.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvMoveArgs a) {
    const int nb = a.c.blocks;
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int part = (int)(t & 7);
    const int64_t blk = t >> 3;
    const int b = (int)(blk % nb);
    const int64_t th = blk / nb;
    const int h = (int)(th % a.c.heads);
    const int64_t tok = th / a.c.heads;
    if (tok >= a.tokens) return;
    const int64_t slot = a.slots[tok];
    const bool is_v = blockIdx.y != 0;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (slot >= 0 && slot < (a.c.pages << a.c.page_shift)) {
        const int at = (int)(slot & (a.c.page_size - 1));
        const int P = a.c.page_size;
        const uint8_t* slab = a.c.data + ((slot >> a.c.page_shift) * a.c.heads + h) * a.c.slab();
        uint32_t packed;
        if (is_v) {
            const uint8_t* codes = slab + P * 32 * nb;
            packed = *reinterpret_cast<const uint16_t*>(codes + v_byte(at, part * 2, b, nb)) |
                     ((uint32_t)*reinterpret_cast<const uint16_t*>(codes + v_byte(at, part * 2 + 1, b, nb)) << 16);
        } else {
            packed = *reinterpret_cast<const uint32_t*>(slab + at * 32 * nb + (part >> 1) * 8 * nb + b * 8 + (part & 1) * 4);
        }
        const float d =
            wide<kBf16>(*reinterpret_cast<const uint16_t*>(slab + P * (is_v ? 66 : 64) * nb + (at * nb + b) * 2)) / 6.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = code_value((packed >> (4 * e)) & 15u) * d;
    }
    const int64_t o = tok * (is_v ? a.ldv : a.ldk) + h * (is_v ? a.hsv : a.hsk) + b * 64 + part * 8;
    void* dst = is_v ? a.v : a.k;
    if (a.out_dtype == I8MP_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + o);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = a.out_dtype == I8MP_DTYPE_BF16 ? narrow<true>(x[2 * e]) | (narrow<true>(x[2 * e + 1]) << 16)
                                                  : narrow<false>(x[2 * e]) | (narrow<false>(x[2 * e + 1]) << 16);
        *reinterpret_cast<uint4*>(static_cast<half_bits*>(dst) + o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

dim3 move_grid(const KvMoveArgs& a) {
    return dim3((unsigned)ceil_div(a.tokens * a.c.heads * a.c.blocks * 8, kThreads), 2);
}

}  // namespace

hipError_t launch_kv_write(const KvMoveArgs& a, hipStream_t stream) {
    if (a.c.bf16)
        hipLaunchKernelGGL(kv_write_kernel<true>, move_grid(a), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(kv_write_kernel<false>, move_grid(a), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvMoveArgs& a, hipStream_t stream) {
    if (a.c.bf16)
        hipLaunchKernelGGL(kv_read_kernel<true>, move_grid(a), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(kv_read_kernel<false>, move_grid(a), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace i8mp
