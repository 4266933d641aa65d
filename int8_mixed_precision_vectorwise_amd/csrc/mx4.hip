// Microscaled 4-bit matrices: quantization of 16-bit matrices by rows and by
// columns, and dequantization.
//
// Elements are E2M1 in blocks of 32 along k under a power of two 2^E, held as the
// byte E + 127:
//   E = max(floor(log2 max |x|) - 2, -127): the block's largest value falls into
//       [4, 8) times 2^E, of which E2M1 reaches 6;
//   code = sign | E2M1 magnitude nearest to |x| / 2^E, ties to even, at most 6;
//   a block that holds a NaN or an infinity has the byte 255 (no number) and codes 0.
// Dividing by a power of two is exact, so every code is decided exactly: the
// hardware's conversion (v_cvt_scalef32_pk_fp4_*) gives the definition's codes for
// all 16-bit values, checked value by value.  Both passes stream: 2 bytes an
// element in, 17/32 of a byte out, and memory bounds them.  4096 x 22016 bfloat16: by
// rows 37 us (6.1 TB/s), by columns 37.5, back 34 (6.7 TB/s); one row of 5120 2.2 and 2.0.
#include "common.h"
#include "launch_limit.h"
#include "mx4.h"
#include "mx4_util.h"
#include "quant_util.h"

namespace i8mp {

namespace {

constexpr int kThreads = 256;

// at any element's address
typedef v4u v4u_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// ---- by rows ------------------------------------------------------------------
// A lane has 8 neighbouring elements, four lanes a block, sixteen a word of scales.  A
// workgroup is kThreads / lanes rows of `lanes` chunks at a time, and takes kRowSteps of
// them: as many 16-byte loads in flight a lane (eight: no faster).  Addresses may be any
// element's: 16-byte loads that are not aligned take 4096 x 22016 39 us instead of 38.
constexpr int kRowSteps = 4;

template <bool kBf16, int kSteps>
__device__ inline void quantize_rows(const MxQuantArgs& a, uint32_t bx, uint32_t by) {
    const int lanes = 1 << a.lane_shift, rows = kThreads >> a.lane_shift;
    const int64_t c = (int64_t)bx * lanes + (threadIdx.x & (lanes - 1));  // chunk of 8 elements
    const int64_t row0 = (int64_t)by * (rows * kSteps) + (threadIdx.x >> a.lane_shift);
    if (c * 8 >= a.q.kp()) return;  // whole words of scales leave: kp is a multiple of 128
    const int64_t left = a.q.k - c * 8;
    v4u x[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        x[i] = v4u{0, 0, 0, 0};
        const int64_t r = row0 + i * rows;
        if (r >= a.q.rows) continue;
        const half_bits* p = a.x + r * a.ldx + c * 8;
        if (left >= 8) {
            x[i] = *reinterpret_cast<const v4u_any*>(p);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) x[i][e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int64_t r = row0 + i * rows;
        if (r >= a.q.rows) continue;
        us2 m = __builtin_elementwise_max(__builtin_elementwise_max(mags(x[i][0]), mags(x[i][1])),
                                          __builtin_elementwise_max(mags(x[i][2]), mags(x[i][3])));
        uint32_t top = m.x > m.y ? m.x : m.y;
        const auto up = [](uint32_t p, uint32_t q) { return p > q ? p : q; };
        top = up(top, (uint32_t)dpp_i32<kDppQuadSwap1>((int32_t)top));
        top = up(top, (uint32_t)dpp_i32<kDppQuadSwap2>((int32_t)top));
        const uint32_t byte = scale_byte<kBf16>(top);
        uint32_t codes = encode8<kBf16>(x[i][0], x[i][1], x[i][2], x[i][3], scale_value(byte));
        if (byte == 255u) codes = 0;
        *reinterpret_cast<uint32_t*>(a.q.codes + r * a.q.ldc + c * 4) = codes;
        uint32_t word = byte << (8 * (threadIdx.x >> 2 & 3));   // four blocks' bytes meet
        word |= (uint32_t)dpp_i32<kDppHalfMirror>((int32_t)word);
        word |= (uint32_t)dpp_i32<kDppRowMirror>((int32_t)word);
        if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(a.q.scales + r * a.q.lds + (c >> 2)) = word;
    }
}

// ---- by columns ------------------------------------------------------------------
// x [k x rows] read as it lies, its transpose quantized: a block is 32 rows of one
// column.  A wave has 32 rows of 128 columns, a lane two columns: the block's
// maximum needs no other lane, and 32 loads of 4 bytes are in flight a lane.  The
// codes (16 bytes a column) meet in LDS, so that a column leaves as 64 contiguous
// bytes.
constexpr int kColCols = 128, kColRows = 32 * kThreads / 64, kColPitch = kColRows / 2 + 16;

// Every lane's dword, the bytes of four rows in turn, becomes one row's bytes of the quad's four lanes
__device__ inline uint32_t transpose4(uint32_t d) {
    const bool upper = threadIdx.x & 2, odd = threadIdx.x & 1;
    d = __builtin_amdgcn_perm((uint32_t)dpp_i32<kDppQuadSwap2>((int32_t)d), d, upper ? 0x03020706u : 0x05040100u);
    return __builtin_amdgcn_perm((uint32_t)dpp_i32<kDppQuadSwap1>((int32_t)d), d, odd ? 0x03070105u : 0x06020400u);
}

// The same 32 rows of two columns a lane, quantized by rows: a block is a row of 16 lanes.  Two rows' maxima share a
// register; a lane has one byte of codes a row, and quads of lanes exchange them into words.
template <bool kBf16>
__device__ inline void quantize_beside(const MxQuantArgs& a, const uint32_t (&x)[kMxBlock], int64_t c0, int64_t r0, uint8_t* scales) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t kept[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kMxBlock; i += 4) {
        uint32_t codes = 0;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const uint32_t u = x[i + j], v = x[i + j + 1];
            us2 m = __builtin_elementwise_max(mags(__builtin_amdgcn_perm(v, u, 0x05040100u)), mags(__builtin_amdgcn_perm(v, u, 0x07060302u)));
            const auto with = [&](uint32_t other) { m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, other)); };
            with((uint32_t)dpp_i32<kDppQuadSwap1>(__builtin_bit_cast(int32_t, m)));
            with((uint32_t)dpp_i32<kDppQuadSwap2>(__builtin_bit_cast(int32_t, m)));
            with((uint32_t)dpp_i32<kDppHalfMirror>(__builtin_bit_cast(int32_t, m)));
            with((uint32_t)dpp_i32<kDppRowMirror>(__builtin_bit_cast(int32_t, m)));
            const uint32_t b0 = scale_byte<kBf16>(m.x), b1 = scale_byte<kBf16>(m.y);
            const uint32_t both = (b0 == 255u ? 0u : encode2<kBf16, 0>(0u, u, scale_value(b0))) |
                                  (b1 == 255u ? 0u : encode2<kBf16, 0>(0u, v, scale_value(b1)) << 8);
            codes |= both << (8 * j);
            if ((lane & 15) == ((i + j) & 15)) kept[(i + j) >> 4] = b0;
            if ((lane & 15) == ((i + j + 1) & 15)) kept[(i + j) >> 4] = b1;
        }
        codes = transpose4(codes);
        const int64_t r = r0 + i + (lane & 3);
        if (r < a.rows.rows) *reinterpret_cast<uint32_t*>(a.rows.codes + r * a.rows.ldc + c0 / 2 + (lane & ~3)) = codes;
        __builtin_amdgcn_sched_barrier(0);   // four rows in registers at a time
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) scales[(wave * kMxBlock + 16 * h + (lane & 15)) * 4 + (lane >> 4)] = (uint8_t)kept[h];
}

template <bool kBf16, bool kAligned, bool kBeside>
__device__ inline void quantize_columns(const MxQuantArgs& a, uint32_t bx, uint32_t by, uint8_t* codes, uint32_t* scales, uint32_t* row_scales) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)bx * kColCols, c = c0 + 2 * lane;
    const int64_t r0 = (int64_t)by * kColRows + wave * kMxBlock;
    uint32_t x[kMxBlock];
    const half_bits* p = a.x + r0 * a.ldx + c;
    const bool two = c + 1 < a.q.rows, one = c < a.q.rows;
    if constexpr (kAligned) {   // rows past the last are out of range, and read as zeros
        const int64_t there = a.q.k - r0 < kMxBlock ? a.q.k - r0 : kMxBlock;
        const int ld = (int)a.ldx * 2, range = there > 0 ? ((int)there - 1) * ld + (int)(a.q.rows - c0 < kColCols ? a.q.rows - c0 : kColCols) * 2 : 0;
        const __amdgpu_buffer_rsrc_t src = range_of(a.x + r0 * a.ldx + c0, __builtin_amdgcn_readfirstlane(range));
        const int at = two ? lane * 4 : kOut;
#pragma unroll
        for (int i = 0; i < kMxBlock; ++i) x[i] = __builtin_amdgcn_raw_buffer_load_b32(src, at + i * ld, 0, 0);
        if (one && !two) {
#pragma unroll
            for (int i = 0; i < kMxBlock; ++i) x[i] = r0 + i < a.q.k ? p[i * a.ldx] : 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kMxBlock; ++i) {
            x[i] = 0;
            if (r0 + i >= a.q.k) continue;
            if (two) x[i] = *reinterpret_cast<const u32_any*>(p + i * a.ldx);
            else if (one) x[i] = p[i * a.ldx];
        }
    }
    if (kBeside && a.rows.codes) quantize_beside<kBf16>(a, x, c0, r0, reinterpret_cast<uint8_t*>(row_scales));
    us2 m = mags(x[0]);
#pragma unroll
    for (int i = 1; i < kMxBlock; ++i) m = __builtin_elementwise_max(m, mags(x[i]));
    const uint32_t b0 = scale_byte<kBf16>(m.x), b1 = scale_byte<kBf16>(m.y);
    const float s0 = scale_value(b0), s1 = scale_value(b1);
    v4u k0, k1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = x[8 * i + 2 * j], v = x[8 * i + 2 * j + 1];
            lo[j] = __builtin_amdgcn_perm(v, u, 0x05040100u);
            hi[j] = __builtin_amdgcn_perm(v, u, 0x07060302u);
        }
        k0[i] = b0 == 255u ? 0u : encode8<kBf16>(lo[0], lo[1], lo[2], lo[3], s0);
        k1[i] = b1 == 255u ? 0u : encode8<kBf16>(hi[0], hi[1], hi[2], hi[3], s1);
    }
    constexpr int kWaves = kThreads / 64;
    static_assert(kWaves == 4, "a word of scales a column");
    *reinterpret_cast<v4u*>(codes + 2 * lane * kColPitch + wave * 16) = k0;
    *reinterpret_cast<v4u*>(codes + (2 * lane + 1) * kColPitch + wave * 16) = k1;
    reinterpret_cast<uint8_t*>(scales)[2 * lane * kWaves + wave] = (uint8_t)b0;
    reinterpret_cast<uint8_t*>(scales)[(2 * lane + 1) * kWaves + wave] = (uint8_t)b1;
    __syncthreads();
    const int64_t first = (int64_t)by * kWaves;   // all four blocks are there: kp is a multiple of 128
#pragma unroll
    for (int t = threadIdx.x; t < kColCols * kWaves; t += kThreads) {
        const int col = t / kWaves, part = t % kWaves;
        if (c0 + col < a.q.rows)
            *reinterpret_cast<v4u*>(a.q.codes + (c0 + col) * a.q.ldc + (first + part) * 16) =
                *reinterpret_cast<const v4u*>(codes + col * kColPitch + part * 16);
    }
    if (threadIdx.x < kColCols && c0 + threadIdx.x < a.q.rows)
        *reinterpret_cast<uint32_t*>(a.q.scales + (c0 + threadIdx.x) * a.q.lds + first) = scales[threadIdx.x];
    const int64_t row = (int64_t)by * kColRows + threadIdx.x;
    if (kBeside && a.rows.codes && threadIdx.x < kColRows && row < a.rows.rows)
        *reinterpret_cast<uint32_t*>(a.rows.scales + row * a.rows.lds + c0 / kMxBlock) = row_scales[threadIdx.x];
}

// Workgroups go to the XCDs in turn; each XCD gets a run of neighbours, two along the rows of x at a time, so that
// the lines they share are found in its L2: those of x where its rows begin anywhere, and those of codes, of which a
// workgroup writes halves.  us of 4096 x 22016: 37.5 (in turn 40), rows that begin at any 4 bytes 38 (53), at any 2
// bytes 47 (56); of 2048 x 4096: 4.8 (4.3), 4.9 (4.8 to 5.8), 7.4 (8 to 12).  So few workgroups stay in turn where
// rows begin at 4 bytes.
__device__ inline void column_place(uint32_t id, uint32_t blocks_x, uint32_t blocks_y, uint32_t& bx, uint32_t& by) {
    constexpr uint32_t kXcds = 8;
    const uint32_t full = blocks_x * blocks_y / kXcds * kXcds;
    const uint32_t t = id < full ? id % kXcds * (full / kXcds) + id / kXcds : id;
    const uint32_t pair = t / (2 * blocks_x), in = t - pair * 2 * blocks_x;
    const bool two = 2 * pair + 1 < blocks_y;
    // divided by vector instructions: back to scalars, which the buffers' descriptors must be
    by = __builtin_amdgcn_readfirstlane(2 * pair + (two ? in & 1 : 0));
    bx = __builtin_amdgcn_readfirstlane(two ? in >> 1 : in);
}

// Up to kMxJobs matrices in one launch: each has its run of workgroups.  kBeside: one of them by rows and by columns at
// once, which takes 88 registers in place of 47.
template <bool kBf16, bool kBeside>
__global__ __launch_bounds__(kThreads) void quantize_kernel(MxQuantJobs jobs) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[kColCols * kColPitch];
    __shared__ uint32_t scales[kColCols], row_scales[kColRows];
    int j = 0;
#pragma unroll
    for (int i = 1; i < kMxJobs; ++i) j += i < jobs.count && blockIdx.x >= jobs.job[i].block0;
    const MxQuantArgs& a = jobs.job[j];
    const uint32_t id = blockIdx.x - a.block0;
    uint32_t by = id / a.blocks_x, bx = id - by * a.blocks_x;
    if (a.columns) {
        if (a.runs) column_place(id, a.blocks_x, a.blocks_y, bx, by);
        if (a.aligned) quantize_columns<kBf16, true, kBeside>(a, bx, by, codes, scales, row_scales);
        else quantize_columns<kBf16, false, kBeside>(a, bx, by, codes, scales, row_scales);
    } else {
        if (a.few) quantize_rows<kBf16, 1>(a, bx, by);
        else quantize_rows<kBf16, kRowSteps>(a, bx, by);
    }
}

// ---- back -----------------------------------------------------------------------

// Outputs that take more than half the last-level cache pass it by: 4096 x 22016 quantized and read back in 72 us
// against 88 (each alone takes 38 and 35 either way), 16384 x 5120 in 67 against 82.  Smaller ones are found there by
// what comes next.
constexpr int64_t kPastCache = 128 << 20;

template <int kType, bool kPast>
__device__ inline void store_out(void* out, int64_t at, const float (&v)[8], int64_t left) {
    if constexpr (kType == I8MP_DTYPE_F32) {
        typedef v4f v4f_any __attribute__((aligned(4)));
        float* p = static_cast<float*>(out) + at;
        if (left >= 8) {
            const v4f lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if constexpr (kPast) {
                __builtin_nontemporal_store(lo, reinterpret_cast<v4f_any*>(p));
                __builtin_nontemporal_store(hi, reinterpret_cast<v4f_any*>(p + 4));
            } else {
                *reinterpret_cast<v4f_any*>(p) = lo;
                *reinterpret_cast<v4f_any*>(p + 4) = hi;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) p[e] = v[e];
        }
    } else {
        half_bits h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (kType == I8MP_DTYPE_BF16) h[e] = __builtin_bit_cast(half_bits, (__bf16)v[e]);
            else h[e] = f2h(v[e]);
        }
        half_bits* p = static_cast<half_bits*>(out) + at;
        if (left >= 8) {
            v4u w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
            if constexpr (kPast) __builtin_nontemporal_store(w, reinterpret_cast<v4u_any*>(p));
            else *reinterpret_cast<v4u_any*>(p) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) p[e] = h[e];
        }
    }
}

template <int kType, bool kPast>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(MxDequantArgs a, int lane_shift) {
    const int lanes = 1 << lane_shift, rows = kThreads >> lane_shift;
    const int64_t c = (int64_t)blockIdx.x * lanes + (threadIdx.x & (lanes - 1));
    const int64_t row0 = (int64_t)blockIdx.y * (rows * kRowSteps) + (threadIdx.x >> lane_shift);
    if (c * 8 >= a.q.k) return;
    uint32_t codes[kRowSteps], byte[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const int64_t r = row0 + i * rows;
        if (r >= a.q.rows) continue;
        codes[i] = *reinterpret_cast<const uint32_t*>(a.q.codes + r * a.q.ldc + c * 4);
        byte[i] = a.q.scales[r * a.q.lds + (c >> 2)];
    }
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const int64_t r = row0 + i * rows;
        if (r >= a.q.rows) continue;
        const float s = scale_value(byte[i]);
        float v[8];
#define I8MP_PAIR(p)                                                                  \
    do {                                                                              \
        const f2 u = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.0f, p);     \
        v[2 * p] = u.x * s;                                                           \
        v[2 * p + 1] = u.y * s;                                                       \
    } while (0)
        I8MP_PAIR(0);
        I8MP_PAIR(1);
        I8MP_PAIR(2);
        I8MP_PAIR(3);
#undef I8MP_PAIR
        store_out<kType, kPast>(a.out, r * a.ldout + c * 8, v, a.q.k - c * 8);
    }
}

// lanes of a workgroup along a row of `chunks`, as a shift: at least 16, since padded rows are whole 16s
int row_lanes(int64_t chunks) {
    int s = 4;
    while (s < 8 && ((int64_t)1 << s) < chunks) ++s;
    return s;
}

// Rows in launches whose grid holds them (a grid's second axis ends at 65535).
template <typename F>
hipError_t by_rows(int64_t rows, int64_t chunks, F launch) {
    const int s = row_lanes(chunks);
    const int64_t per = (int64_t)(kThreads >> s) * kRowSteps, most = per * 65535;
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most;
        launch(r, n, dim3((unsigned)ceil_div(chunks, (int64_t)1 << s), (unsigned)ceil_div(n, per)), s);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

// the workgroups of a matrix
int64_t set_blocks(MxQuantArgs& a) {
    int64_t x, y;
    if (a.columns) {
        a.aligned = a.ldx % 2 == 0 && reinterpret_cast<uintptr_t>(a.x) % 4 == 0 && a.ldx <= (int64_t)1 << 24;   // 32 rows stay below 2^31 bytes
        x = ceil_div(a.q.rows, kColCols);
        y = ceil_div(a.q.k, kColRows);
        a.runs = !a.aligned || x * y > 1024;
    } else {
        a.lane_shift = row_lanes(a.q.kp() / 8);
        x = ceil_div(a.q.kp() / 8, (int64_t)1 << a.lane_shift);
        // too few rows to fill the chip with kRowSteps a lane: one each (16 rows of 13824: 3.2 us, four a lane 4.0)
        const int64_t rows = kThreads >> a.lane_shift;
        a.few = x * ceil_div(a.q.rows, rows * kRowSteps) < 256;
        y = ceil_div(a.q.rows, a.few ? rows : rows * kRowSteps);
    }
    a.blocks_x = (uint32_t)x;
    a.blocks_y = (uint32_t)y;
    return x * y;
}

template <bool kBeside>
hipError_t launch_kind(const MxQuantJobs& jobs, int64_t blocks, bool bf16, hipStream_t stream) {
    if (bf16) hipLaunchKernelGGL((quantize_kernel<true, kBeside>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, jobs);
    else hipLaunchKernelGGL((quantize_kernel<false, kBeside>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, jobs);
    return hipGetLastError();
}
hipError_t launch_jobs(const MxQuantJobs& jobs, int64_t blocks, bool bf16, hipStream_t stream) {
    bool beside = false;
    for (int i = 0; i < jobs.count; ++i) beside = beside || jobs.job[i].rows.codes;
    return beside ? launch_kind<true>(jobs, blocks, bf16, stream) : launch_kind<false>(jobs, blocks, bf16, stream);
}

// One matrix of more workgroups than a launch takes: rows of it at a time.
hipError_t in_pieces(const MxQuantArgs& args, hipStream_t stream) {
    const int64_t all = args.columns ? args.q.k : args.q.rows;
    MxQuantArgs a = args;
    int64_t most = all;
    while (set_blocks(a) > i8mp_launch_blocks && most > kMxPad) {
        most = round_up(most / 2, kMxPad);
        (args.columns ? a.q.k : a.q.rows) = most;
    }
    for (int64_t r = 0; r < all; r += most) {
        a = args;
        a.x += r * a.ldx;
        (args.columns ? a.q.k : a.q.rows) = all - r < most ? all - r : most;
        a.q.codes += args.columns ? r / 2 : r * a.q.ldc;
        a.q.scales += args.columns ? r / kMxBlock : r * a.q.lds;
        if (a.rows.codes) {
            a.rows.codes += r * a.rows.ldc;
            a.rows.scales += r * a.rows.lds;
            a.rows.rows = a.q.k;
        }
        MxQuantJobs jobs{};
        jobs.job[0] = a;
        jobs.count = 1;
        const int64_t blocks = set_blocks(jobs.job[0]);
        if (hipError_t e = launch_jobs(jobs, blocks, args.bf16, stream); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int kType>
hipError_t dequantize(const MxDequantArgs& args, hipStream_t stream) {
    constexpr int kElem = kType == I8MP_DTYPE_F32 ? 4 : 2;
    const bool past = args.q.rows * args.q.k * kElem > kPastCache;
    return by_rows(args.q.rows, ceil_div(args.q.k, 8), [&](int64_t r, int64_t n, dim3 grid, int s) {
        MxDequantArgs a = args;
        a.q.codes += r * a.q.ldc;
        a.q.scales += r * a.q.lds;
        a.q.rows = n;
        a.out = static_cast<uint8_t*>(a.out) + r * a.ldout * kElem;
        if (past) hipLaunchKernelGGL((dequantize_kernel<kType, true>), grid, dim3(kThreads), 0, stream, a, s);
        else hipLaunchKernelGGL((dequantize_kernel<kType, false>), grid, dim3(kThreads), 0, stream, a, s);
    });
}

}  // namespace

// Rows and columns at once save a read of x, and a wave works longer on what it has read.  us of a captured backward, at
// once / apart, fp16 (bfloat16 differs by 1 %), by the workgroups that x takes:
//    128   512 x  4096 x 1024   20.0 /  17.7         512  2048 x  4096 x 4096   61.9 /  61.9
//    256  1024 x  4096 x 1024   25.6 /  23.1         605  1333 x  7001 x  900   54.3 /  56.4
//    320  1000 x  5000 x  600   27.2 /  24.1         688  1024 x 11008 x 4096   112  / 114
//    384  1536 x  4096 x 4096   54.9 /  54.2        1024  4096 x  4096 x 4096   97.8 / 100.6
//    430   640 x 11008 x 2048   61.4 /  59.6        4902  7189 x 11008 x 1024   177  / 202
// They cross near 512.  Where x's rows begin at odd elements a second read costs more, and at once is faster by 1 to 7 %
// from 128 workgroups on (2048 x 2560 x 2560, rows of 2563: 38.6 / 40.7); 512 holds for those too.
bool mx4_quantize_both(int64_t rows, int64_t cols) { return ceil_div(rows, kColRows) * ceil_div(cols, kColCols) >= 512; }

hipError_t launch_mx4_quantize(const MxQuantArgs* args, int count, hipStream_t stream) {
    MxQuantJobs jobs{};
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        if (args[i].q.rows == 0 || args[i].q.k == 0) continue;
        MxQuantArgs& a = jobs.job[jobs.count];
        a = args[i];
        const int64_t more = set_blocks(a);
        if (more > i8mp_launch_blocks / kMxJobs) {
            if (hipError_t e = in_pieces(args[i], stream); e != hipSuccess) return e;
            continue;
        }
        a.block0 = (uint32_t)blocks;
        blocks += more;
        ++jobs.count;
    }
    return jobs.count > 0 ? launch_jobs(jobs, blocks, args[0].bf16, stream) : hipSuccess;
}

hipError_t launch_mx4_dequantize(const MxDequantArgs& a, hipStream_t stream) {
    return a.out_dtype == I8MP_DTYPE_F32   ? dequantize<I8MP_DTYPE_F32>(a, stream)
           : a.out_dtype == I8MP_DTYPE_F16 ? dequantize<I8MP_DTYPE_F16>(a, stream)
                                           : dequantize<I8MP_DTYPE_BF16>(a, stream);
}

}  // namespace i8mp
