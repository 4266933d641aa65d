// Internal declarations of the 4-bit key/value cache: its layout, and the
// write, read and attention kernels (gfx950 only).
#pragma once

#include "common.h"

namespace i8mp {

// ---- cache layout -------------------------------------------------------------
// One page of one kv head is a slab: page_size tokens of head_dim = 64 NB
// dimensions, quantized in blocks of 64.  Its four parts:
//   K codes   per token 32 NB bytes: [4 groups g][NB blocks b][8 bytes], dims 64 b + 16 g + 0..15
//   V codes   per 4 tokens 128 NB bytes: [16 groups m][NB blocks b][tokens 0, 2, 1, 3][2 bytes],
//             dims 64 b + 4 m + 0..3
//   K scales  [page_size][NB] block absmax, 2 bytes each;  V scales  the same
// The even element is in a byte's low nibble.  Both code parts are in the order
// in which the attention's matrix operands take them, so a lane's share of a
// tile is one contiguous load: K rows feed the operand of Q K^T (a lane holds
// one token's dims of group g, whole blocks apart so that each block's sum gets
// its own scale); four tokens of V's dims stand together for the operand of
// P V, whose contraction runs over tokens.  A token owns whole bytes in both,
// so writing one never reads another's.
struct KvCache {
    uint8_t* data;
    int64_t pages;
    int32_t heads;
    int32_t page_size, page_shift;   // 16 .. 256, a power of two
    int32_t blocks;                  // NB = head_dim / 64: 1, 2 or 4
    bool bf16;                       // scales (and the 16-bit tensors beside the cache) are bfloat16
    __host__ __device__ int64_t slab() const { return (int64_t)page_size * blocks * 68; }
};

struct KvMoveArgs {
    KvCache c;
    const int64_t* slots;            // [tokens], outside [0, pages * page_size): skipped / read as zeros
    int64_t tokens;
    void* k; int64_t ldk, hsk;       // strides of a token and of a head, in elements
    void* v; int64_t ldv, hsv;
    int32_t out_dtype;               // read only
};
hipError_t launch_kv_write(const KvMoveArgs& a, hipStream_t stream);
hipError_t launch_kv_read(const KvMoveArgs& a, hipStream_t stream);

struct KvAttnArgs {
    KvCache c;
    const half_bits* q; int64_t ldq, hsq;
    half_bits* out; int64_t ldo, hso;
    float* lse;                      // nullable [tokens x q_heads]
    const int32_t* table; int64_t ldt; int32_t table_cols;
    const int32_t* lengths;          // [batch]
    const int32_t* q_offsets;        // nullable [batch + 1]
    const float* alibi;              // nullable [q_heads]
    const int32_t* prefix;           // nullable [batch]
    int32_t batch, q_heads, group;   // group = q_heads / kv heads
    int32_t max_q, window;           // window 0: none
    int64_t tokens;                  // rows of q
    float scale, softcap;            // softcap 0: none
    int64_t max_len;                 // bound on the lengths
    bool fill;                       // zeros for rows of q that are no sequence's queries
    // set by the launcher
    float to_s, to_y, to_e;          // factors of a product of q with E2M1 values and scales A: to its score, in units
                                     // of log2 e, to y = score / cap, and to 2 y in the same units
    float cap;                       // softcap in units of log2 e
    int32_t tile_rows, row_tiles;    // rows of a row tile, row tiles of the longest sequence
    int32_t waves;                   // waves of a workgroup
    int32_t chunk_tiles, chunks;     // key tiles of a part, most parts of a segment (kv head of a row tile)
    int32_t slot_rows;               // rows that a part leaves (up to tile_rows)
    int32_t join_rows, join_groups;  // rows of a workgroup of the join, its workgroups for a segment
    uint32_t block0;                 // first workgroup of the launch
    float* part;                     // [segments][chunks][slot_rows][head_dim] partial sums
    float* part_ml;                  // [segments][chunks][slot_rows][maximum, sum]
};
// workspace of one call (0: none needed)
size_t kv_attention_workspace(const KvAttnArgs& a);
hipError_t launch_kv_attention(const KvAttnArgs& a, void* workspace, hipStream_t stream);
hipError_t launch_kv_attention_bf16(const KvAttnArgs& a, hipStream_t stream);  // its bfloat16 part, with the cut made

}  // namespace i8mp
