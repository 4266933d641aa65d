// Attention over the 4-bit key/value cache: the cut of a call into workgroups, and
// the fp16 kernels.
#include <cfloat>
#include <cmath>

#include "attention_kernels.h"

namespace i8mp {

namespace {

// How the keys are cut.  A part costs its workgroup a prologue and epilogue of about
// 4 us and the join its launch and sums, so there are no more parts than fill the chip
// once (one sequence: all parts are alike) or twice (several, which may differ in length:
// 64 sequences of 2048 to 8192 tokens, 64 / 8 heads of 128, took 89 us at 0.75, 80 at 2
// and 78 us at 4 times the chip's 1024 workgroups; equal ones 109, 113 and 116; one
// sequence of 131072 tokens 29, 32 and 39).
//
// Contexts of up to whole_tiles() are not cut, the join costs more than a longer loop.  Few
// segments (one kv head of one row tile each) leave most CUs idle so, and the limit is low
// (8 of them, 1024 tokens: 10.2 us whole, 11.9 cut; 2048: 15.1 and 12.0); many fill the
// chip whole (128 of 2048 tokens: 16 and 21 us; 256 of 4096: 27 and 33).  Whole contexts
// of up to 256 segments take workgroups of 8 waves (256 of 2048 tokens: 17.9 us, 19.8
// with 4, 20.2 with 16; 512: 29.4 and 27.9).  Row tiles of several sets of rows (T > 1):
// 176 segments of 1000 tokens 21 us whole, 29 and 5 cut, 64 of 4000 49 us, 24 and 5.
int whole_tiles(int64_t segments, int T, int NB) {
    const int n = segments < 64 ? 32 : segments < 128 || T > 1 ? 64 : 128;
    return NB == 4 ? n / 2 : n;
}

// Row tiles that there are, where batch * row_tiles counts every sequence as the longest.
int64_t real_segments(const KvAttnArgs& a) {
    const int64_t most = (int64_t)a.batch * a.row_tiles, some = a.tokens * a.group / a.tile_rows + a.batch;
    return (some < most ? some : most) * a.c.heads;
}

// Prompts of so many row tiles that single waves fill the chip 3/2 times (head_dim 128:
// it holds 2048) take workgroups of one wave, which has its row tile's keys for itself: a
// quarter of the prologues, no sums to join.  Waves of 4 / 1, us: 5504 row tiles of a
// 4096-token prompt 422 / 368, 3520 of 8 prompts of 512 97 / 82, 2752 of a 2048-token
// one 138 / 127, but 2736 behind 2048 tokens 301 / 296, with a distance bias 378 / 411,
// and 1500 of ragged pieces 239 / 282.
// head_dim 64 (3 waves a SIMD): 5504 row tiles 223 / 244, so 4 there.
void plan(KvAttnArgs& a) {
    const int64_t rows = (int64_t)a.max_q * a.group;
    const int NB = a.c.blocks;
    const int T = NB == 4 || rows <= kCols ? 1 : rows <= 2 * kCols ? 2 : 3;
    a.tile_rows = kCols * T;
    a.row_tiles = (int32_t)ceil_div(rows, a.tile_rows);
    const int64_t segments = (int64_t)a.batch * a.row_tiles * a.c.heads;
    // keys that a row tile sees: beside a window, those of the prefix are not known here
    int64_t near = a.max_len;
    if (a.window > 0 && a.window + (int64_t)a.max_q + 2 * kTile < near) near = a.window + (int64_t)a.max_q + 2 * kTile;
    const int64_t chip = 256 * simd_waves(NB, T);
    const int64_t tiles = ceil_div(near, kTile), most = ceil_div(a.prefix ? a.max_len : near, kTile);
    const int64_t fill = a.batch > 1 ? 2 * chip : chip;
    int64_t per = ceil_div(tiles * segments, fill);
    per = per < 4 ? 4 : per;
    if (most <= whole_tiles(segments, T, NB) || segments >= 4 * chip) per = most > 0 ? most : 1;
    a.chunk_tiles = (int32_t)per;
    // No more parts than fill the chip, whatever a prefix beside a window may reach (all of a
    // table of 131072 tokens took 64 sequences of 64 / 8 heads 926 MiB of workspace and 233000
    // workgroups for 35 tiles each, 354 us; 8 MiB and 33 us so): where it does reach further,
    // the parts are longer.
    const int64_t parts = ceil_div(most > 0 ? most : 1, per), full = ceil_div(fill, segments);
    a.chunks = (int32_t)(parts < full ? parts : full);
    a.waves = T == 1 && a.chunks == 1 && segments <= 256 && most >= 8 ? 8 : 4;
    if (T == 3 && NB == 2 && a.chunks == 1 && real_segments(a) * 2 >= 1024 * simd_waves(NB, T) * 3) a.waves = 1;
    a.slot_rows = (int32_t)(rows < a.tile_rows ? rows : a.tile_rows);
    a.join_rows = 1;
    // a row's parts are shared by as many sets of lanes as have two each (one workgroup a row
    // whatever the parts: 10 to 21 us for 64 to 176 segments of 48 rows, so 5); with many
    // segments there are rows enough, and a workgroup takes all it can
    while (a.join_rows < 16 && a.join_rows < a.slot_rows && (segments >= 256 || 16 / a.join_rows * 2 > a.chunks))
        a.join_rows *= 2;
    a.join_groups = (int32_t)ceil_div(a.slot_rows, a.join_rows);
}

}  // namespace

size_t kv_attention_workspace(const KvAttnArgs& args) {
    KvAttnArgs a = args;
    plan(a);
    return a.chunks == 1 ? 0 : (size_t)a.batch * a.row_tiles * a.c.heads * a.chunks * a.slot_rows * (64 * a.c.blocks + 2) * 4;
}

hipError_t launch_kv_attention(const KvAttnArgs& args, void* workspace, hipStream_t stream) {
    KvAttnArgs a = args;
    plan(a);
    const float f = a.scale / 6.0f;
    a.to_s = f * kLog2e;
    // a cap past 1e20 leaves scores as one of 1e20 does; y is finite, so that a score of 0 stays 0 under the smallest
    const float cap = std::fmin(a.softcap, 1e20f);
    const auto finite = [](float y) { return std::fmax(std::fmin(y, FLT_MAX), -FLT_MAX); };
    a.to_y = cap > 0.0f ? finite(f / cap) : 0.0f;
    a.to_e = finite(2.0f * kLog2e * a.to_y);
    a.cap = cap * kLog2e;
    a.part = static_cast<float*>(workspace);
    a.part_ml = a.part + (a.chunks == 1 ? 0 : (int64_t)a.batch * a.row_tiles * a.c.heads * a.chunks * a.slot_rows * 64 * a.c.blocks);
    if (a.c.bf16) return launch_kv_attention_bf16(a, stream);
    return a.c.blocks == 1 ? launch<false, 1>(a, stream) : a.c.blocks == 2 ? launch<false, 2>(a, stream) : launch<false, 4>(a, stream);
}

}  // namespace i8mp
