// How an attention call is laid out, from sizes alone: plain host arithmetic, shared by
// the launchers and (compiled by itself) their CPU test.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/tq2_attn.h"
#include "tq2_pages.h"

namespace tq2 {

constexpr int kTileRows = 128;           // of a block of the tiled form

// Most blocks of the tiled form's steps, all sequences and key heads together.  The
// steps are those of the longest sequence, or of all of q's rows if it is not given: many
// short sequences then start mostly blocks that find no row, at about 1.5 ns each, and a
// long one among them needs blocks.  1,024 sequences of 64 tokens, 32 heads of 128 on 8
// key heads: 1.3 ms, with 2^18 blocks 1.0, with 2^20 2.1 (0.42 with the longest given); one of
// 32,768 tokens and 1,023 of one: 11.6 ms, 15.4, 12.0.
constexpr int64_t kTileBlocks = int64_t(1) << 19;

// Blocks along each axis of a launch.  An axis holds fewer than 2^32 threads: of 256 to a
// block, 2^24 - 1 blocks.
struct Grid {
  uint32_t x, y, z;
};
constexpr int64_t kAxisBlocks = (int64_t(1) << 24) - 1;

struct AttnPlan {
  bool tiled;                            // the form for many rows (new tokens times heads of a key head)
  int32_t row_tiles;                     // streaming form: 16-row tiles of a step
  int32_t steps;                         // steps of max_q new tokens
  int32_t splits, split_keys;
  size_t workspace;                      // bytes
};

inline int64_t pieces(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline AttnPlan plan_attention(const tq2_paged_attention_args& a) {
  const tq2_paged_cache& c = a.cache;
  AttnPlan plan;
  const int64_t max_q = a.max_q < 1 ? 1 : (a.max_q < c.tokens ? a.max_q : c.tokens);
  const int64_t rows = max_q * (c.q_heads / c.kv_heads);
  // The tiled form reads keys and values once for 128 rows: 64 rows over 16 caches of 4,096
  // take 64 us (103 streaming), 36 rows over 4 of them 27 (35).
  plan.tiled = rows > 32;
  // Two row tiles share the loads of keys and values; wider heads' outputs leave no registers for a second.
  plan.row_tiles = rows <= 16 || c.head_dim > 128 ? 1 : 2;
  const int64_t steps = pieces(rows, plan.tiled ? kTileRows : plan.row_tiles * 16);
  // Steps past the room of the grid are walked over by its blocks.
  const int64_t room = plan.tiled ? kTileBlocks / (c.kv_heads * c.batch) : 65535 / c.kv_heads;
  plan.steps = int32_t(steps < room ? steps : (room < 1 ? 1 : room));
  const int64_t span = a.window ? a.window + max_q + 31 : a.max_kv;  // that a sequence's rows see
  const int64_t most = a.max_kv < kMaxKeys ? a.max_kv : kMaxKeys;
  const int64_t keys = span < most ? span : most;
  const int64_t blocks = c.batch * c.kv_heads * plan.steps;
  const double joined = double(c.tokens) * double(c.q_heads) * double(c.head_dim + 4) * 8.0 / 3e6;  // us a part
  int64_t per, splits;
  if (plan.tiled) {
    // The number of parts with the least time: a block takes about 4.5 us to start and
    // end and 1.9 us for 64 keys of 128 components in 16 bits, twice that in 32; two
    // blocks fit on a CU, or one of wide heads; parts that are joined cost 6 us and
    // their way to memory and back at 3 TB/s (measured; 36 rows over 1,000 keys: 12.5 us in
    // parts of 128 keys, 19.4 of 512; 1,200 rows over 300 keys: 14.3 us whole, 22.6 in two).
    const bool wide = c.act_type == TQ2_TYPE_F32;
    const int64_t slots = c.head_dim > 128 || (wide && c.head_dim > 64) ? 256 : 512;
    const double tile = 1.9 * double(c.head_dim) / 128.0 * (wide ? 2.0 : 1.0);
    double least = 0.0;
    per = 128;
    for (int64_t parts = 1; parts <= 64; parts += parts < 4 ? 1 : parts / 2) {
      const int64_t each = keys < 1 ? 128 : pieces(pieces(keys, parts), 128) * 128, count = keys < 1 ? 1 : pieces(keys, each);
      const double time = double(pieces(blocks * count, slots)) * (4.5 + tile * double(each) / 64.0) +
                          (count > 1 ? 6.0 + joined * double(count) : 0.0);
      if (parts == 1 || time < least) {
        least = time;
        per = each;
      }
    }
  } else {
    // 1, 2, 4 or 8 tiles of 32 keys for each of a block's four waves, by the least time:
    // two blocks fit on a CU, a block takes about 4.5 us to start and end and 1.4 us a
    // tile, and joining parts takes 4 us and their way to memory and back at 3 TB/s
    // (measured).  Longer parts leave CUs idle at the end of ragged batches: 16 sequences of
    // up to 16,000 tokens take 102 us with 1024 keys a part, 113 with 2048, 129 with 4096.
    double least = 0.0;
    per = 128;
    for (int64_t tiles = 1; tiles <= 8; tiles *= 2) {
      const int64_t parts = keys < 1 ? 1 : pieces(keys, 128 * tiles), rounds = pieces(blocks * parts, 512);
      const double time = double(rounds) * (4.5 + 1.4 * double(tiles)) + (parts > 1 ? 4.0 + joined * double(parts) : 0.0);
      if (tiles == 1 || time < least) {
        least = time;
        per = 128 * tiles;
      }
    }
    // No more than a dozen blocks for each place on the card, which bounds the parts'
    // memory: ragged batches' ends even out by themselves there (1,024 sequences of up to
    // 2,048 tokens whole 684 us, in two parts 705, all of that length 1301 and 1380; 128 of
    // up to 8,192 in parts of 1408 keys 358, of 1024 341, all of that length 645 and 647).
    const int64_t dozen = 12 * 512 / blocks, each = pieces(pieces(keys, dozen < 1 ? 1 : dozen), 128) * 128;
    if (per < each) per = each;
  }
  splits = keys < 1 ? 1 : pieces(keys, per);
  if (splits > 512) splits = 512;
  plan.splits = int32_t(splits);
  plan.split_keys = int32_t(per);
  const int64_t fit = kAxisBlocks / (c.kv_heads * splits);
  if (plan.tiled && plan.steps > fit) plan.steps = int32_t(fit);
  plan.workspace = splits == 1 ? 0 : size_t(c.tokens) * size_t(c.q_heads) * size_t(splits) * size_t(c.head_dim + 4) * 4;
  return plan;
}

// Key heads vary fastest, then parts, then steps; sequences have an axis of their own.
inline Grid tile_grid(const AttnPlan& plan, int64_t kv_heads, int64_t batch) {
  return Grid{uint32_t(kv_heads * plan.splits * plan.steps), uint32_t(batch), 1};
}

// Blocks of the streaming form: key heads (and row steps) along x, sequences along y, parts
// along z.  Blocks go round the 8 dies and the 4 engines of each by their number, whether
// they find work or not, and short sequences have fewer parts: with parts fastest, those of
// 64 sequences of up to 8,192 tokens (one to eight parts) crowded the first dies (260 us in
// parts of 1024 keys, 188 now; with all at 8,192 346 both ways).  The number of sequences is
// rounded up to an odd one: 131,071 tokens beside three short sequences would leave all
// blocks with work on one engine of each die (240 us, 113 now).
inline Grid stream_grid(const AttnPlan& plan, int64_t kv_heads, int64_t batch) {
  return Grid{uint32_t(plan.steps * kv_heads), uint32_t(plan.splits > 1 ? batch | 1 : batch), uint32_t(plan.splits)};
}

// Blocks numbered along x and then y, 2^20 to a row: block (y << kRowShift) + x, with no
// size to be loaded first.  The last row's blocks may be past the last one.
constexpr int kRowShift = 20;
inline Grid row_grid(int64_t blocks) {
  const int64_t row = int64_t(1) << kRowShift;
  return Grid{uint32_t(blocks < row ? blocks : row), uint32_t(pieces(blocks, row)), 1};
}

// Blocks of the append: of `per_block` tokens, numbered like that along x and z, with a
// token's heads (`rounds` of a block's threads) shared out along y.  Few tokens: their heads
// are spread until there are eight blocks for each CU (1,640 tokens of 48 heads: 7.3 us,
// with sixteen 8.8).
inline Grid append_grid(int64_t tokens, int64_t per_block, int64_t rounds) {
  const int64_t blocks = pieces(tokens, per_block), share = 2048 / blocks;
  const Grid g = row_grid(blocks);
  return Grid{g.x, uint32_t(share < 1 ? 1 : (share < rounds ? share : rounds)), g.y};
}

}  // namespace tq2
