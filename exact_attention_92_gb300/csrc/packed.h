// Attention over packed sequences: what the planning kernel, the forward kernel
// and the merge share.
//
// Rows.  Queries are taken in tiles of 128 rows that hold `tile_tokens` tokens
// of `group_heads` query heads of one key/value head (row = token * group_heads
// + head), so that K and V are read once for all of these; a block is two tiles.
// A head group is a (key/value head, run of group_heads of its query heads).
//
// Units.  An entry is a block of query tokens with the keys it takes (the shared
// prefix's, then the sequence's own), a unit is an entry for one head group.
// There are two lists of them, each head group by head group:
//   whole blocks   (more than one tile of rows): both element-wise warpgroups of a
//                  CTA take a tile of rows each and share the K, V tiles;
//   small blocks   (at most one tile: decoding, the ends of sequences): each
//                  warpgroup, with its own loads and products, takes units alone,
//                  so that one's start and end overlap the other's steps.
// The lists' 128-key tiles, weighted by what they take, make one line of places,
// of which every CTA takes an equal stretch (its two warpgroups halve what of it
// are small blocks).  That depends on nothing but the lengths, so results are the
// same from run to run.  What a cut leaves in parts is written as fp32 partial
// results, two slots a stretch, and merged.
//
// Sequence ends.  A tile of a sequence's last keys must read as zeros where it
// has no keys: the rows there are another sequence's, or memory of no sequence,
// and may hold NaN, which a weight of 0 does not silence.  Tensor maps check
// coordinates, not sequences, so the row is given by two coordinates of the same
// stride, the tile's first row and the row within the tile.  A tile with n < 128
// keys left starts at n - 128 in the second: what lies before 0 is outside and
// reads as zero, and the n keys take the tile's last n places.  (Clipping at the
// other end would take a map whose base lies ahead of the tensor.  Such a map
// faults where that address is not mapped, whatever coordinates are loaded.)
#pragma once

#include <cstdint>

#include "fa_common.h"

namespace fa {

constexpr int kSlotRows = 256;   // query rows of a whole block; half of it of a small one
constexpr int kDirectSeqs = 32;  // sequences of a call without a plan
constexpr int kMostGrid = 340;   // CTAs of the forward kernel: the merges keep their starts in shared memory

// Places of a key tile and of a unit's start and end: an eighth of a tile of a whole
// block (1.4 us at d = 128; small blocks run two at a time).  16 prompts of 16 Ki
// tokens, a server's batch and 64 answers behind a prefix (d = 128) and 32 sentences
// of d = 96 take 211, 212, 48.4 and 55.4 us over changing inputs; with 16 for a whole
// unit 217, 213, 48.2 and 55.9, with 6 for a small one 211, 217, 49.9 and 55.2, with
// 7 for a small tile 212, 222, 50.8 and 55.3.  (At d = 64 not measured apart.)
__host__ __device__ constexpr int tile_places(int list) { return list ? 6 : 8; }
__host__ __device__ constexpr int unit_places(int list) { return list ? 4 : 14; }

// A cut leaves at least so many tiles on either side.  (With 2 of a small block 64
// steps over 512 keys, 4 tiles, take 38 us in place of 31; with 3 of a whole one
// prompts take 208 in place of 211, but a server's batch 213 and not 212, sentences
// 55.8 and not 55.4.)
__host__ __device__ constexpr int least_tiles(int list) { return list ? 3 : 2; }

struct PackedEntry {
  int q_row, q_len;  // first token and tokens of the block
  int k_row, k_len;  // first key row and keys of the sequence
  int prefix;        // tiles of the prefix, ahead of the sequence's own
  int tiles;         // tiles in all that the block's last token sees
  int pos;           // causal: token j of the block sees own keys < pos + j + 1
  int kind;          // 1: block over the prefix alone (its rows get a second part)
};
static_assert(sizeof(PackedEntry) == 32, "read as two 16-byte words");

// Where a CTA's stretch starts: unit and tile.
struct PackedStart {
  int unit, tile;
};

struct PackedSeqs {
  const int* cu_q;
  const int* cu_k;
  const int* used_k;  // or null
  int B, Tq, Tk;
  int causal;         // FA_CAUSAL_*
  unsigned int* status;
};

constexpr int kWhole = 0, kSmall = 1;  // the lists

struct PackedHeader {
  int entries[2];        // of each list
  int over[2];           // of these, over the prefix alone (the first ones)
  int first, rows;       // query tokens that those cover
};

struct PackedPlan {
  PackedSeqs s;
  int tile_tokens;
  int prefix_tiles;   // 0: no prefix
  int shared;         // 1: the prefix has blocks of its own
  int head_groups;
  int grid;
  int whole;          // 1: no cuts
  int* seq_base[2];        // [B + 1] first entry of each sequence (where it does not fit shared memory)
  PackedEntry* entries[2];
  long long* cum;          // [entries of both + 1] places ahead of each entry (likewise)
  PackedStart* starts[2];  // [grid + 1], [2 grid + 1]
  PackedHeader* header;
};

struct PackedFwd {
  PackedSeqs s;
  int direct;         // 1: no plan; CTAs take units in turn
  int halves;         // direct: small blocks may be halved between a CTA's warpgroups
  int head_groups, prefix_tiles;
  int H, Hkv;
  int group;          // query heads of a key/value head
  int group_heads;    // of them in a tile
  int chunks;         // ceil(group / group_heads)
  int tile_tokens;
  int Tq;
  int prefix_len;
  int causal;         // 0 or 1
  int shared;
  float scale_log2;
  const PackedEntry* entries[2];
  const PackedStart* starts[2];
  const PackedHeader* header;
  int grid;
  void* o;
  long long o_row, o_head;  // strides in elements
  float* lse;               // [H, Tq]
  int store32;
  int tile_store;     // a warp's 32 rows are a box of o's tensor map (32 / group_heads tokens)
  float* o_slot[2];   // [2 stretches][D / 4][rows][4]
  float* lse_slot[2];  // [2 stretches][rows]
  float* o_part;      // shared: [2][Tq][H][D], of the prefix and of the own keys
  float* lse_part;    // shared: [2][H][Tq]
  unsigned int* status;
  unsigned long long timeout_ns;
};

}  // namespace fa
