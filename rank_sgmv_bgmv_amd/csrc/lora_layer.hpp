// Internal declarations of the norm, the 8-bit cache and the attention that
// reads it (include/lora_layer.h).  Not part of the public ABI.
#pragma once

#include "lora_internal.hpp"
#include "lora_layer.h"

namespace lora {

struct NormArgs {
  const void *x, *residual;  // residual may be nullptr
  const float *weight;
  void *total, *y;  // may be nullptr
  int8_t *q;        // may be nullptr
  float *scale;
  int64_t ldx, ldr, ldt, ldy, ldq;
  double eps;
  int rows, d;
};
hipError_t launch_norm(const NormArgs &a, int dtype, hipStream_t stream);

inline int cache_pitch(int head_dim) { return (head_dim + 15) / 16 * 16; }

struct CacheArgs {
  lora_cache c;
  int pitch, page_bits;  // page_size = 1 << page_bits
  const int32_t *slots;
  lora_heads k, v;
  int T;
};
hipError_t launch_cache_write(const CacheArgs &a, int dtype, hipStream_t stream);
hipError_t launch_cache_read(const CacheArgs &a, int dtype, hipStream_t stream);

// ---------------------------------------------------------------- attention --
// Keys are taken in tiles of 64 whose first one is a multiple of 64.  The rows
// of a sequence and cache head are (query, query head) pairs, the head the
// faster.  A unit is a tile of such rows with the key tiles that they see; it
// is cut into nsplit pieces of key tiles, the items.  Each item is done for
// every cache head.
constexpr int kKeyTile = 64;

struct AttnUnit {
  int q0, n, len;      // first row in the batch, queries and keys of the sequence
  int row0, rows;      // the unit's rows among the n * group of the sequence
  int seq;
  int ntiles, sink_tiles, main;  // tile v is v < sink_tiles ? v : main + v - sink_tiles
  int nsplit, slot;    // pieces, and where those of a cut unit leave their results (nsplit > 1)
  int pad[5];
};
static_assert(sizeof(AttnUnit) == 64, "read as four 16-byte pieces");

// Two kinds of units: those of few rows (one tile a sequence) and of many.
enum { ATTN_FEW = 0, ATTN_MANY = 1, ATTN_KINDS = 2 };

// Plan header words beyond those of the adapters' plan that lora_read_device_errors reads (H_ERR).
enum {
  A_ITEMS = 0,   // [ATTN_KINDS]
  A_CUT = 4,     // units of more than one piece [ATTN_KINDS]
  A_KEY = 8,     // what the plan was made for [A_KEYS]
  A_KEYS = 12
};
static_assert(H_ERR == 2 && H_WORDS >= A_KEY + A_KEYS, "the words of a plan's header");
constexpr int kAttnMagic = 0x41747450;

struct AttnShape {
  int T, S, group, kv_heads, head_dim, dp;  // dp: head_dim padded to the kernels' 64, 128 or 256
  int few_blocks;                           // row blocks of 16 that the kernel for few rows takes; 0: not launched
  int few_rows, many_rows;                  // rows of a unit of either kind; many_rows 0: not launched
  int units[ATTN_KINDS], items[ATTN_KINDS], cut[ATTN_KINDS];  // most that a batch of this shape can have
  int target[ATTN_KINDS], least[ATTN_KINDS];  // pieces a head that a launch aims at, tiles that a piece has at least
  // byte offsets in the plan
  size_t toff, unit[ATTN_KINDS], item[ATTN_KINDS], cutlist[ATTN_KINDS], plan_bytes;
  // in the workspace: results of pieces [slot][head][rows][dp] and their maxima and sums [slot][head][rows][2], floats
  size_t part[ATTN_KINDS], stat[ATTN_KINDS], ws_bytes;
};

struct AttnPlanArgs {
  AttnShape s;
  const int32_t *q_off, *lens;
  int *plan;
  int max_q, capacity;  // of queries and keys of a sequence
  int window, sinks, tree;
  int key[A_KEYS];
};
hipError_t launch_attention_plan(const AttnPlanArgs &a, hipStream_t stream);

struct AttnArgs {
  AttnShape s;
  lora_cache c;
  int pitch, page_bits;  // page_size = 1 << page_bits
  lora_heads q, out;
  const int32_t *pages;
  int64_t ld_pages;
  const uint64_t *tree;
  int *plan;  // the error word alone is written
  char *ws;
  int window, sinks;  // window: 0 became the largest int
  float scale;                 // of the scores, times log2 e
  int key[A_KEYS];
};
hipError_t launch_attention(const AttnArgs &a, int dtype, hipStream_t stream);

}  // namespace lora
