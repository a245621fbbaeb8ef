// Internal types of the packed ragged step over bf16 paged caches: rotary positions, append and
// attention. Not part of the public ABI.
#pragma once

#include "duo_internal.h"

namespace duo {

constexpr int kRopeHalf = 0, kRopeInterleaved = 1;

// Rows of a packed batch, bf16 [tokens, heads, D]; stride: elements from a token to the next.
struct RaggedRows {
  const uint16_t* in;
  uint16_t* out;  // rotated rows (q, and k of a rotation alone)
  int64_t in_stride;
  int64_t out_stride;
  int heads;
};

struct RopeParams {
  const uint64_t* turns;  // per pair: angle per position, in units of 2^-64 of a full turn
  int rotary;             // leading dims that are rotated, a multiple of 16 (0: none)
  int layout;
  float scale;
};

// A rotation of q and k, or (append) of q and of k on its way into the caches, v copied beside it.
struct RopeAppendParams {
  RaggedRows q;  // heads = 0: none
  RaggedRows k;
  RaggedRows v;
  RopeParams rope;
  const int32_t* positions;  // token_pos of an append; below 0: the token is skipped
  int tokens;
  int chunk;  // tokens per CTA, up to kRopeChunk
  // append only
  const int32_t* cu_new;
  const int32_t* token_seq;
  const int64_t* slots;
  uint16_t* k_pool;  // [rows, D]
  uint16_t* v_pool;
  uint16_t* k_sr;
  uint16_t* v_sr;
  int32_t* pos;
  int64_t rows;  // of each pool
  Shape sh;
  HeadTable heads;
};
constexpr int kRopeChunk = 8;
cudaError_t launch_rope(const RopeAppendParams& p, cudaStream_t stream);
cudaError_t launch_append_ragged(const RopeAppendParams& p, cudaStream_t stream);
cudaError_t append_ragged_read_clear_error(uint32_t* code);

}  // namespace duo
