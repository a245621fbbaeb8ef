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

// ------------------------------------------------------------------ attention
constexpr int kRaggedRows = 256;  // packed query rows (token x head of a KV head) of an item at most
// Places on the line of work (attn_ragged.cu), of some 0.17 us each: a retrieval tile's with two query tiles
// and with one, a streaming tile's (most are masked) likewise, and an item's own, likewise. What they are decides
// how evenly the CTAs are loaded, and they are fitted over chunks, mixed batches and decodes of either head dim.
// (With one figure for either kind of items 32 mixed sequences took 249 us, with two 239; 4096 tokens over 28672
// 390 and 382.) One thing is more than balance: a tile takes no more places than a CTA's share has at least, so
// that every CTA between an item's first and last one begins a tile of it and leaves the part that the merge reads.
struct RaggedPlaces {
  int two, one, stream_two, stream_one, item_two, item_one;
};
constexpr RaggedPlaces kRaggedPlaces128 = {8, 6, 10, 6, 28, 16}, kRaggedPlaces64 = {8, 6, 11, 8, 22, 20};
constexpr int kRaggedLeast = 24;  // places of a CTA's share at least
constexpr bool tiles_fit_a_share(RaggedPlaces p) {
  return p.two <= kRaggedLeast && p.one <= kRaggedLeast && p.stream_two <= kRaggedLeast && p.stream_one <= kRaggedLeast;
}
static_assert(tiles_fit_a_share(kRaggedPlaces128) && tiles_fit_a_share(kRaggedPlaces64), "a part would be missing");
constexpr int kRaggedShort = 4;   // tiles of an item that is not shared at most

// An item whose key tiles several CTAs share, noted by the CTA that begins it (last < 0: it begins none):
// CTA `at` has the first part in its place 2 at + 1, CTAs at + 1 ... last the others in place 2 c.
struct RaggedJob {
  int last;
  int tok;   // first token of the packed batch
  int rows;  // packed query rows
  int head;  // first query head
};

struct RaggedAttnParams {
  CUtensorMap tm_q;      // 3-D over q [N, Hq, D], box 64 x g x 128 / g, 128B swizzle
  CUtensorMap tm_q8;     // the same, box 64 x g x 8 / g: the tokens of up to 8 rows
  CUtensorMap tm_k;      // 3-D over k [N, Hkv, D], box 64 x 1 x 128 (chunks only)
  CUtensorMap tm_v;
  CUtensorMap tm_kpool;  // 3-D over the pools [num_blocks, block_size, D], box 64 x 128 x 1
  CUtensorMap tm_vpool;
  CUtensorMap tm_ksr;    // 3-D over the rings [B n_str, S + R, D]
  CUtensorMap tm_vsr;
  uint16_t* o;           // bf16 [N, Hq, D]
  // chunks: sequence b has tokens cu_new[b] ... cu_new[b + 1] - 1, the first one at position
  // token_pos[cu_new[b]], which is also what its caches hold; single tokens (cu_new = nullptr): token b is
  // the last of the seq_lens[b] (clamped to [0, max_len]) that its caches hold
  const int32_t* cu_new;
  const int32_t* token_pos;
  const int32_t* seq_lens;
  int64_t max_len;
  const int32_t* pos;    // int32 [B, S+R]
  int tokens;            // N
  int log2_g;
  // a streaming head's window of tb + R - 1 positions, seen from a block of tb = 256 / g tokens: 16 x the
  // tiles it touches at least, + a bit for each of the 128 / tb places in a tile a block may begin at (place
  // 0 alone where tb is 128 or 256): one tile more
  int window;
  RaggedPlaces places;
  int ctas;
  int part_rows;         // rows a part has room for
  float scale_log2;      // log2(e) / sqrt(D)
  float* part_o;         // [2 ctas][D / 4][part_rows][4], unnormalised
  float2* part_ml;       // [2 ctas][part_rows] (max, sum)
  RaggedJob* jobs;       // [ctas], or nullptr: no item is long enough to be shared
  Shape sh;
  HeadTable heads;
  PagedLayout pg;
};
// Bytes of parts and jobs for items of up to `rows` rows on `ctas` CTAs.
size_t ragged_workspace_bytes(int ctas, int rows, int D);
cudaError_t launch_attn_ragged(const RaggedAttnParams& p, int device, cudaStream_t stream);
cudaError_t attn_ragged_read_clear_error(uint32_t* code);

}  // namespace duo
