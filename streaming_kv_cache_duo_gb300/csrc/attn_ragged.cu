// duo_attn_prefill_ragged and duo_attn_decode_paged_varlen: attention of a packed batch over bf16 paged
// caches, every length read on the device.
//
// What it computes: sequence b's query at position i attends to the keys its caches hold and to the new
// tokens of its own sequence, by the visibility rule of the library (retrieval j <= i; streaming also
// j < S or i - j < R). Chunks: the caches as they were before the call, then the new tokens. Single
// tokens: the caches alone, the query's token appended before.
//
// Items. Query rows are packed, row = token x g + head of a KV head, so that one token's g heads share
// every K and V tile and a short chunk fills the rows of a tile. An item is up to 256 rows of one
// (sequence, KV head), and what it reads is a list of 128-key tiles: of the cache, then of the new
// tokens. All items' tiles are laid end to end on a line, retrieval items before streaming ones, with
// room before each item for what it costs apart from its tiles, and CTA c of C (one an SM) takes the
// tiles that begin in [c W / C, (c + 1) W / C). So a batch of one long and many short sequences is as
// balanced as a uniform one, however long a context is. Nothing is planned on the host or by a kernel
// before: where a sequence, a head and a block of queries begin on the line follows from the lengths in
// closed form, so each CTA sums the sequences' lengths and finds its own first item. An item that
// several CTAs share leaves parts (output, maximum, sum) that a second kernel merges; a CTA has at most
// two: one that goes on with an item, one that begins one.
//
// One CTA, 12 warps (setmaxnreg moves registers from the third warpgroup to the two softmax ones):
//   warp 11     walks the CTA's share of the line, and hands descriptors of its segments (an item's tiles
//               or some of them) to the others through a ring of four
//   warp 8      TMA producer: Q, then K and V tiles (128-byte swizzle) into rings of kNS stages, running
//               ahead over segments' ends
//   warp 9      MMA: the whole warp follows the tiles, one elected lane issues tcgen05.mma
//   warp 10     writes zeros for single-token sequences that hold nothing
//   warps 0-3, 4-7  softmax: thread r has query row r (TMEM lane r), with its running maximum and sum
// Segments of more than 128 rows have two query tiles, one a softmax warpgroup, and every K/V tile serves
// both: S0(j), S1(j), PV0(j), S0(j+1), PV1(j), S1(j+1), ... Shorter ones (decodes, short chunks) have
// one query tile and the two warpgroups take the key tiles by turns, each with its own output
// accumulator, so that one's softmax runs beside the other's products all the same; at the end the
// warpgroups read both accumulators (same TMEM lanes), half of the dims each, and merge them. A decode
// uses few of the 128 rows: a tile's products take 0.7 us of the tensor core, its 64 KB 1.5 us of an SM's
// share of HBM, so wasted rows cost nothing that bounds it. What does is the way from a tile's scores to
// its P, as V's stage waits for it: up to eight rows are loaded once for each warp, which takes 32 of a tile's
// 128 keys (a million tokens 167.3 -> 164.4 us, 128 short sequences of 64-dim heads 78 -> 64).
//
// What lies behind a sequence's last row in a tile (another sequence's tokens, padding, rows of a block
// never written) may be anything. Scores there are masked by selection; for V, zero times an infinity or
// NaN would not do, so the product stops after the 16 rows that hold the last one, and the MMA warp
// writes zeros over what is left of those. A block id outside the pool: its rows are left out.
//
// P is rounded to bf16 (its sum is of the unrounded values, in fp32), as the matrix unit takes operands of
// one type and V is bf16: that is what parts the outputs of chunks (0.0021 to 0.0023 of their norm from
// 64 bits) from those of a product in fp32, rounded once (0.0017). A second term would make the products
// 1.5 times as many. With up to eight rows it costs nothing, being other rows of the same product, and single
// tokens are as exact as a product in fp32. Scores, maxima, sums and outputs are fp32.
//
// Measured (graphs replayed one by one; measured peaks 6.77 TB/s and 1904 TFLOP/s):
//   16384 tokens, 32 heads over 8, all retrieval, D = 128: 1270 us, 1730 TFLOP/s (the uniform prefill 1380);
//     D = 64: 990 us (the uniform prefill 1166), where a tile's way through softmax (1240 cycles) and the
//     MMA warp's own instructions take the time, not the products (512). All streaming: 151 us, an item of
//     four masked tiles 11, some 2 of them its end.
//   4096 tokens over 28672, MHA 32 heads, 8 of them retrieval: 379 us
//   one sequence of 1048576 tokens, one token: 162 to 164 us, 6.6 TB/s; 48 of up to 32000: 116 to 118 us, the
//     floor of their bytes
//   128 short ones, D = 64: 56 us where their bytes take 30: each item is Q, a few tiles and an end, one
//     after the other. Two sequences of a few blocks: 9.5 us, of which 5 go by before the first segment is
//     known, most of it first reads of the instructions.
// Of the ways tried, with the times before and after at that point, us, for the first case unless said: one
// thread that issues, with counters and descriptors of its own, 1330 -> 1712 (they were carried to uniform
// registers one by one); two issuing warps, one a query tile, 1712 -> 1828 (the softmaxes fall into phase); scores
// masked and summed in rolled loops of chunks, and dead chunks skipped, 1330 -> 1415 (spills); one loop of
// steps for both kinds of segments 1324 -> 1470; an eighth of the exponentials by a polynomial 1345 -> 1365,
// and 1015 -> 1067 for D = 64; four partial sums, or the exponentials in between the sums by hand, 1301 ->
// 1320 to 1345 (spills); a third place of scores for D = 64, so that a softmax finds its next tile ready,
// 990 -> 1045; new tokens' tiles classed as seen whole or not at all before they are masked, 183 -> 187 for
// streaming heads. Streaming items shared out over all CTAs beside the retrieval ones: 80 -> 65 for 128 short
// decodes, but 121 -> 125 for the 48 long ones, as every CTA then begins twice.
#include <atomic>

#include "duo_device.cuh"
#include "ragged_internal.h"

namespace duo {
namespace {

__device__ unsigned int g_attn_ragged_err;

constexpr int BM = 128;  // rows per query tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpZero = 10, kWarpLine = 11;
// 2 x 128 x 200 + 128 x 104 = 384 x 168 = 64512, the launch's registers
constexpr int kLaunchRegs = 168, kRegsSoftmax = 200, kRegsCtl = 104;
constexpr uint32_t kTmemCols = 512;
constexpr int kBox = 128 * 128;  // bytes of a 128-row x 64-column bf16 box
constexpr int kSegs = 4;         // descriptors in flight
constexpr int kWarpBatch = 32;   // sequences that the line's warp sums alone
constexpr int kFew = 8;          // rows of a segment whose tiles the four warps of a warpgroup share at most
constexpr int kSegUsers = 10;    // producer, MMA, eight softmax warps

__host__ __device__ constexpr uint32_t col_s(int x) { return (uint32_t)x * 256u; }
__host__ __device__ constexpr uint32_t col_o(int x) { return (uint32_t)x * 256u + 128u; }

template <int D>
struct Cfg {
  static constexpr int NBOX = D / 64;
  static constexpr int kNS = D == 64 ? 4 : 2;  // K/V stages
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + kNS * KV_BYTES;
  static constexpr int OFF_ML = OFF_V + kNS * KV_BYTES;  // float2 [2][BM]
  static constexpr int OFF_VIS = OFF_ML + 2 * BM * 8;  // uint4 per softmax thread
  static constexpr int PITCH = D / 2 + 4;  // floats from a row to the next (16 bytes on in the banks)
  static constexpr int OFF_SUM = OFF_VIS + 2 * BM * 16;  // float [2][4 warps][kFew][PITCH]
  static constexpr int OFF_BAR = OFF_SUM + 2 * 4 * kFew * PITCH * 4;
  static constexpr size_t SMEM = (size_t)OFF_BAR + 1024 + 1024;  // + alignment slack
};

// What a segment is. Cache rows are [0, held) of the pool's plane or of the ring.
struct Seg {
  int last;       // no more segments
  int b, tok0, T, n;  // sequence: its first token of the packed batch, new tokens, cached ones
  int q0, rows;   // first token (of the sequence) and packed rows of the item
  int kvh, cidx, streaming;
  int j0, j1;     // tiles of the item
  int n_cache, sink_eff, w_lo;
  // the tiles not all of whose rows hold a token of the sequence (-1: none): the last one of the cache and
  // the last one of the new tokens, and the rows that do
  int cut_cache, rows_cache, cut_new, rows_new;
  int part;       // place of its part, -1: the whole item
  int bad;        // a block of its tiles does not exist (written later than the rest: seg_known)
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t pair_ml[4], pair_done[4];
  uint64_t meet_both, meet_one[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs], seg_known[kSegs];
  uint64_t drain;
  uint32_t tmem_base;
  int stop;  // an earlier CTA gave up a wait
  // the line: places of all items, and where this CTA's share begins
  long long sums[2][kThreads / 32];
  long long places, places_r, start_at;
  int start_b;
  Seg seg[kSegs];
};
static_assert(sizeof(Bars) <= 1024, "barrier area");

// ---------------------------------------------------------------- the line
struct Sequence {
  int tok0, T, n;
};

// Sequence b; T = 0 where it has nothing to compute. report: note what cannot be.
__device__ __forceinline__ Sequence sequence_at(const RaggedAttnParams& p, int b, bool report) {
  Sequence s{0, 0, 0};
  if (!p.cu_new) {
    const int64_t len = p.seq_lens[b];
    s.tok0 = b;
    s.n = (int)(len < 0 ? 0 : (len > p.max_len ? p.max_len : len));
    s.T = s.n > 0;
    return s;
  }
  const int first = p.cu_new[b], end = p.cu_new[b + 1];
  bool good = first >= 0 && end >= first;
  if (good && (end == first || first >= p.tokens)) return s;  // (behind the batch: turned down)
  if (good) {
    const int pos = p.token_pos[first];
    if (pos < 0) return s;  // turned down
    const int64_t cap = (int64_t)p.pg.block_size * p.pg.max_blocks;
    good = end <= p.tokens && end - first <= 0x7fffffff - pos && (p.sh.n_ret == 0 || pos <= cap);
    if (good) s = Sequence{first, end - first, pos};
  }
  if (!good && report) atomicOr(&g_attn_ragged_err, kErrBadLength);
  return s;
}

__device__ __forceinline__ int tiles_of(int64_t rows) { return (int)((rows + BN - 1) / BN); }

// Places on the line of a head's first m items (all, if it has no more), in the order of their tokens. An
// item reads cache tiles and the new tokens' tiles up to its last token, ceil(min(T, (k + 1) tb) / 128)
// for block k of tb tokens; a streaming head's, from the first block on whose every query is past the
// ring but for the sinks, tiles of sinks and of a window (p.window). Never fewer than its items read, which would
// lose tiles, but some more: sinks among the new tokens are counted beside a window that still reaches them. And
// places go by the sequence, though its last block, of 128 rows or fewer, runs with one query tile and not two.
// Both cost balance alone. Out of line, and with few instructions: when a CTA begins, none of them is in its SM's
// cache, and each costs some 30 cycles the first time.
__device__ __noinline__ long long line_upto(int T, int n, bool streaming, int m, int place, int item, int log2_g,
                                            bool chunks, int S, int R, int window) {
  const int shift = 8 - log2_g;  // tb = 2^shift
  const int blocks = (int)(((unsigned)T + (1u << shift) - 1u) >> shift);
  m = min(m, blocks);
  int held = n, whole = blocks;  // blocks that see the cache whole
  if (streaming) {
    held = min(n, S + R);
    if (chunks) whole = min(blocks, (R - 1 + (1 << shift) - 1) >> shift);
  }
  const int e = min(m, whole);
  long long tiles = (long long)e * tiles_of(held);
  if (chunks && e > 0) {
    const unsigned f = e == blocks ? e - 1 : e;
    const int l = max(0, log2_g - 1);  // 2^l blocks a tile, or (tb = 256) a block two tiles
    const unsigned q = f >> l, rest = f & ((1u << l) - 1u);
    const long long half = (long long)q * (q + 1) / 2;
    tiles += log2_g == 0 ? 2 * half : (half << l) + (long long)rest * (q + 1);
    if (e == blocks) tiles += tiles_of(T);
  }
  if (m > e) {
    const int sinks = tiles_of(min(held, S)) + (n < S ? tiles_of(S - n) : 0);
    const int l = max(0, log2_g - 1);
    const unsigned longer = window & 15, in = (1u << l) - 1u;
    const auto ones = [&](unsigned k) { return (int)((k >> l) * __popc(longer) + __popc(longer & ((1u << (k & in)) - 1u))); };
    tiles += (long long)(m - e) * (sinks + (window >> 4)) + ones(m) - ones(e);
  }
  return (long long)m * item + place * tiles;
}
// Places of a tile, and of an item apart from its tiles.
__device__ __forceinline__ bool two_query_tiles(const RaggedAttnParams& p, int T) { return T > (BM >> p.log2_g); }
__device__ __forceinline__ int item_of(const RaggedAttnParams& p, int T) {
  return two_query_tiles(p, T) ? p.places.item_two : p.places.item_one;
}
__device__ __forceinline__ int place_of(const RaggedAttnParams& p, int T, bool streaming) {
  const bool two = two_query_tiles(p, T);
  return streaming ? (two ? p.places.stream_two : p.places.stream_one) : (two ? p.places.two : p.places.one);
}
__device__ __forceinline__ long long line_upto(const RaggedAttnParams& p, const Sequence& s, bool streaming, int m) {
  return line_upto(s.T, s.n, streaming, m, place_of(p, s.T, streaming), item_of(p, s.T), p.log2_g, p.cu_new != nullptr,
                   p.sh.S, p.sh.R, p.window);
}
constexpr int kAllItems = 0x7fffffff;
// Places of all items of a sequence's heads of one kind.
__device__ __forceinline__ long long places_of(const RaggedAttnParams& p, const Sequence& s, bool streaming) {
  return (streaming ? p.sh.n_str : p.sh.n_ret) * line_upto(p, s, streaming, kAllItems);
}

// The tiles of block `blk` of a sequence and kind: cache tiles 0 ... n_cache - 1, then of the new tokens
// [0, sink_eff) and [w_lo, ...].
__device__ __forceinline__ int plan_item(const RaggedAttnParams& p, const Sequence& s, bool streaming, int blk, Seg* g) {
  const int tb = kRaggedRows >> p.log2_g;
  const int q0 = blk * tb;
  const int tokens = min(tb, s.T - q0);
  g->q0 = q0;
  g->rows = tokens << p.log2_g;
  const int held = streaming ? min(s.n, p.sh.S + p.sh.R) : s.n;
  g->n_cache = tiles_of(held);
  g->sink_eff = 0;
  g->w_lo = 0;
  g->cut_new = -1;
  g->rows_new = BN;
  if (p.cu_new && streaming && q0 + 1 >= p.sh.R) g->n_cache = tiles_of(min(p.sh.S, held));  // only sinks are still seen
  g->rows_cache = min(BN, held - (g->n_cache - 1) * BN);
  g->cut_cache = g->n_cache > 0 && g->rows_cache < BN ? g->n_cache - 1 : -1;
  if (!p.cu_new) return g->n_cache;
  if (streaming) {
    const int first = q0 - p.sh.R + 1;
    g->w_lo = first > 0 ? first / BN : 0;
    const int sinks = p.sh.S > s.n ? tiles_of(p.sh.S - s.n) : 0;  // new tokens that are sinks
    g->sink_eff = min(sinks, g->w_lo);
  }
  const int last = (q0 + tokens - 1) / BN;
  const int total = g->n_cache + g->sink_eff + last - g->w_lo + 1;
  if ((int64_t)(last + 1) * BN > s.T) {
    g->cut_new = total - 1;
    g->rows_new = s.T - last * BN;
  }
  return total;
}

// a / b for a >= 0, b > 0 (64-bit divisions take several times as long)
__device__ __noinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// CTAs that share a line of W places, the first place of CTA c of them, and the CTA of place x.
__device__ __forceinline__ int sharers(int64_t W) {
  return (int)min((int64_t)gridDim.x, max((int64_t)1, divide(W, kRaggedLeast)));
}
__device__ __forceinline__ int64_t bound(int64_t W, int ctas, int c) { return divide(c * W, ctas); }
__device__ __forceinline__ int owner(int64_t W, int ctas, int64_t x) { return (int)divide((x + 1) * ctas + W - 1, W) - 1; }
struct Share {
  int ctas;
  int64_t lo, hi;  // of this CTA
};
__device__ __noinline__ Share share_of(int64_t W) {
  const int ctas = sharers(W), c = blockIdx.x;
  return Share{ctas, c < ctas ? bound(W, ctas, c) : W, c < ctas ? bound(W, ctas, c + 1) : W};
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Tile j of an item: of the cache or of the new tokens, and which one of these.
struct Tile {
  bool cache;
  int k;
};
__device__ __forceinline__ Tile tile_at(const Seg& g, int j) {
  Tile t;
  t.cache = j < g.n_cache;
  j -= t.cache ? 0 : g.n_cache;
  t.k = t.cache || j < g.sink_eff ? j : g.w_lo + (j - g.sink_eff);
  return t;
}
// Rows of it that hold a token of the sequence.
__device__ __forceinline__ int rows_of(const Seg& g, int j) {
  return j == g.cut_cache ? g.rows_cache : (j == g.cut_new ? g.rows_new : BN);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bits_below(int hi) {  // (shl gives 0 for 32 and more)
  uint32_t above;
  asm("shl.b32 %0, %1, %2;" : "=r"(above) : "r"(0xffffffffu), "r"(max(hi, 0)));
  return ~above;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Which of the 32 keys from column c0 of a tile on a row sees, as a mask. New tokens, whose positions are
// consecutive (column 0 is d positions before the row): at most two runs, sinks and (i - R, i], from a few
// shifts.
__device__ __forceinline__ uint32_t visible_new(const RaggedAttnParams& p, bool streaming, int i_abs, int d, int c0) {
  const int sinks = streaming ? p.sh.S - (i_abs - d) : 0, out = streaming ? d - p.sh.R + 1 : 0;
  return bits_below(d + 1 - c0) & (bits_below(sinks - c0) | ~bits_below(out - c0));
}
// Cached ones: of `rows` in the tile all are visible to a retrieval head. Ring slots: jp is the position slot
// c0 + lane holds, -1 if none; most are seen by all of the warp's rows or by none (rows' positions rise with
// the lane), the few others are compared row by row.
__device__ __forceinline__ uint32_t visible_held(const RaggedAttnParams& p, bool streaming, int rows, int c0, int i_abs,
                                                 int jp) {
  if (!streaming) return bits_below(rows - c0);
  const int S = p.sh.S, R = p.sh.R;
  const int i0 = __shfl_sync(0xffffffffu, i_abs, 0), i1 = __shfl_sync(0xffffffffu, i_abs, 31);
  const bool all = jp >= 0 && jp <= i0 && (jp < S || i1 - jp < R);
  const bool none = jp < 0 || jp > i1 || (jp >= S && i0 - jp >= R);
  uint32_t vis = __ballot_sync(0xffffffffu, all);
  for (uint32_t some = __ballot_sync(0xffffffffu, !all && !none); some; some &= some - 1) {
    const int e = __ffs((int)some) - 1;
    const int j = __shfl_sync(0xffffffffu, jp, e);
    vis |= (uint32_t)(j <= i_abs && (j < S || i_abs - j < R)) << e;
  }
  return vis;
}

// Position of packed row `row` of a segment's item; a row past the item takes the last one's.
__device__ __forceinline__ int position(const RaggedAttnParams& p, const Seg& g, int row) {
  return p.cu_new ? g.n + g.q0 + (min(row, g.rows - 1) >> p.log2_g) : g.n - 1;
}

// Bounded waits as mbar_wait and mbar_wait_warp, in fewer instructions (they are written out some forty
// times: with those the kernel was 164 KB of code, more than an SM's instruction caches hold, and what
// runs now and then, a segment's beginning and end, took several times as long as it should).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, DevError err, uint32_t code) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if (i & 255u) continue;  // (the clock is slow to read)
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitLimitNs) {
      atomicOr(err.word, code);
      return false;
    }
  }
  return true;
}
// By all 32 lanes together, which get one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, DevError err, uint32_t code) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i) {
    if (i & 255u) continue;
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
      atomicOr(err.word, code);
      return false;
    }
  }
  return true;
}

// A value that is the same in all lanes, known to be so by the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Reads the descriptors in order: done() gives one back.
struct SegReader {
  Bars* bars;
  int count = 0;
  __device__ __forceinline__ explicit SegReader(Bars* b) : bars(b) {}
  __device__ __forceinline__ const Seg& seg() const { return bars->seg[count % kSegs]; }
  __device__ __forceinline__ uint64_t* full() const { return &bars->seg_full[count % kSegs]; }
  __device__ __forceinline__ uint64_t* known() const { return &bars->seg_known[count % kSegs]; }
  __device__ __forceinline__ uint32_t parity() const { return (uint32_t)((count / kSegs) & 1); }
  __device__ __forceinline__ void done() {  // by one lane
    mbar_arrive(&bars->seg_empty[count % kSegs]);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_ragged_kernel(const __grid_constant__ RaggedAttnParams p) {
  using C = Cfg<D>;
  constexpr int kNS = C::kNS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  float2* sML = reinterpret_cast<float2*>(smem + C::OFF_ML);
  uint4* sVis = reinterpret_cast<uint4*>(smem + C::OFF_VIS);
  float* sSum = reinterpret_cast<float*>(smem + C::OFF_SUM);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);

  const DevError err{&g_attn_ragged_err};
  const int warp = uniform(threadIdx.x >> 5);  // (with roles that are the warps' own, shuffles need no care: 157 -> 146 KB)
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 1);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_full[s], 4);
      mbar_init(&bars->o_final[s], 1);
      mbar_init(&bars->meet_one[s], 4);
    }
    mbar_init(&bars->meet_both, 8);
    for (int s = 0; s < kNS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&bars->seg_full[s], 1);
      mbar_init(&bars->seg_empty[s], kSegUsers);
      mbar_init(&bars->seg_known[s], 1);
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&bars->pair_ml[w], 2);
      mbar_init(&bars->pair_done[w], 2);
    }
    mbar_init(&bars->drain, 1);
    fence_mbarrier_init();
    // After any CTA gave up a wait, later ones do no work, so that a failure ends in about one wait limit.
    // (Bad lengths and block ids, recorded in the same word, concern their sequences alone.)
    bars->stop = (*(volatile unsigned int*)err.word & ~(kErrBadBlock | kErrBadLength)) != 0u;
    bars->start_b = -1;
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // the merge may be scheduled now; nothing that earlier grids write is read before they have ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---------------------------------------------------------------- this CTA's share of the line
  // A batch of few sequences is summed by the line's warp alone (two barriers of the whole CTA and
  // their way through memory cost a small decode 2 us); of many, by all threads: the places of either
  // kind, and the sequence where the CTA's share begins.
  const int B = p.sh.B;
  if (B > kWarpBatch) {
    long long mine[2] = {0, 0};  // places of this thread's sequences: retrieval, streaming
#pragma unroll 1
    for (int b = threadIdx.x; b < B; b += kThreads) {
      const Sequence s = sequence_at(p, b, blockIdx.x == 0);
      mine[0] += places_of(p, s, false);
      mine[1] += places_of(p, s, true);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long v = warp_sum(mine[k]);
      if (lane == 0) bars->sums[k][warp] = v;
    }
    __syncthreads();
    int64_t W_r = 0, W = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) W_r += bars->sums[0][w], W += bars->sums[1][w];
    W += W_r;
    const Share sh = share_of(W);
    const bool streaming = sh.lo >= W_r;
    if (sh.lo < sh.hi) {  // (the same for all threads) the sequence whose items of that kind hold place lo
      const int64_t x = streaming ? sh.lo - W_r : sh.lo;
      long long before = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        long long v = 0;
        if (B <= kThreads) v = streaming ? mine[1] : mine[0];
        else if (b < B) v = places_of(p, sequence_at(p, b, false), streaming);
        long long upto = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += u;
        }
        __syncthreads();  // sums have been read
        if (lane == 31) bars->sums[0][warp] = upto;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w < warp) upto += bars->sums[0][w];
          all += bars->sums[0][w];
        }
        if (before + upto - v <= x && x < before + upto) {
          bars->start_b = b;
          bars->start_at = before + upto - v;
        }
        before += all;
        if (before > x) break;  // (the same for all threads)
      }
    }
    if (threadIdx.x == 0) {
      bars->places = W;
      bars->places_r = W_r;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp >= 8) {
    // ================================================ warpgroup 2: TMA, MMA, zeros, the line
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (warp == kWarpLine) {
      // ------------------------------------------------------------ segments
      int count = 0;
      RaggedJob job{-1, 0, 0, 0};
      bool ok = true;
      int64_t W_r = bars->places_r, W = bars->places;
      // a window of 32 sequences, one a lane, from `base` on; with few sequences it is all of them, and
      // says itself where the share begins
      int base = 0, w = 0, kind = 0;
      int64_t at = 0;  // where sequence base + w begins
      Sequence s{0, 0, 0};
      long long v[2] = {0, 0};
      auto window = [&]() {
        s = Sequence{0, 0, 0};
        if (base + lane < B) s = sequence_at(p, base + lane, B <= kWarpBatch && blockIdx.x == 0);
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const long long x = places_of(p, s, k == 1);
          if (k == 0) v[0] = x;
          else v[1] = x;
        }
      };
      if (B <= kWarpBatch) {
        window();
        long long upto[2] = {v[0], v[1]};
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const long long a = __shfl_up_sync(0xffffffffu, upto[0], o), b = __shfl_up_sync(0xffffffffu, upto[1], o);
          upto[0] += lane >= o ? a : 0;
          upto[1] += lane >= o ? b : 0;
        }
        W_r = __shfl_sync(0xffffffffu, upto[0], 31);
        W = W_r + __shfl_sync(0xffffffffu, upto[1], 31);
        const Share sh = share_of(W);
        kind = sh.lo >= W_r;
        const long long end = kind ? W_r + upto[1] : upto[0], from = end - (kind ? v[1] : v[0]);
        w = max(0, __ffs((int)__ballot_sync(0xffffffffu, from <= sh.lo && sh.lo < end)) - 1);
        at = __shfl_sync(0xffffffffu, from, w);
      } else {
        kind = share_of(W).lo >= W_r;
        base = bars->start_b;
        at = bars->start_at + (kind ? W_r : 0);
        if (base >= 0) window();
      }
      const Share sh = share_of(W);
      const int ctas = sh.ctas;
      const int64_t lo = sh.lo, hi = sh.hi;
      if (lo < hi && !bars->stop && base >= 0) {
        int64_t cur = lo;
        while (ok && cur < hi) {
          const Sequence q{__shfl_sync(0xffffffffu, s.tok0, w), __shfl_sync(0xffffffffu, s.T, w),
                           __shfl_sync(0xffffffffu, s.n, w)};
          const int64_t places = __shfl_sync(0xffffffffu, kind ? v[1] : v[0], w);
          if (places > 0) {
            const int place = place_of(p, q.T, kind == 1);
            const int heads = kind ? p.sh.n_str : p.sh.n_ret;
            const int blocks = (int)(((unsigned)q.T + (kRaggedRows >> p.log2_g) - 1u) >> (8 - p.log2_g));
            const int64_t per_head = line_upto(p, q, kind == 1, kAllItems);
            // its first item that ends behind cur (the first one of all, but where the share begins)
            int h = 0, blk = 0;
            int64_t head_at = at, begin = at;
            if (cur > at) {
              h = (int)divide(cur - at, per_head);
              head_at += h * per_head;
#pragma unroll 1
              for (int top = blocks; top - blk > 1;) {
                const int mid = blk + (top - blk) / 2;
                if (head_at + line_upto(p, q, kind == 1, mid) <= cur) blk = mid;
                else top = mid;
              }
              begin = head_at + line_upto(p, q, kind == 1, blk);
            }
#pragma unroll 1
            while (h < heads && cur < hi) {
              const int64_t end = head_at + line_upto(p, q, kind == 1, blk + 1);
              Seg g;
              g.last = 0;
              g.b = base + w;
              g.tok0 = q.tok0;
              g.T = q.T;
              g.n = q.n;
              g.cidx = h;
              g.streaming = kind;
              g.kvh = kind ? p.heads.str_head[h] : p.heads.ret_head[h];
              const int total = plan_item(p, q, kind == 1, blk, &g);
              // tile j's place is begin + item + j place
              const int64_t first = begin + item_of(p, q.T);
              g.j0 = 0;
              g.j1 = total;
              if (total <= kRaggedShort) {
                if (begin < lo) g.j1 = 0;  // the CTA's where it begins
              } else {
                const int64_t a = cur - first, e = min(hi, end) - first;
                if (a > 0) g.j0 = (int)min((int64_t)total, divide(a + place - 1, place));
                if (hi < end) g.j1 = e > 0 ? (int)min((int64_t)total, divide(e + place - 1, place)) : 0;
              }
              cur = begin = end;
              if (++blk == blocks) {
                blk = 0;
                ++h;
                head_at = end;
              }
              if (g.j0 >= g.j1) continue;
              g.part = -1;
              if (g.j0 > 0) {
                g.part = 2 * blockIdx.x;
              } else if (g.j1 < total) {
                g.part = 2 * blockIdx.x + 1;
                job = RaggedJob{owner(W, ctas, first + (int64_t)(total - 1) * place), g.tok0 + g.q0, g.rows,
                                g.kvh << p.log2_g};
              }
              const int slot = count % kSegs;
              if (!wait_warp(&bars->seg_empty[slot], (uint32_t)(((count / kSegs) & 1) ^ 1), err, kErrPrefillProducer)) {
                ok = false;
                break;
              }
              if (lane == 0) {
                bars->seg[slot] = g;
                mbar_arrive(&bars->seg_full[slot]);
              }
              // while Q and the first tiles are on their way: do all of its blocks exist?
              bool bad = false;
              if (kind == 0 && g.j0 < g.n_cache) {
                const int32_t* row = p.pg.table + ((int64_t)g.b * p.sh.n_ret + g.cidx) * p.pg.max_blocks;
                const int tpb = p.pg.block_size / BN, end_blk = (min(g.j1, g.n_cache) - 1) / tpb;
#pragma unroll 1
                for (int i = g.j0 / tpb + lane; i <= end_blk; i += 32) {
                  const int id = row[i];
                  bad |= id < 0 || id >= p.pg.num_blocks;
                }
              }
              bad = __any_sync(0xffffffffu, bad);
              if (lane == 0) {
                if (bad) atomicOr(&g_attn_ragged_err, kErrBadBlock);
                bars->seg[slot].bad = bad;
                mbar_arrive(&bars->seg_known[slot]);
              }
              ++count;
            }
            at += places;
          }
          if (++w == 32 || base + w >= B) {  // on to the next sequences, or to the streaming items (from W_r on)
            if (base + w >= B) {
              if (kind == 1) break;
              kind = 1;
              at = W_r;
              w = 0;
              if (base == 0) continue;
              base = 0;
            } else {
              base += 32;
              w = 0;
            }
            window();
          }
        }
      }
      const int slot = count % kSegs;
      if (ok && wait_warp(&bars->seg_empty[slot], (uint32_t)(((count / kSegs) & 1) ^ 1), err, kErrPrefillProducer) &&
          lane == 0) {
        bars->seg[slot].last = 1;
        mbar_arrive(&bars->seg_full[slot]);
      }
      if (lane == 0 && p.jobs) p.jobs[blockIdx.x] = job;
    } else if (warp == kWarpZero) {
      // ------------------------------------------------------------ sequences without a token: zeros
      if (!p.cu_new) {
#pragma unroll 1
        for (int b = blockIdx.x; b < B; b += gridDim.x) {
          if (p.seq_lens[b] > 0) continue;
          uint4* o = reinterpret_cast<uint4*>(p.o + (int64_t)b * p.sh.Hq * D);
#pragma unroll 1
          for (int e = lane; e < p.sh.Hq * D / 8; e += 32) o[e] = make_uint4(0, 0, 0, 0);
        }
      }
    } else if (warp == kWarpTma) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        const uint64_t pol_again = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
        SegReader in(bars);
        bool ok = true;
        int jt = 0;                // tiles so far
        uint32_t used = 0, qp = 3;  // places of query tiles: used at all, and the phases of q_empty (a bit each)
        int slot = 0;               // the place of the next single query tile
        while (ok) {
          if (!wait_for(in.full(), in.parity(), err, kErrPrefillProducer)) {
            ok = false;
            break;
          }
          const Seg g = in.seg();
          if (g.last) break;
          const bool two = g.rows > BM;
          // a sequence's other blocks of queries read the tiles again
          const uint64_t pol_kv = (int64_t)g.T << p.log2_g > kRaggedRows ? pol_again : pol_once;
#pragma unroll 1
          for (int x = 0; x < (two ? 2 : 1) && ok; ++x) {
            const int s = two ? x : slot;
            if (!wait_for(&bars->q_empty[s], (qp >> s) & 1u, err, kErrPrefillProducer)) {
              ok = false;
              break;
            }
            qp ^= 1u << s;
            used |= 1u << s;
            // a few rows: eight times, as rows 0-7 and 8-15 of each warp's 32
            const bool few = g.rows <= kFew;
            const int head = g.kvh << p.log2_g, tok = g.tok0 + g.q0 + x * (BM >> p.log2_g);
            mbar_arrive_expect_tx(&bars->q_full[s], few ? C::NBOX * 8 * 1024 : C::Q_BYTES);
#pragma unroll
            for (int bx = 0; bx < C::NBOX; ++bx) {
              uint8_t* dst = sQ + s * C::Q_BYTES + bx * kBox;
              if (!few) tma_load_3d(dst, &p.tm_q, bx * 64, head, tok, &bars->q_full[s]);
#pragma unroll 1
              for (int c = 0; few && c < 8; ++c)
                tma_load_3d(dst + (c >> 1) * 4096 + (c & 1) * 1024, &p.tm_q8, bx * 64, head, tok, &bars->q_full[s]);
            }
          }
          if (!two) slot ^= 1;
          const int32_t* row = p.pg.table + ((int64_t)g.b * p.sh.n_ret + g.cidx) * p.pg.max_blocks;
          const unsigned tpb = (unsigned)p.pg.block_size / BN;
          const bool paged = !g.streaming;
          int blk_next = paged && g.j0 < g.n_cache ? row[(unsigned)g.j0 / tpb] : 0;
#pragma unroll 1
          for (int j = g.j0; j < g.j1 && ok; ++j, ++jt) {
            const Tile t = tile_at(g, j);
            int blk = blk_next, prow = 0;
            if (paged && t.cache) {
              prow = (int)((unsigned)t.k % tpb) * BN;
              if (blk < 0 || blk >= p.pg.num_blocks) blk = (int)p.pg.num_blocks;  // out of range: zeros
              if (j + 1 < g.n_cache && j + 1 < g.j1) blk_next = row[(unsigned)(t.k + 1) / tpb];
            }
            const int s = jt % kNS;
            const uint32_t ph = (uint32_t)((jt / kNS) & 1);
            // (row and plane of the tile in whichever tensor it is in)
            const int c1 = !t.cache ? g.kvh : (paged ? prow : t.k * BN);
            const int c2 = !t.cache ? g.tok0 + t.k * BN : (paged ? blk : g.b * p.sh.n_str + g.cidx);
            auto load = [&](uint8_t* dst, uint64_t* bar, const CUtensorMap* fresh, const CUtensorMap* pool,
                            const CUtensorMap* ring) {
              const CUtensorMap* map = !t.cache ? fresh : (paged ? pool : ring);
              mbar_arrive_expect_tx(bar, C::KV_BYTES);
#pragma unroll
              for (int bx = 0; bx < C::NBOX; ++bx) tma_load_3d_hint(dst + bx * kBox, map, bx * 64, c1, c2, bar, pol_kv);
            };
            if (!wait_for(&bars->k_empty[s], ph ^ 1u, err, kErrPrefillProducer)) {
              ok = false;
              break;
            }
            load(sK + s * C::KV_BYTES, &bars->k_full[s], &p.tm_k, &p.tm_kpool, &p.tm_ksr);
            if (!wait_for(&bars->v_empty[s], ph ^ 1u, err, kErrPrefillProducer)) {
              ok = false;
              wait_for(&bars->k_full[s], ph, err, kErrPrefillProducer);  // in flight
              break;
            }
            load(sV + s * C::KV_BYTES, &bars->v_full[s], &p.tm_v, &p.tm_vpool, &p.tm_vsr);
          }
          in.done();
          ++in.count;
        }
        if (!ok) {
          // after an early exit, let the copies already issued land before the CTA ends
#pragma unroll 1
          for (int s = 0; s < 2; ++s)
            if ((used >> s) & 1u) wait_for(&bars->q_full[s], (qp >> s) & 1u, err, kErrPrefillProducer);
#pragma unroll 1
          for (int jj = (jt > kNS ? jt - kNS : 0); jj < jt; ++jj) {
            wait_for(&bars->k_full[jj % kNS], (uint32_t)((jj / kNS) & 1), err, kErrPrefillProducer);
            wait_for(&bars->v_full[jj % kNS], (uint32_t)((jj / kNS) & 1), err, kErrPrefillProducer);
          }
        }
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp follows the tiles and one lane issues. What decides where it goes is read through
      // shuffles, so that the compiler knows it to be the same for all lanes and keeps counters, barrier
      // addresses and descriptors in uniform registers, where the products need them: with one lane
      // following alone, they went there one by one, and a tile took 500 cycles more.
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
      const uint32_t tmem = uniform(*(volatile uint32_t*)&bars->tmem_base);
      // (a k-step only moves the start address, in the descriptors' low bits)
      const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(sV), kBox, 1024);
      // S_x = Q K^T, Q in place qs, K in stage s
      auto issue_s = [&](int x, int qs, int s) {
        const uint64_t dq = dq0 + (uint64_t)((qs * C::Q_BYTES) >> 4);
        const uint64_t dk = dk0 + (uint64_t)((s * C::KV_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t koff = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
          mma_ss(tmem + col_s(x), dq + koff, dk + koff, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(&bars->s_full[x]);
      };
      // O_x (+)= P_x V, V in stage s, over the first `rows` keys (in groups of 16)
      auto issue_pv = [&](int x, int s, bool first, int rows) {
        const uint64_t dv = dv0 + (uint64_t)((s * C::KV_BYTES) >> 4);
        if (rows == BN) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + col_o(x), tmem + col_s(x) + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                   (!first || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < (rows + 15) >> 4; ++kk)
            mma_ts(tmem + col_o(x), tmem + col_s(x) + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                   (!first || kk > 0) ? 1u : 0u);
        }
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, err, kErrPrefillMma); };
      SegReader in(bars);
      int jt = 0;                // tiles so far: tile jt is in stage jt % kNS
      uint32_t pp = 0, qp = 0;   // phases of p_full and q_full, a bit each
      int slot = 0, turn = 0;    // of segments with one query tile: Q's place, and x of the next tile
      bool ok = true;
      while (ok) {
        if (!(ok = ready(in.full(), in.parity()))) break;
        const Seg& g = in.seg();
        if (uniform(g.last)) break;
        const int nt = uniform(g.j1 - g.j0), rows = uniform(g.rows);
        const int cut_c = uniform(g.cut_cache - g.j0), cut_n = uniform(g.cut_new - g.j0);
        const int rows_c = uniform(g.rows_cache), rows_n = uniform(g.rows_new);
        if (elect_one()) in.done();
        ++in.count;
        auto k_ready = [&](int j) { return ready(&bars->k_full[j % kNS], (uint32_t)((j / kNS) & 1)); };
        auto v_ready = [&](int j) { return ready(&bars->v_full[j % kNS], (uint32_t)((j / kNS) & 1)); };
        // rows of tile t's V to multiply; what no token owns of their last 16 is set to zero first
        // (whole 128-byte rows of the boxes, so the swizzle does not matter)
        auto rows_to_use = [&](int t, int s) {
          if (t != cut_c && t != cut_n) return BN;
          const int r = t == cut_c ? rows_c : rows_n, pad = 16 - (r & 15);
          if (pad < 16) {
            uint8_t* v = sV + s * C::KV_BYTES + r * 128;
#pragma unroll 1
            for (int e = lane; e < pad * 8 * C::NBOX; e += 32)
              *reinterpret_cast<uint4*>(v + (e / (pad * 8)) * kBox + e % (pad * 8) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_shared();  // read by the tensor core next
            __syncwarp();
          }
          return r;
        };
        if (rows > BM) {
          // two query tiles, each K/V tile for both
          ok = ready(&bars->q_full[0], qp & 1u) && ready(&bars->q_full[1], (qp >> 1) & 1u) && k_ready(jt);
          qp ^= 3u;
          if (!ok) break;
          if (elect_one()) {
            tc_fence_after();
            issue_s(0, 0, jt % kNS);
            issue_s(1, 1, jt % kNS);
            tc_commit(&bars->k_empty[jt % kNS]);
            if (nt == 1) {
              tc_commit(&bars->q_empty[0]);
              tc_commit(&bars->q_empty[1]);
            }
          }
#pragma unroll 1
          for (int t = 0; t < nt; ++t, ++jt) {
            const bool more = t + 1 < nt;
            const int s = jt % kNS, sn = (jt + 1) % kNS;
            // A look at a barrier takes the warp 110 to 150 cycles, also when its phase is long over. D = 128, where
            // the tensor core bounds it: at three in one go (16384 tokens 1323 -> 1287 us). D = 64, where the
            // softmaxes do: not, as the later products keep the two of them out of phase (990; 1048 with it).
            bool there = false;
            if constexpr (D == 128) {
              const bool v = mbar_try_wait(&bars->v_full[s], (uint32_t)((jt / kNS) & 1));
              const bool k = !more || mbar_try_wait(&bars->k_full[sn], (uint32_t)(((jt + 1) / kNS) & 1));
              const bool p0 = mbar_try_wait(&bars->p_full[0], pp & 1u);
              there = __all_sync(0xffffffffu, v && k && p0);
            }
            if (!there && !(ok = v_ready(jt) && (!more || k_ready(jt + 1)))) break;
            const int v_rows = rows_to_use(t, s);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || (!(x == 0 && there) && !(ok = ready(&bars->p_full[x], (pp >> x) & 1u)))) break;
              if (elect_one()) {
                tc_fence_after();
                issue_pv(x, s, t == 0, v_rows);
                if (more) issue_s(x, x, sn);
                else tc_commit(&bars->o_final[x]);
                if (x == 1) {
                  tc_commit(&bars->v_empty[s]);
                  if (more) tc_commit(&bars->k_empty[sn]);
                }
                if (t + 2 == nt) tc_commit(&bars->q_empty[x]);  // the last scores of Q
              }
            }
            if (!ok) break;
            pp ^= 3u;
          }
        } else {
          // one query tile; the key tiles by turns with S_0 and O_0, and with S_1 and O_1 (across segments, so
          // that the end of one with a single tile runs beside the next one's softmax)
          const int qs = slot;
          slot ^= 1;
          ok = ready(&bars->q_full[qs], (qp >> qs) & 1u);
          qp ^= 1u << qs;
#pragma unroll 1
          for (int t = -2; t < nt && ok; ++t) {
            // P_x V of tile t (from 0 on), then the scores of tile t + 2
            const int x = (t ^ turn) & 1, j = jt + t;
            if (t >= 0) {
              if (!(ok = v_ready(j))) break;
              const int v_rows = rows_to_use(t, j % kNS);
              if (!(ok = ready(&bars->p_full[x], (pp >> x) & 1u))) break;
              pp ^= 1u << x;
              if (elect_one()) {
                tc_fence_after();
                issue_pv(x, j % kNS, t < 2, v_rows);
                tc_commit(&bars->v_empty[j % kNS]);
                if (t + 2 >= nt) tc_commit(&bars->o_final[x]);
              }
            }
            if (t + 2 < nt) {  // (K is waited for behind the product that gives V's stage back)
              if (!(ok = k_ready(j + 2))) break;
              if (elect_one()) {
                tc_fence_after();
                issue_s(x, qs, (j + 2) % kNS);
                tc_commit(&bars->k_empty[(j + 2) % kNS]);
                if (t + 3 == nt) tc_commit(&bars->q_empty[qs]);
              }
            }
          }
          turn ^= nt & 1;
          jt += nt;
        }
      }
      // every MMA issued here has finished before TMEM is released
      if (elect_one()) {
        tc_commit(&bars->drain);
        wait_for(&bars->drain, 0, err, kErrPrefillMma);
      }
    }
  } else {
    // ================================================ warpgroups 0, 1: softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int x = uniform(warp >> 2);
    const int r = (warp & 3) * 32 + lane;  // row within the query tile == TMEM lane
    const uint32_t lane_base = *(volatile uint32_t*)&bars->tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t sbase = lane_base + col_s(x);
    const uint32_t obase = lane_base + col_o(x);
    const float sl2 = p.scale_log2;
    SegReader in(bars);
    // phases of the barriers waited for, a bit each
    uint32_t phase = 0;
    constexpr uint32_t kPhS = 1, kPhO0 = 2, kPhO1 = 4, kPhPair = 8, kPhBoth = 16, kPhOne = 32;
    // the warps of both warpgroups, or of this one, wait for one another
    auto meet = [&](bool both) {
      const uint32_t bit = both ? kPhBoth : kPhOne;
      uint64_t* bar = both ? &bars->meet_both : &bars->meet_one[x];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      const bool met = wait_warp(bar, (phase & bit) != 0, err, kErrPrefillSoftmax);
      phase ^= bit;
      return met;
    };
    int turn = 0;  // of segments with one query tile: x of the next tile
    bool ok = true;
    while (ok) {
      if (!wait_warp(in.full(), in.parity(), err, kErrPrefillSoftmax)) break;
      const Seg& g = in.seg();
      if (uniform(g.last)) break;
      if (!wait_warp(in.known(), in.parity(), err, kErrPrefillSoftmax)) break;
      const bool two = uniform(g.rows) > BM;
      const int j0 = uniform(g.j0), nt = uniform(g.j1) - j0;
      const int step = two ? 1 : 2, t0 = two ? 0 : x ^ turn;  // its tiles: t0, t0 + step, ...
      const int row = two ? x * BM + r : r;            // of the item
      const bool mine_any = uniform(row) < uniform(g.rows);
      // tiles below plain are seen whole by every row, and so are those from n_cache on below diag, the first
      // one of the new tokens that some row of this query tile does not see whole; a streaming head's are
      // all masked, and so are those of a segment with a block that does not exist
      const int n_cache = uniform(g.n_cache);
      const int plain = uniform(g.streaming || g.bad ? 0 : (g.cut_cache >= 0 ? n_cache - 1 : n_cache));
      const int diag = uniform(g.streaming ? 0 : n_cache + (g.q0 + ((two ? x * BM : 0) >> p.log2_g)) / BN);
      float m_run = -INFINITY, l_run = 0.f;
      const bool few = uniform(g.rows) <= kFew;
      if (few) {
        // A few rows (single tokens): they stand in each warp's lanes 0-7 and again in 8-15. A warp takes 32 of
        // a tile's keys, with a maximum and a sum of its own, and leaves zeros for the others' keys in its rows
        // of P; lanes 8-15 write what the bf16 of lanes 0-7 leaves of P. The rows of O are added up at the
        // segment's end.
        const int w = warp & 3;
#pragma unroll 1
        for (int t = t0; t < nt; t += 2) {
          const int j = j0 + t;
          uint32_t vis = ~0u;
          if (j >= plain && (j < n_cache || j >= diag)) {
            const Tile tl = tile_at(g, j);
            bool gone = false;
            if (g.bad && tl.cache) {
              const int id = p.pg.table[((int64_t)g.b * p.sh.n_ret + g.cidx) * p.pg.max_blocks + tl.k / (p.pg.block_size / BN)];
              gone = id < 0 || id >= p.pg.num_blocks;
            }
            const int c = tl.k * BN + w * 32 + lane;
            const bool slot = g.streaming && tl.cache && c < min(g.n, p.sh.S + p.sh.R);
            const int jp = slot ? p.pos[(int64_t)g.b * (p.sh.S + p.sh.R) + c] : -1;
            const int i_abs = position(p, g, lane & 7);
            if (!tl.cache) vis = visible_new(p, g.streaming, i_abs, i_abs - (g.n + tl.k * BN), w * 32);
            else vis = gone ? 0u : visible_held(p, g.streaming, rows_of(g, j), w * 32, i_abs, jp);
          }
          const bool masked = __any_sync(0xffffffffu, vis != ~0u);
          if (!wait_warp(&bars->s_full[x], phase & kPhS, err, kErrPrefillSoftmax)) {
            ok = false;
            break;
          }
          phase ^= kPhS;
          tc_fence_after();
          float v[32];
          {
            uint32_t raw[32];
            tmem_ld32_sync(sbase + w * 32, raw);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
            const uint32_t none[16] = {};
#pragma unroll
            for (int i = 1; i < 4; ++i) tmem_st16(sbase + ((w + i) & 3) * 16, none);
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((vis >> e) & 1u)) v[e] = -INFINITY;
          }
          float mx = v[0], mx2 = v[1];
#pragma unroll
          for (int e = 2; e < 32; e += 4) {
            mx = max3(mx, v[e], v[e + 1]);
            if (e + 3 < 32) mx2 = max3(mx2, v[e + 2], v[e + 3]);
          }
          mx = fmaxf(mx, mx2) * sl2;
          float f = 1.f;
          if (mx > m_run + 8.f) {
            f = ex2_approx(m_run - mx);
            l_run *= f;
            m_run = mx;
          }
          if (__any_sync(0xffffffffu, lane < kFew && f != 1.f && t > t0)) {
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t ov[32];
              tmem_ld32_sync(obase + q4 * 32, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
              tmem_st32(obase + q4 * 32, ov);
            }
          }
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const float2 sl2x2 = make_float2(sl2, sl2), negm2 = make_float2(-m_use, -m_use);
          const float less = lane & kFew ? -1.f : 0.f;
          float2 ls = make_float2(0.f, 0.f);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(make_float2(v[2 * e], v[2 * e + 1]), sl2x2, negm2);
            const float2 pe = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            ls = __fadd2_rn(ls, pe);
            const uint32_t hi = pack_bf16x2(pe.x, pe.y);
            const float2 rest = __ffma2_rn(make_float2(bf16lo(hi), bf16hi(hi)), make_float2(less, less), pe);
            pk[e] = pack_bf16x2(rest.x, rest.y);
          }
          l_run += ls.x + ls.y;
          tmem_st16(sbase + w * 16, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[x]);
        }
      } else if (!mine_any) {
        // no rows: what its rows of S hold goes for P, and their O is not read
#pragma unroll 1
        for (int t = t0; t < nt && ok; t += step) {
          ok = wait_warp(&bars->s_full[x], phase & kPhS, err, kErrPrefillSoftmax);
          phase ^= kPhS;
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars->p_full[x]);
        }
      } else {
#pragma unroll 1
        for (int t = t0; t < nt; t += step) {
          const int j = j0 + t;
          uint32_t masked = 0;  // 32-key chunks in which some row of the warp does not see some key
          if (j >= plain && (j < n_cache || j >= diag)) {
            // the masks first, while the scores are on their way; they wait in shared memory
            const Tile tl = tile_at(g, j);
            const int i_abs = position(p, g, row);
            const int32_t* held = p.pos + (int64_t)g.b * (p.sh.S + p.sh.R);
            const int slots = min(g.n, p.sh.S + p.sh.R), keys = rows_of(g, j);
            if (j >= n_cache) {
              const int d = i_abs - (g.n + tl.k * BN);
              uint32_t vis[4];
#pragma unroll
              for (int q4 = 0; q4 < BN / 32; ++q4) {
                vis[q4] = visible_new(p, g.streaming, i_abs, d, q4 * 32);
                masked |= (uint32_t)__any_sync(0xffffffffu, vis[q4] != ~0u) << q4;
              }
              sVis[threadIdx.x] = make_uint4(vis[0], vis[1], vis[2], vis[3]);
            } else {
              bool gone = false;
              if (g.bad) {
                const int id = p.pg.table[((int64_t)g.b * p.sh.n_ret + g.cidx) * p.pg.max_blocks + tl.k / (p.pg.block_size / BN)];
                gone = id < 0 || id >= p.pg.num_blocks;
              }
              int jp = 0, jp_next = 0;
              const auto slot_pos = [&](int q4) {
                const int c = tl.k * BN + q4 * 32 + lane;
                return g.streaming && c < slots ? held[c] : -1;
              };
              jp_next = slot_pos(0);
#pragma unroll 1
              for (int q4 = 0; q4 < BN / 32; ++q4) {
                jp = jp_next;
                if (q4 < 3) jp_next = slot_pos(q4 + 1);
                const uint32_t vis = gone ? 0u : visible_held(p, g.streaming, keys, q4 * 32, i_abs, jp);
                masked |= (uint32_t)__any_sync(0xffffffffu, vis != ~0u) << q4;
                reinterpret_cast<uint32_t*>(&sVis[threadIdx.x])[q4] = vis;
              }
            }
          }
          if (!wait_warp(&bars->s_full[x], phase & kPhS, err, kErrPrefillSoftmax)) {
            ok = false;
            break;
          }
          phase ^= kPhS;
          tc_fence_after();
          float v[BN];
          {
            uint32_t raw[BN];
            tmem_ld128_sync(sbase, raw);
#pragma unroll
            for (int e = 0; e < BN; ++e) v[e] = __uint_as_float(raw[e]);
          }
          if (masked) {
#pragma unroll
            for (int q4 = 0; q4 < BN / 32; ++q4) {
              if (!((masked >> q4) & 1u)) continue;
              const uint32_t vis = reinterpret_cast<const uint32_t*>(&sVis[threadIdx.x])[q4];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) v[q4 * 32 + e] = -INFINITY;
            }
          }
          float mxa = v[0], mxb = v[1];
#pragma unroll
          for (int e = 2; e < BN; e += 4) {
            mxa = max3(mxa, v[e], v[e + 1]);
            if (e + 3 < BN) mxb = max3(mxb, v[e + 2], v[e + 3]);
          }
          const float mx_s = fmaxf(mxa, mxb) * sl2;
          float f = 1.f;
          if (mx_s > m_run + 8.f) {
            f = ex2_approx(m_run - mx_s);  // 0 while nothing was visible
            l_run *= f;
            m_run = mx_s;
          }
          // O rescale (rare); the last P V of this accumulator is complete since this S is
          if (__any_sync(0xffffffffu, f != 1.f && t > t0)) {
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t ov[32];
              tmem_ld32_sync(obase + q4 * 32, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
              tmem_st32(obase + q4 * 32, ov);
            }
          }
          // P = exp2(s scale - m), written over the first 64 columns of S
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          float2 ls = make_float2(0.f, 0.f);
          const float2 sl2x2 = make_float2(sl2, sl2), negm2 = make_float2(-m_use, -m_use);
#pragma unroll
          for (int q4 = 0; q4 < BN / 32; ++q4) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = __ffma2_rn(make_float2(v[q4 * 32 + 2 * e], v[q4 * 32 + 2 * e + 1]), sl2x2, negm2);
              const float p0 = ex2_approx(y.x);
              const float p1 = ex2_approx(y.y);
              ls = __fadd2_rn(ls, make_float2(p0, p1));
              pk[e] = pack_bf16x2(p0, p1);
            }
            tmem_st16(sbase + q4 * 16, pk);
          }
          l_run += ls.x + ls.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[x]);
        }
      }
      // ---------------------------------------------------------------- the segment's end
      const bool both = !two && nt > 1;  // two accumulators of the same rows
      const int part = uniform(g.part);
      if (few && ok && (both || x == turn)) {
        // row r: the sum over the warps (and the accumulators), half of the dims at a time (two accumulators: a
        // half by either warpgroup)
        const int w = warp & 3;
        if (lane < kFew) sML[x * BM + w * 32 + lane] = make_float2(m_run, l_run);
        ok = meet(both) && (!(both || x == 0) || wait_warp(&bars->o_final[0], (phase & kPhO0) != 0, err, kErrPrefillSoftmax)) &&
             (!(both || x == 1) || wait_warp(&bars->o_final[1], (phase & kPhO1) != 0, err, kErrPrefillSoftmax));
        if (ok) {
          tc_fence_after();
          // (lane: the parts of warp lane / 8)
          const float2 none = make_float2(-INFINITY, 0.f), *mls = sML + (lane & 7) + (lane >> 3) * 32;
          const float2 a0 = both || x == 0 ? mls[0] : none, a1 = both || x == 1 ? mls[BM] : none;
          float m = fmaxf(a0.x, a1.x);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          float f0 = a0.x == -INFINITY ? 0.f : ex2_approx(a0.x - m), f1 = a1.x == -INFINITY ? 0.f : ex2_approx(a1.x - m);
          float l = f0 * a0.y + f1 * a1.y;
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const float inv = part >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);  // (no key at all: zeros)
          f0 = __shfl_sync(0xffffffffu, f0, w * 8 + (lane & 7)) * inv;  // of this warp's own parts
          f1 = __shfl_sync(0xffffffffu, f1, w * 8 + (lane & 7)) * inv;
          if (part >= 0 && w == 0 && lane < g.rows && (!both || x == 0))
            p.part_ml[(int64_t)part * p.part_rows + lane] = make_float2(m, l);
          float* sum = sSum + (x * 4 * kFew) * C::PITCH;
          const int unit = w * 32 + lane, urow = unit / (D / 8), vec = unit % (D / 8);
#pragma unroll 1
          for (int h = both ? x : 0; ok && h < (both ? x + 1 : 2); ++h) {
#pragma unroll 1
            for (int u = 0; u < D / 64; ++u) {
              const uint32_t col = (uint32_t)(h * (D / 2) + u * 32);
              float ov[32] = {};
#pragma unroll 1
              for (int i = both ? 0 : x; i < (both ? 2 : x + 1); ++i) {
                uint32_t raw[32];
                tmem_ld32_sync(lane_base + col_o(i) + col, raw);
                const float fi = i ? f1 : f0;
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = fmaf(__uint_as_float(raw[e]), fi, ov[e]);
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] += __shfl_xor_sync(0xffffffffu, ov[e], kFew);
              if (lane < kFew) {
                float4* to = reinterpret_cast<float4*>(sum + (w * kFew + lane) * C::PITCH + u * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
              }
            }
            // (the accumulators have been read, too: the next segment's products may write them)
            tc_fence_before();
            if (!(ok = meet(both))) break;
            if (urow < g.rows) {
              float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 a = *reinterpret_cast<const float4*>(sum + (i * kFew + urow) * C::PITCH + vec * 4);
                o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
              }
              const int at4 = h * (D / 8) + vec;
              if (part >= 0) {
                reinterpret_cast<float4*>(p.part_o + (int64_t)part * p.part_rows * D)[(int64_t)at4 * p.part_rows + urow] = o;
              } else {
                const int64_t at = (int64_t)(g.tok0 + g.q0 + (urow >> p.log2_g)) * p.sh.Hq + (g.kvh << p.log2_g) +
                                   (urow & ((1 << p.log2_g) - 1));
                reinterpret_cast<uint2*>(p.o + at * D)[at4] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
              }
            }
            ok = meet(both);  // the sums have been read
          }
        }
      } else if (!few && ok && mine_any && (two || both || x == turn)) {
        // weights of the accumulators, and the dims this warp reads: all of its own, or half of both
        float f0 = 1.f, f1 = 0.f, m = m_run, l = l_run;
        if (both) {
          sML[x * BM + r] = make_float2(m_run, l_run);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->pair_ml[warp & 3]);
          ok = wait_warp(&bars->pair_ml[warp & 3], (phase & kPhPair) != 0, err, kErrPrefillSoftmax) &&
               wait_warp(&bars->o_final[0], (phase & kPhO0) != 0, err, kErrPrefillSoftmax) &&
               wait_warp(&bars->o_final[1], (phase & kPhO1) != 0, err, kErrPrefillSoftmax);
          if (ok) {
            const float2 a = sML[r], b = sML[BM + r];
            m = fmaxf(a.x, b.x);
            f0 = a.x == -INFINITY ? 0.f : ex2_approx(a.x - m);
            f1 = b.x == -INFINITY ? 0.f : ex2_approx(b.x - m);
            l = f0 * a.y + f1 * b.y;
          }
        } else {
          ok = wait_warp(&bars->o_final[x], (phase & (x ? kPhO1 : kPhO0)) != 0, err, kErrPrefillSoftmax);
        }
        if (ok) {
          tc_fence_after();
          const bool store = row < g.rows;
          // four rows whose chunks the lane stores: from `left` on behind the item; 4 divides g or g divides 4, so
          // where they lie apart is the same for all lanes
          const int four = row - (lane & 3), left = g.rows - four;
          const int64_t at = (int64_t)(g.tok0 + g.q0 + (four >> p.log2_g)) * p.sh.Hq + (g.kvh << p.log2_g) +
                             (four & ((1 << p.log2_g) - 1));
          uint4* orow = reinterpret_cast<uint4*>(p.o + at * D) + (lane & 3);
          int next_row[4];
#pragma unroll
          for (int a = 0; a < 4; ++a)
            next_row[a] = ((a >> p.log2_g) * p.sh.Hq + (a & ((1 << p.log2_g) - 1))) * (D / 8);
          if (part < 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;  // (no key at all: zeros)
            f0 *= inv;
            f1 *= inv;
          }
          const int q_first = both ? x * (D / 64) : 0, q_end = both ? q_first + D / 64 : D / 32;
          float4* prow = reinterpret_cast<float4*>(p.part_o + (int64_t)part * p.part_rows * D) + row;
#pragma unroll 1
          for (int q4 = q_first; q4 < q_end; ++q4) {
            float ov[32];
            {
              uint32_t raw[32];
              tmem_ld32_sync((both ? lane_base + col_o(0) : obase) + q4 * 32, raw);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __uint_as_float(raw[e]) * f0;
              if (both) {
                tmem_ld32_sync(lane_base + col_o(1) + q4 * 32, raw);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = fmaf(__uint_as_float(raw[e]), f1, ov[e]);
              }
            }
            if (store && part >= 0) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                prow[(int64_t)(q4 * 8 + e) * p.part_rows] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
            } else if (part < 0) {
              // four lanes exchange their rows' 64 bytes, so that each store has these of a row side by side
              // (32 rows of 16 bytes a store took 32 wavefronts)
              uint32_t w[4][4];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e / 4][e % 4] = pack_bf16x2(ov[2 * e], ov[2 * e + 1]);
#pragma unroll
              for (int k = 1; k < 4; k *= 2) {
                const bool up = lane & k;
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                  if (a & k) continue;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[a][e] : w[a + k][e], k);
                    w[a][e] = up ? got : w[a][e];
                    w[a + k][e] = up ? w[a + k][e] : got;
                  }
                }
              }
#pragma unroll
              for (int a = 0; a < 4; ++a)  // chunk lane % 4 of row `four` + a
                if (a < left) orow[next_row[a] + q4 * 4] = make_uint4(w[a][0], w[a][1], w[a][2], w[a][3]);
            }
          }
          if (store && part >= 0 && (!both || x == 0)) p.part_ml[(int64_t)part * p.part_rows + row] = make_float2(m, l);
          if (both) {
            // neither accumulator is written again before both warps have read it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->pair_done[warp & 3]);
            ok = wait_warp(&bars->pair_done[warp & 3], (phase & kPhPair) != 0, err, kErrPrefillSoftmax);
            phase ^= kPhPair;
          }
        }
      }
      phase ^= two || both ? kPhO0 | kPhO1 : (turn ? kPhO1 : kPhO0);
      if (!two) turn ^= nt & 1;
      __syncwarp();
      if (lane == 0) in.done();
      ++in.count;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(bars->tmem_base, kTmemCols);
  }
}

// The parts of an item: O = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s. A CTA takes 32 rows and 32 dims of
// an item: a lane a row, a warp four dims; with fewer rows the lanes left over share the parts. Eight
// parts are on their way at a time.
template <int D>
__global__ void __launch_bounds__(256) merge_ragged_kernel(const __grid_constant__ RaggedAttnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int NB = 8;
  const RaggedJob job = p.jobs[blockIdx.x];
  const int r0 = (int)blockIdx.y / (D / 32) * 32;
  if (job.last < 0 || r0 >= job.rows) return;
  const int lane = threadIdx.x & 31, vec = (int)blockIdx.y % (D / 32) * 8 + (threadIdx.x >> 5);
  int share = 1;  // lanes per row
  while (share < 32 && job.rows * share * 2 <= 32) share *= 2;
  const int width = 32 / share;
  const int row = r0 + lane % width, first = lane / width;
  const int parts = job.last - (int)blockIdx.x + 1;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  if (row < job.rows) {
    for (int s0 = first; s0 < parts; s0 += NB * share) {
      float2 ml[NB];
      float4 o[NB];
      float mn = M;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int s = s0 + k * share;
        const int64_t at = s == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * (int64_t)(blockIdx.x + s);
        ml[k] = make_float2(-INFINITY, 0.f);
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < parts) {
          ml[k] = __ldcg(p.part_ml + at * p.part_rows + row);
          o[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * p.part_rows * D) + (int64_t)vec * p.part_rows + row);
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) mn = fmaxf(mn, ml[k].x);
      const float keep = M == -INFINITY ? 0.f : ex2_approx(M - mn);
      l *= keep;
      acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float f = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - mn);
        l = fmaf(f, ml[k].y, l);
        acc.x = fmaf(f, o[k].x, acc.x);
        acc.y = fmaf(f, o[k].y, acc.y);
        acc.z = fmaf(f, o[k].z, acc.z);
        acc.w = fmaf(f, o[k].w, acc.w);
      }
      M = mn;
    }
  }
  for (int o = width; o < 32; o *= 2) {
    const float M2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float x2 = __shfl_xor_sync(0xffffffffu, acc.x, o), y2 = __shfl_xor_sync(0xffffffffu, acc.y, o);
    const float z2 = __shfl_xor_sync(0xffffffffu, acc.z, o), w2 = __shfl_xor_sync(0xffffffffu, acc.w, o);
    const float mn = fmaxf(M, M2);
    const float a = M == -INFINITY ? 0.f : ex2_approx(M - mn), b = M2 == -INFINITY ? 0.f : ex2_approx(M2 - mn);
    M = mn;
    l = a * l + b * l2;
    acc = make_float4(a * acc.x + b * x2, a * acc.y + b * y2, a * acc.z + b * z2, a * acc.w + b * w2);
  }
  if (row < job.rows && first == 0) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = ((int64_t)(job.tok + (row >> p.log2_g)) * p.sh.Hq + job.head + (row & ((1 << p.log2_g) - 1))) * D;
    reinterpret_cast<uint2*>(p.o + at)[vec] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

// The kernel's attributes on a device: set, and looked at, the first time.
template <int D>
cudaError_t prepare_t(int device) {
  static std::atomic<uint64_t> done{0};  // a bit per device (those past the last bit are prepared every time)
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaError_t e =
      cudaFuncSetAttribute(attn_ragged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, attn_ragged_kernel<D>)) != cudaSuccess) return e;
  // the setmaxnreg split is sized for exactly this launch allocation
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  done.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

template <int D>
cudaError_t launch_t(const RaggedAttnParams& p, int device, cudaStream_t stream) {
  using C = Cfg<D>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  cudaError_t e = prepare_t<D>(device);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, attn_ragged_kernel<D>, p)) != cudaSuccess || !p.jobs) return e;
  cfg.gridDim = dim3((unsigned)p.ctas, (unsigned)((p.part_rows + 31) / 32 * (D / 32)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, merge_ragged_kernel<D>, p);
}

}  // namespace

size_t ragged_workspace_bytes(int ctas, int rows, int D) {
  return (size_t)2 * ctas * rows * (D * sizeof(float) + sizeof(float2)) + (size_t)ctas * sizeof(RaggedJob);
}

cudaError_t launch_attn_ragged(const RaggedAttnParams& p, int device, cudaStream_t stream) {
  if (p.sh.D == 128) return launch_t<128>(p, device, stream);
  if (p.sh.D == 64) return launch_t<64>(p, device, stream);
  return cudaErrorInvalidValue;
}

cudaError_t attn_ragged_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_ragged_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_attn_ragged_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
