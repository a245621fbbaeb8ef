// duo_attn_decode_kv8: one query token per sequence over 8-bit caches (codes with one scale
// per 64 rows of a head, the open block in a bf16 tail) and the streaming heads' bf16 rings.
//
// A unit is one (sequence, KV head). Its keys are cut into tiles of 64 KB: 256 keys of codes (512
// at D = 64), or 128 bf16 rows of a ring or a tail (32 KB at D = 64). All tiles of all units, laid
// end to end in unit order with one tile's worth of room before each unit for what a unit costs
// apart from its keys (q, the merge of the warps), are shared out evenly over one CTA per SM:
// CTA c takes those that start in [c W / C, (c + 1) W / C). With lengths on the device every CTA
// sums the units' tiles itself, so a batch of ragged lengths is as balanced as a uniform one and
// nothing is planned on the host but the launch shape. (With the streaming units laid end to end
// without that room, the last CTAs had most of them: 119 us for a million tokens, 100 us with it.)
//
// Eight warps, each with its own slice of every tile (32 or 64 keys of codes, or 16 bf16 rows) and
// its own ring of two stages (K and V, 8 KB together) that it refills itself; no warp waits for
// another. Two, for fairness: with three, 128 KB or more on their way into every SM, some SMs got
// their bytes a fifth slower than others and the last one ended late (eight sequences of 131072
// tokens, e4m3: 75 us on average, 85 at most; 93 us against 86 in all).
// Codes come by TMA through a swizzled map, so that the matrix loads below are free of bank
// conflicts while the rows in HBM stay plain row-major, their two scales by 4-byte asynchronous
// copies on the same barrier; bf16 rows by 16-byte ones, swizzled by their addresses.
// (Twelve warps of 168 registers with two stages each were no faster: 93 us against 88 us for a
// million tokens then. D = 64 with 32-key slices paid every slice's fixed cost twice: 59 us against 35 us
// for 11 x 110556 tokens.)
//
// Per slice, on warp-level tensor-core products (a decode has one to eight query heads per
// KV head: 8 columns, far too few rows to fill a 128-row tcgen05 tile, and the time is
// HBM's: the products take a fraction of it):
//     S^T = K Q^T        rows = 16 keys, cols = heads, over the dims
//     O^T += s_v V^T P^T rows = 16 dims, cols = heads, over the keys
// Codes become fp16 exactly (int8: the byte with its sign bit flipped under the exponent of
// 1024, minus 1152; e4m3: the hardware conversion), the scales multiply the fp32 results: K's
// the scores, V's the slice's own fresh accumulator as it is added to the running one, so no
// scale passes through 16 bits and no accumulator grows long in the tensor core. q enters
// as fp16 after a scaling by a power of two of its own (exact), p as fp16 with 7 bits of
// headroom taken from above (p <= 2^15, flushed below 2^-31 of the maximum).
//
// K's fragments come by ldmatrix, V's by its transposing form for bytes, whose rows are named in
// the order that makes each lane's four bytes the keys of its P fragment: no byte is shuffled.
//
// bf16 rows (at most 63 of a tail, S + R of a ring) take bf16 products, p as two terms. Only these need
// masks.
//
// Bound by HBM: one million tokens with two retrieval heads, int8: 86 us in replayed graphs, one after the
// other = 6.25 TB/s of the 538 MB stored (0.92 of the measured copy rate), 83 us (0.95) among other calls,
// whose starts and merges overlap; a CTA works through a tile in 1.3 us, 7.5 TB/s in all. What is left is
// fixed: 2.8 us until a CTA's first tiles are under way, a merge of 0.8 us, the second kernel and two
// launches, 8 us. (The figures above and below are of replayed graphs.)
//
// Merge: as the bf16 decode. The warps of a CTA merge in shared memory; a unit split over
// CTAs leaves (o, max, sum) parts for a second kernel, launched as a programmatic dependent.
// A CTA has at most one part that goes on with a unit begun by another (its first) and one that
// begins a unit it does not end (its last): two places each. So there is one job for the second
// kernel at most per CTA of the first, however many units there are.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_decode_kv8_err;

constexpr int kWarps = kKv8Warps;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
// units of at most this many tiles are not split (their merge would cost more)
constexpr int kShortTiles = 4;
// weight of a place of a retrieval unit on the line of tiles, and the least that a CTA's share
// weighs: 2.5 places, so two of them whole wherever it begins
constexpr int kPlace = 8;
constexpr int kLeast = 20;
// p is kept times 2^kPShift: fp16 then holds it down to 2^-(24 + kPShift) of the row maximum,
// and up to 2^8 (lazy rescale) x 2^kPShift = 2^15
constexpr float kPShift = 7.f;

template <int D, int G>
struct Cfg {
  static constexpr int ROWS = kv8_slice_rows(D);  // keys of a slice of codes
  static constexpr int TK = ROWS * kWarps;        // and of a tile of them
  static constexpr int SLICE = ROWS * D;          // bytes of a warp's K (or V) codes
  static constexpr int STAGE = 2 * SLICE;
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int HR = G < 4 ? G : 4;  // heads merged at a time
  static constexpr int RED = kWarps * HR * (D + 2);
  static constexpr int PS = D + 4;  // floats per head of a part
  static constexpr int OFF_RED = RING;
  static constexpr int OFF_BAR = OFF_RED + 2 * RED * 4;  // (two merge buffers)
  static constexpr int OFF_SCALE = OFF_BAR + kWarps * kStages * 16;
  static constexpr size_t SMEM = (size_t)OFF_SCALE + kWarps * kStages * 8 + 1024;  // + alignment
};

__device__ __forceinline__ void tma_load_2d_hint(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar,
                                                 uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

// 4 bytes to shared memory, counted by the barrier's arrival below
__device__ __forceinline__ void copy4_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// one (already expected) arrival once this thread's earlier cp.async copies have landed
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8x8 matrices of 16-bit values (rows of 16 bytes, lane l naming row l % 8 of matrix l / 8):
// lane (gid, tig) gets the four bytes at 4 tig of row gid of each. Transposed: the values of
// rows 2 tig and 2 tig + 1 in column gid.
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared::cta.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Two 16x16 matrices of bytes, transposed (lane l names row l % 16 of matrix l / 16): of each, the
// bytes of rows 4 tig ... 4 tig + 3 in column gid, and in column gid + 8.
__device__ __forceinline__ void ldm2_trans8(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared::cta.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// 8x8 transpose of 16-bit values in fragment layout
__device__ __forceinline__ uint32_t transpose8x8(uint32_t m) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(m));
  return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes as two fp16 pairs, exactly. Which bytes make a pair is up to the code: e4m3's
// conversion takes neighbours (0, 1) and (2, 3); int8 takes (0, 2) and (1, 3), each pair one
// masked xor (a byte with its sign bit flipped under the exponent of 1024 reads as 1152 + code)
// after a shift for the second. byte_of: the byte in place i of pair j.
template <int CODE>
__host__ __device__ constexpr int byte_of(int j, int i) {
  return CODE == kKv8E4m3 ? 2 * j + i : j + 2 * i;
}
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& p0, uint32_t& p1) {
  if constexpr (CODE == kKv8E4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(p0), "=r"(p1)
        : "r"(w));
  } else {
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));  // 1152
    uint32_t l, h;
    asm("lop3.b32 %0, %1, 0x00FF00FF, 0x64806480, 0x6A;" : "=r"(l) : "r"(w));  // (w & mask) ^ magic
    asm("lop3.b32 %0, %1, 0x00FF00FF, 0x64806480, 0x6A;" : "=r"(h) : "r"(w >> 8));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
    p0 = *reinterpret_cast<const uint32_t*>(&a);
    p1 = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// Byte offset of 16-byte chunk c of row `row` of a slice as TMA's swizzle leaves it (rows of
// D bytes: the 128-byte pattern for D = 128, the 64-byte one for D = 64).
template <int D>
__device__ __forceinline__ int chunk_at(int row, int c) {
  return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

// The same for a bf16 slice, as its copies place it (rows of 2 D bytes).
template <int D>
__device__ __forceinline__ int chunk16_at(int row, int c) {
  return row * D * 2 + ((c ^ (row & 7)) << 4);
}

__device__ __forceinline__ int seq_len(const Kv8DecodeParams& p, int b) {
  if (!p.seq_lens) return (int)p.n;
  const int v = p.seq_lens[b];
  return v < 0 ? 0 : (v > p.n ? (int)p.n : v);
}

// Tiles of a retrieval / streaming unit of a sequence of n tokens (at least one, so that
// every unit's output is written).
__host__ __device__ __forceinline__ int code_rows_of(int n) { return n & ~(kKv8Block - 1); }
template <int D>
__host__ __device__ __forceinline__ int tiles_codes(int n) {
  constexpr uint32_t TK = Cfg<D, 1>::TK;
  return (int)(((uint32_t)code_rows_of(n) + TK - 1) / TK);
}
template <int D>
__host__ __device__ __forceinline__ int tiles_ret(int n) {
  const int t = tiles_codes<D>(n) + ((n & (kKv8Block - 1)) > 0);
  return t > 0 ? t : 1;
}
__host__ __device__ __forceinline__ int tiles_str(int n, int SR) {
  const int rows = n < SR ? n : SR;
  return rows > 0 ? (int)(((uint32_t)rows + kKv8TKBf16 - 1) / kKv8TKBf16) : 1;
}

struct Unit {
  int u, b, idx;  // idx: its index among the heads of its kind
  int n;          // tokens of the sequence
  int tiles, tc;  // tiles, and those of codes among them
  bool streaming;
};
template <int D>
__device__ __forceinline__ Unit unit_of(const Kv8DecodeParams& p, int u) {
  Unit x;
  x.u = u;
  x.streaming = u >= p.U_r;
  const uint32_t k = x.streaming ? u - p.U_r : u, heads = x.streaming ? p.sh.n_str : p.sh.n_ret;
  x.b = (int)(k / heads);
  x.idx = (int)(k - x.b * heads);
  x.n = seq_len(p, x.b);
  x.tiles = x.streaming ? tiles_str(x.n, p.sh.S + p.sh.R) : tiles_ret<D>(x.n);
  x.tc = x.streaming ? 0 : tiles_codes<D>(x.n);
  return x;
}
// Its query heads' first row in q and o.
template <int G>
__device__ __forceinline__ int64_t head_row(const Kv8DecodeParams& p, const Unit& x) {
  const int kvh = x.streaming ? p.heads.str_head[x.idx] : p.heads.ret_head[x.idx];
  return (int64_t)x.b * p.sh.Hq + kvh * G;
}
// Rows of a unit that are bf16: a streaming unit's ring slots, or the tail of the open block.
__device__ __forceinline__ int bf16_rows(const Kv8DecodeParams& p, const Unit& x) {
  const int SR = p.sh.S + p.sh.R;
  return x.streaming ? (x.n < SR ? x.n : SR) : x.n & (kKv8Block - 1);
}

// Places on the line of all tiles: a unit whose first tile is at ub takes tiles + 1 places, tile
// lt >= 1 is at ub + lt + 1. Tiles of a unit of T tiles that lie before place ub + y:
__device__ __forceinline__ int tiles_before(int64_t y, int T) {
  const int64_t t = y > 1 ? y - 1 : y;
  return t <= 0 ? 0 : (t < T ? (int)t : T);
}

// a b / c for a, b, c >= 0; in 32 bits where it fits (64-bit divisions on a CTA's way in and
// out cost a microsecond).
__device__ __noinline__ int64_t div64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  const int64_t ab = a * b;
  if (((ab | c) >> 32) == 0) return (int64_t)((uint32_t)ab / (uint32_t)c);
  return div64(ab, c);
}

// This CTA's share of the line of Wr places of retrieval units and W - Wr of streaming ones, places
// [x0, x1), starting in unit u at ub. The line is cut by weight: a retrieval place weighs kPlace, a
// streaming one p.str_place, WW in all. Each of the C CTAs that share
// it gets at least two places, so none inside a unit's span is left without a tile of it.
struct Share {
  int64_t W, Wr, WW, x0, x1, ub;
  int C, u;
};
// The CTA with place x.
__device__ __forceinline__ int cta_of(const Kv8DecodeParams& p, const Share& s, int64_t x) {
  const int64_t str = x + 1 - s.Wr;
  const int64_t end = str > 0 ? s.Wr * kPlace + str * p.str_place : (x + 1) * kPlace;  // weight up to its end
  return (int)mul_div(end * s.C - 1, 1, s.WW);
}
// The place in which weight w lies.
__device__ __forceinline__ int64_t place_at(const Kv8DecodeParams& p, const Share& s, int64_t w) {
  const int64_t str = w - s.Wr * kPlace;
  return str >= 0 ? s.Wr + mul_div(str, 1, p.str_place) : w / kPlace;
}
__device__ __forceinline__ void cut(const Kv8DecodeParams& p, Share& s, int64_t Wr, int64_t Ws) {
  const int c = blockIdx.x;
  s.Wr = Wr;
  s.W = Wr + Ws;
  s.WW = Wr * kPlace + Ws * p.str_place;
  const int64_t most = s.WW / kLeast;
  s.C = (int)(p.C < most ? p.C : (most > 1 ? most : 1));
  s.x0 = c < s.C ? place_at(p, s, mul_div(c, s.WW, s.C)) : s.W;
  s.x1 = c < s.C ? place_at(p, s, mul_div(c + 1, s.WW, s.C)) : s.W;
}

template <int D>
__device__ Share share_of(const Kv8DecodeParams& p, int64_t* scratch) {
  Share s;
  if (p.whole) {
    s.W = s.Wr = s.WW = s.x0 = s.x1 = s.ub = 0;
    s.C = p.C;
    s.u = blockIdx.x;
    return s;
  }
  if (!p.seq_lens) {
    cut(p, s, p.line_r, p.line_s);
    const bool in_r = s.x0 < p.line_r;
    const int64_t at = in_r ? s.x0 : s.x0 - p.line_r;
    const int64_t per = (in_r ? p.tiles_r : p.tiles_s) + 1;
    const int64_t k = mul_div(at, 1, per);
    s.u = (int)k + (in_r ? 0 : p.U_r);
    s.ub = s.x0 - at + k * per;
    return s;
  }
  const int SR = p.sh.S + p.sh.R;
  // lengths on the device: thread t sums the places of sequences [t per, (t + 1) per), then
  // the thread whose sums hold x0 finds the unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.sh.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.sh.B), b1 = min(b0 + per, p.sh.B);
  int64_t r = 0, q = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = seq_len(p, b);
    r += (int64_t)p.sh.n_ret * (tiles_ret<D>(n) + 1);
    q += (int64_t)p.sh.n_str * (tiles_str(n, SR) + 1);
  }
  const int64_t r_own = r, q_own = q;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, q, o);
    if (lane >= o) r += a, q += b;
  }
  if (lane == 31) {
    scratch[warp] = r;
    scratch[kWarps + warp] = q;
  }
  __syncthreads();
  int64_t Wr = 0, Wq = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) r += scratch[w], q += scratch[kWarps + w];
    Wr += scratch[w];
    Wq += scratch[kWarps + w];
  }
  cut(p, s, Wr, Wq);
  const bool in_r = s.x0 < Wr && s.x0 >= r - r_own && s.x0 < r;
  const bool in_q = s.x0 >= Wr && s.x0 - Wr >= q - q_own && s.x0 - Wr < q;
  if (in_r || in_q) {
    const int heads = in_r ? p.sh.n_ret : p.sh.n_str;
    int64_t base = in_r ? r - r_own : Wr + q - q_own;
    for (int b = b0; b < b1; ++b) {
      const int n = seq_len(p, b);
      const int64_t T = (in_r ? tiles_ret<D>(n) : tiles_str(n, SR)) + 1;
      if (s.x0 < base + heads * T) {
        const int64_t k = mul_div(s.x0 - base, 1, T);
        scratch[2 * kWarps] = (in_r ? 0 : p.U_r) + (int64_t)b * heads + k;
        scratch[2 * kWarps + 1] = base + k * T;
        break;
      }
      base += heads * T;
    }
  }
  __syncthreads();
  // (a CTA without a share starts past the end)
  s.u = s.x0 < s.x1 ? (int)scratch[2 * kWarps] : p.U_r + p.U_s;
  s.ub = s.x0 < s.x1 ? scratch[2 * kWarps + 1] : s.W;
  return s;
}

// A unit and this CTA's tiles of it.
template <int D>
struct Segment {
  Unit x;
  int64_t ub;
  int lt0, lt1;
  bool live;
  // from the unit (u, ub) on, the first of which the share has tiles
  __device__ __forceinline__ void find(const Kv8DecodeParams& p, const Share& s, int u, int64_t at) {
    ub = at;
    for (;; ++u) {
      live = p.whole ? u == s.u : ub < s.x1;
      if (!live) return;
      x = unit_of<D>(p, u);
      lt0 = p.whole ? 0 : tiles_before(s.x0 - ub, x.tiles);
      lt1 = p.whole ? x.tiles : tiles_before(s.x1 - ub, x.tiles);
      if (lt0 < lt1) return;
      ub += x.tiles + 1;  // (the share starts behind its last tile)
    }
  }
};

// The slices this warp takes, in order, over the CTA's share: one tile further each time, across
// units.
template <int D>
struct Cursor {
  static constexpr int TK = Cfg<D, 1>::TK;
  Unit x;
  int64_t ub, x1;
  int lt, lt1;      // next tile of the unit, and the end of the share's tiles in it
  int row, rows;    // first row of the slice in its codes (kv8_slice_rows(D) of them), or in its bf16 rows (1 to 16)
  int code_rows;    // rows of codes of the unit
  const int32_t* pages;  // paged codes: the unit's row of the block table,
  int blk;               // and the id of the page the slice lies in
  int warp;
  bool live, codes;

  // from this CTA's first segment on
  __device__ __forceinline__ void init(const Kv8DecodeParams& p, const Share& s, const Segment<D>& first, int w) {
    warp = w;
    live = first.live;
    if (!live) return;
    x = first.x;
    ub = first.ub;
    x1 = s.x1;
    lt = first.lt0;
    lt1 = first.lt1;
    settle(p);
  }
  // from tile lt on, the first with a slice for this warp
  __device__ __forceinline__ void settle(const Kv8DecodeParams& p) {
    for (;;) {
      if (lt < x.tc && lt < lt1) {
        code_rows = code_rows_of(x.n);
        const int64_t r = (int64_t)lt * TK + warp * Cfg<D, 1>::ROWS;
        if (r < code_rows) {
          row = (int)r;
          codes = true;
          if (p.pg.table) {
            pages = p.pg.table + ((int64_t)x.b * p.sh.n_ret + x.idx) * p.pg.max_blocks;
            blk = pages[(uint32_t)row / (uint32_t)p.pg.block_size];
          }
          return;
        }
        lt = x.tc;  // none in the last, partial tile of codes: on to the tail
      }
      if (lt < lt1) {
        const int64_t r = (int64_t)(lt - x.tc) * kKv8TKBf16 + warp * 16;
        const int have = bf16_rows(p, x);
        if (r < have) {
          row = (int)r;
          rows = min(16, have - row);
          codes = false;
          return;
        }
      }
      // nothing (more) for this warp in the unit
      ub += x.tiles + 1;
      if (p.whole || ub >= x1) {
        live = false;
        return;
      }
      x = unit_of<D>(p, x.u + 1);
      lt = 0;
      lt1 = tiles_before(x1 - ub, x.tiles);
    }
  }
  __device__ __forceinline__ void advance(const Kv8DecodeParams& p) {
    ++lt;
    if (codes && lt < lt1 && (int64_t)row + TK < code_rows) {  // (the most frequent case, kept short)
      row += TK;
      if (p.pg.table) blk = pages[(uint32_t)row / (uint32_t)p.pg.block_size];
      return;
    }
    settle(p);
  }
};

// Copies the cursor's slice of codes into a stage (lane 0). False: its page does not exist.
template <int D, int G>
__device__ __forceinline__ bool issue_codes(const Kv8DecodeParams& p, const Cursor<D>& cur, uint8_t* stage, float* scales,
                                            uint64_t* bar, uint64_t pol) {
  using C = Cfg<D, G>;
  int64_t row;
  if (p.pg.table) {
    if (cur.blk < 0 || cur.blk >= p.pg.num_blocks) {
      atomicOr(&g_decode_kv8_err, kErrBadBlock);
      mbar_arrive_expect_tx(bar, 0);
      mbar_arrive(bar);
      return false;
    }
    row = (int64_t)cur.blk * p.pg.block_size + (uint32_t)cur.row % (uint32_t)p.pg.block_size;
  } else {
    row = ((int64_t)cur.x.b * p.sh.n_ret + cur.x.idx) * p.cap64 + cur.row;
  }
  mbar_arrive_expect_tx(bar, C::STAGE);
  tma_load_2d_hint(stage, &p.tm_k, 0, (int)row, bar, pol);
  tma_load_2d_hint(stage + C::SLICE, &p.tm_v, 0, (int)row, bar, pol);
  copy4_async(scales, p.k_scale + row / kKv8Block);
  copy4_async(scales + 1, p.v_scale + row / kKv8Block);
  arrive_after_copies(bar);
  return true;
}

// Copies the cursor's bf16 rows into a stage (every lane; every lane arrives).
template <int D, int G>
__device__ __forceinline__ void issue_rows(const Kv8DecodeParams& p, const Cursor<D>& cur, uint8_t* stage, uint64_t* bar,
                                           int lane) {
  constexpr int CPR = D / 8;  // 16-byte chunks per row
  const int64_t first = cur.x.streaming ? ((int64_t)cur.x.b * p.sh.n_str + cur.x.idx) * (p.sh.S + p.sh.R) + cur.row
                                        : ((int64_t)cur.x.b * p.sh.n_ret + cur.x.idx) * kKv8Block + cur.row;
  const uint16_t* k = (cur.x.streaming ? p.k_sr : p.k_tail) + first * D;
  const uint16_t* v = (cur.x.streaming ? p.v_sr : p.v_tail) + first * D;
#pragma unroll
  for (int e = 0; e < 16 * CPR / 32; ++e) {
    const int i = lane + 32 * e, row = i / CPR, c = i % CPR;
    if (row < cur.rows) {
      copy16_async(stage + chunk16_at<D>(row, c), k + i * 8);
      copy16_async(stage + Cfg<D, G>::SLICE + chunk16_at<D>(row, c), v + i * 8);
    }
  }
  arrive_after_copies(bar);
}

// A warp's running softmax over the keys it has seen. Lane (gid, tig) = (lane / 4, lane % 4)
// holds, of heads 2 tig and 2 tig + 1, the maximum and its own part of the sum, and of O^T
// m-tile i the dims 16 i + gid (+ 8).
template <int D, int G>
struct State {
  static constexpr int MT = D / 16;  // m-tiles of O^T
  float o[MT][4];
  float m[2], l[2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // x[k]: scores in log2 units, head 2 tig + k % 2; replaced by p 2^kPShift. vis: bit k set
  // where the key is visible.
  template <int N, bool kMask>
  __device__ __forceinline__ void softmax(float (&x)[N], uint32_t vis) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (kMask && !((vis >> k) & 1u)) x[k] = -INFINITY;
      mx[k & 1] = fmaxf(mx[k & 1], x[k]);
    }
#pragma unroll
    for (int s = 4; s < 32; s <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], s));
    // the maximum moves only when a score passes it by 2^8
    const bool g0 = mx[0] > m[0] + 8.f, g1 = mx[1] > m[1] + 8.f;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float f0 = g0 ? ex2_approx(m[0] - mx[0]) : 1.f;
      const float f1 = g1 ? ex2_approx(m[1] - mx[1]) : 1.f;
      if (g0) m[0] = mx[0], l[0] *= f0;
      if (g1) m[1] = mx[1], l[1] *= f1;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f1;
        o[i][2] *= f0;
        o[i][3] *= f1;
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float pk = (!kMask || ((vis >> k) & 1u)) ? ex2_approx(x[k] - (m[k & 1] - kPShift)) : 0.f;
      x[k] = pk;
      l[k & 1] += pk;
    }
  }

  // One slice of codes, every key visible (addresses in shared memory). qb: q in B
  // fragments; kf: K's scale times the heads' factors.
  template <int CODE>
  __device__ __forceinline__ void codes(uint32_t sk, uint32_t sv, const uint32_t (&qb)[D / 16][2], float kf0, float kf1,
                                        float vs, int lane) {
    constexpr int NG = Cfg<D, G>::ROWS / 16;  // 16-key groups
    float x[4 * NG];
    // K: a fragment's words are the bytes 4 tig ... of rows gid and gid + 8, one 16-dim chunk each
    const int krow = lane & 15, kch = lane >> 4;
#pragma unroll
    for (int h = 0; h < NG; ++h) {  // keys 16 h + gid and 16 h + gid + 8
      float sc[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[c][k] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
        uint32_t w[4];
        ldm4(sk + chunk_at<D>(16 * h + krow, j + kch), w);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t a0, a1, a2, a3;
          decode4<CODE>(w[2 * c], a0, a2);
          decode4<CODE>(w[2 * c + 1], a1, a3);
          mma<true>(sc[c], a0, a1, a2, a3, qb[j + c][0], qb[j + c][1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = (sc[0][k] + sc[1][k]) * ((k & 1) ? kf1 : kf0);
    }
    softmax<4 * NG, false>(x, 0u);
    uint32_t pb[2 * NG];  // P^T: keys 16 h + 2 tig (+ 1) and + 8 (+ 9) of head gid
#pragma unroll
    for (int k = 0; k < 2 * NG; ++k) pb[k] = transpose8x8(pack_half2(x[2 * k], x[2 * k + 1]));
    // V: matrix row 4 t + e is the key whose byte lands in byte e of the words of lanes tig = t,
    // which is to be key 2 t (+ 1) in the first pair and 2 t + 8 (+ 9) in the second
    const int e = lane & 3, t = (lane >> 2) & 3;
    const int pair = CODE == kKv8E4m3 ? e >> 1 : e & 1, place = CODE == kKv8E4m3 ? e & 1 : e >> 1;
    const int vrow = 2 * t + place + 8 * pair, vch = lane >> 4;
    constexpr int HALF = MT / 2;  // m-tiles at a time: a slice's own accumulators stay few
#pragma unroll
    for (int i0 = 0; i0 < MT; i0 += HALF) {
      float acc[HALF][4];
#pragma unroll
      for (int i = 0; i < HALF; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
#pragma unroll
      for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int i = 0; i < HALF; i += 2) {
          uint32_t w[4];
          ldm2_trans8(sv + chunk_at<D>(16 * h + vrow, i0 + i + vch), w);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t a0, a1, a2, a3;
            decode4<CODE>(w[2 * c], a0, a2);
            decode4<CODE>(w[2 * c + 1], a1, a3);
            mma<true>(acc[i + c], a0, a1, a2, a3, pb[2 * h], pb[2 * h + 1]);
          }
        }
#pragma unroll
      for (int i = 0; i < HALF; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i0 + i][k] = fmaf(acc[i][k], vs, o[i0 + i][k]);
    }
  }

  // A slice of up to 16 bf16 rows. vis: bit k set where value k's key is visible (keys gid and
  // gid + 8, heads 2 tig and + 1); what lies in the other rows is not used.
  __device__ __forceinline__ void rows16(uint32_t sk, uint32_t sv, uint32_t vis, const uint32_t (&qa)[D / 16][2],
                                         float qf, int lane) {
    const int tig = lane & 3;
    float sc[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[c][k] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t w[4];
      ldm4(sk + chunk16_at<D>(lane & 15, 2 * j + (lane >> 4)), w);
      mma<false>(sc[j & 1], w[0], w[1], w[2], w[3], qa[j][0], qa[j][1]);
    }
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (sc[0][k] + sc[1][k]) * qf;
    softmax<4, true>(x, vis);
    // p in two bf16 terms, 2^-17 of it left out: one alone, 2^-9, was most of the decode's error (outputs
    // 0.0022 of their norm off, the streaming heads' above all, where the output's rounding is 0.0017)
    const uint32_t p01 = pack_bf16x2(x[0], x[1]), p23 = pack_bf16x2(x[2], x[3]);
    const uint32_t pb0 = transpose8x8(p01), pb1 = transpose8x8(p23);
    const uint32_t pl0 = transpose8x8(pack_bf16x2(x[0] - bf16lo(p01), x[1] - bf16hi(p01)));
    const uint32_t pl1 = transpose8x8(pack_bf16x2(x[2] - bf16lo(p23), x[3] - bf16hi(p23)));
    // a value row nobody sees (an empty or evicted slot) may hold anything: out of the product.
    // Lane (g, .) knows of keys g and g + 8; the V fragments hold keys 2 tig, 2 tig + 1 (+ 8).
    const uint32_t seen = __ballot_sync(0xffffffffu, vis & 1u);          // bit 4 g: key g
    const uint32_t seen8 = __ballot_sync(0xffffffffu, (vis >> 2) & 1u);  // bit 4 g: key g + 8
    const uint32_t m0 = ((seen >> (8 * tig)) & 1u) * 0xFFFFu | ((seen >> (8 * tig + 4)) & 1u) * 0xFFFF0000u;
    const uint32_t m8 = ((seen8 >> (8 * tig)) & 1u) * 0xFFFFu | ((seen8 >> (8 * tig + 4)) & 1u) * 0xFFFF0000u;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t w[4];  // dims 16 i + gid and + 8, keys below 8; the same, keys from 8
      ldm4_trans(sv + chunk16_at<D>((lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)), w);
      const uint32_t v0 = w[0] & m0, v1 = w[1] & m0, v2 = w[2] & m8, v3 = w[3] & m8;
      mma<false>(o[i], v0, v1, v2, v3, pl0, pl1);
      mma<false>(o[i], v0, v1, v2, v3, pb0, pb1);
    }
  }

  // the sums of the warp's lanes
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int s = 4; s < 32; s <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += __shfl_xor_sync(0xffffffffu, l[e], s);
  }
  // (o, max, sum) of heads [h0, h0 + HR) into the CTA's merge buffer: red[(warp HR + h - h0) (D + 2) + d]
  __device__ __forceinline__ void write(float* red, int h0, int warp, int gid, int tig) {
    constexpr int HR = Cfg<D, G>::HR;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 2 * tig + e - h0;
      if (h < 0 || h >= HR) continue;
      float* r = red + (warp * HR + h) * (D + 2);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        r[16 * i + gid] = o[i][e];
        r[16 * i + gid + 8] = o[i][2 + e];
      }
      if (gid == 0) *reinterpret_cast<float2*>(r + D) = make_float2(m[e], l[e]);
    }
  }
};

// q of head gid (nullptr past the last) as bf16 B fragments for rows16, and as fp16 ones for
// codes: scaled by 2^(8 - e), e the exponent of the head's largest |q|, so that every bf16
// value down to 2^-22 of the largest stays exact. Returns 2^(e - 8).
template <int D, int CODE>
__device__ __forceinline__ float convert_q(uint32_t (&qb)[D / 16][2]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) m = __vmaxu2(m, __vmaxu2(qb[j][0] & 0x7FFF7FFFu, qb[j][1] & 0x7FFF7FFFu));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  int e = (int)(max(m & 0xFFFFu, m >> 16) >> 7);  // biased exponent
  e = e < 9 ? 9 : (e > 254 ? 254 : e);
  const float f = __uint_as_float((uint32_t)(262 - e) << 23);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const float v[4] = {bf16lo(qb[j][0]) * f, bf16hi(qb[j][0]) * f, bf16lo(qb[j][1]) * f, bf16hi(qb[j][1]) * f};
#pragma unroll
    for (int k = 0; k < 2; ++k) qb[j][k] = pack_half2(v[byte_of<CODE>(k, 0)], v[byte_of<CODE>(k, 1)]);
  }
  return __uint_as_float((uint32_t)(e - 8) << 23);
}

// Entry of the merge's jobs, behind the parts: by unit (its first CTA, its number of parts) if
// p.merge_units, else by CTA (a unit it begins and does not end, or -1; its number of parts).
__device__ __forceinline__ int2* job_of(const Kv8DecodeParams& p, int i) {
  return reinterpret_cast<int2*>(p.partials + (int64_t)2 * p.C * p.sh.g * (p.sh.D + 4)) + i;
}

// What a lane needs of q's row of head gid (nullptr past the last): for codes dims 16 j + 4 tig
// ... + 3 (convert_q makes the fragments), for bf16 rows the fragments themselves.
template <int D>
__device__ __forceinline__ void fetch_q(const uint16_t* qh, bool codes, uint32_t (&q)[D / 16][2], int tig) {
  const uint16_t* a = qh ? qh + (codes ? 4 * tig : 2 * tig) : nullptr;
  const int second = codes ? 2 : 8;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    q[j][0] = a ? __ldg(reinterpret_cast<const uint32_t*>(a + 16 * j)) : 0u;
    q[j][1] = a ? __ldg(reinterpret_cast<const uint32_t*>(a + 16 * j + second)) : 0u;
  }
}

// Positions held by ring slots gid and gid + 8 of a warp's slice, which starts at slot r0 (-1
// past the last; any position does for a tail's rows).
__device__ __forceinline__ void fetch_pos(const Kv8DecodeParams& p, const Unit& x, int r0, int have, int gid, int (&at)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = r0 + gid + 8 * k;
    at[k] = row >= have ? -1 : (x.streaming ? p.pos[(int64_t)x.b * (p.sh.S + p.sh.R) + row] : 0);
  }
}

template <int D, int G, int CODE>
__global__ void __launch_bounds__(kThreads, 1) decode_kv8_kernel(const __grid_constant__ Kv8DecodeParams p) {
  using C = Cfg<D, G>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  const DevError err{&g_decode_kv8_err};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * kStages * C::STAGE;
  // per stage one barrier for codes (the bulk copies' bytes, and the two scales' arrival) and
  // one for bf16 rows (every lane's arrival)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * kStages * 2;
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE) + warp * kStages * 2;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[2 * s], 2);
      mbar_init(&bars[2 * s + 1], 32);
    }
    fence_mbarrier_init();
    if (p.U_r > 0) {
      prefetch_tmap(&p.tm_k);
      prefetch_tmap(&p.tm_v);
    }
  }
  __syncthreads();
  // Launched as a programmatic dependent: nothing the grid before it writes is read earlier, and none of
  // it (lengths, tables, ring positions) through the read-only path, which may assume that it does not
  // change while this kernel lives.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Share sh = share_of<D>(p, reinterpret_cast<int64_t*>(red));
  __syncthreads();  // (share_of's scratch is the merge buffer)
  const uint64_t pol = l2_policy_evict_first();  // codes are read once

  Cursor<D> cur;
  Segment<D> sg;
  sg.find(p, sh, sh.u, sh.ub);
  cur.init(p, sh, sg, warp);
  int fill = 0, use = 0;             // stages to fill and to use next
  uint32_t pending = 0, phases = 0;  // bit of a barrier: copies under way; the phase to wait for
  uint32_t bad = 0;                  // lane 0: bit s set if stage s was not copied
  bool rows_seen = false;
  auto refill = [&]() {
    uint8_t* stage = ring + fill * C::STAGE;
    if (cur.codes) {
      if (lane == 0) {
        if (rows_seen) fence_proxy_async_shared();  // a stage may have held rows written by cp.async
        const bool there = issue_codes<D, G>(p, cur, stage, scales + 2 * fill, &bars[2 * fill], pol);
        bad = there ? bad & ~(1u << fill) : bad | (1u << fill);
      }
      pending |= 1u << (2 * fill);
    } else {
      issue_rows<D, G>(p, cur, stage, &bars[2 * fill + 1], lane);
      pending |= 2u << (2 * fill);
      rows_seen = true;
    }
    fill = fill + 1 == kStages ? 0 : fill + 1;
    cur.advance(p);
  };
  for (int s = 0; s < kStages - 1 && cur.live; ++s) refill();

  bool ok = true;  // of this warp: a wait that ran out stops its copies, not the CTA's barriers
  State<D, G> st;
  auto wait = [&](int b) {
    const bool done = mbar_wait_warp(&bars[b], (phases >> b) & 1u, err, kErrDecodeConsumer);
    phases ^= 1u << b;
    pending &= ~(1u << b);
    return done;
  };
  // next slice: refills the stage of the one before, and waits for its own
  auto next = [&](int kind) {
    if (cur.live && ok) refill();
    const int s = use;
    if (ok) ok = wait(2 * s + kind);
    use = use + 1 == kStages ? 0 : use + 1;
    return s;
  };
  // fetched ahead for the unit that comes next, while the warps of this one are merged
  uint32_t q[D / 16][2];
  int at[2];
  int64_t hrow = 0;
  auto fetch = [&]() {
    hrow = head_row<G>(p, sg.x);
    const bool codes = sg.lt0 < sg.x.tc;
    fetch_q<D>(gid < G ? p.q + (hrow + gid) * D : nullptr, codes, q, tig);
    if (!codes) fetch_pos(p, sg.x, (sg.lt0 - sg.x.tc) * kKv8TKBf16 + warp * 16, bf16_rows(p, sg.x), gid, at);
  };
  if (sg.live) fetch();
  int buf = 0;
  int2 job = make_int2(-1, 0);  // for the merge: a unit this CTA begins and does not end, its parts
  while (sg.live) {
    const Unit x = sg.x;
    const int lt0 = sg.lt0, lt1 = sg.lt1, tc = x.tc;
    const int64_t ub = sg.ub, orow = hrow;
    st.reset();
    if (lt0 < tc) {
      const float f = convert_q<D, CODE>(q) * p.scale_log2;
      const float f0 = __shfl_sync(0xffffffffu, f, 8 * tig), f1 = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
      int left = (lt1 < tc ? lt1 : tc) - lt0;  // this warp's slices: none in a tile it lies behind
      if ((int64_t)(lt0 + left - 1) * C::TK + warp * C::ROWS >= code_rows_of(x.n)) --left;
      for (; left > 0; --left) {
        const int s = next(0);
        const bool skip = !ok || ((__shfl_sync(0xffffffffu, bad, 0) >> s) & 1u);
        if (!skip) {
          const uint32_t sk = smem_u32(ring + s * C::STAGE);
          const float ks = scales[2 * s], vs = scales[2 * s + 1];
          st.template codes<CODE>(sk, sk + C::SLICE, q, f0 * ks, f1 * ks, vs, lane);
        }
        __syncwarp();
      }
      if (lt1 > tc) {  // the tail's tile follows
        fetch_q<D>(gid < G ? p.q + (orow + gid) * D : nullptr, false, q, tig);
        fetch_pos(p, x, warp * 16, bf16_rows(p, x), gid, at);
      }
    }
    const int have = bf16_rows(p, x);
    for (int lt = lt0 > tc ? lt0 : tc; lt < lt1; ++lt) {  // a streaming unit's tiles, or the tail's one
      const int r0 = (lt - tc) * kKv8TKBf16 + warp * 16;
      if (r0 >= have) break;
      uint32_t vis = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool v = at[k] >= 0 && (!x.streaming || (at[k] < x.n && (at[k] < p.sh.S || x.n - 1 - at[k] < p.sh.R)));
        vis |= (v ? 3u : 0u) << (2 * k);
      }
      if (lt + 1 < lt1) fetch_pos(p, x, r0 + kKv8TKBf16, have, gid, at);
      const int s = next(1);
      const uint32_t sk = smem_u32(ring + s * C::STAGE);
      if (ok) st.rows16(sk, sk + C::SLICE, vis, q, p.scale_log2, lane);
      __syncwarp();
    }
    sg.find(p, sh, x.u + 1, ub + x.tiles + 1);
    if (sg.live) fetch();

    // merge of the warps, HR heads at a time, in two buffers in turn: a warp may write the next
    // one while another still reads this one, and is past the barrier between before its turn
    st.finish();
    int n_parts = 1;
    if (!p.whole && (lt0 > 0 || lt1 < x.tiles)) n_parts = cta_of(p, sh, ub + x.tiles) - cta_of(p, sh, ub) + 1;
    float* part = p.partials + (int64_t)(2 * blockIdx.x + (lt0 == 0)) * G * C::PS;
    if (lt0 == 0 && p.merge_units) {
      if (tid == 0) *job_of(p, x.u) = make_int2(blockIdx.x, n_parts);
    } else if (lt0 == 0 && n_parts > 1) {
      job = make_int2(x.u, n_parts);
    }
#pragma unroll 1
    for (int h0 = 0; h0 < G; h0 += C::HR) {
      float* rb = red + buf * C::RED;
      buf ^= 1;
      st.write(rb, h0, warp, gid, tig);
      __syncthreads();
      // a thread two dims of a head, everything it needs in flight together
      for (int e = tid; e < C::HR * D / 2; e += kThreads) {
        const int h = e / (D / 2), d = 2 * (e % (D / 2));
        float2 ml[kWarps], ov[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* r = rb + (w * C::HR + h) * (D + 2);
          ml[w] = *reinterpret_cast<const float2*>(r + D);
          ov[w] = *reinterpret_cast<const float2*>(r + d);
        }
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w].x);
        float n0 = 0.f, n1 = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ml[w].x == -INFINITY && !(ml[w].y != 0.f) ? 0.f : ex2_approx(ml[w].x - M);
          n0 = fmaf(f, ov[w].x, n0);
          n1 = fmaf(f, ov[w].y, n1);
          den = fmaf(f, ml[w].y, den);
        }
        float* ph = part + (h0 + h) * C::PS;
        if (n_parts == 1) {
          const float inv = den != 0.f ? 1.f / den : 0.f;
          *reinterpret_cast<uint32_t*>(p.o + (orow + h0 + h) * D + d) = pack_bf16x2(n0 * inv, n1 * inv);
        } else {
          *reinterpret_cast<float2*>(ph + d) = make_float2(n0, n1);
          if (d == 0) *reinterpret_cast<float2*>(ph + D) = make_float2(M, den);
        }
      }
    }
  }
  if (!p.whole && !p.merge_units && tid == 0) *job_of(p, blockIdx.x) = job;
  // copies still in flight (after a wait that ran out) land before the CTA ends
#pragma unroll 1
  for (int b = 0; b < 2 * kStages; ++b)
    if ((pending >> b) & 1u) wait(b);
  __syncthreads();
}

// Merge of the units whose tiles were split over CTAs, launched as the decode's programmatic
// dependent. Two shapes:
//   kWide: few units, with up to one part per SM each. A CTA takes 32 dims of one unit's head;
//          four warps take every fourth part, up to 20 of them in flight each.
//   else:  many units, few parts each. A CTA takes the unit that CTA blockIdx.x of the decode has
//          begun and not ended, all its heads; the warps of a head take the parts in turn.
template <int D, int G, bool kWide>
__global__ void __launch_bounds__(kWide ? 128 : 256) decode_kv8_merge_kernel(const __grid_constant__ Kv8DecodeParams p) {
  constexpr int PS = Cfg<D, G>::PS, V = kWide ? 1 : D / 32;  // dims per lane
  constexpr int NW = kWide ? 4 : 8, NG = kWide ? 4 : 8 / G;  // warps, and those of one head
  constexpr int NB = kWide ? 20 : 4;                         // parts in flight per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = kWide ? warp : warp / G;
  const int h = kWide ? blockIdx.x / (D / 32) % G : warp % G;
  const int d = kWide ? blockIdx.x % (D / 32) * 32 + lane : lane * V;
  const int key = kWide ? blockIdx.x / (D / 32 * G) : blockIdx.x;
  __shared__ float s_o[NW][32 * V], s_m[NW], s_l[NW];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 job = __ldcg(job_of(p, key));
  const int u = kWide ? key : job.x, c = kWide ? job.x : key, n_parts = job.y;
  if (n_parts <= 1) return;
  const float* cont = p.partials + ((int64_t)2 * c * G + h) * PS;  // part i >= 1: 2 i G PS further
  const float* head = cont + G * PS;
  float acc[V], M = -INFINITY, den = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int i0 = grp; i0 < n_parts; i0 += NG * NB) {
    float mb[NB], lb[NB], ob[NB][V];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int k = i0 + i * NG;
      const float* r = k == 0 ? head : cont + (int64_t)2 * k * G * PS;
      mb[i] = -INFINITY;
      lb[i] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) ob[i][v] = 0.f;
      if (k < n_parts) {
        mb[i] = __ldcg(r + D);
        lb[i] = __ldcg(r + D + 1);
#pragma unroll
        for (int v = 0; v < V; ++v) ob[i][v] = __ldcg(r + d + v);
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < NB; ++i) mn = fmaxf(mn, mb[i]);
    const float fo = M == -INFINITY && !(den != 0.f) ? 0.f : ex2_approx(M - mn);
    den *= fo;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= fo;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const float f = mb[i] == -INFINITY && !(lb[i] != 0.f) ? 0.f : ex2_approx(mb[i] - mn);
      den = fmaf(f, lb[i], den);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(f, ob[i][v], acc[v]);
    }
    M = mn;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = acc[v];
  if (lane == 0) s_m[warp] = M, s_l[warp] = den;
  __syncthreads();
  if (grp == 0) {
    constexpr int STEP = kWide ? 1 : G;  // warps between those of a head
    float T = -INFINITY, num[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) num[v] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) T = fmaxf(T, s_m[g * STEP + warp]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int w = g * STEP + warp;
      const float f = s_m[w] == -INFINITY && !(s_l[w] != 0.f) ? 0.f : ex2_approx(s_m[w] - T);
      sum = fmaf(f, s_l[w], sum);
#pragma unroll
      for (int v = 0; v < V; ++v) num[v] = fmaf(f, s_o[w][lane * V + v], num[v]);
    }
    const bool streaming = u >= p.U_r;
    const int us = streaming ? u - p.U_r : u, nk = streaming ? p.sh.n_str : p.sh.n_ret;
    const int b = us / nk;
    const int kvh = streaming ? p.heads.str_head[us - b * nk] : p.heads.ret_head[us - b * nk];
    uint16_t* out = p.o + ((int64_t)b * p.sh.Hq + (int64_t)kvh * G + h) * D + d;
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = __bfloat16_as_ushort(__float2bfloat16_rn(sum != 0.f ? num[v] / sum : 0.f));
  }
}

template <int D, int G, int CODE>
cudaError_t launch_t(const Kv8DecodeParams& p, cudaStream_t stream) {
  using C = Cfg<D, G>;
  static_assert(C::SMEM <= 232448, "shared memory");
  // the attribute belongs to a device's copy of the kernel
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(decode_kv8_kernel<D, G, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_kv8_kernel<D, G, CODE>, p);
  if (e != cudaSuccess || p.whole) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3((unsigned)(p.merge_units ? (p.U_r + p.U_s) * G * (D / 32) : p.C));
  cfg.blockDim = dim3(p.merge_units ? 128 : 256);
  return p.merge_units ? cudaLaunchKernelEx(&cfg, decode_kv8_merge_kernel<D, G, true>, p)
                       : cudaLaunchKernelEx(&cfg, decode_kv8_merge_kernel<D, G, false>, p);
}

template <int D, int CODE>
cudaError_t launch_g(const Kv8DecodeParams& p, cudaStream_t stream) {
  switch (p.sh.g) {
    case 1: return launch_t<D, 1, CODE>(p, stream);
    case 2: return launch_t<D, 2, CODE>(p, stream);
    case 4: return launch_t<D, 4, CODE>(p, stream);
    case 8: return launch_t<D, 8, CODE>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

void plan_decode_kv8(Kv8DecodeParams* p, int num_sms) {
  const int64_t U = (int64_t)p->U_r + p->U_s;
  p->tiles_r = p->sh.D == 128 ? tiles_ret<128>((int)p->n) : tiles_ret<64>((int)p->n);
  p->tiles_s = tiles_str((int)p->n, p->sh.S + p->sh.R);
  p->line_r = (int64_t)p->U_r * (p->tiles_r + 1);
  p->line_s = (int64_t)p->U_s * (p->tiles_s + 1);
  p->whole = U <= num_sms && (p->U_r == 0 || p->tiles_r <= kShortTiles) && (p->U_s == 0 || p->tiles_s <= kShortTiles);
  // int8 codes take a fifth longer per tile than e4m3's or a ring's rows (a streaming unit of one
  // tile costs its two places all the same): 128 ragged sequences of up to 700 tokens 49.2 us with
  // even places, 46.5 so; 48 of up to 32000 84.3, 83.1; e4m3 so 79.3 instead of 75.6
  p->str_place = p->code_type == kKv8Int8 && p->sh.S + p->sh.R > kKv8TKBf16 ? kPlace - 1 : kPlace;
  const int64_t most = std::max<int64_t>(1, (p->line_r * kPlace + p->line_s * p->str_place) / kLeast);
  p->C = (int)(p->whole ? U : (most < num_sms ? most : num_sms));
  // merge by unit, 32 dims a CTA, where that is no more than a CTA per SM
  p->merge_units = U <= p->C && U * p->sh.g * (p->sh.D / 32) <= num_sms;
}

size_t decode_kv8_workspace_bytes(const Kv8DecodeParams& p) {
  if (p.whole) return 0;
  const size_t part = (size_t)p.sh.g * (p.sh.D + 4) * sizeof(float);
  return 2 * (size_t)p.C * part + (p.merge_units ? (size_t)p.U_r + p.U_s : (size_t)p.C) * sizeof(int2);
}

cudaError_t launch_decode_kv8(const Kv8DecodeParams& p, cudaStream_t stream) {
  if (p.sh.D == 128)
    return p.code_type == kKv8E4m3 ? launch_g<128, kKv8E4m3>(p, stream) : launch_g<128, kKv8Int8>(p, stream);
  if (p.sh.D == 64)
    return p.code_type == kKv8E4m3 ? launch_g<64, kKv8E4m3>(p, stream) : launch_g<64, kKv8Int8>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t decode_kv8_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_kv8_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_decode_kv8_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
