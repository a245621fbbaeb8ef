// duo_attn_decode_kv8: one query token per sequence over 8-bit caches (codes with one scale
// per 64 rows of a head, the open block in a bf16 tail) and the streaming heads' bf16 rings.
//
// A unit is one (sequence, KV head). Its keys are cut into tiles of 64 KB (at D = 128): 256
// keys of codes, or 128 bf16 rows of a ring or a tail. All tiles of all units, laid end to end
// in unit order with one tile's worth of room before each unit for what a unit costs apart from
// its keys (q, the merge of the warps), are shared out evenly over one CTA per SM: CTA c takes
// those that start in [c W / C, (c + 1) W / C). With lengths on the device every CTA sums the
// units' tiles itself, so a batch of ragged lengths is as balanced as a uniform one and
// nothing is planned on the host but the launch shape.
//
// Eight warps, each with its own slice of every tile (32 keys of codes or 16 bf16 rows) and
// its own ring of three stages (K and V, 8 KB together at D = 128) that it refills itself; no
// warp waits for another. Codes come by TMA through a swizzled map, so that both fragment
// reads below are free of bank conflicts while the rows in HBM stay plain row-major, their two
// scales by 4-byte asynchronous copies on the same barrier; bf16 rows by plain bulk copies.
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
// bf16 rows (at most 63 of a tail, S + R of a ring) take bf16 products. Only these need masks.
//
// Merge: as the bf16 decode. The warps of a CTA merge in shared memory; a unit split over
// CTAs leaves (o, max, sum) parts for a second kernel, launched as a programmatic dependent.
// A part that starts a unit sits at the unit's index, a continuation at its CTA's (a CTA has
// one at most), and the first part names the CTAs of the others.
#include <cuda_fp16.h>

#include <atomic>

#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_decode_kv8_err;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = kKv8TK / kWarps;  // keys of a slice: 32
constexpr int kStages = 3;
// units of at most this many tiles are not split (their merge would cost more)
constexpr int kShortTiles = 4;
// p is kept times 2^kPShift: fp16 then holds it down to 2^-(24 + kPShift) of the row maximum,
// and up to 2^8 (lazy rescale) x 2^kPShift = 2^15
constexpr float kPShift = 7.f;

template <int D, int G>
struct Cfg {
  static constexpr int SLICE = kRows * D;  // bytes of a warp's K (or V) codes
  static constexpr int STAGE = 2 * SLICE;
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int RED = kWarps * G * (D + 2);
  static constexpr int PS = D + 4;  // floats per head of a part
  static constexpr int OFF_RED = RING;
  static constexpr int OFF_BAR = OFF_RED + RED * 4;
  static constexpr int OFF_SCALE = OFF_BAR + kWarps * kStages * 8;
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

// The codes in bytes 0, 1 and 2, 3 of w as two fp16 pairs, exactly.
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == kKv8E4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));  // 1152
    const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// Byte offset of 16-byte chunk c of row `row` of a slice as TMA's swizzle leaves it (rows of
// D bytes: the 128-byte pattern for D = 128, the 64-byte one for D = 64).
template <int D>
__device__ __forceinline__ int chunk_at(int row, int c) {
  return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ int64_t seq_len(const Kv8DecodeParams& p, int b) {
  if (!p.seq_lens) return p.n;
  const int64_t v = __ldg(p.seq_lens + b);
  return v < 0 ? 0 : (v > p.n ? p.n : v);
}

// Tiles of a retrieval / streaming unit of a sequence of n tokens (at least one, so that
// every unit's output is written).
__host__ __device__ __forceinline__ int64_t tiles_codes(int64_t n) { return (n / kKv8Block + 3) / 4; }
__host__ __device__ __forceinline__ int64_t tiles_ret(int64_t n) {
  const int64_t t = tiles_codes(n) + (n % kKv8Block > 0);
  return t > 0 ? t : 1;
}
__host__ __device__ __forceinline__ int64_t tiles_str(int64_t n, int SR) {
  const int64_t rows = n < SR ? n : SR;
  return rows > 0 ? (rows + kKv8TKBf16 - 1) / kKv8TKBf16 : 1;
}

struct Unit {
  int u, b, kvh, idx;  // idx: its index among the heads of its kind
  bool streaming;
  int64_t n;      // tokens of the sequence
  int64_t tiles;
};
__device__ __forceinline__ Unit unit_of(const Kv8DecodeParams& p, int u) {
  Unit x;
  x.u = u;
  x.streaming = u >= p.U_r;
  if (!x.streaming) {
    x.b = u / p.sh.n_ret;
    x.idx = u - x.b * p.sh.n_ret;
    x.kvh = p.heads.ret_head[x.idx];
    x.n = seq_len(p, x.b);
    x.tiles = tiles_ret(x.n);
  } else {
    const int us = u - p.U_r;
    x.b = us / p.sh.n_str;
    x.idx = us - x.b * p.sh.n_str;
    x.kvh = p.heads.str_head[x.idx];
    x.n = seq_len(p, x.b);
    x.tiles = tiles_str(x.n, p.sh.S + p.sh.R);
  }
  return x;
}

// Rows of a unit that are bf16: a streaming unit's ring slots, or the tail of the open block.
__device__ __forceinline__ int bf16_rows(const Kv8DecodeParams& p, const Unit& x) {
  const int SR = p.sh.S + p.sh.R;
  return x.streaming ? (int)(x.n < SR ? x.n : SR) : (int)(x.n % kKv8Block);
}

// Places on the line of all tiles: a unit whose first tile is at ub takes tiles + 1 places, tile
// lt >= 1 is at ub + lt + 1. Tiles of a unit of T tiles that lie before place ub + y:
__device__ __forceinline__ int64_t tiles_before(int64_t y, int64_t T) {
  const int64_t t = y > 1 ? y - 1 : y;
  return t <= 0 ? 0 : (t < T ? t : T);
}

// This CTA's share of the line, places [x0, x1) of W, shared by C CTAs (each gets at least two
// places, so none inside a unit's span is left without a tile of it), starting in unit u at ub.
struct Share {
  int64_t W, x0, x1, ub;
  int C, u;
};
__device__ __forceinline__ int cta_of(const Share& s, int64_t x) { return (int)(((x + 1) * s.C - 1) / s.W); }
__device__ __forceinline__ void cut(Share& s, int ctas) {
  const int c = blockIdx.x;
  s.C = (int)(ctas < s.W / 2 ? ctas : s.W / 2);
  s.x0 = c < s.C ? c * s.W / s.C : s.W;
  s.x1 = c < s.C ? (c + 1) * s.W / s.C : s.W;
}

__device__ Share share_of(const Kv8DecodeParams& p, int64_t* scratch) {
  Share s;
  const int SR = p.sh.S + p.sh.R;
  if (p.whole) {
    s.W = s.x0 = s.x1 = s.ub = 0;
    s.C = p.C;
    s.u = blockIdx.x;
    return s;
  }
  if (!p.seq_lens) {
    const int64_t tr = tiles_ret(p.n) + 1, ts = tiles_str(p.n, SR) + 1, Wr = tr * p.U_r;
    s.W = Wr + ts * p.U_s;
    cut(s, p.C);
    if (s.x0 < Wr) {
      s.u = (int)(s.x0 / tr);
      s.ub = s.u * tr;
    } else {
      s.u = p.U_r + (int)((s.x0 - Wr) / ts);
      s.ub = Wr + (s.u - p.U_r) * ts;
    }
    return s;
  }
  // lengths on the device: thread t sums the places of sequences [t per, (t + 1) per), then
  // the thread whose sums hold x0 finds the unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.sh.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.sh.B), b1 = min(b0 + per, p.sh.B);
  int64_t r = 0, q = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t n = seq_len(p, b);
    r += p.sh.n_ret * (tiles_ret(n) + 1);
    q += p.sh.n_str * (tiles_str(n, SR) + 1);
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
  s.W = Wr + Wq;
  cut(s, p.C);
  const bool in_r = s.x0 < Wr && s.x0 >= r - r_own && s.x0 < r;
  const bool in_q = s.x0 >= Wr && s.x0 - Wr >= q - q_own && s.x0 - Wr < q;
  if (in_r || in_q) {
    const int heads = in_r ? p.sh.n_ret : p.sh.n_str;
    int64_t base = in_r ? r - r_own : Wr + q - q_own;
    for (int b = b0; b < b1; ++b) {
      const int64_t n = seq_len(p, b);
      const int64_t T = (in_r ? tiles_ret(n) : tiles_str(n, SR)) + 1;
      if (s.x0 < base + heads * T) {
        const int64_t k = (s.x0 - base) / T;
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

// The slices this warp takes, in order, over the CTA's share: one tile further each time, across
// units.
struct Cursor {
  Unit x;
  int64_t ub, x0, x1;
  int64_t lt, lt1;  // next tile of the unit, and the end of the share's tiles in it
  int row, rows;    // first row of the slice in its codes (32 rows), or in its bf16 rows (1 to 16)
  bool live, codes;
  int blk;  // paged codes: the id of the page the slice lies in
  int warp;

  __device__ __forceinline__ void init(const Kv8DecodeParams& p, const Share& s, int w) {
    warp = w;
    live = p.whole || s.x0 < s.x1;
    if (!live) return;
    x = unit_of(p, s.u);
    x0 = s.x0;
    x1 = s.x1;
    ub = s.ub;
    lt = p.whole ? 0 : tiles_before(x0 - ub, x.tiles);
    lt1 = p.whole ? x.tiles : tiles_before(x1 - ub, x.tiles);
    settle(p);
  }
  // from tile lt on, the first with a slice for this warp
  __device__ __forceinline__ void settle(const Kv8DecodeParams& p) {
    for (;;) {
      if (lt < lt1) {
        const int64_t tc = x.streaming ? 0 : tiles_codes(x.n);
        if (lt < tc) {
          const int64_t r = lt * kKv8TK + warp * kRows;
          if (r < x.n / kKv8Block * kKv8Block) {
            row = (int)r;
            codes = true;
            if (p.pg.table)
              blk = __ldg(p.pg.table + ((int64_t)x.b * p.sh.n_ret + x.idx) * p.pg.max_blocks +
                          (uint32_t)row / (uint32_t)p.pg.block_size);
            return;
          }
          lt = tc;  // none in the last, partial tile of codes: on to the tail
          continue;
        }
        const int r = (int)(lt - tc) * kKv8TKBf16 + warp * 16;
        const int have = bf16_rows(p, x);
        if (r < have) {
          row = r;
          rows = min(16, have - r);
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
      x = unit_of(p, x.u + 1);
      lt = 0;
      lt1 = tiles_before(x1 - ub, x.tiles);
    }
  }
  __device__ __forceinline__ void advance(const Kv8DecodeParams& p) {
    ++lt;
    settle(p);
  }
};

// Copies the cursor's slice into a stage (lane 0). False: its page does not exist.
template <int D, int G>
__device__ __forceinline__ bool issue(const Kv8DecodeParams& p, const Cursor& cur, uint8_t* stage, float* scales,
                                      uint64_t* bar, uint64_t pol) {
  using C = Cfg<D, G>;
  if (!cur.codes) {
    const int64_t first = cur.x.streaming ? ((int64_t)cur.x.b * p.sh.n_str + cur.x.idx) * (p.sh.S + p.sh.R) + cur.row
                                          : ((int64_t)cur.x.b * p.sh.n_ret + cur.x.idx) * kKv8Block + cur.row;
    const uint32_t bytes = (uint32_t)cur.rows * D * 2;
    mbar_arrive_expect_tx(bar, 2 * bytes);
    bulk_g2s(stage, (cur.x.streaming ? p.k_sr : p.k_tail) + first * D, bytes, bar);
    bulk_g2s(stage + C::SLICE, (cur.x.streaming ? p.v_sr : p.v_tail) + first * D, bytes, bar);
    mbar_arrive(bar);
    return true;
  }
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

// A warp's running softmax over the keys it has seen. Lane (gid, tig) = (lane / 4, lane % 4)
// holds, of heads 2 tig and 2 tig + 1, the maximum and its own part of the sum, and of O^T
// m-tile i the dims DT gid + 2 i (+ 1).
template <int D, int G>
struct State {
  static constexpr int MT = D / 16;  // m-tiles of O^T
  static constexpr int DT = D / 8;   // dims of a lane
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

  // One 32-key slice of codes, every key visible. qb: q in B fragments; kf: K's scale times
  // the heads' factors.
  template <int CODE>
  __device__ __forceinline__ void codes(const uint8_t* sk, const uint8_t* sv, const uint32_t (&qb)[D / 16][2],
                                        float kf0, float kf1, float vs, int gid, int tig) {
    float x[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // keys 16 h + gid and 16 h + gid + 8
      float sc[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[c][k] = 0.f;
      const int ra = 16 * h + gid, rb = ra + 8;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        const uint4 va = *reinterpret_cast<const uint4*>(sk + chunk_at<D>(ra, tig + 4 * u));
        const uint4 vb = *reinterpret_cast<const uint4*>(sk + chunk_at<D>(rb, tig + 4 * u));
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          decode4<CODE>(wa[i], a0, a2);
          decode4<CODE>(wb[i], a1, a3);
          mma<true>(sc[i & 1], a0, a1, a2, a3, qb[4 * u + i][0], qb[4 * u + i][1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = (sc[0][k] + sc[1][k]) * ((k & 1) ? kf1 : kf0);
    }
    softmax<8, false>(x, 0u);
    uint32_t pb[4];  // P^T: keys 16 h + 2 tig (+ 1) and + 8 (+ 9) of head gid
#pragma unroll
    for (int k = 0; k < 4; ++k) pb[k] = transpose8x8(pack_half2(x[2 * k], x[2 * k + 1]));
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4][DT / 4];  // the lane's dims of keys 2 tig, + 1, + 8, + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * h + 2 * tig + (k & 1) + 8 * (k >> 1);
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(sv + chunk_at<D>(row, gid));
          w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(sv + chunk_at<D>(row, gid >> 1) + (gid & 1) * 8);
          w[k][0] = v.x, w[k][1] = v.y;
        }
      }
#pragma unroll
      for (int j = 0; j < DT / 4; ++j) {
        // bytes of one dim of two neighbouring keys side by side: (dim, dim + 1) per word
        uint32_t a[2], b[2], c[2], d[2];
        decode4<CODE>(__byte_perm(w[0][j], w[1][j], 0x5140), a[0], b[0]);
        decode4<CODE>(__byte_perm(w[0][j], w[1][j], 0x7362), a[1], b[1]);
        decode4<CODE>(__byte_perm(w[2][j], w[3][j], 0x5140), c[0], d[0]);
        decode4<CODE>(__byte_perm(w[2][j], w[3][j], 0x7362), c[1], d[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) mma<true>(acc[2 * j + e], a[e], b[e], c[e], d[e], pb[2 * h], pb[2 * h + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = fmaf(acc[i][k], vs, o[i][k]);
  }

  // A slice of up to 16 bf16 rows. vis: bit k set where value k's key is visible (keys gid and
  // gid + 8, heads 2 tig and + 1); what lies in the other rows is not used.
  __device__ __forceinline__ void rows16(const uint8_t* sk, const uint8_t* sv, uint32_t vis,
                                         const uint32_t (&qa)[D / 16][2], float qf, int gid, int tig) {
    float sc[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[c][k] = 0.f;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const uint4 ka = *reinterpret_cast<const uint4*>(sk + gid * D * 2 + (tig + 4 * u) * 16);
      const uint4 kb = *reinterpret_cast<const uint4*>(sk + (gid + 8) * D * 2 + (tig + 4 * u) * 16);
      mma<false>(sc[0], ka.x, kb.x, ka.y, kb.y, qa[2 * u][0], qa[2 * u][1]);
      mma<false>(sc[1], ka.z, kb.z, ka.w, kb.w, qa[2 * u + 1][0], qa[2 * u + 1][1]);
    }
    uint32_t w[4][MT];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 2 * tig + (k & 1) + 8 * (k >> 1);
#pragma unroll
      for (int c = 0; c < MT / 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(sv + row * D * 2 + DT * 2 * gid + 16 * c);
        w[k][4 * c] = v.x, w[k][4 * c + 1] = v.y, w[k][4 * c + 2] = v.z, w[k][4 * c + 3] = v.w;
      }
    }
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (sc[0][k] + sc[1][k]) * qf;
    softmax<4, true>(x, vis);
    const uint32_t pb0 = transpose8x8(pack_bf16x2(x[0], x[1]));
    const uint32_t pb1 = transpose8x8(pack_bf16x2(x[2], x[3]));
    // a value row nobody sees (an empty or evicted slot) may hold anything: out of the product.
    // Value k's key is held by lane (gid, tig); the V fragments want it by row.
    const uint32_t seen = __ballot_sync(0xffffffffu, vis & 1u);         // bit 4 g: key g
    const uint32_t seen8 = __ballot_sync(0xffffffffu, (vis >> 2) & 1u); // bit 4 g: key g + 8
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int g = 2 * tig + (k & 1);
      if (!(((k >> 1) ? seen8 : seen) >> (4 * g) & 1u)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) w[k][i] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
      mma<false>(o[i], __byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[0][i], w[1][i], 0x7632),
                 __byte_perm(w[2][i], w[3][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x7632), pb0, pb1);
  }

  // (o, max, sum) per head into the CTA's merge buffer: red[(warp G + h) (D + 2) + d]
  __device__ __forceinline__ void write(float* red, int warp, int gid, int tig) {
#pragma unroll
    for (int s = 4; s < 32; s <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += __shfl_xor_sync(0xffffffffu, l[e], s);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 2 * tig + e;
      if (h >= G) continue;
      float* r = red + (warp * G + h) * (D + 2);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<float2*>(r + DT * gid + 2 * i) = make_float2(o[i][e], o[i][2 + e]);
      if (gid == 0) *reinterpret_cast<float2*>(r + D) = make_float2(m[e], l[e]);
    }
  }
};

// q of head gid (nullptr past the last) as bf16 B fragments for rows16, and as fp16 ones for
// codes: scaled by 2^(8 - e), e the exponent of the head's largest |q|, so that every bf16
// value down to 2^-22 of the largest stays exact. Returns 2^(e - 8).
template <int D>
__device__ __forceinline__ float load_q16(const uint16_t* qh, uint32_t (&qb)[D / 16][2], int tig) {
  uint32_t w[D / 64][8];  // dims 16 (tig + 4 u) ... + 15
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < D / 64; ++u) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 v = qh ? __ldg(reinterpret_cast<const uint4*>(qh + (tig + 4 * u) * 16 + 8 * c)) : make_uint4(0, 0, 0, 0);
      w[u][4 * c] = v.x, w[u][4 * c + 1] = v.y, w[u][4 * c + 2] = v.z, w[u][4 * c + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[u][k] & 0x7FFF7FFFu);
  }
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  int e = (int)(max(m & 0xFFFFu, m >> 16) >> 7);  // biased exponent
  e = e < 9 ? 9 : (e > 254 ? 254 : e);
  const float f = __uint_as_float((uint32_t)(262 - e) << 23);
#pragma unroll
  for (int u = 0; u < D / 64; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // word i of a chunk of codes: dims 4 i ... 4 i + 3
      qb[4 * u + i][0] = pack_half2(bf16lo(w[u][2 * i]) * f, bf16hi(w[u][2 * i]) * f);
      qb[4 * u + i][1] = pack_half2(bf16lo(w[u][2 * i + 1]) * f, bf16hi(w[u][2 * i + 1]) * f);
    }
  return __uint_as_float((uint32_t)(e - 8) << 23);
}

template <int D>
__device__ __forceinline__ void load_qbf16(const uint16_t* qh, uint32_t (&qa)[D / 16][2], int tig) {
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    const uint4 v = qh ? __ldg(reinterpret_cast<const uint4*>(qh + (tig + 4 * u) * 8)) : make_uint4(0, 0, 0, 0);
    qa[2 * u][0] = v.x, qa[2 * u][1] = v.y, qa[2 * u + 1][0] = v.z, qa[2 * u + 1][1] = v.w;
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * kStages;
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE) + warp * kStages * 2;
  if (lane == 0) {
    // a stage is full after the bulk copies' bytes and the two scales' arrival
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 2);
    fence_mbarrier_init();
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  __syncthreads();
  // Launched as a programmatic dependent: nothing the grid before it writes is read earlier.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Share sh = share_of(p, reinterpret_cast<int64_t*>(red));
  __syncthreads();  // (share_of's scratch is the merge buffer)
  const uint64_t pol = l2_policy_evict_first();  // codes are read once

  Cursor cur;
  cur.init(p, sh, warp);
  uint32_t issued = 0, used = 0, landed = 0;  // slices; landed: waited for
  uint32_t bad = 0;                           // lane 0: bit s set if stage s was not copied
  auto refill = [&]() {
    const int s = (int)(issued % kStages);
    if (lane == 0) {
      const bool ok = issue<D, G>(p, cur, ring + s * C::STAGE, scales + 2 * s, &bars[s], pol);
      bad = ok ? bad & ~(1u << s) : bad | (1u << s);
    }
    ++issued;
    cur.advance(p);
  };
  for (int s = 0; s < kStages - 1 && cur.live; ++s) refill();

  const int U = p.U_r + p.U_s;
  const int SR = p.sh.S + p.sh.R;
  bool ok = true;  // of this warp: a wait that ran out stops its copies, not the CTA's barriers
  State<D, G> st;
  int64_t ub = sh.ub;
  // next slice: refills the stage of the one before, and waits for its own
  auto next = [&]() {
    if (cur.live && ok) refill();
    const int s = (int)(used % kStages);
    if (ok) ok = mbar_wait(&bars[s], (used / kStages) & 1u, err, kErrDecodeConsumer);
    if (ok) ++landed;
    ++used;
    return s;
  };
  for (int u = sh.u; p.whole ? u == sh.u : ub < sh.x1; ++u) {
    const Unit x = unit_of(p, u);
    const int64_t lt0 = p.whole ? 0 : tiles_before(sh.x0 - ub, x.tiles);
    const int64_t lt1 = p.whole ? x.tiles : tiles_before(sh.x1 - ub, x.tiles);
    if (lt0 >= lt1) {  // (the share starts behind its last tile)
      ub += x.tiles + 1;
      continue;
    }
    st.reset();
    const uint16_t* qh = gid < G ? p.q + ((int64_t)x.b * p.sh.Hq + (int64_t)x.kvh * G + gid) * D : nullptr;
    const int64_t tc = x.streaming ? 0 : tiles_codes(x.n);
    if (lt0 < tc) {
      uint32_t qb[D / 16][2];
      const float f = load_q16<D>(qh, qb, tig) * p.scale_log2;
      const float f0 = __shfl_sync(0xffffffffu, f, 8 * tig), f1 = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
      const int64_t full = x.n / kKv8Block * kKv8Block;
      for (int64_t lt = lt0; lt < lt1 && lt < tc; ++lt) {
        if (lt * kKv8TK + warp * kRows >= full) break;
        const int s = next();
        const bool skip = !ok || ((__shfl_sync(0xffffffffu, bad, 0) >> s) & 1u);
        if (!skip) {
          const uint8_t* sk = ring + s * C::STAGE;
          const float ks = scales[2 * s], vs = scales[2 * s + 1];
          st.template codes<CODE>(sk, sk + C::SLICE, qb, f0 * ks, f1 * ks, vs, gid, tig);
        }
        __syncwarp();
      }
    }
    const int64_t tb = lt0 > tc ? lt0 : tc;  // bf16 tiles: a streaming unit's, or the tail's one
    if (tb < lt1) {
      uint32_t qa[D / 16][2];
      load_qbf16<D>(qh, qa, tig);
      const int have = bf16_rows(p, x);
      for (int64_t lt = tb; lt < lt1; ++lt) {
        const int r0 = (int)(lt - tc) * kKv8TKBf16 + warp * 16;
        if (r0 >= have) break;
        int64_t at[2];  // positions of keys gid and gid + 8
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int key = gid + 8 * k;
          at[k] = r0 + key >= have ? -1 : (x.streaming ? __ldg(p.pos + (int64_t)x.b * SR + r0 + key) : 0);
        }
        const int s = next();
        uint32_t vis = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool v = at[k] >= 0 && (!x.streaming || (at[k] < x.n && (at[k] < p.sh.S || x.n - 1 - at[k] < p.sh.R)));
          vis |= (v ? 3u : 0u) << (2 * k);
        }
        const uint8_t* sk = ring + s * C::STAGE;
        if (ok) st.rows16(sk, sk + C::SLICE, vis, qa, p.scale_log2, gid, tig);
        __syncwarp();
      }
    }

    // merge of the eight warps
    st.write(red, warp, gid, tig);
    __syncthreads();
    int c_first = 0, n_parts = 1;
    if (!p.whole) {
      c_first = cta_of(sh, ub);
      n_parts = cta_of(sh, x.tiles > 1 ? ub + x.tiles : ub) - c_first + 1;
    }
    float* part = p.partials + (int64_t)(lt0 == 0 ? u : U + (int)blockIdx.x) * G * C::PS;
    for (int e = tid; e < G * D; e += kThreads) {
      const int h = e / D, d = e % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * G + h) * (D + 2) + D]);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* r = red + (w * G + h) * (D + 2);
        const float f = r[D] == -INFINITY && !(r[D + 1] != 0.f) ? 0.f : ex2_approx(r[D] - M);
        num = fmaf(f, r[d], num);
        den = fmaf(f, r[D + 1], den);
      }
      if (n_parts == 1)
        p.o[((int64_t)x.b * p.sh.Hq + (int64_t)x.kvh * G + h) * D + d] =
            __bfloat16_as_ushort(__float2bfloat16_rn(den != 0.f ? num / den : 0.f));
      if (n_parts > 1) part[h * C::PS + d] = num;
      if (d == 0 && !p.whole && (n_parts > 1 || lt0 == 0)) {
        part[h * C::PS + D] = M;
        part[h * C::PS + D + 1] = den;
        part[h * C::PS + D + 2] = __int_as_float(c_first);
        part[h * C::PS + D + 3] = __int_as_float(n_parts);
      }
    }
    __syncthreads();  // the buffer is the next unit's
    ub += x.tiles + 1;
  }
  // copies still in flight (after a wait that ran out) land before the CTA ends
  if (lane == 0)
    for (uint32_t j = landed; j < issued; ++j) mbar_wait(&bars[j % kStages], (j / kStages) & 1u, err, kErrDecodeConsumer);
  __syncthreads();
}

// Units whose tiles were split over CTAs: one CTA per (unit, head), warp w takes parts w,
// w + 8, ...; a lane holds D / 32 dims. Launched as the decode's programmatic dependent.
template <int D, int G>
__global__ void __launch_bounds__(kThreads) decode_kv8_merge_kernel(const __grid_constant__ Kv8DecodeParams p) {
  constexpr int PS = Cfg<D, G>::PS, V = D / 32;
  const int h = blockIdx.x % G, u = blockIdx.x / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* head = p.partials + ((int64_t)u * G + h) * PS;
  const int n_parts = __float_as_int(__ldcg(head + D + 3));
  if (n_parts <= 1) return;
  const int c_first = __float_as_int(__ldcg(head + D + 2));
  const int U = p.U_r + p.U_s;
  float acc[V], M = -INFINITY, den = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
  for (int i = warp; i < n_parts; i += kWarps) {
    const float* r = i == 0 ? head : p.partials + ((int64_t)(U + c_first + i) * G + h) * PS;
    const float m = __ldcg(r + D), l = __ldcg(r + D + 1);
    float ov[V];
#pragma unroll
    for (int v = 0; v < V; ++v) ov[v] = __ldcg(r + lane * V + v);
    const float mn = fmaxf(M, m);
    const float fo = M == -INFINITY && !(den != 0.f) ? 0.f : ex2_approx(M - mn);
    const float fi = m == -INFINITY && !(l != 0.f) ? 0.f : ex2_approx(m - mn);
    den = den * fo + l * fi;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = acc[v] * fo + ov[v] * fi;
    M = mn;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = acc[v];
  if (lane == 0) s_m[warp] = M, s_l[warp] = den;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float T = -INFINITY, num = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) T = fmaxf(T, s_m[w]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY && !(s_l[w] != 0.f) ? 0.f : ex2_approx(s_m[w] - T);
      num = fmaf(f, s_o[w][d], num);
      sum = fmaf(f, s_l[w], sum);
    }
    const bool streaming = u >= p.U_r;
    const int us = streaming ? u - p.U_r : u, nk = streaming ? p.sh.n_str : p.sh.n_ret;
    const int b = us / nk;
    const int kvh = streaming ? p.heads.str_head[us - b * nk] : p.heads.ret_head[us - b * nk];
    p.o[((int64_t)b * p.sh.Hq + (int64_t)kvh * G + h) * D + d] =
        __bfloat16_as_ushort(__float2bfloat16_rn(sum != 0.f ? num / sum : 0.f));
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
  cfg.gridDim = dim3((unsigned)((p.U_r + p.U_s) * G));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, decode_kv8_merge_kernel<D, G>, p);
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
  const int SR = p->sh.S + p->sh.R;
  const int64_t tr = p->U_r ? tiles_ret(p->n) : 0, ts = p->U_s ? tiles_str(p->n, SR) : 0;
  const int64_t U = (int64_t)p->U_r + p->U_s;
  p->whole = U <= num_sms && tr <= kShortTiles && ts <= kShortTiles;
  const int64_t W = tr * p->U_r + ts * p->U_s;  // (a CTA's share is at least one tile)
  p->C = (int)(p->whole ? U : (W < num_sms ? W : num_sms));
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
