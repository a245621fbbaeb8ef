// duo_kv_append_kv8: new tokens into 8-bit caches (codes with one fp32 scale per block of
// 64 tokens of a head) and into the bf16 sink + ring caches of the streaming heads.
//
// A block is rounded once, when its 64th row arrives: amax over its 64 x D values, scale =
// amax / 127 (int8) or amax / 448 (e4m3), code = x / scale rounded to nearest even (two
// roundings, both in fp32: the scale's, then the quotient's before it becomes a code).
// Until then its rows wait in bf16 in the tail. So the cache does not depend on how the
// tokens were split into calls, and nothing stored is ever rounded again.
//
// Work: grid (chunk of consecutive tokens, one row of CTAs for the ring, then K and V of each
// retrieval plane). The CTA that holds the token completing a block does
// that block: rows of this call from the packed input, earlier ones from the tail. The rows of
// the block left open are written by the CTA of the sequence's last token, except when an
// earlier block of this call reads the tail rows they replace: then by the CTA that read them,
// after it. One pass: the block sits in registers (16 KB over 128 threads) between the maximum
// and the codes. HBM-bound for prompts: 2 D bytes in, D out per row. A prompt of 32K tokens with four
// retrieval heads, D = 128, e4m3: 25.4 us (replayed graphs, one after the other; 22.7 among other calls,
// whose starts and ends overlap); HBM's share is 15. As many CTAs per SM as registers allow without
// spills in the loops: seven (72 registers) at D = 128, ten at 64 (48, 4 bytes spilled). K and V in one
// CTA of 256 threads took 27.1 us, and 20.2 instead of 17.4 for 2 x 8192 tokens, eight heads, D = 64;
// CTAs that fetch the next block's rows while they round the ones they have 32 / 28 (graphs as well).
#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_append_kv8_err;

constexpr int kThreads = 128;
constexpr int kBlk = kKv8Block;

// Codes of values over their block's scale, rounded from the fp32 quotient x / scale. A division
// per value costs more than all the rest (a 32K prompt took 93 us with it; HBM's share is 15 us),
// so each value is rounded from two products instead, with 1 / scale made a little smaller and a
// little larger: by 2^-21, where u = 2^-24 bounds the relative error of 1 / scale, of each product
// and of the fp32 quotient itself. The quotient lies between them, and rounding to a code is
// monotone: where both give the same code it is the quotient's. Where they do not (a border
// between two codes is that near: about one value in 10^5) the division is done, as it is for
// scales so small that their reciprocal could overflow.
constexpr float kTinyScale = 1e-30f;
struct Inverse {
  float lo, hi;
};
__device__ __forceinline__ Inverse inverse_of(float scale) {
  const float r = 1.f / scale;
  return Inverse{r * (1.f - 4.76837158203125e-7f), r * (1.f + 4.76837158203125e-7f)};
}

// Codes of eight values (two per word of w). The low byte of 1.5 2^23 + v, an fp32 sum rounded to
// nearest even, is the integer nearest to v (|v| <= 127).
__device__ __forceinline__ uint32_t pack_bytes(const float (&v)[4]) {
  const uint32_t a = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
template <int CODE>
__device__ __forceinline__ uint2 encode8(const uint32_t (&w)[4], float scale, const Inverse inv, bool tiny) {
  uint32_t c[2];
  uint32_t differ = 0;
  constexpr float kRound = 12582912.f;  // 1.5 2^23
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float x[4] = {bf16lo(w[2 * h]), bf16hi(w[2 * h]), bf16lo(w[2 * h + 1]), bf16hi(w[2 * h + 1])};
    if constexpr (CODE == kKv8E4m3) {
      c[h] = e4m3x2(x[0] * inv.lo, x[1] * inv.lo) | (e4m3x2(x[2] * inv.lo, x[3] * inv.lo) << 16);
      differ |= c[h] ^ (e4m3x2(x[0] * inv.hi, x[1] * inv.hi) | (e4m3x2(x[2] * inv.hi, x[3] * inv.hi) << 16));
    } else {
      float a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = fmaf(x[k], inv.lo, kRound);
        differ |= __float_as_uint(a[k]) ^ __float_as_uint(fmaf(x[k], inv.hi, kRound));
      }
      c[h] = pack_bytes(a);
    }
  }
  if (differ || tiny) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t v = w[2 * h + (k >> 1)];
        q[k] = __fdiv_rn((k & 1) ? bf16hi(v) : bf16lo(v), scale);
        if (CODE != kKv8E4m3) q[k] = fminf(fmaxf(q[k], -127.f), 127.f) + kRound;
      }
      c[h] = CODE == kKv8E4m3 ? e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16) : pack_bytes(q);
    }
  }
  return make_uint2(c[0], c[1]);
}

// One token of the call: its sequence, position, and the packed index of its sequence's
// first and last token. ok = stored by this call.
struct Token {
  bool ok;
  int b, pos, first, last;
};
__device__ __forceinline__ Token token_at(const Kv8AppendParams& p, int i) {
  Token t;
  if (!p.token_seq) {
    t.b = i / p.T;
    t.first = t.b * p.T;
    t.last = t.first + p.T - 1;
    t.pos = (int)(p.n + (i - t.first));
    t.ok = true;
    return t;
  }
  t.b = p.token_seq[i];
  t.pos = p.token_pos[i];
  t.ok = t.pos >= 0;
  t.first = t.last = i;
  if (!t.ok) return t;
  bool good = t.b >= 0 && t.b < p.sh.B;
  if (good) {
    t.first = p.cu_new[t.b];
    t.last = p.cu_new[t.b + 1] - 1;
    // (the sequence's length before and after the call follow from these, in 32 bits)
    good = t.first >= 0 && t.first <= i && t.last >= i && t.last < p.tokens && t.pos >= i - t.first &&
           t.last - i < 0x7fffffff - t.pos;
  }
  if (!good) {
    atomicOr(&g_append_kv8_err, kErrBadBlock);
    t.ok = false;
  }
  return t;
}

// First row of the codes of the block that token i (the block's 64th) completes, -1 if none.
__device__ __forceinline__ int64_t block_row(const Kv8AppendParams& p, const Token& t, int i, int r) {
  int64_t row;
  if (p.token_seq) {
    row = p.slots[(int64_t)i * p.sh.n_ret + r] - (kBlk - 1);
  } else {
    const int64_t plane = (int64_t)t.b * p.sh.n_ret + r;
    const int64_t first = t.pos - (kBlk - 1);
    if (!p.pg.table) return plane * p.cap64 + first;
    const int64_t blk = p.pg.table[plane * p.pg.max_blocks + first / p.pg.block_size];
    row = blk < 0 || blk >= p.pg.num_blocks ? -1 : blk * p.pg.block_size + first % p.pg.block_size;
  }
  return row >= 0 && row % kBlk == 0 && row + kBlk <= p.rows ? row : -1;
}

// s_max: one word per warp.
template <int D, int CODE>
__device__ __forceinline__ void complete_block(const Kv8AppendParams& p, const Token& t, int i, int r, int tid,
                                               const uint16_t* in, const uint16_t* tail, uint8_t* codes, float* scales,
                                               uint32_t* s_max) {
  constexpr int VPR = D / 8;                   // 16-byte vectors per row
  constexpr int NV = kBlk * VPR / kThreads;       // vectors per thread
  constexpr int RS = kThreads / VPR;              // rows between a thread's vectors
  const int64_t row0 = block_row(p, t, i, r);  // (the same for every thread)
  if (row0 < 0) {
    if (tid == 0) atomicOr(&g_append_kv8_err, kErrBadBlock);
    return;
  }
  // row `row` of the block is packed token first + row; before the call's first it is in the tail
  const int first = i - (kBlk - 1), row_of = tid / VPR, v = tid % VPR;
  const uint16_t* src = in + ((int64_t)(first + row_of) * p.sh.Hkv + p.heads.ret_head[r]) * D + v * 8;
  const int64_t step = (int64_t)RS * p.sh.Hkv * D;
  uint4 x[NV];
  if (first >= t.first) {
#pragma unroll
    for (int k = 0; k < NV; ++k) x[k] = __ldg(reinterpret_cast<const uint4*>(src + k * step));
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int row = row_of + k * RS;
      x[k] = first + row >= t.first ? *reinterpret_cast<const uint4*>(src + k * step)
                                    : *reinterpret_cast<const uint4*>(tail + row * D + v * 8);
    }
  }
  uint32_t m = 0;
  // |x| as 16-bit integers order as the values do; infinities and NaN come out on top
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) m = __vmaxu2(m, w[c] & 0x7FFF7FFFu);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();  // the last block's readers are done with s_max
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = __vmaxu2(m, s_max[w]);
  m = max(m & 0xFFFFu, m >> 16);
  float scale = __fdiv_rn(__uint_as_float(m << 16), CODE == kKv8E4m3 ? 448.f : 127.f);
  const bool finite = m < 0x7F80u;
  if (!finite) scale = __uint_as_float(0x7FC00000u);
  const bool zero = !finite || scale == 0.f;
  if (tid == 0) scales[row0 / kBlk] = scale;
  uint8_t* dst = codes + row0 * D + tid * 8;
  const Inverse inv = inverse_of(scale);
  const bool tiny = scale < kTinyScale;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
    const uint2 c = zero ? make_uint2(0, 0) : encode8<CODE>(w, scale, inv, tiny);
    *reinterpret_cast<uint2*>(dst + k * (kThreads * 8)) = c;
  }
}

// The sequence's new rows of the block it leaves open, into the tail.
template <int D>
__device__ __forceinline__ void write_tail(const Kv8AppendParams& p, const Token& t, int i, int r, int tid,
                                           const uint16_t* in, uint16_t* tail) {
  constexpr int VPR = D / 8;
  const int end = t.pos + (t.last - i) + 1;  // length after the call
  const int start = t.pos - (i - t.first);   // and before it
  const int lo = max(end / kBlk * kBlk, start);
  const int head = p.heads.ret_head[r];
  for (int e = tid; e < (end - lo) * VPR; e += kThreads) {
    const int pos = lo + e / VPR, v = e % VPR;
    const int64_t src = t.first + (pos - start);
    *reinterpret_cast<uint4*>(tail + (pos % kBlk) * D + v * 8) =
        *reinterpret_cast<const uint4*>(in + (src * p.sh.Hkv + head) * D + v * 8);
  }
}

template <int D, int CODE>
__global__ void __launch_bounds__(kThreads, D == 64 ? 10 : 7) append_kv8_kernel(const Kv8AppendParams p) {
  // as append_kernel: dependents may be scheduled now, and nothing is touched before the
  // grid before this one (a decode reading the tail or the ring) has ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i0 = blockIdx.x * p.chunk;
  const int i1 = min(i0 + p.chunk, p.tokens);
  const int n_ret = p.sh.n_ret;
  constexpr int VPR = D / 8;

  // the ring's CTAs come first: the few with something to copy take longest
  const bool ring = p.sh.n_str > 0 && blockIdx.y == 0;
  // what there is to do, token by token: blocks completed and sequences' last tokens, or for
  // the ring the tokens a streaming head still holds after the call
  __shared__ Token s_tok[kBlk];
  __shared__ uint32_t s_todo[kBlk / 32];
  __shared__ uint32_t s_max[kThreads / 32];
  __shared__ uint8_t s_list[kBlk];  // ring: the tokens in s_todo, one after the other
  bool todo = false;
  if (threadIdx.x < kBlk) {
    const int i = i0 + (int)threadIdx.x;
    if (i < i1) {
      const Token t = token_at(p, i);
      s_tok[threadIdx.x] = t;
      const int left = t.last - i;  // tokens of the sequence behind this one
      todo = t.ok && (ring ? t.pos < p.sh.S || left < p.sh.R : t.pos % kBlk == kBlk - 1 || left == 0);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, todo);
    if ((threadIdx.x & 31) == 0) s_todo[threadIdx.x >> 5] = m;
  }
  __syncthreads();
  const uint64_t all = s_todo[0] | ((uint64_t)s_todo[1] << 32);
  if (ring) {
    if (todo) s_list[__popcll(all & (((uint64_t)1 << threadIdx.x) - 1))] = (uint8_t)threadIdx.x;
    __syncthreads();
    const int n_str = p.sh.n_str;
    const int SR = p.sh.S + p.sh.R;
    const int per = n_str * VPR;
    const int count = __popcll(all);
    // (all vectors of the chunk side by side: token after token would wait for memory each time)
#pragma unroll 4
    for (int e = threadIdx.x; e < count * per; e += kThreads) {
      const int k = s_list[e / per], f = e % per;
      const Token t = s_tok[k];
      const int slot = t.pos < p.sh.S ? t.pos : p.sh.S + (t.pos - p.sh.S) % p.sh.R;
      const int si = f / VPR, v = f % VPR;
      const int64_t src = ((int64_t)(i0 + k) * p.sh.Hkv + p.heads.str_head[si]) * VPR + v;
      const int64_t dst = (((int64_t)t.b * n_str + si) * SR + slot) * VPR + v;
      reinterpret_cast<uint4*>(p.k_sr)[dst] = __ldg(reinterpret_cast<const uint4*>(p.k_new) + src);
      reinterpret_cast<uint4*>(p.v_sr)[dst] = __ldg(reinterpret_cast<const uint4*>(p.v_new) + src);
      if (f == 0) p.pos[(int64_t)t.b * SR + slot] = t.pos;
    }
    return;
  }

  const int y = (int)blockIdx.y - (p.sh.n_str > 0);
  const int r = y >> 1;
  const bool is_v = y & 1;
  const int tid = threadIdx.x;
  const uint16_t* in = is_v ? p.v_new : p.k_new;
  uint16_t* tails = is_v ? p.v_tail : p.k_tail;
  uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  float* scales = is_v ? p.v_scale : p.k_scale;
  for (uint64_t todo = all; todo; todo &= todo - 1) {
    const int i = i0 + __ffsll((long long)todo) - 1;
    const Token t = s_tok[i - i0];
    const int row = t.pos % kBlk;
    const int end_row = (t.pos + (t.last - i)) % kBlk;  // row of the sequence's last token
    const int start = t.pos - (i - t.first);
    uint16_t* tail = tails + ((int64_t)t.b * n_ret + r) * kBlk * D;
    if (row == kBlk - 1) {
      complete_block<D, CODE>(p, t, i, r, tid, in, tail, codes, scales, s_max);
      // the block took rows from the tail: the new open block's rows go there after it
      if (t.pos - (kBlk - 1) < start && end_row != kBlk - 1) {
        __syncthreads();
        write_tail<D>(p, t, i, r, tid, in, tail);
      }
    } else if (i == t.last) {
      const int open = t.pos / kBlk * kBlk;  // first position of the open block
      if (start % kBlk == 0 || start >= open) write_tail<D>(p, t, i, r, tid, in, tail);
    }
  }
}

template <int D, int CODE>
cudaError_t launch_t(const Kv8AppendParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tokens + p.chunk - 1) / p.chunk), (unsigned)(2 * p.sh.n_ret + (p.sh.n_str > 0)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kv8_kernel<D, CODE>, p);
}

}  // namespace

cudaError_t launch_append_kv8(const Kv8AppendParams& p, cudaStream_t stream) {
  if (p.sh.D == 128)
    return p.code_type == kKv8E4m3 ? launch_t<128, kKv8E4m3>(p, stream) : launch_t<128, kKv8Int8>(p, stream);
  if (p.sh.D == 64)
    return p.code_type == kKv8E4m3 ? launch_t<64, kKv8E4m3>(p, stream) : launch_t<64, kKv8Int8>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t append_kv8_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_kv8_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_append_kv8_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
