// duo_kv_append_kv8: new tokens into 8-bit caches (codes with one fp32 scale per block of
// 64 tokens of a head) and into the bf16 sink + ring caches of the streaming heads.
//
// A block is rounded once, when its 64th row arrives: amax over its 64 x D values, scale =
// amax / 127 (int8) or amax / 448 (e4m3), code = x / scale rounded to nearest even (two
// roundings, both in fp32: the scale's, then the quotient's before it becomes a code).
// Until then its rows wait in bf16 in the tail. So the cache does not depend on how the
// tokens were split into calls, and nothing stored is ever rounded again.
//
// Work: grid (chunk of consecutive tokens, retrieval plane x {K, V}, then one row of CTAs
// for the ring). The CTA that holds the token completing a block does that block: rows of
// this call from the packed input, earlier ones from the tail. The rows of the block left
// open are written by the CTA of the sequence's last token, except when an earlier block of
// this call reads the tail rows they replace: then by the CTA that read them, after it.
// One pass: the block sits in registers (16 KB over 256 threads) between the maximum and
// the codes. HBM-bound for prompts: 2 D bytes in, D out per row.
#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_append_kv8_err;

constexpr int kThreads = 256;
constexpr int kBlk = kKv8Block;

// Two codes of one byte each from two values over the block's scale.
template <int CODE>
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  if constexpr (CODE == kKv8E4m3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  } else {
    const int ia = max(-127, min(127, __float2int_rn(a)));
    const int ib = max(-127, min(127, __float2int_rn(b)));
    return (uint32_t)(ia & 0xFF) | ((uint32_t)(ib & 0xFF) << 8);
  }
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
  bool good = t.b >= 0 && t.b < p.sh.B && t.pos < 0x7fffffff;
  if (good) {
    t.first = p.cu_new[t.b];
    t.last = p.cu_new[t.b + 1] - 1;
    good = t.first >= 0 && t.first <= i && t.last >= i && t.last < p.tokens && t.pos >= i - t.first;
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

template <int D, int CODE>
__device__ void complete_block(const Kv8AppendParams& p, const Token& t, int i, int r, const uint16_t* in,
                               const uint16_t* tail, uint8_t* codes, float* scales, uint32_t* s_max) {
  constexpr int VPR = D / 8;                       // 16-byte vectors per row
  constexpr int NV = kBlk * VPR / kThreads;        // vectors per thread
  const int64_t row0 = block_row(p, t, i, r);      // (the same for every thread)
  if (row0 < 0) {
    if (threadIdx.x == 0) atomicOr(&g_append_kv8_err, kErrBadBlock);
    return;
  }
  const int head = p.heads.ret_head[r];
  uint4 x[NV];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = threadIdx.x + k * kThreads;
    const int row = e / VPR, v = e % VPR;
    const int src = i - (kBlk - 1) + row;  // packed token of the row; before the call's first: in the tail
    const uint16_t* a = src >= t.first ? in + ((int64_t)src * p.sh.Hkv + head) * D : tail + (int64_t)row * D;
    x[k] = *reinterpret_cast<const uint4*>(a + v * 8);
  }
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
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = __vmaxu2(m, s_max[w]);
  m = max(m & 0xFFFFu, m >> 16);
  float scale = __fdiv_rn(__uint_as_float(m << 16), CODE == kKv8E4m3 ? 448.f : 127.f);
  const bool finite = m < 0x7F80u;
  if (!finite) scale = __uint_as_float(0x7FC00000u);
  const bool zero = !finite || scale == 0.f;
  if (threadIdx.x == 0) scales[row0 / kBlk] = scale;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = threadIdx.x + k * kThreads;
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = zero ? 0u : encode2<CODE>(__fdiv_rn(bf16lo(w[j]), scale), __fdiv_rn(bf16hi(w[j]), scale));
    *reinterpret_cast<uint2*>(codes + row0 * D + (int64_t)e * 8) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
}

// The sequence's new rows of the block it leaves open, into the tail.
template <int D>
__device__ void write_tail(const Kv8AppendParams& p, const Token& t, int i, int r, const uint16_t* in, uint16_t* tail) {
  constexpr int VPR = D / 8;
  const int end = t.pos + (t.last - i) + 1;  // length after the call
  const int start = t.pos - (i - t.first);   // and before it
  const int lo = max(end / kBlk * kBlk, start);
  const int head = p.heads.ret_head[r];
  for (int e = threadIdx.x; e < (end - lo) * VPR; e += kThreads) {
    const int pos = lo + e / VPR, v = e % VPR;
    const int64_t src = t.first + (pos - start);
    *reinterpret_cast<uint4*>(tail + (pos % kBlk) * D + v * 8) =
        *reinterpret_cast<const uint4*>(in + (src * p.sh.Hkv + head) * D + v * 8);
  }
}

template <int D, int CODE>
__global__ void __launch_bounds__(kThreads) append_kv8_kernel(const Kv8AppendParams p) {
  // as append_kernel: dependents may be scheduled now, and nothing is touched before the
  // grid before this one (a decode reading the tail or the ring) has ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i0 = blockIdx.x * p.chunk;
  const int i1 = min(i0 + p.chunk, p.tokens);
  const int n_ret = p.sh.n_ret;
  constexpr int VPR = D / 8;

  if ((int)blockIdx.y == 2 * n_ret) {
    // ring: the tokens a streaming head still holds after the call, as 16-byte vectors
    const int n_str = p.sh.n_str;
    const int SR = p.sh.S + p.sh.R;
    const int per = n_str * VPR;
    for (int e = threadIdx.x; e < (i1 - i0) * per; e += kThreads) {
      const int i = i0 + e / per;
      const Token t = token_at(p, i);
      if (!t.ok) continue;
      const int end = t.pos + (t.last - i) + 1;
      if (t.pos >= p.sh.S && t.pos < end - p.sh.R) continue;
      const int slot = t.pos < p.sh.S ? t.pos : p.sh.S + (t.pos - p.sh.S) % p.sh.R;
      const int si = e % per / VPR, v = e % VPR;
      const int64_t src = ((int64_t)i * p.sh.Hkv + p.heads.str_head[si]) * VPR + v;
      const int64_t dst = (((int64_t)t.b * n_str + si) * SR + slot) * VPR + v;
      reinterpret_cast<uint4*>(p.k_sr)[dst] = __ldg(reinterpret_cast<const uint4*>(p.k_new) + src);
      reinterpret_cast<uint4*>(p.v_sr)[dst] = __ldg(reinterpret_cast<const uint4*>(p.v_new) + src);
      if (si == 0 && v == 0) p.pos[(int64_t)t.b * SR + slot] = t.pos;
    }
    return;
  }

  const int r = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const uint16_t* in = is_v ? p.v_new : p.k_new;
  uint16_t* tails = is_v ? p.v_tail : p.k_tail;
  uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  float* scales = is_v ? p.v_scale : p.k_scale;
  __shared__ Token s_tok[kBlk];
  __shared__ uint32_t s_max[kThreads / 32];
  if ((int)threadIdx.x < i1 - i0) s_tok[threadIdx.x] = token_at(p, i0 + threadIdx.x);
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    const Token t = s_tok[i - i0];
    if (!t.ok) continue;
    const int row = t.pos % kBlk;
    const int end_row = (t.pos + (t.last - i)) % kBlk;  // row of the sequence's last token
    const int start = t.pos - (i - t.first);
    uint16_t* tail = tails + ((int64_t)t.b * n_ret + r) * kBlk * D;
    if (row == kBlk - 1) {
      complete_block<D, CODE>(p, t, i, r, in, tail, codes, scales, s_max);
      // the block took rows from the tail: the new open block's rows go there after it
      if (t.pos - (kBlk - 1) < start && end_row != kBlk - 1) {
        __syncthreads();
        write_tail<D>(p, t, i, r, in, tail);
      }
    } else if (i == t.last) {
      const int open = t.pos / kBlk * kBlk;  // first position of the open block
      if (start % kBlk == 0 || start >= open) write_tail<D>(p, t, i, r, in, tail);
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
