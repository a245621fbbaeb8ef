// duo_rope_rotate and duo_kv_append_ragged: rotary positions of a packed batch, alone or on the way
// into bf16 paged caches.
//
// Pair i of a row (a, b) at position p becomes scale (a cos t - b sin t, b cos t + a sin t), t = p f_i.
// The pairs are (i, i + rotary / 2) or (2 i, 2 i + 1) of the row's first `rotary` dims; the other dims
// pass through. A far position leaves p f_i few bits for its fraction of a turn (p f_i = 10^6 rad in
// fp32 is off by 0.06 rad), so f_i comes as a fraction of a full turn in 64-bit fixed point: p f_i is
// one integer product, wrapped as angles wrap, and exact for every int32 position. Its upper 32 bits
// as a signed number of half turns go to sincospif (the fp32 rounding there is 2^-25 of half a turn).
//
// An append writes K rotated and V as it is: retrieval heads to the pool rows the slot map names,
// streaming heads to their sink + ring slots (token t to slot t if t < S, else S + (t - S) mod R; of a
// call's tokens only those still held when it ends). With q given, q is rotated beside them: a decode
// step's one launch between the projection and the attention.
//
// HBM-bound: rows in and out once. A CTA takes a few tokens: their cosines and sines go to shared memory
// once for all heads (a thread per pair), then a thread moves 32 bytes of a row, two 16-byte vectors that
// lie half a (rotated or unrotated) part apart, which for the one layout are the two halves of eight pairs
// and for the other four whole pairs each. Measured: 24001 tokens of 40 heads of 128 dims 80 us = 6.16 TB/s
// (0.91 of a copy); 8 tokens a CTA there, fewer where a call has not enough for every SM. 64 tokens: 2.5 to 2.8 us
// alone, 3.7 with the append, and 12 to 17 among other calls that make their outputs, where the host is what takes
// the time. Nothing rotated: 64 tokens 2.7 us (6.4 to 7 among others), four prompts of 20480 tokens, 4 of 8 heads
// retrieval, 19.5 us where their rows take 13.3.
#include "duo_device.cuh"
#include "ragged_internal.h"

namespace duo {
namespace {

__device__ unsigned int g_append_ragged_err;

constexpr int kThreads = 256;

// Two vectors of a row, eight dims each, rotated: cs holds the pairs' (cos, sin). Half layout: dims d
// and d + rotary / 2 are pair d; interleaved: neighbours.
template <bool kInter>
__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float2* cs, int u, int units) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[u * 4 + i], d = cs[(u + units) * 4 + i];
      const float a0 = bf16lo(a[i]), a1 = bf16hi(a[i]), b0 = bf16lo(b[i]), b1 = bf16hi(b[i]);
      a[i] = pack_bf16x2(a0 * c.x - a1 * c.y, a1 * c.x + a0 * c.y);
      b[i] = pack_bf16x2(b0 * d.x - b1 * d.y, b1 * d.x + b0 * d.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = *reinterpret_cast<const float4*>(cs + u * 8 + 2 * i);
      const float a0 = bf16lo(a[i]), a1 = bf16hi(a[i]), b0 = bf16lo(b[i]), b1 = bf16hi(b[i]);
      a[i] = pack_bf16x2(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w);
      b[i] = pack_bf16x2(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w);
    }
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}

// One token of the call: its sequence, position, and how many tokens of its sequence come behind it.
struct Token {
  int b, pos, behind;
};
__device__ __forceinline__ Token token_at(const RopeAppendParams& p, int i) {
  Token t{0, p.positions[i], 0};
  if (t.pos < 0) return t;
  t.b = p.token_seq[i];
  bool good = t.b >= 0 && t.b < p.sh.B;
  if (good) {
    const int first = p.cu_new[t.b], last = p.cu_new[t.b + 1] - 1;
    t.behind = last - i;
    // (the sequence's length before and after the call follow from these, in 32 bits)
    good = first >= 0 && first <= i && last >= i && last < p.tokens && t.pos >= i - first && t.behind < 0x7fffffff - t.pos;
  }
  if (!good) {
    atomicOr(&g_append_ragged_err, kErrBadBlock);
    t.pos = -1;
  }
  return t;
}

template <int D, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
  // as append_kernel: dependents may be scheduled now, and nothing is touched before the grid before
  // this one has ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) float2 s_cs[kRopeChunk][D / 2];
  __shared__ Token s_tok[kRopeChunk];
  const int i0 = blockIdx.x * p.chunk;
  const int count = min(p.chunk, p.tokens - i0);
  const int half = p.rope.rotary / 2;
  if ((int)threadIdx.x < count) {
    if (kAppend) {
      const Token t = token_at(p, i0 + threadIdx.x);
      s_tok[threadIdx.x] = t;
      if (t.pos >= 0 && p.sh.n_str > 0 && (t.pos < p.sh.S || t.behind < p.sh.R))
        p.pos[(int64_t)t.b * (p.sh.S + p.sh.R) + (t.pos < p.sh.S ? t.pos : p.sh.S + (t.pos - p.sh.S) % p.sh.R)] = t.pos;
    } else {
      s_tok[threadIdx.x].pos = p.positions[i0 + threadIdx.x];
    }
  }
  for (int e = threadIdx.x; e < count * half; e += kThreads) {
    const int k = e / half, i = e - k * half;
    const int pos = p.positions[i0 + k];
    const uint64_t phase = (uint64_t)(uint32_t)pos * p.rope.turns[i];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns in [-1, 1]
    s_cs[k][i] = make_float2(c * p.rope.scale, s * p.rope.scale);
  }
  __syncthreads();

  constexpr int UPR = D / 16;  // units per row
  const int rot = p.rope.rotary / 16;
  const int rows = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int total = count * rows * UPR;
  for (int e = threadIdx.x; e < total; e += kThreads) {
    const int u = e % UPR, r = e / UPR;
    const int k = r / rows;
    int h = r - k * rows;
    const int pos = s_tok[k].pos;
    if (pos < 0) continue;
    const int i = i0 + k;
    const bool is_q = h < p.q.heads;
    if (!is_q) h -= p.q.heads;
    const bool is_v = kAppend && !is_q && h >= p.k.heads;
    if (is_v) h -= p.k.heads;
    const RaggedRows& rw = is_q ? p.q : (is_v ? p.v : p.k);
    uint16_t* dst;
    if (!kAppend || is_q) {
      dst = rw.out + (int64_t)i * rw.out_stride + (int64_t)h * D;
    } else {
      const int idx = p.heads.kidx[h];
      if (p.heads.kind[h]) {
        const int64_t row = p.slots[(int64_t)i * p.sh.n_ret + idx];
        if (row < 0 || row >= p.rows) {
          atomicOr(&g_append_ragged_err, kErrBadBlock);
          continue;
        }
        dst = (is_v ? p.v_pool : p.k_pool) + row * D;
      } else {
        if (pos >= p.sh.S && s_tok[k].behind >= p.sh.R) continue;  // not held when the call ends
        const int slot = pos < p.sh.S ? pos : p.sh.S + (pos - p.sh.S) % p.sh.R;
        dst = (is_v ? p.v_sr : p.k_sr) + (((int64_t)s_tok[k].b * p.sh.n_str + idx) * (p.sh.S + p.sh.R) + slot) * D;
      }
    }
    const uint4* src = reinterpret_cast<const uint4*>(rw.in + (int64_t)i * rw.in_stride + (int64_t)h * D);
    const bool turned = !is_v && u < rot;
    // the two vectors of unit u: of the rotated part, or of what passes through
    const int v0 = turned || is_v ? u : rot + u;
    const int v1 = v0 + (is_v ? UPR : (turned ? rot : UPR - rot));
    if (!kAppend && !turned && dst == rw.in + (int64_t)i * rw.in_stride + (int64_t)h * D) continue;  // in place
    uint4 x = src[v0], y = src[v1];
    if (turned) rotate<kInter>(x, y, s_cs[k], u, rot);
    reinterpret_cast<uint4*>(dst)[v0] = x;
    reinterpret_cast<uint4*>(dst)[v1] = y;
  }
}

template <int D, bool kInter, bool kAppend>
cudaError_t launch_t(const RopeAppendParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tokens + p.chunk - 1) / p.chunk));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, kInter, kAppend>, p);
}

template <bool kAppend>
cudaError_t launch_any(const RopeAppendParams& p, cudaStream_t stream) {
  const bool inter = p.rope.layout == kRopeInterleaved;
  if (p.sh.D == 128) return inter ? launch_t<128, true, kAppend>(p, stream) : launch_t<128, false, kAppend>(p, stream);
  if (p.sh.D == 64) return inter ? launch_t<64, true, kAppend>(p, stream) : launch_t<64, false, kAppend>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeAppendParams& p, cudaStream_t stream) { return launch_any<false>(p, stream); }
cudaError_t launch_append_ragged(const RopeAppendParams& p, cudaStream_t stream) { return launch_any<true>(p, stream); }

cudaError_t append_ragged_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_ragged_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_append_ragged_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
