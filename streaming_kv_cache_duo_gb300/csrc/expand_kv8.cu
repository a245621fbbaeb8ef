// Rows of 8-bit caches as bf16, for the prefill: plane by plane into a caller's workspace,
// [planes, ceil(n / 64) 64, D], the open block's rows as they stand in the tail. Of a block's scale the
// power of two goes with the codes, which stay exact; what is left, in [1, 2), is a factor per block
// that the prefill applies in fp32. (Rows of code * scale rounded to bf16 doubled the error of its
// outputs, 0.0036 against 0.0017 of their norm.) The prefill reads the rows with TMA as it reads a
// bf16 cache.
//
// Why not inside the prefill, as the 4-bit caches do it: there every CTA that reads a cache tile
// dequantizes it again (16 q blocks of a 4096-token chunk, times the query heads of a KV head),
// and its 192 dequantizing threads are what a tile waits for: 722 us for that chunk over 28672
// cached tokens (8 of 32 heads), 2.9 us a tile against 1.6 us from a bf16 cache. Done once, it
// is a copy, HBM-bound: 3 bytes moved per value.
//
// A CTA per block of 64 rows, plane after plane; half of a CTA's threads do K, half V. A thread
// turns 8 codes into 16 bytes at a time, all its loads in flight together.
#include <cuda_fp16.h>

#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_expand_kv8_err;

constexpr int kThreads = 256;
constexpr int kHalf = kThreads / 2;

// Four codes times a power of two as bf16.
template <int CODE>
__device__ __forceinline__ uint2 expand4(uint32_t w, float scale) {
  float2 a, b;
  if constexpr (CODE == kKv8E4m3) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  } else {
    // a code with its sign bit flipped under the float exponent of 2^23 reads as 2^23 + 128 + code
    const uint32_t u = w ^ 0x80808080u;
    constexpr float kBias = 8388736.f;
    a = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)) - kBias,
                    __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541)) - kBias);
    b = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)) - kBias,
                    __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543)) - kBias);
  }
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

template <int D, int CODE>
__global__ void __launch_bounds__(kThreads) expand_kv8_kernel(const Kv8ExpandParams p) {
  // (a prefill launched as a programmatic dependent waits for this grid before it reads a row)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool is_v = threadIdx.x >= kHalf;
  const int tid = threadIdx.x % kHalf;
  const uint32_t blocks = ((uint32_t)p.n + kKv8Block - 1) / kKv8Block;  // of a plane
  const int64_t plane = blockIdx.x / blocks;
  const int r0 = (int)(blockIdx.x - (uint32_t)plane * blocks) * kKv8Block;
  uint16_t* out = (is_v ? p.v_out : p.k_out) + (int64_t)blockIdx.x * kKv8Block * D;
  constexpr int N = kKv8Block * D / 8 / kHalf;  // pieces of 8 values per thread
  float* fac = (is_v ? p.v_fac : p.k_fac) + blockIdx.x;
  if (p.n - r0 < kKv8Block) {  // the open block
    if (tid == 0) *fac = is_v ? 0.f : 1.f;
    const uint4* tail = reinterpret_cast<const uint4*>((is_v ? p.v_tail : p.k_tail) + plane * kKv8Block * D);
    for (int i = tid; i < (p.n - r0) * (D / 8); i += kHalf) reinterpret_cast<uint4*>(out)[i] = tail[i];
    return;
  }
  int64_t row = plane * p.cap64 + r0;
  if (p.pg.table) {
    const int bi = (int)((uint32_t)r0 / (uint32_t)p.pg.block_size);
    const int64_t id = __ldg(p.pg.table + plane * p.pg.max_blocks + bi);
    row = id * p.pg.block_size + (r0 - bi * p.pg.block_size);
    if (id < 0 || id >= p.pg.num_blocks) {  // no such block: the prefill leaves its rows out
      if (tid == 0) {
        atomicOr(&g_expand_kv8_err, kErrBadBlock);
        *fac = is_v ? -INFINITY : 1.f;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) reinterpret_cast<uint4*>(out)[tid + k * kHalf] = make_uint4(0, 0, 0, 0);
      return;
    }
  }
  const float whole = __ldg((is_v ? p.v_scale : p.k_scale) + row / kKv8Block);
  // the power of two (2^-126 for a subnormal scale), and the rest; a scale of 0 has codes of 0, NaN stays
  const uint32_t bits = __float_as_uint(whole), exponent = bits >> 23;
  const float scale = exponent == 255 ? 1.f : __uint_as_float((exponent ? exponent : 1u) << 23);
  if (tid == 0) {
    const float left = whole == 0.f || exponent == 255 ? whole : whole / scale;
    *fac = whole == 0.f ? (is_v ? 0.f : 1.f) : (is_v ? log2f(left) : left);
  }
  const uint2* codes = reinterpret_cast<const uint2*>((is_v ? p.v_codes : p.k_codes) + row * D);
  uint2 w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = __ldg(codes + tid + k * kHalf);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint2 a = expand4<CODE>(w[k].x, scale), b = expand4<CODE>(w[k].y, scale);
    reinterpret_cast<uint4*>(out)[tid + k * kHalf] = make_uint4(a.x, a.y, b.x, b.y);
  }
}

}  // namespace

cudaError_t launch_expand_kv8(const Kv8ExpandParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)p.n + kKv8Block - 1) / kKv8Block * p.planes);  // < 2^31, checked on the host
  if (grid == 0) return cudaSuccess;
  if (p.D == 128 && p.code_type == kKv8E4m3)
    expand_kv8_kernel<128, kKv8E4m3><<<grid, kThreads, 0, stream>>>(p);
  else if (p.D == 128)
    expand_kv8_kernel<128, kKv8Int8><<<grid, kThreads, 0, stream>>>(p);
  else if (p.D == 64 && p.code_type == kKv8E4m3)
    expand_kv8_kernel<64, kKv8E4m3><<<grid, kThreads, 0, stream>>>(p);
  else if (p.D == 64)
    expand_kv8_kernel<64, kKv8Int8><<<grid, kThreads, 0, stream>>>(p);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

cudaError_t expand_kv8_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_expand_kv8_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_expand_kv8_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
