// duo_block_tables_update: block tables, slot maps, free list and lengths of a serving
// step, from the requests' lengths, on the device.
//
// With s = block_size, L_b the length and new_b the new tokens of sequence b, it holds
// ceil(L_b / s) blocks a plane and needs planes (ceil((L_b + new_b) / s) - ceil(L_b / s))
// more. Three prefix sums over the sequences decide everything: the new tokens (cu_new),
// the blocks needed (first come, first served: a sequence is served iff it needs none or
// the sum up to it fits) and the blocks given back. The k-th new block is entry
// avail - 1 - k of the free list, so every table entry and slot follows from the sums
// without an atomic and the result does not depend on the order of threads.
//
// Latency-bound: a few KB of lengths in, 8 + 8 planes bytes a token out. One CTA does the sums
// (each thread one sequence, warp shuffles, a carry between rounds), in shared memory for up
// to kSmall sequences: the sums are bisected to find the sequence of an entry or a token, and
// each step of that is a round trip to wherever they are. A small step (kFuseWork outputs) is
// finished by the same CTA in the same launch; larger ones by a second grid, launched as the
// first one's programmatic dependent.
#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_tables_err;

constexpr int kScanThreads = 1024;  // at most
constexpr int kSmall = 1024;        // sequences whose sums fit in shared memory
// outputs (table entries and slots) up to which the scanning CTA writes them itself
constexpr int64_t kFuseWork = 8192;
constexpr int kPlanes = 4;  // planes whose slots a thread writes

// Scratch, int32: [0] free blocks after the returns, [1] blocks handed out, [2] tokens in
// the packed batch (at most max_tokens), then per sequence the old length (-1: turned down
// or finished), and the prefix sums of needed and returned blocks, B + 1 entries each.
struct Scratch {
  int32_t* head;
  int32_t* old_len;
  int32_t* need_base;
  int32_t* rel_base;
  const int32_t* cu_new;  // (an output as well)
};
__device__ __forceinline__ Scratch scratch_at(int32_t* at, int B, const int32_t* cu_new) {
  Scratch s;
  s.head = at;
  s.old_len = at + 4;
  s.need_base = s.old_len + B;
  s.rel_base = s.need_base + B + 1;
  s.cu_new = cu_new;
  return s;
}

// (len and bs are below 2^31)
__device__ __forceinline__ int blocks_of(int64_t len, int bs) { return (int)(((uint32_t)len + bs - 1) / (uint32_t)bs); }

// Largest i in [0, n) with base[i] <= v (base non-decreasing, base[0] = 0 <= v).
__device__ __forceinline__ int bisect(const int32_t* base, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Inclusive sums of three values over the CTA's threads; total: those of all of them.
struct Sums {
  int64_t tok;
  int32_t need, rel;
};
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v.tok, o);
    const int32_t a = __shfl_up_sync(0xffffffffu, v.need, o);
    const int32_t r = __shfl_up_sync(0xffffffffu, v.rel, o);
    if (lane >= o) v.tok += t, v.need += a, v.rel += r;
  }
  __syncthreads();  // the last round's readers are done with warp_sums
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  if (warp == 0) {
    Sums w = lane < warps ? warp_sums[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, w.tok, o);
      const int32_t a = __shfl_up_sync(0xffffffffu, w.need, o);
      const int32_t r = __shfl_up_sync(0xffffffffu, w.rel, o);
      if (lane >= o) w.tok += t, w.need += a, w.rel += r;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  if (warp > 0) {
    const Sums w = warp_sums[warp - 1];
    v.tok += w.tok, v.need += w.need, v.rel += w.rel;
  }
  total = warp_sums[warps - 1];
  return v;
}

// Writes the new blocks' table entries and the tokens' maps, both shared out among `step`
// threads, of which this is number `first`.
__device__ void fill(const BlockTablesParams& p, const Scratch& s, int64_t first, int64_t step) {
  const int avail = s.head[0], handed = s.head[1], tokens = s.head[2];
  for (int64_t e = first; e < handed; e += step) {
    const int b = bisect(s.need_base, p.B, (int)e);
    const int have = blocks_of(s.old_len[b], p.bs);
    const int per = (s.need_base[b + 1] - s.need_base[b]) / p.planes;
    const int k = (int)e - s.need_base[b];
    const int id = p.free_list[avail - 1 - (int)e];
    if (id < 0 || id >= p.num_blocks) atomicOr(&g_tables_err, kErrBadBlock);
    p.table[((int64_t)b * p.planes + k / per) * p.max_blocks + have + k % per] = id;
  }
  // a thread takes a token's slots for kPlanes planes: its sequence is found once, and 32 bytes a
  // thread fill whole lines
  const int groups = (p.planes + kPlanes - 1) / kPlanes;
  const int64_t items = (int64_t)p.max_tokens * groups;
  for (int64_t it = first; it < items; it += step) {
    const int i = (int)((it >> 32) ? it / groups : (uint32_t)it / (uint32_t)groups);
    const int p0 = (int)(it - (int64_t)i * groups) * kPlanes;
    int seq = -1, pos = -1;
    int64_t slot[kPlanes] = {-1, -1, -1, -1};
    if (i < tokens) {
      seq = bisect(s.cu_new, p.B, i);
      const int old = s.old_len[seq];
      if (old >= 0) {
        pos = old + (i - s.cu_new[seq]);
        const int have = blocks_of(old, p.bs);
        const int j = (int)((uint32_t)pos / (uint32_t)p.bs);
        const int nb = s.need_base[seq];
        const int per = (int)((uint32_t)(s.need_base[seq + 1] - nb) / (uint32_t)p.planes);
        int id[kPlanes];
#pragma unroll
        for (int k = 0; k < kPlanes; ++k)
          if (p0 + k < p.planes)
            id[k] = j < have ? p.table[((int64_t)seq * p.planes + p0 + k) * p.max_blocks + j]
                             : p.free_list[avail - 1 - (nb + (p0 + k) * per + (j - have))];
#pragma unroll
        for (int k = 0; k < kPlanes; ++k)
          if (p0 + k < p.planes) {
            if (id[k] < 0 || id[k] >= p.num_blocks)
              atomicOr(&g_tables_err, kErrBadBlock);
            else
              slot[k] = (int64_t)id[k] * p.bs + (pos - j * p.bs);
          }
      }
    }
    if (p0 == 0) {
      p.token_seq[i] = seq;
      p.token_pos[i] = pos;
    }
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
      if (p0 + k < p.planes) p.slots[(int64_t)i * p.planes + p0 + k] = slot[k];
  }
}

__global__ void __launch_bounds__(kScanThreads) block_tables_scan_kernel(const BlockTablesParams p, int fuse) {
  // as the appends: dependents may be scheduled now, nothing is touched before the grid before this
  // one has ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ Sums warp_sums[32];
  __shared__ int s_handed;
  __shared__ int32_t s_sums[4 + 3 * kSmall + 2], s_cu[kSmall + 1];
  const bool small = p.B <= kSmall;
  const Scratch s = scratch_at(small ? s_sums : p.scratch, p.B, small ? s_cu : p.cu_new);
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t cap = (int64_t)p.max_blocks * p.bs;
  uint32_t err = 0;
  int count = *p.free_count;

  // the sums: tokens, blocks needed, blocks given back
  int64_t c_tok = 0;
  int32_t c_need = 0, c_rel = 0;
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    const int b = b0 + tid;
    Sums v{0, 0, 0};
    int len = 0, nw = 0, kind = 2;  // 0 takes tokens, 1 finished, 2 turned down
    if (b < p.B) {
      len = p.seq_lens[b];
      nw = p.new_lens[b];
      if (len < 0 || len > cap || nw < -1)
        err |= kErrBadLength;
      else if (nw == -1)
        kind = 1;
      else if (len + (int64_t)nw > cap)
        err |= kErrPoolFull;
      else
        kind = 0;
      v.tok = nw > 0 ? nw : 0;
      if (kind == 0) v.need = p.planes * (blocks_of(len + (int64_t)nw, p.bs) - blocks_of(len, p.bs));
      if (kind == 1) v.rel = p.planes * blocks_of(len, p.bs);
    }
    Sums total;
    Sums u = block_scan(v, warp_sums, total);
    // a sequence whose tokens pass the packed batch is turned down before it asks for blocks
    const bool past = kind == 0 && nw > 0 && c_tok + u.tok > p.max_tokens;
    if (__syncthreads_or(past)) {
      if (past) {
        kind = 2;
        v.need = 0;
        err |= kErrPoolFull;
      }
      u = block_scan(v, warp_sums, total);
    }
    if (b < p.B) {
      const int64_t begin = c_tok + u.tok - v.tok;
      const int cu = (int)(begin < 0x7fffffff ? begin : 0x7fffffff);
      p.cu_new[b] = cu;
      if (small) s_cu[b] = cu;
      s.need_base[b] = c_need + u.need - v.need;
      s.rel_base[b] = c_rel + u.rel - v.rel;
      s.old_len[b] = kind == 0 ? len : (kind == 1 ? -2 - len : -1);
    }
    c_tok += total.tok;
    c_need += total.need;
    c_rel += total.rel;
  }
  if (tid == 0) {
    const int cu = (int)(c_tok < 0x7fffffff ? c_tok : 0x7fffffff);
    p.cu_new[p.B] = cu;
    if (small) s_cu[p.B] = cu;
    s.need_base[p.B] = c_need;
    s.rel_base[p.B] = c_rel;
    s_handed = 0;
  }
  if (count < 0 || count > p.num_blocks) {
    err |= kErrBadLength;
    count = count < 0 ? 0 : (int)p.num_blocks;
  }
  __syncthreads();

  // returned blocks, in order, dropping ids that are none
  int avail = count;
  for (int e0 = 0; e0 < c_rel; e0 += threads) {
    const int e = e0 + tid;
    int id = -1;
    if (e < c_rel) {
      const int b = bisect(s.rel_base, p.B, e);
      const int have = blocks_of(-2 - s.old_len[b], p.bs);
      const int k = e - s.rel_base[b];
      id = p.table[((int64_t)b * p.planes + k / have) * p.max_blocks + k % have];
      if (id < 0 || id >= p.num_blocks) {
        err |= kErrBadBlock;
        id = -1;
      }
    }
    Sums total;
    const Sums u = block_scan(Sums{0, id >= 0, 0}, warp_sums, total);
    const int64_t at = (int64_t)avail + u.need - 1;
    if (id >= 0 && at < p.num_blocks) p.free_list[at] = id;
    const int64_t next = (int64_t)avail + total.need;
    if (next > p.num_blocks) err |= kErrBadBlock;  // more blocks than the pool has: one came back twice
    avail = (int)(next < p.num_blocks ? next : p.num_blocks);
  }

  // who is served
  for (int b = tid; b < p.B; b += threads) {
    const int old = s.old_len[b];
    const int end = s.need_base[b + 1];
    const bool asks = end > s.need_base[b];
    int len = p.seq_lens[b];
    if (old >= 0) {
      if (!asks || end <= avail) {
        len = old + p.new_lens[b];
        if (asks) atomicMax(&s_handed, end);
      } else {
        s.old_len[b] = -1;
        err |= kErrPoolFull;
      }
    } else if (old <= -2) {
      len = 0;
    }
    p.seq_lens_out[b] = len;
  }
  __syncthreads();
  if (tid == 0) {
    s.head[0] = avail;
    s.head[1] = s_handed;
    s.head[2] = (int)(c_tok < p.max_tokens ? c_tok : p.max_tokens);
    *p.free_count_out = avail - s_handed;
  }
  if (err) atomicOr(&g_tables_err, err);
  if (fuse) {
    __syncthreads();
    fill(p, s, tid, threads);
  } else if (small) {  // for the second grid
    __syncthreads();
    for (int i = tid; i < 4 + 2 * p.B + 1; i += threads) p.scratch[i] = s_sums[i];
  }
}

__global__ void __launch_bounds__(256) block_tables_fill_kernel(const BlockTablesParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fill(p, scratch_at(p.scratch, p.B, p.cu_new), (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

}  // namespace

size_t block_tables_scratch_bytes(int B) { return ((size_t)4 + 3 * (size_t)B + 2) * 4; }

cudaError_t launch_block_tables(const BlockTablesParams& p, int num_sms, cudaStream_t stream) {
  // table entries of the new blocks: at most one partly filled block a plane and sequence
  // beside the full ones
  const int64_t work = (int64_t)p.max_tokens * p.planes + (int64_t)p.B * p.planes;
  const bool fuse = work <= kFuseWork;
  // threads: one per sequence, and in a fused step one per output, as far as they go
  const int64_t want = fuse && work > p.B ? work : p.B;
  const int threads = want >= kScanThreads ? kScanThreads : (want <= 128 ? 128 : (int)((want + 31) / 32 * 32));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, block_tables_scan_kernel, p, fuse ? 1 : 0);
  if (e != cudaSuccess || fuse) return e;
  const int64_t items = (int64_t)p.max_tokens * ((p.planes + kPlanes - 1) / kPlanes) + (int64_t)p.B * p.planes;
  int64_t blocks = (items + 255) / 256;
  if (blocks > (int64_t)num_sms * 8) blocks = (int64_t)num_sms * 8;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, block_tables_fill_kernel, p);
}

cudaError_t block_tables_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tables_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_tables_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
