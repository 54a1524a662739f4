// Moving rows to their experts and back, for gfx950.
//
// dispatch: entry i = t * k + j is token t's j-th choice idx[t][j]; an index
//   outside [0, experts) is a dropped entry.  With the entries in the stable
//   order of their expert (dropped ones last), row r of the output is the
//   r-th entry's:  offsets[e] = entries of experts below e,
//   pos[t][j] = r, or -2 - r for a dropped entry,  token[r] = t (-1: dropped),
//   out[r] = x[t] with its scales (dropped: zero bytes and the scale of a
//   zero tile).  The order depends on idx alone: counts and prefix sums, no
//   atomics whose order could show.
// combine: out[t] = base[t] + sum_j w[t][j] z[pos[t][j]] over the places
//   >= 0, summed in fp32 in the order of j.
// combine's gradient: dz[pos[t][j]] = w[t][j] dy[t], dw[t][j] = <dy[t], z[pos[t][j]]>;
//   a dropped entry's row gets zeros.  The gradient of dispatch is combine
//   without weights.
//
// All are bound by HBM.  A row is moved by the workgroup of its token, so
// that x and dy are read once for the token's k places.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"

namespace fp8fg {

namespace {

constexpr int kChunkThreads = 256;
constexpr int kChunkWaves = kChunkThreads / 64;
constexpr int kMaxChunks = 256;
constexpr int kMinChunk = 1024;
constexpr int kMaxBuckets = 1025;  // experts and the bucket of dropped entries

struct Plan {
  const int32_t* idx;
  int64_t ld_idx;
  int64_t entries;
  int64_t chunk;  // entries per chunk, a multiple of kChunkThreads
  int k, experts;
  int32_t* counts;
  int32_t* offsets;
  int32_t* pos;
  int32_t* token;
};

__device__ __forceinline__ int bucket_of(const Plan& p, int64_t i) {
  const int64_t t = i / p.k;
  const int e = p.idx[t * p.ld_idx + (i - t * p.k)];
  return (uint32_t)e < (uint32_t)p.experts ? e : p.experts;
}

// counts[chunk][e]
__global__ __launch_bounds__(kChunkThreads) void count_kernel(Plan p) {
  __shared__ int32_t n[kMaxBuckets];
  const int B = p.experts + 1;
  for (int e = threadIdx.x; e < B; e += kChunkThreads) n[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.chunk;
  const int64_t i1 = i0 + p.chunk < p.entries ? i0 + p.chunk : p.entries;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kChunkThreads) atomicAdd(&n[bucket_of(p, i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += kChunkThreads) p.counts[(int64_t)blockIdx.x * B + e] = n[e];
}

// Lanes of the wave whose bucket is this lane's, among the `valid` ones.
__device__ __forceinline__ uint64_t same_bucket(int b, bool valid, int bits) {
  uint64_t m = __builtin_amdgcn_ballot_w64(valid);
  for (int i = 0; i < bits; ++i) {
    const uint64_t one = __builtin_amdgcn_ballot_w64((b >> i) & 1);
    m &= (b >> i) & 1 ? one : ~one;
  }
  return m;
}

// Each chunk: start of every bucket (all chunks' counts), then the entries
// in order: wave w takes the w-th quarter of the chunk, 64 at a time.
__global__ __launch_bounds__(kChunkThreads) void place_kernel(Plan p) {
  __shared__ int32_t start[kMaxBuckets];
  __shared__ int32_t base[kChunkWaves][kMaxBuckets];
  __shared__ int32_t wsum[kChunkWaves];
  const int B = p.experts + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // counts of the whole list and of the chunks before this one
  int32_t carry = 0;
  for (int e0 = 0; e0 < B; e0 += kChunkThreads) {
    const int e = e0 + tid;
    int32_t total = 0, before = 0;
    if (e < B)
      for (int c = 0; c < (int)gridDim.x; ++c) {
        const int32_t n = p.counts[(int64_t)c * B + e];
        total += n;
        before += c < (int)blockIdx.x ? n : 0;
      }
    int32_t incl = total;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int32_t o = __shfl_up(incl, m);
      incl += lane >= m ? o : 0;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int32_t first = carry + incl - total;
    for (int w = 0; w < wave; ++w) first += wsum[w];
    if (e < B) {
      start[e] = first + before;
      if (blockIdx.x == 0) p.offsets[e] = first;  // offsets[experts]: entries with an expert
    }
    for (int w = 0; w < kChunkWaves; ++w) carry += wsum[w];
    __syncthreads();
  }
  for (int e = tid; e < B; e += kChunkThreads)
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) base[w][e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.chunk + wave * (p.chunk / kChunkWaves);
  const int64_t i1 = min(i0 + p.chunk / kChunkWaves, p.entries);
  int bits = 0;
  while ((1 << bits) < B) ++bits;
  // the wave's own counts
  for (int64_t i = i0; i < i1; i += 64) {
    const bool valid = i + lane < i1;
    if (valid) atomicAdd(&base[wave][bucket_of(p, i + lane)], 1);
  }
  __syncthreads();
  for (int e = tid; e < B; e += kChunkThreads) {
    int32_t at = start[e];
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) {
      const int32_t n = base[w][e];
      base[w][e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 64) {
    const bool valid = i + lane < i1;
    const int b = valid ? bucket_of(p, i + lane) : 0;
    const uint64_t same = same_bucket(b, valid, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int32_t r = 0;
    if (valid) r = base[wave][b] + rank;
    wave_fence();  // every lane has read before the first of its bucket adds
    if (valid && rank == 0) base[wave][b] += __popcll(same);
    wave_fence();
    if (valid) {
      const int32_t t = (int32_t)((i + lane) / p.k);
      p.pos[i + lane] = b < p.experts ? r : -2 - r;
      p.token[r] = b < p.experts ? t : -1;
    }
  }
}

struct Move {
  const uint8_t* x;
  int64_t pitch;       // bytes
  int64_t vecs;        // 16-byte vectors per row
  const float* xs;
  int64_t xs_rs, xs_ts;
  int tiles;           // scales per row (0: none)
  int64_t tokens;
  int k;
  const int32_t* pos;
  uint8_t* out;
  int64_t opitch;
  float* os;
  int64_t os_rs, os_ts;
};

// One workgroup per token: the row is read once and written to its k places.
__global__ __launch_bounds__(256) void move_kernel(Move p) {
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const int32_t* pos = p.pos + t * p.k;
    for (int64_t v = threadIdx.x; v < p.vecs; v += 256) {
      const uint4 w = ld_nt16(p.x + t * p.pitch + v * 16);
      for (int j = 0; j < p.k; ++j) {
        const int32_t r = pos[j];
        if (r >= 0)
          st_nt16(p.out + (int64_t)r * p.opitch + v * 16, w);
        else
          st_nt16(p.out + (int64_t)(-2 - r) * p.opitch + v * 16, make_uint4(0, 0, 0, 0));
      }
    }
    for (int i = threadIdx.x; i < p.tiles; i += 256) {
      const float s = p.xs[t * p.xs_rs + i * p.xs_ts];
      for (int j = 0; j < p.k; ++j) {
        const int32_t r = pos[j];
        p.os[(r >= 0 ? r : -2 - r) * p.os_rs + i * p.os_ts] = r >= 0 ? s : kFltMinNormal;
      }
    }
  }
}

template <int XT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p) {
  const int nvec = (int)(p.cols >> 3);
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int v = threadIdx.x; v < nvec; v += 256) {
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int32_t r = p.pos[t * p.k + j];
        if (r < 0 || r >= p.z_rows) continue;
        const float w = p.w ? p.w[t * p.ldw + j] : 1.0f;
        float z[8];
        load8<XT>(p.z, r * p.ldz + v * 8, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += w * z[e];
      }
      if (p.base) {
        float b[8];
        load8<XT>(p.base, t * p.ldb + v * 8, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += b[e];
      }
      store_raw8<XT, true>(p.out, t * p.ldo + v * 8, encode8<XT>(acc));
    }
  }
}

template <int XT>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineGradArgs p) {
  __shared__ float part[4];
  const int nvec = (int)(p.cols >> 3);
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j = 0; j < p.k; ++j) {
      const int32_t r = p.pos[t * p.k + j];
      const bool here = r >= 0 && r < p.z_rows;
      const int64_t row = here ? r : -2 - (int64_t)r;
      const bool zero = !here && row >= 0 && row < p.z_rows;
      const float w = p.w ? p.w[t * p.ldw + j] : 1.0f;
      float dot = 0.0f;
      for (int v = threadIdx.x; v < nvec; v += 256) {
        float d[8];
        if (here) {
          load8<XT>(p.dy, t * p.lddy + v * 8, d);
          if (p.dw) {
            float z[8];
            load8<XT>(p.z, row * p.ldz + v * 8, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot += d[e] * z[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = 0.0f;
        }
        if (here || zero) store_raw8<XT, true>(p.dz, row * p.lddz + v * 8, encode8<XT>(d));
      }
      if (p.dw) {
        dot = wave_sum(dot);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (threadIdx.x == 0) p.dw[t * p.lddw + j] = ((part[0] + part[1]) + part[2]) + part[3];
        __syncthreads();
      }
    }
  }
}

constexpr int64_t kMaxTokenBlocks = 1 << 20;

dim3 token_grid(int64_t tokens) { return dim3((unsigned)(tokens < kMaxTokenBlocks ? tokens : kMaxTokenBlocks)); }

}  // namespace

// At most kMaxChunks chunks: each chunk's workgroup reads all their counts.
int64_t dispatch_chunks(int64_t entries) {
  const int64_t n = (entries + kMinChunk - 1) / kMinChunk;
  return n < 1 ? 1 : n < kMaxChunks ? n : kMaxChunks;
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st) {
  const int64_t entries = a.tokens * a.k;
  const int64_t chunks = dispatch_chunks(entries);
  const int64_t per = (entries + chunks - 1) / chunks;
  const int64_t chunk = (per + kChunkThreads - 1) / kChunkThreads * kChunkThreads;
  const Plan p{a.idx, a.ld_idx, entries, chunk, a.k, a.experts, a.counts, a.offsets, a.pos, a.token};
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)chunks), dim3(kChunkThreads), 0, st, p);
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)chunks), dim3(kChunkThreads), 0, st, p);
  if (a.x && a.tokens > 0) {
    const int size = a.x_type == 2 ? 1 : a.x_type == 0 ? 2 : 4;
    const Move m{reinterpret_cast<const uint8_t*>(a.x), a.ldx * size, a.cols * size / 16, a.xs, a.xs_rs, a.xs_ts,
                 a.x_type == 2 ? (int)(a.cols / 128) : 0, a.tokens, a.k, a.pos,
                 reinterpret_cast<uint8_t*>(a.out), a.ldo * size, a.os, a.os_rs, a.os_ts};
    hipLaunchKernelGGL(move_kernel, token_grid(a.tokens), dim3(256), 0, st, m);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
  if (a.type == 0)
    hipLaunchKernelGGL(combine_kernel<0>, token_grid(a.tokens), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(combine_kernel<1>, token_grid(a.tokens), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t st) {
  if (a.type == 0)
    hipLaunchKernelGGL(combine_grad_kernel<0>, token_grid(a.tokens), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(combine_grad_kernel<1>, token_grid(a.tokens), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace fp8fg
