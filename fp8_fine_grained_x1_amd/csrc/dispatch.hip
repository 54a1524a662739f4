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

constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kMaxChunks = 256;
constexpr int kMinChunk = 1024;
constexpr int kMaxBuckets = 1025;  // experts and the bucket of dropped entries
// Short lists are placed by every token's workgroup for itself, in the launch
// that moves the rows: work for each token and entry (reading the list, k
// comparisons), so that tokens x entries bounds it where k is small and the
// entries alone where it is not.  In one launch and in three, us, 256 experts,
// rows of 7168 / 2048 bytes:
//   k = 1    1536 entries  10.8, 12.3 / 10.0, 10.2     2048  15.3, 13.0 / 13.7, 10.4
//   k = 2    2048  10.4, 12.5 / 9.3, 10.0              2560  12.6, 12.9 / 12.0, 10.6
//   k = 4    2560  10.9, 12.2 / 9.4, 10.3              3584  15.8, 13.3 / 14.0, 10.8
//   k = 8    2560  11.3, 13.8 / 9.7, 11.1              4096  15.0, 14.7 / 12.6, 11.8
//   k = 16   2560  12.6, 15.3 / 10.8, 11.8             3584  16.4, 16.2 / 13.4, 12.3
constexpr int64_t kSmallReads = 2400000;
constexpr int64_t kSmallEntries = 3000;
constexpr int kSmallK = 16;

struct Plan {
  const int32_t* idx;
  int64_t ld_idx;
  int entries;
  int chunk;    // entries per chunk, a multiple of kPlanThreads
  int chunks;
  int pitch;    // of counts: chunks, rounded up to 4
  int k, experts;
  int32_t* counts;  // [bucket][chunk]
  int32_t* offsets;
  int32_t* pos;
  int32_t* token;
};

__device__ __forceinline__ int bucket_at(const Plan& p, int64_t at) {
  const int e = p.idx[at];
  return (uint32_t)e < (uint32_t)p.experts ? e : p.experts;
}

__device__ __forceinline__ int bucket_of(const Plan& p, int i) {
  if (p.ld_idx == p.k) return bucket_at(p, i);
  const int t = i / p.k;
  return bucket_at(p, t * p.ld_idx + (i - t * p.k));
}

// counts[e][chunk]: a bucket's counts lie side by side for place_kernel.
__global__ __launch_bounds__(kPlanThreads) void count_kernel(Plan p) {
  __shared__ int32_t n[kMaxBuckets];
  const int B = p.experts + 1;
  for (int e = threadIdx.x; e < B; e += kPlanThreads) n[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.chunk;
  const int64_t i1 = i0 + p.chunk < p.entries ? i0 + p.chunk : p.entries;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kPlanThreads) atomicAdd(&n[bucket_of(p, (int)i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += kPlanThreads) {
    p.counts[(int64_t)e * p.pitch + blockIdx.x] = n[e];
    // the padding that place_kernel reads with the last chunks
    if ((int)blockIdx.x == p.chunks - 1)
      for (int c = p.chunks; c < p.pitch; ++c) p.counts[(int64_t)e * p.pitch + c] = 0;
  }
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

// Exclusive prefix sum over the workgroup, plus `carry`, which grows by the
// workgroup's sum.  Ends behind a barrier.
template <int WAVES>
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t* wsum, int32_t& carry) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t incl = v;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int32_t o = __shfl_up(incl, m);
    incl += lane >= m ? o : 0;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int32_t first = carry + incl - v;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int32_t n = wsum[w];
    first += w < wave ? n : 0;
    carry += n;
  }
  __syncthreads();
  return first;
}

// Each chunk: start of every bucket (all chunks' counts), then the entries
// in order: wave w takes the w-th eighth of the chunk, 64 at a time, and
// ranks an entry among its 64 by ballots over the bits of the bucket.
__global__ __launch_bounds__(kPlanThreads) void place_kernel(Plan p) {
  __shared__ int32_t start[kMaxBuckets];
  __shared__ int32_t base[kPlanWaves][kMaxBuckets];
  __shared__ int32_t wsum[kPlanWaves];
  const int B = p.experts + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t carry = 0;
  for (int e0 = 0; e0 < B; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int32_t total = 0, before = 0;
    if (e < B) {
      const int4* row = reinterpret_cast<const int4*>(p.counts + (int64_t)e * p.pitch);
#pragma unroll 8
      for (int c = 0; c < p.pitch; c += 4) {
        const int4 n = row[c >> 2];
        const int b = (int)blockIdx.x - c;
        total += n.x + n.y + n.z + n.w;
        before += (b > 0 ? n.x : 0) + (b > 1 ? n.y : 0) + (b > 2 ? n.z : 0) + (b > 3 ? n.w : 0);
      }
    }
    const int32_t first = block_prefix<kPlanWaves>(total, wsum, carry);
    if (e < B) {
      start[e] = first + before;
      if (blockIdx.x == 0) p.offsets[e] = first;  // offsets[experts]: entries with an expert
    }
  }
  for (int e = tid; e < B; e += kPlanThreads)
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) base[w][e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.chunk + wave * (p.chunk / kPlanWaves);
  const int64_t i1 = min(i0 + p.chunk / kPlanWaves, (int64_t)p.entries);
  int bits = 0;
  while ((1 << bits) < B) ++bits;
  for (int64_t i = i0 + lane; i < i1; i += 64) atomicAdd(&base[wave][bucket_of(p, (int)i)], 1);
  __syncthreads();
  for (int e = tid; e < B; e += kPlanThreads) {
    int32_t at = start[e];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t n = base[w][e];
      base[w][e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 64) {
    const bool valid = i + lane < i1;
    const int at = (int)(i + lane);
    const int b = valid ? bucket_of(p, at) : 0;
    const uint64_t same = same_bucket(b, valid, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int32_t r = 0;
    if (valid) r = base[wave][b] + rank;
    wave_fence();  // every lane has read before the first of its bucket adds
    if (valid && rank == 0) base[wave][b] += __popcll(same);
    wave_fence();
    if (valid) {
      p.pos[at] = b < p.experts ? r : -2 - r;
      p.token[r] = b < p.experts ? at / p.k : -1;
    }
  }
}

constexpr int kMoveThreads = 256;

struct Move {
  const uint8_t* x;    // null: nothing to move
  int64_t pitch;       // bytes
  int vecs;            // 16-byte vectors per row
  const float* xs;
  int64_t xs_rs, xs_ts;
  int tiles;           // scales per row (0: none)
  int64_t tokens;
  int rows;            // tokens * k
  int k;
  const int32_t* pos;
  const int32_t* token;
  uint8_t* out;
  int64_t opitch;
  float* os;
  int64_t os_rs, os_ts;
  int scale_blocks;    // workgroups that move scales by output row (0: the tokens' do)
};

// The row of token t to its places: read once, written k times.  The read is
// an ordinary one, which gains where the rows lie in the caches (8192 x 8 rows of
// 7168 bytes that do: 115 us, 130 past them) and costs nothing where they do
// not, as after the norm and the quantizers, which store them past the caches
// (norm and dispatch together: 217 us, 220); the writes are non-temporal (ordinary ones take 12% more time).
__device__ __forceinline__ uint4 row_vec(const Move& p, int64_t t, int v) {
  return *reinterpret_cast<const uint4*>(p.x + t * p.pitch + (int64_t)v * 16);
}

// `first`: this thread's first vector, loaded ahead.
__device__ __forceinline__ void move_row(const Move& p, int64_t t, const int32_t* pos, uint4 first) {
  for (int v = threadIdx.x; v < p.vecs; v += blockDim.x) {
    const uint4 w = v == (int)threadIdx.x ? first : row_vec(p, t, v);
    for (int j = 0; j < p.k; ++j) {
      const int32_t r = pos[j];
      const int64_t row = r >= 0 ? r : -2 - r;
      st_nt16(p.out + row * p.opitch + (int64_t)v * 16, r >= 0 ? w : make_uint4(0, 0, 0, 0));
    }
  }
}

__device__ __forceinline__ void move_scales_of(const Move& p, int64_t t, const int32_t* pos) {
  for (int i = threadIdx.x; i < p.tiles; i += blockDim.x) {
    const float s = p.xs[t * p.xs_rs + i * p.xs_ts];
    for (int j = 0; j < p.k; ++j) {
      const int32_t r = pos[j];
      p.os[(r >= 0 ? r : -2 - r) * p.os_rs + i * p.os_ts] = r >= 0 ? s : kFltMinNormal;
    }
  }
}

// 8192 tokens to 8 of 256 experts, rows of 7168 bytes: 103.5 us with the
// counts and places (12), that is 5.3 TB/s of rows and scales, most of it
// writes.  (By output row, gathering: 145 us.)
//
// Workgroups 0 .. scale_blocks - 1 move the scales of 64 output rows each, a
// lane to a row: with group-major scales a wave then writes 256 contiguous
// bytes, where a token's workgroup would write single floats into lines that
// it shares with 15 other tokens.  The others take a token each.
__global__ __launch_bounds__(kMoveThreads) void move_kernel(Move p) {
  if ((int)blockIdx.x < p.scale_blocks) {
    const int waves = blockDim.x >> 6;
    for (int64_t r = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63); r < p.rows; r += (int64_t)p.scale_blocks * 64) {
      const int32_t t = p.token[r];
#pragma unroll 4
      for (int i = threadIdx.x >> 6; i < p.tiles; i += waves) {
        const float s = t >= 0 ? p.xs[t * p.xs_rs + i * p.xs_ts] : kFltMinNormal;
        p.os[r * p.os_rs + i * p.os_ts] = s;
      }
    }
    return;
  }
  const int64_t step = gridDim.x - p.scale_blocks;
  for (int64_t t = (int64_t)blockIdx.x - p.scale_blocks; t < p.tokens; t += step) {
    move_row(p, t, p.pos + t * p.k, (int)threadIdx.x < p.vecs ? row_vec(p, t, threadIdx.x) : uint4{});
    if (p.scale_blocks == 0) move_scales_of(p, t, p.pos + t * p.k);
  }
}

// The whole dispatch of a short list in one launch: workgroup t counts, for
// each of token t's entries, the entries before it in the order; the last
// workgroup writes the offsets.
__global__ __launch_bounds__(512) void dispatch_small_kernel(Plan p, Move m) {
  __shared__ int32_t n[kMaxBuckets];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int64_t)blockIdx.x == m.tokens) {
    __shared__ int32_t wsum[kPlanWaves];
    const int B = p.experts + 1;
    for (int e = tid; e < B; e += kPlanThreads) n[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.entries; i += kPlanThreads) atomicAdd(&n[bucket_of(p, i)], 1);
    __syncthreads();
    int32_t carry = 0;
    for (int e0 = 0; e0 < B; e0 += kPlanThreads) {
      const int32_t first = block_prefix<kPlanWaves>(e0 + tid < B ? n[e0 + tid] : 0, wsum, carry);
      if (e0 + tid < B) p.offsets[e0 + tid] = first;
    }
    return;
  }
  const int t = blockIdx.x;
  __shared__ int32_t part[kPlanWaves][kSmallK];
  __shared__ int32_t place[kSmallK];
  int before[kSmallK], mine[kSmallK];
#pragma unroll
  for (int j = 0; j < kSmallK; ++j) {
    before[j] = 0;
    mine[j] = j < p.k ? bucket_at(p, t * p.ld_idx + j) : 0;
  }
  const uint4 first = m.x && tid < m.vecs ? row_vec(m, t, tid) : uint4{};
  for (int i0 = wave * 64; i0 < p.entries; i0 += kPlanThreads) {
    const int i = i0 + lane;
    const int b = i < p.entries ? bucket_of(p, i) : kMaxBuckets;
#pragma unroll
    for (int j = 0; j < kSmallK; ++j)
      if (j < p.k) before[j] += __popcll(__builtin_amdgcn_ballot_w64(b < mine[j] || (b == mine[j] && i < t * p.k + j)));
  }
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < kSmallK; ++j) part[wave][j] = before[j];
  __syncthreads();
  if (tid < p.k) {
    int32_t r = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) r += part[w][tid];
    const bool here = bucket_at(p, t * p.ld_idx + tid) < p.experts;
    place[tid] = here ? r : -2 - r;
    p.pos[t * p.k + tid] = place[tid];
    p.token[r] = here ? t : -1;
  }
  __syncthreads();
  if (!m.x) return;
  move_row(m, t, place, first);
  move_scales_of(m, t, place);
}

// A lane sums 16 bytes of the row over the token's places, the loads of
// kAhead of them in flight together; the columns are spread over workgroups
// of one wave, which suits a decode batch's few tokens and the many of a long
// one alike.  Large z is read past the caches, base ordinarily (its producer
// has just left it), the result stored past them.  4096 x 8 rows of 4096 f32
// with base: 101 us (6.6 TB/s); workgroups of two waves 103, of four 105; 32
// bytes a lane, in two loads, 117; z ordinarily +7, base past the caches +5,
// the result ordinarily +3.
constexpr int kAhead = 8;
constexpr int kCombineThreads = 64;

template <int XT, bool NT>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs p, int64_t units, int blocks) {
  constexpr int N = kPer16<XT>;
  const int nvec = (int)(p.cols / N);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t t = u / blocks;
    const int v = (int)(u - t * blocks) * kCombineThreads + threadIdx.x;
    if (v >= nvec) continue;
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    uint4 base = {};
    if (p.base) base = load16<XT, false>(p.base, t * p.ldb + (int64_t)v * N);
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
      uint4 z[kAhead];
      float w[kAhead];
      bool here[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t r = j0 + j < p.k ? p.pos[t * p.k + j0 + j] : -1;
        here[j] = r >= 0 && r < p.z_rows;
        z[j] = {};
        w[j] = 1.0f;
        if (here[j]) {
          z[j] = load16<XT, NT>(p.z, r * p.ldz + (int64_t)v * N);
          if (p.w) w[j] = p.w[t * p.ldw + j0 + j];
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (!here[j]) continue;
        float f[N];
        decode16<XT>(z[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = __builtin_fmaf(w[j], f[e], acc[e]);
      }
    }
    if (p.base) {
      float f[N];
      decode16<XT>(base, f);
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] += f[e];
    }
    store16<XT, true>(p.out, t * p.ldo + (int64_t)v * N, encode16<XT>(acc));
  }
}

// A workgroup per token: dy's vector is read once for kAhead places, whose
// rows of z are in flight together; the places' dot products stay in
// registers and meet once per kAhead of them.  Large z is read past the
// caches (4096 x 8 rows of 7168 bf16: 179 us; ordinarily 196), dy ordinarily
// (past them 188), dz stored past them (ordinarily 198).
template <int XT, bool NT>
__global__ __launch_bounds__(512) void combine_grad_kernel(CombineGradArgs p) {
  __shared__ float part[8][kAhead];
  constexpr int N = kPer16<XT>;
  const int nvec = (int)(p.cols / N);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
      int64_t row[kAhead];  // -1: nothing to write
      float w[kAhead], dot[kAhead];
      bool here[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t r = j0 + j < p.k ? p.pos[t * p.k + j0 + j] : -1;
        here[j] = r >= 0 && r < p.z_rows;
        row[j] = r >= 0 ? r : -2 - r;
        if (row[j] >= p.z_rows) row[j] = -1;
        w[j] = here[j] && p.w ? p.w[t * p.ldw + j0 + j] : 1.0f;
        dot[j] = 0.0f;
      }
      for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        float d[N];
        const uint4 dy = load16<XT, false>(p.dy, t * p.lddy + (int64_t)v * N);
        uint4 z[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          z[j] = {};
          if (here[j] && p.dw) z[j] = load16<XT, NT>(p.z, row[j] * p.ldz + (int64_t)v * N);
        }
        decode16<XT>(dy, d);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (row[j] < 0) continue;
          float f[N];
          if (here[j]) {
            decode16<XT>(z[j], f);
#pragma unroll
            for (int e = 0; e < N; ++e) dot[j] = __builtin_fmaf(d[e], f[e], dot[j]);
          }
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] = here[j] ? w[j] * d[e] : 0.0f;
          store16<XT, true>(p.dz, row[j] * p.lddz + (int64_t)v * N, encode16<XT>(f));
        }
      }
      if (p.dw) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          dot[j] = wave_sum(dot[j]);
          if (lane == 0) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kAhead && j0 + (int)threadIdx.x < p.k) {
          float s = part[0][threadIdx.x];
          for (int i = 1; i < waves; ++i) s += part[i][threadIdx.x];
          p.dw[t * p.lddw + j0 + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
  }
}

constexpr int64_t kMaxTokenBlocks = 1 << 20;
constexpr int64_t kMaxCombineBlocks = 1 << 24;  // (x 64 threads: below 2^32 work-items)

unsigned token_blocks(int64_t tokens) { return (unsigned)(tokens < kMaxTokenBlocks ? tokens : kMaxTokenBlocks); }

// Threads (at most 512, whole waves) that split `vecs` evenly.
unsigned row_threads(int64_t vecs) {
  const int64_t rounds = (vecs + 511) / 512;
  const int64_t t = rounds > 0 ? (vecs + rounds - 1) / rounds : 1;
  return (unsigned)((t + 63) / 64 * 64);
}

}  // namespace

// At most kMaxChunks chunks: each chunk's workgroup reads all their counts.
static int64_t dispatch_chunks(int64_t entries) {
  const int64_t n = (entries + kMinChunk - 1) / kMinChunk;
  return n < 1 ? 1 : n < kMaxChunks ? n : kMaxChunks;
}

static int64_t count_pitch(int64_t chunks) { return (chunks + 3) / 4 * 4; }

int64_t dispatch_counts(int64_t entries, int64_t experts) {
  return count_pitch(dispatch_chunks(entries)) * (experts + 1);
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st) {
  const int64_t entries = a.tokens * a.k;
  const int64_t chunks = dispatch_chunks(entries);
  const int64_t per = (entries + chunks - 1) / chunks;
  const int64_t chunk = (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  const Plan p{a.idx,    a.ld_idx,  (int)entries, (int)chunk, (int)chunks, (int)count_pitch(chunks), a.k,
               a.experts, a.counts, a.offsets,    a.pos,      a.token};
  const int size = a.x_type == 2 ? 1 : a.x_type == 0 ? 2 : 4;
  Move m{reinterpret_cast<const uint8_t*>(a.x), a.ldx * size, (int)(a.cols * size / 16), a.xs, a.xs_rs, a.xs_ts,
         a.x_type == 2 ? (int)(a.cols / 128) : 0, a.tokens, (int)entries, a.k, a.pos, a.token,
         reinterpret_cast<uint8_t*>(a.out), a.ldo * size, a.os, a.os_rs, a.os_ts, 0};
  if (entries <= kSmallEntries && a.tokens * entries <= kSmallReads && a.k <= kSmallK) {
    hipLaunchKernelGGL(dispatch_small_kernel, dim3((unsigned)a.tokens + 1), dim3(kPlanThreads), 0, st, p, m);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)chunks), dim3(kPlanThreads), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)chunks), dim3(kPlanThreads), 0, st, p);
  e = hipGetLastError();
  if (e == hipSuccess && a.x) {
    if (m.tiles > 0 && a.os_rs == 1) m.scale_blocks = (int)token_blocks((entries + 63) / 64);
    hipLaunchKernelGGL(move_kernel, dim3(m.scale_blocks + token_blocks(a.tokens)), dim3(kMoveThreads), 0, st, m);
    e = hipGetLastError();
  }
  return e;
}

template <int XT>
static void combine_t(const CombineArgs& a, hipStream_t st) {
  const int64_t blocks = (a.cols / kPer16<XT> + kCombineThreads - 1) / kCombineThreads;
  const int64_t units = a.tokens * blocks;
  const unsigned grid = (unsigned)(units < kMaxCombineBlocks ? units : kMaxCombineBlocks);
  if (past_caches(a.tokens, a.k, a.cols, XT == 0 ? 2 : 4))
    hipLaunchKernelGGL((combine_kernel<XT, true>), dim3(grid), dim3(kCombineThreads), 0, st, a, units, (int)blocks);
  else
    hipLaunchKernelGGL((combine_kernel<XT, false>), dim3(grid), dim3(kCombineThreads), 0, st, a, units, (int)blocks);
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
  if (a.type == 0)
    combine_t<0>(a, st);
  else
    combine_t<1>(a, st);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t st) {
  const dim3 grid(token_blocks(a.tokens)), block(row_threads(a.cols / (a.type == 0 ? kPer16<0> : kPer16<1>)));
  const bool stream = past_caches(a.tokens, a.k, a.cols, a.type == 0 ? 2 : 4);
  if (a.type == 0 && stream)
    hipLaunchKernelGGL((combine_grad_kernel<0, true>), grid, block, 0, st, a);
  else if (a.type == 0)
    hipLaunchKernelGGL((combine_grad_kernel<0, false>), grid, block, 0, st, a);
  else if (stream)
    hipLaunchKernelGGL((combine_grad_kernel<1, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((combine_grad_kernel<1, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace fp8fg
