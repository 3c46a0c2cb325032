// Log probabilities of given tokens, with entropy and top alternatives (sm_100a).
//
// What a server answers beside the tokens that the acceptance emitted, from the logit rows of the
// LM head ("Gemma 4 MTP: drafter drafts, target verifies", section "basic structure of
// speculative decoding": the target's own distribution p is what the emitted tokens follow).
//
// Mathematics, x = z / T: with m = max z, t_v = (z_v - m) log2(e) / T, S = sum 2^t, A = sum t 2^t,
//   ln p(token) = (z_token - m) / T - ln S,     entropy = ln S - ln(2) A / S.
// (m, S, A) of two parts merge as S = S_1 w_1 + S_2 w_2, A = sum w_i (A_i + d_i S_i) with d_i the
// shift of m_i to the common maximum and w_i = 2^d_i, all in float32.
//
// Bound by HBM: the 4 V bytes of a row are read once.  A CTA streams a chunk of one row in tiles of 16
// logits a thread, the next tile's loads in flight meanwhile.  Every thread keeps its own (m, S, A), so
// nothing is exchanged until the chunk's end.  The top n are found without sorting: the n-th largest of
// the first tile's thread maxima (of at most 8 a warp) is a logit that at least n reach.  Only logits
// that reach the bound are gathered as (logit, id) keys, a comparison with the thread's maximum for most
// threads; where many are, they are ranked by counting and the n-th becomes the bound.  A second
// kernel, one CTA per row, merges the chunks' sums and ranks their keys.
#include <algorithm>

#include "common.cuh"
#include "host.cuh"

namespace sdv {
namespace lp {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kTileLogits = 16 * kThreads;
constexpr int kCap = 1024;  // gathered keys; a tile that brings more (rising logits) is gathered again, 256
                            // keys at a time with thinning in between
constexpr int kHigh = 512;  // more than these after a tile are thinned out
constexpr int kDump = 64;   // keys that a chunk leaves for the merge, in any order

typedef unsigned long long u64;

struct Params {
  int rows, V, ld, top, chunks, chunk_logits;
  float c;     // log2(e) / T
  float invT;
  const float *z;
  const int32_t *tokens;
  float *logprob, *entropy, *top_lp;
  int32_t *top_ids;
  float4 *part;  // [rows][chunks] (m, S, A, -)
  u64 *cand;     // [rows][chunks][kDump]
  int *status;
};

// Keys rise with the logit and, among equal logits (-0 = 0), fall with the id; 0 is no key.
__device__ __forceinline__ u64 key_of(float z, int id) {
  const uint32_t b = __float_as_uint(z + 0.f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((u64)o << 32) | (uint32_t)~(uint32_t)id;
}
__device__ __forceinline__ int key_id(u64 k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_logit(u64 k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

struct Select {
  u64 keys[kCap];
  u64 best[kMaxTop];
  float tau[8 * kWarps];
  float bound;
  int count;
};

// A logit that at least n of the CTA's logits reach (-inf where there are fewer): the n-th largest of the
// warps' min(n, 8) largest thread maxima.  `mine` is the thread's largest.  Every thread of the CTA
// calls it; it ends behind a barrier.
__device__ __forceinline__ float block_bound(Select &s, int n, float mine) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = min(n, 8);
  float left = mine, kept = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const float top = warp_max(left);
    const unsigned who = __ballot_sync(0xffffffffu, left == top);
    if (lane == __ffs(who) - 1) left = -INFINITY;
    if (lane == i) kept = top;
  }
  if (lane < per) s.tau[warp * per + lane] = kept == kept ? kept : -INFINITY;
  if (tid == 0) s.bound = -INFINITY;
  __syncthreads();
  if (tid < kWarps * per) {
    const float v = s.tau[tid];
    int rank = 0;
    for (int i = 0; i < kWarps * per; ++i) rank += s.tau[i] > v || (s.tau[i] == v && i < tid);
    if (rank == n - 1) s.bound = v;
  }
  __syncthreads();
  return s.bound;
}

// The n largest of s.keys[0 .. count) to s.best in their order (0 behind the last key).  Callers have
// a barrier before and after.
__device__ __forceinline__ void block_rank(Select &s, int n, int count) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (i >= count) s.best[i] = 0;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const u64 k = s.keys[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s.keys[j] > k;
    if (rank < n) s.best[rank] = k;
  }
}

// Keeps the n largest of s.keys[0 .. count), sorted in s.best too; returns the smallest of them (or 1).
__device__ __noinline__ u64 block_thin(Select &s, int n, int count) {
  float mine = -INFINITY;
  u64 held[kCap / kThreads];
#pragma unroll
  for (int i = 0; i < kCap / kThreads; ++i) {
    const int at = threadIdx.x + i * kThreads;
    held[i] = at < count ? s.keys[at] : 0;
    if (held[i]) mine = fmaxf(mine, key_logit(held[i]));
  }
  const float bound = block_bound(s, n, mine);
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCap / kThreads; ++i)
    if (held[i] && key_logit(held[i]) >= bound) s.keys[atomicAdd(&s.count, 1)] = held[i];
  __syncthreads();
  const int left = s.count;
  block_rank(s, n, left);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) s.keys[i] = s.best[i];
  if (threadIdx.x == 0) s.count = min(n, left);
  const u64 last = s.best[n - 1];
  __syncthreads();
  return last == 0 ? 1 : last;
}

// One key more of a thread (0: none) where it reaches the bound; barriers around it are the caller's.
__device__ __forceinline__ void gather(Select &s, u64 k, u64 bound) {
  if (k < bound) return;
  const int at = atomicAdd(&s.count, 1);
  if (at < kCap) s.keys[at] = k;
}

__device__ __forceinline__ float block_max(float v, float *red) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[w]);
  return v;
}

// Both sums, in a fixed order; red holds 2 * kWarps floats of its own.
__device__ __forceinline__ void block_sum2(float &a, float &b, float *red) {
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = a;
    red[kWarps + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    a += red[w];
    b += red[kWarps + w];
  }
}

constexpr float kLowest = -1e4f;  // 2^kLowest is 0, and 0 * kLowest is 0
constexpr float kFloor = -3.402823466e38f;  // maximum of no logits: -inf minus it is -inf, not NaN

// Answers of one row from its (m, S, A); bad rows get NaN.
__device__ __forceinline__ void answer(const Params &p, int row, int token, float m, float S,
                                       float A, bool bad) {
  const float nan = __int_as_float(0x7fc00000);
  const float lnS = logf(S);
  p.logprob[row] = bad ? nan : (p.z[(size_t)row * p.ld + token] - m) * p.invT - lnS;
  if (p.entropy) p.entropy[row] = bad ? nan : lnS - 0.69314718056f * (A / S);
}

__device__ __forceinline__ void answer_top(const Params &p, int row, int rank, u64 key, float m,
                                           float lnS, bool bad) {
  const size_t at = (size_t)row * p.top + rank;
  p.top_ids[at] = bad ? -1 : key_id(key);
  p.top_lp[at] = bad ? __int_as_float(0x7fc00000) : (key_logit(key) - m) * p.invT - lnS;
}

// The row's token; false (and the row's outputs written by the CTA that owns them) where there is
// nothing to score.
__device__ __forceinline__ bool scored(const Params &p, int row, int &token, bool owner) {
  token = p.tokens[row];
  if (token >= 0 && token < p.V) return true;
  if (owner) {
    if (threadIdx.x == 0) {
      if (token >= p.V) record_status(p.status, SD_ERR_DEVICE);
      p.logprob[row] = 0.f;
      if (p.entropy) p.entropy[row] = 0.f;
    }
    for (int i = threadIdx.x; i < p.top; i += kThreads) {
      p.top_ids[(size_t)row * p.top + i] = -1;
      p.top_lp[(size_t)row * p.top + i] = -INFINITY;
    }
  }
  return false;
}

// Sixteen logits of a thread; element e has id base + tile_id(e).
template <bool VEC>
__device__ __forceinline__ int tile_id(int e) {
  return VEC ? (e / 4) * (4 * kThreads) + 4 * (int)threadIdx.x + e % 4
             : e * kThreads + (int)threadIdx.x;
}
template <bool VEC>
__device__ __forceinline__ void load_tile(const float *z, int base, int V, float (&x)[16]) {
  if (base + kTileLogits <= V) {
#pragma unroll
    for (int e = 0; e < 16; e += VEC ? 4 : 1) {
      if constexpr (VEC) {
        const float4 f = __ldcs(reinterpret_cast<const float4 *>(z + base + tile_id<VEC>(e)));
        x[e] = f.x, x[e + 1] = f.y, x[e + 2] = f.z, x[e + 3] = f.w;
      } else {
        x[e] = __ldcs(z + base + tile_id<VEC>(e));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int v = base + tile_id<VEC>(e);
      x[e] = v < V ? __ldcs(z + v) : -INFINITY;
    }
  }
}

// One chunk of one row, in float4 quads where VEC (rows 16-byte aligned).  With one chunk a row the
// kernel writes the answers itself.
template <bool VEC, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) chunk_kernel(const __grid_constant__ Params p) {
  __shared__ Select sel;
  __shared__ float red[3 * kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const float *z = p.z + (size_t)row * p.ld;
  const int begin = chunk * p.chunk_logits, end = min(p.V, begin + p.chunk_logits);
  int token;
  if (!scored(p, row, token, p.chunks == 1)) return;
  float x[16];
  load_tile<VEC>(z, begin, end, x);  // behind the token: the memory of a row without one may be missing
  if (TOP && tid == 0) sel.count = 0;
  float m = kFloor, S = 0.f, A = 0.f;
  u64 bound = 1;        // keys below it are not gathered,
  float bound_z = 0.f;  // nor logits below it
  for (int base = begin; base < end; base += kTileLogits) {
    float next[16];
    if (base + kTileLogits < end) load_tile<VEC>(z, base + kTileLogits, end, next);
    float mt = x[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mt = fmaxf(mt, x[e]);
    if (mt > m) {
      const float d = fmaxf((m - mt) * p.c, kLowest), w = ex2_approx(d);
      A = S > 0.f ? w * fmaf(d, S, A) : 0.f;
      S *= w;
      m = mt;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float t = (x[e] - m) * p.c;  // NaN or +inf: S becomes NaN
      const float w = ex2_approx(t);
      S += w;
      A = fmaf(w, fmaxf(t, kLowest), A);
    }
    if (TOP) {
      if (base == begin) bound_z = block_bound(sel, p.top, mt);
      const int before = sel.count;  // the last write is behind a barrier
      __syncthreads();
      if (mt >= bound_z) {
        uint32_t mask = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) mask |= x[e] >= bound_z ? 1u << e : 0u;
        for (; mask; mask &= mask - 1) {  // few: their logits are read again
          const int v = base + tile_id<VEC>(__ffs(mask) - 1);
          if (v < end) gather(sel, key_of(z[v], v), bound);
        }
      }
      __syncthreads();
      int count = sel.count;
      if (__builtin_expect(count > kCap, 0)) {
        // more than there is room for: 256 keys at a time, thinned out in between
        __syncthreads();
        if (tid == 0) sel.count = before;
        for (int e = 0; e < 16; ++e) {
          __syncthreads();
          const int v = base + tile_id<VEC>(e);
          if (v < end) gather(sel, key_of(z[v], v), bound);
          __syncthreads();
          count = sel.count;
          if (count > kHigh) {
            bound = block_thin(sel, p.top, count);
            count = p.top;
          }
        }
        if (bound > 1) bound_z = key_logit(bound);
      }
      // A higher bound spares later tiles the gathering (every gathered key stalls its warp for a
      // read): ranking at 4 n keys rather than at 512 took 192 rows from 54 to 50 us.
      if (__builtin_expect(count > max(kDump, 4 * p.top), 0) && base + kTileLogits < end) {
        bound = block_thin(sel, p.top, count);
        if (bound > 1) bound_z = key_logit(bound);
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = next[e];
  }
  const float M = block_max(m, red);
  const float d = fmaxf((m - M) * p.c, kLowest), w = ex2_approx(d);
  A = S > 0.f ? w * fmaf(d, S, A) : 0.f;
  S *= w;
  block_sum2(S, A, red + kWarps);
  const bool one = p.chunks == 1;
  const bool bad = !(S > 0.f) || !(S < INFINITY);
  if (tid == 0) {
    if (one) answer(p, row, token, M, S, A, bad);
    else p.part[blockIdx.x] = make_float4(M, S, A, 0.f);
  }
  if (!TOP) return;
  const int count = sel.count;
  if (one || count > kDump) block_thin(sel, p.top, count);
  if (!one) {
    if (tid < kDump) p.cand[(size_t)blockIdx.x * kDump + tid] = tid < sel.count ? sel.keys[tid] : 0;
  } else if (tid < p.top) {
    answer_top(p, row, tid, sel.best[tid], M, logf(S), bad || sel.best[tid] == 0);
  }
}

// Merges the chunks of one row.
constexpr int kHeld = 6;  // candidates a thread requests with its first loads (24 chunks)
__global__ void __launch_bounds__(kThreads) merge_kernel(const __grid_constant__ Params p) {
  __shared__ Select sel;
  __shared__ float red[3 * kWarps];
  pdl_wait();
  const int tid = threadIdx.x, row = blockIdx.x;
  const float4 *part = p.part + (size_t)row * p.chunks;
  const u64 *cand = p.cand + (size_t)row * p.chunks * kDump;
  const int n = p.top > 0 ? p.chunks * kDump : 0;
  // the first values of each kind are requested together
  const float4 first = tid < p.chunks ? part[tid] : make_float4(kFloor, 0.f, 0.f, 0.f);
  u64 held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = tid + i * kThreads < n ? cand[tid + i * kThreads] : 0;
  int token;
  if (!scored(p, row, token, true)) return;
  if (tid == 0) sel.count = 0;
  float m = first.x;
  for (int i = tid + kThreads; i < p.chunks; i += kThreads) m = fmaxf(m, part[i].x);
  const float M = block_max(m, red);
  float S = 0.f, A = 0.f;
  for (int i = tid; i < p.chunks; i += kThreads) {
    const float4 v = i == tid ? first : part[i];
    const float d = fmaxf((v.x - M) * p.c, kLowest);
    const float w = ex2_approx(d);
    S = fmaf(v.y, w, S);
    A = fmaf(w, fmaf(d, v.y, v.z), A);
  }
  block_sum2(S, A, red + kWarps);
  const bool bad = !(S > 0.f) || !(S < INFINITY);
  if (tid == 0) answer(p, row, token, M, S, A, bad);
  if (p.top == 0) return;
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (held[i]) f(held[i]);
    for (int i = tid + kHeld * kThreads; i < n; i += kThreads) {
      const u64 k = cand[i];
      if (k) f(k);
    }
  };
  float mine = -INFINITY;
  each([&](u64 k) { mine = fmaxf(mine, key_logit(k)); });
  const float bound = block_bound(sel, p.top, mine);
  each([&](u64 k) {
    if (key_logit(k) >= bound) gather(sel, k, 1);
  });
  __syncthreads();
  if (sel.count > kCap) {
    __syncthreads();
    if (tid == 0) sel.count = 0;
    u64 least = 1;
    for (int i = 0; i < n; i += kThreads) {
      __syncthreads();
      if (i + tid < n) gather(sel, cand[i + tid], least);
      __syncthreads();
      const int count = sel.count;
      if (count > kHigh) least = block_thin(sel, p.top, count);
    }
    __syncthreads();
  }
  block_rank(sel, p.top, sel.count);
  __syncthreads();
  const float lnS = logf(S);
  if (tid < p.top) answer_top(p, row, tid, sel.best[tid], M, lnS, bad || sel.best[tid] == 0);
}

// ------------------------------------------------------------------------------- host side

struct Split {
  int chunk_logits, chunks;
};

// Chunks of whole tiles: as many a row as give one wave of four CTAs an SM (192 rows of 262144: 3 of 22
// tiles), and no longer than 24 tiles, so that more rows than CTAs still spread evenly.
static Split split(const sd_logprobs_desc *d) {
  const long long ctas = 4ll * std::max(sm_count(), 1);
  const long long tiles = ((long long)d->vocab + kTileLogits - 1) / kTileLogits;
  const long long want = std::min(std::max(ctas / std::max(d->rows, 1), 1ll), tiles);
  const long long per = std::min((tiles + want - 1) / want, 24ll);
  Split s;
  s.chunk_logits = (int)(per * kTileLogits);
  s.chunks = (int)((tiles + per - 1) / per);
  return s;
}

static sd_status validate(const sd_logprobs_desc *d) {
  if (!d || d->rows < 0 || d->vocab < 1 || d->top_n < 0) return SD_ERR_INVALID_ARG;
  if (d->ld_logits != 0 && d->ld_logits < d->vocab) return SD_ERR_INVALID_ARG;
  if (!(d->temperature > 0.f) || !(1.4426950408889634f / d->temperature <= 3.4e38f) ||
      !(d->temperature <= 3.4e38f))
    return SD_ERR_INVALID_ARG;
  if (d->top_n > d->vocab) return SD_ERR_INVALID_ARG;
  if (d->top_n > kMaxTop) return SD_ERR_UNSUPPORTED;
  // ids and one row's candidates are counted in 32 bits
  if (d->vocab > (1 << 28)) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

static size_t part_bytes(const sd_logprobs_desc *d, const Split &s) {
  return round_up((size_t)d->rows * s.chunks * sizeof(float4), 256);
}

}  // namespace lp
}  // namespace sdv

extern "C" {

size_t sd_logprobs_workspace_size(const sd_logprobs_desc *desc) {
  using namespace sdv::lp;
  if (validate(desc) != SD_OK || desc->rows == 0) return 0;
  const Split s = split(desc);
  if (s.chunks == 1) return 0;
  return part_bytes(desc, s) +
         (desc->top_n > 0 ? (size_t)desc->rows * s.chunks * kDump * sizeof(u64) : 0);
}

sd_status sd_logprobs(const sd_logprobs_desc *desc, const float *logits, const int32_t *tokens,
                      float *logprob, float *entropy, int32_t *top_ids, float *top_logprobs,
                      void *ws, size_t ws_bytes, sd_stream stream) {
  using namespace sdv;
  using namespace sdv::lp;
  const sd_status st = validate(desc);
  if (st != SD_OK) return st;
  if (desc->rows == 0) return SD_OK;
  if (!logits || !tokens || !logprob) return SD_ERR_INVALID_ARG;
  if (desc->top_n > 0 && (!top_ids || !top_logprobs)) return SD_ERR_INVALID_ARG;
  const Split s = split(desc);
  if ((long long)desc->rows * s.chunks > 0x7fffffffll) return SD_ERR_UNSUPPORTED;
  const size_t need = sd_logprobs_workspace_size(desc);
  if (need > 0 && (!ws || ws_bytes < need)) return SD_ERR_WORKSPACE;
  if (need > 0 && !aligned16(ws)) return SD_ERR_INVALID_ARG;
  Params p{};
  p.rows = desc->rows;
  p.V = desc->vocab;
  p.ld = desc->ld_logits ? desc->ld_logits : desc->vocab;
  p.top = desc->top_n;
  p.chunks = s.chunks;
  p.chunk_logits = s.chunk_logits;
  p.invT = 1.f / desc->temperature;
  p.c = 1.4426950408889634f / desc->temperature;
  p.z = logits;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_lp = top_logprobs;
  if (need > 0) {
    p.part = reinterpret_cast<float4 *>(ws);
    p.cand = reinterpret_cast<u64 *>(reinterpret_cast<uint8_t *>(ws) + part_bytes(desc, s));
  }
  p.status = device_status_word();
  const bool vec = aligned16(logits) && p.ld % 4 == 0;
  const dim3 grid((unsigned)(p.rows * p.chunks)), block(kThreads);
  const cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e;
  if (p.top > 0)
    e = vec ? launch(chunk_kernel<true, true>, grid, block, 0, cs, p)
            : launch(chunk_kernel<false, true>, grid, block, 0, cs, p);
  else
    e = vec ? launch(chunk_kernel<true, false>, grid, block, 0, cs, p)
            : launch(chunk_kernel<false, false>, grid, block, 0, cs, p);
  if (e != cudaSuccess) return SD_ERR_CUDA;
  if (p.chunks == 1) return SD_OK;
  return cuda_status(launch(merge_kernel, dim3((unsigned)p.rows), block, 0, cs, p));
}

}  // extern "C"
