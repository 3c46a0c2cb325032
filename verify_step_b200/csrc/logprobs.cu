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
// Bound by HBM: the 4 V bytes of a row are read once.  A CTA takes a chunk of 256 * EPT logits of
// one row into registers and makes three passes over them: maximum, sums, candidates.  The top n
// are found without sorting: every thread's largest (logit, id) key is a lower bound of the
// ranks it holds, so the smallest over the warps of the ceil(n / warps)-th largest thread key
// has at least n keys at or above it; the few keys not below it are gathered and ranked by
// counting.  A second kernel, one CTA per row, merges the chunks the same way.
#include <algorithm>

#include "common.cuh"
#include "host.cuh"

namespace sdv {
namespace lp {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kCap = 512;  // gathered keys; more of them (rows of a special pattern) are bisected

typedef unsigned long long u64;

struct Params {
  int rows, V, ld, top, chunks;
  float c;     // log2(e) / T
  float invT;
  const float *z;
  const int32_t *tokens;
  float *logprob, *entropy, *top_lp;
  int32_t *top_ids;
  float4 *part;  // [rows][chunks] (m, S, A, -)
  u64 *cand;     // [rows][chunks][top]
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

__device__ __forceinline__ u64 warp_max(u64 v) {
  for (int o = 16; o > 0; o >>= 1) {
    const u64 u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

struct Select {
  u64 keys[kCap];
  u64 tau[kWarps];
  int count;
};

// The n largest of the CTA's keys, handed to out(rank, key).  each(f) calls f on all keys that
// the thread holds, `mine` is their largest.  Every thread of the CTA calls it.
template <typename Each, typename Out>
__device__ __forceinline__ void block_top(Select &s, int n, u64 mine, const Each &each,
                                          const Out &out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kWarps - 1) / kWarps;
  u64 left = mine, top = 0;
  for (int i = 0; i < per; ++i) {
    top = warp_max(left);
    if (left == top) left = 0;  // keys differ, so one lane gives up its own
  }
  if (lane == 0) s.tau[warp] = top;
  if (tid == 0) s.count = 0;
  __syncthreads();
  u64 tau = s.tau[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) tau = min(tau, s.tau[w]);
  if (tau == 0) tau = 1;  // 0 is no key
  if (mine >= tau)
    each([&](u64 k) {
      if (k >= tau) {
        const int at = atomicAdd(&s.count, 1);
        if (at < kCap) s.keys[at] = k;
      }
    });
  __syncthreads();
  int count = s.count;
  if (count > kCap) {
    // the n-th largest key, bit by bit: the largest threshold that n keys reach
    u64 t = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 v = t | (1ull << bit);
      int have = 0;
      if (mine >= v) each([&](u64 k) { have += k >= v; });
      for (int o = 16; o > 0; o >>= 1) have += __shfl_xor_sync(0xffffffffu, have, o);
      __syncthreads();
      if (tid == 0) s.count = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(&s.count, have);
      __syncthreads();
      if (s.count >= n) t = v;
    }
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    if (t == 0) t = 1;
    if (mine >= t)
      each([&](u64 k) {
        if (k >= t) s.keys[atomicAdd(&s.count, 1)] = k;  // n of them: the keys differ
      });
    __syncthreads();
    count = s.count;
  }
  for (int i = tid; i < count; i += kThreads) {
    const u64 k = s.keys[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s.keys[j] > k;
    if (rank < n) out(rank, k);
  }
  for (int i = count + tid; i < n; i += kThreads) out(i, (u64)0);  // fewer than n keys at all
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

// One chunk of one row.  EPT logits a thread, in float4 quads where VEC (rows 16-byte aligned).
// With one chunk a row the kernel writes the answers itself.
template <int EPT, bool VEC>
__global__ void __launch_bounds__(kThreads) chunk_kernel(const __grid_constant__ Params p) {
  __shared__ Select sel;
  __shared__ float red[3 * kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  int token;
  if (!scored(p, row, token, p.chunks == 1)) return;
  const float *z = p.z + (size_t)row * p.ld;
  const int base = chunk * (kThreads * EPT);
  float x[EPT];
  // element e of the thread has id base + id_of(e)
  auto id_of = [&](int e) {
    return VEC ? (e / 4) * (4 * kThreads) + 4 * tid + e % 4 : e * kThreads + tid;
  };
  if constexpr (VEC) {
#pragma unroll
    for (int q = 0; q < EPT / 4; ++q) {
      const int v = base + q * 4 * kThreads + 4 * tid;
      if (v + 3 < p.V) {
        const float4 f = __ldcs(reinterpret_cast<const float4 *>(z + v));
        x[4 * q] = f.x, x[4 * q + 1] = f.y, x[4 * q + 2] = f.z, x[4 * q + 3] = f.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * q + e] = v + e < p.V ? z[v + e] : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int v = base + e * kThreads + tid;
      x[e] = v < p.V ? __ldcs(z + v) : -INFINITY;
    }
  }
  float m = -INFINITY;
  bool odd = false;  // NaN or +inf
  int arg = 0;       // element of the thread's largest key: the first of its largest logit
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    odd |= !(x[e] < INFINITY);
    if (x[e] > m) {
      m = x[e];
      arg = e;
    }
  }
  odd = __syncthreads_or(odd);
  const float M = block_max(m, red);
  float S = 0.f, A = 0.f;
  if (!odd && M > -INFINITY) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const float t = fmaxf((x[e] - M) * p.c, kLowest);
      const float w = ex2_approx(t);
      S += w;
      A = fmaf(w, t, A);
    }
  }
  block_sum2(S, A, red + kWarps);
  const bool one = p.chunks == 1;
  const bool bad = odd || S == 0.f;
  if (tid == 0) {
    if (one)
      answer(p, row, token, M, S, A, bad);
    else
      p.part[blockIdx.x] = make_float4(odd ? __int_as_float(0x7fc00000) : M, S, A, 0.f);
  }
  if (p.top == 0) return;
  const float lnS = logf(S);
  // a thread whose first element lies behind the row's end holds no key
  const u64 mine = base + id_of(arg) < p.V ? key_of(m, base + id_of(arg)) : 0;
  block_top(
      sel, p.top, odd ? 0 : mine,
      [&](auto f) {
#pragma unroll
        for (int e = 0; e < EPT; ++e)
          if (base + id_of(e) < p.V) f(key_of(x[e], base + id_of(e)));
      },
      [&](int rank, u64 k) {
        if (one)
          answer_top(p, row, rank, k, M, lnS, bad || k == 0);
        else
          p.cand[(size_t)blockIdx.x * p.top + rank] = k;
      });
}

// Merges the chunks of one row.
__global__ void __launch_bounds__(kThreads) merge_kernel(const __grid_constant__ Params p) {
  __shared__ Select sel;
  __shared__ float red[3 * kWarps];
  pdl_wait();
  const int tid = threadIdx.x, row = blockIdx.x;
  int token;
  if (!scored(p, row, token, true)) return;
  const float4 *part = p.part + (size_t)row * p.chunks;
  float m = -INFINITY;
  bool odd = false;
  for (int i = tid; i < p.chunks; i += kThreads) {
    const float v = part[i].x;
    odd |= v != v;
    m = fmaxf(m, v);
  }
  odd = __syncthreads_or(odd);
  const float M = block_max(m, red);
  float S = 0.f, A = 0.f;
  if (!odd && M > -INFINITY)
    for (int i = tid; i < p.chunks; i += kThreads) {
      const float4 v = part[i];
      const float d = fmaxf((v.x - M) * p.c, kLowest);
      const float w = ex2_approx(d);
      S = fmaf(v.y, w, S);
      A = fmaf(w, fmaf(d, v.y, v.z), A);
    }
  block_sum2(S, A, red + kWarps);
  const bool bad = odd || S == 0.f;
  if (tid == 0) answer(p, row, token, M, S, A, bad);
  if (p.top == 0) return;
  const float lnS = logf(S);
  const u64 *cand = p.cand + (size_t)row * p.chunks * p.top;
  const int n = p.chunks * p.top;
  auto each = [&](auto f) {
    for (int i = tid; i < n; i += kThreads) {
      const u64 k = cand[i];
      if (k) f(k);
    }
  };
  u64 mine = 0;
  if (!odd) each([&](u64 k) { mine = k > mine ? k : mine; });
  block_top(sel, p.top, mine, each, [&](int rank, u64 k) {
    answer_top(p, row, rank, k, M, lnS, bad || k == 0);
  });
}

// ------------------------------------------------------------------------------- host side

struct Split {
  int ept, chunks;
};

// 8192 logits a CTA, fewer while that leaves SMs idle (one row of 262144: 32 CTAs; with 2048
// logits each, 128).
static Split split(const sd_logprobs_desc *d) {
  const long long sms = std::max(sm_count(), 1);
  Split s{32, 0};
  for (;; s.ept /= 2) {
    s.chunks = (int)(((long long)d->vocab + kThreads * s.ept - 1) / (kThreads * s.ept));
    if (s.ept == 8 || (long long)s.chunks * d->rows >= sms) return s;
  }
}

static sd_status validate(const sd_logprobs_desc *d) {
  if (!d || d->rows < 0 || d->vocab < 1 || d->top_n < 0) return SD_ERR_INVALID_ARG;
  if (d->ld_logits != 0 && d->ld_logits < d->vocab) return SD_ERR_INVALID_ARG;
  if (!(d->temperature > 0.f) || !(1.f / d->temperature <= 3.4e38f) ||
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
  return part_bytes(desc, s) + (size_t)desc->rows * s.chunks * desc->top_n * sizeof(u64);
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
  if (s.ept == 32)
    e = vec ? launch(chunk_kernel<32, true>, grid, block, 0, cs, p)
            : launch(chunk_kernel<32, false>, grid, block, 0, cs, p);
  else if (s.ept == 16)
    e = vec ? launch(chunk_kernel<16, true>, grid, block, 0, cs, p)
            : launch(chunk_kernel<16, false>, grid, block, 0, cs, p);
  else
    e = vec ? launch(chunk_kernel<8, true>, grid, block, 0, cs, p)
            : launch(chunk_kernel<8, false>, grid, block, 0, cs, p);
  if (e != cudaSuccess) return SD_ERR_CUDA;
  if (p.chunks == 1) return SD_OK;
  return cuda_status(launch(merge_kernel, dim3((unsigned)p.rows), block, 0, cs, p));
}

}  // extern "C"
