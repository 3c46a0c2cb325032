// Rotary positions and the append of new K/V rows to the paged cache (sm_100a).
//
// The target's layers turn their queries and keys by the position before attention reads them,
// and the cache that target and drafter share ("Gemma 4 MTP: drafter drafts, target verifies",
// section "drafter internal architecture") holds the turned keys.  The pages give no formula for
// positions; this is the standard rotary embedding (Su et al., "RoFormer"), with the two usual
// ways to stretch the context: frequencies divided by a factor, or divided by parts (Peng et al.,
// "YaRN": fast dimensions keep their frequency, slow ones are divided, a ramp between).
//
// Angles.  A frequency is held as a 64-bit fraction of a turn, so position x frequency modulo one
// turn is one integer product, exact for every int32 position: a float angle of position 10^6
// would be off by 0.03 rad.  The product is reduced to the nearest quarter turn in integers, and
// Taylor's series give sine and cosine of the pi / 4 at most that is left.
//
// Rows (sd_rope, and the append to a cache of the rows' own type): a thread owns one unit of a
// row, V rotating pairs (two 16-byte vectors), computes its V sines and cosines once and turns
// that unit of several heads.  Bound by HBM: every element is read and written once.
//
// The append to an e4m3 cache: a CTA owns one (block, heads, K or V), so the block's scale has one
// writer.  It goes from head to head, the next head's rows in flight while this one's maximum is
// joined; a thread has the same elements of every head and keeps their sines and cosines in shared
// memory.  Bound by issue slots and latency, not by HBM: 53.5 us for 190 MB (3.6 TB/s, blocks of 16
// rows, 4 heads of 512 elements), 48 without a rotation (V, never turned, is half of the work and goes
// through the same unpacking and float maxima as K); leaving out the stores alone changed nothing.
// Staging a block's rows in shared memory and going over them twice took 61 us, with copies a block
// ahead 59, and with loops in place of unrolled heads 81.
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "host.cuh"

namespace sdv {
namespace app {

constexpr int kMaxThreads = 256;    // rows_kernel
constexpr int kQuantThreads = 512;  // quant_kernel
constexpr int kMaxRows = INT_MAX - kMaxThreads;  // rows are counted up to whole CTAs

struct Rot {
  const unsigned long long *freqs;  // null: no rotation
  int half;                         // rotating pairs of a head
  int inter;                        // 0: pairs (i, i + half); 1: pairs (2i, 2i + 1)
  float amp;
};

// One group of heads of the rows: source rows [rows][heads][D], destination rows of the same
// form or rows of the paged cache.
struct Seg {
  const void *src;
  void *dst;
  int64_t ld_src, ld_dst;
  int heads;
  int rotate, to_cache;
};

struct Params {
  int rows, B, D, units, nrot;  // units of a row, the first nrot of them rotating
  Rot rot;
  // positions: pos[row], else ctx_len[b] + j + q_offset
  const int32_t *pos, *ctx_len, *cu;
  int per_seq, q_offset;
  Seg seg[3];
  int heads_total, heads_per_cta, rows_per_cta;
  // paged cache
  const int32_t *table;
  int hkv, bs, mbps, num_blocks;
  // e4m3 append
  const void *k_new, *v_new;
  int64_t ld_k, ld_v;
  uint8_t *kc, *vc;
  float *ks, *vs;
  int items, chunks, heads_per_quant, quant_ctas;
  int *status;
};

// cos and sin of position * frequency, times amp.  The series up to x^9 and x^10 leave at most
// x^11 / 11! = 1.8e-9 and x^12 / 12! = 1.2e-10 at pi / 4, a 16th of the half step of a float there.
// (sincospif reduces its argument once more: with it and a division and single products in the rounding
// to codes the prompts of the header took 58.0 us, without 54.4.)
__device__ __forceinline__ void turn(unsigned long long freq, int pos, float amp, float &c,
                                     float &s) {
  const unsigned long long ph = freq * (unsigned long long)(long long)pos;
  const unsigned q = (unsigned)((ph + (1ull << 61)) >> 62);
  // what is left of the nearest quarter turn: bits 30 to 61, signed, in 2^-34 turns
  const float x = (float)(int)(unsigned)(ph >> 30) * (6.2831853071795864769f * 0x1p-34f);
  const float y = x * x;
  float s0 = 1.f / 362880.f;
  s0 = fmaf(s0, y, -1.f / 5040.f);
  s0 = fmaf(s0, y, 1.f / 120.f);
  s0 = fmaf(s0, y, -1.f / 6.f);
  s0 = fmaf(s0 * y, x, x);
  float c0 = -1.f / 3628800.f;
  c0 = fmaf(c0, y, 1.f / 40320.f);
  c0 = fmaf(c0, y, -1.f / 720.f);
  c0 = fmaf(c0, y, 1.f / 24.f);
  c0 = fmaf(c0, y, -0.5f);
  c0 = fmaf(c0, y, 1.f);
  const float a = (q & 1) ? -s0 : c0, b = (q & 1) ? c0 : s0;
  c = ((q & 2) ? -a : a) * amp;
  s = ((q & 2) ? -b : b) * amp;
}

template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    r = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Vec<float, 4> {
  float4 r;
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
  }
  __device__ __forceinline__ void set(const float (&x)[4]) {
    r = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 r;
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = __bfloat162float(r); }
  __device__ __forceinline__ void set(const float (&x)[1]) { r = __float2bfloat16_rn(x[0]); }
};
template <>
struct Vec<float, 1> {
  float r;
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = r; }
  __device__ __forceinline__ void set(const float (&x)[1]) { r = x[0]; }
};

// Unit u of a row: its two V-element vectors start at p0 and p1.
struct Unit {
  int p0, p1;
  bool rot, two;
};
template <int V>
__device__ __forceinline__ Unit unit_of(const Params &p, int u) {
  Unit x;
  x.rot = u < p.nrot;
  if (x.rot) {
    x.p0 = p.rot.inter ? 2 * u * V : u * V;
    x.p1 = p.rot.inter ? x.p0 + V : x.p0 + p.rot.half;
    x.two = true;
  } else {
    x.p0 = 2 * p.rot.half + (u - p.nrot) * 2 * V;
    x.p1 = x.p0 + V;
    x.two = x.p1 < p.D;
  }
  return x;
}

template <int V>
__device__ __forceinline__ void unit_turns(const Params &p, int u, int pos, float (&c)[V],
                                           float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) turn(p.rot.freqs[u * V + i], pos, p.rot.amp, c[i], s[i]);
}

// Turns the V pairs of a unit (one rounding per product and sum, float32).
template <int V>
__device__ __forceinline__ void unit_rotate(int inter, const float (&c)[V], const float (&s)[V],
                                            float (&a)[V], float (&b)[V]) {
  if (inter && V > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {  // pair i: elements 2i, 2i + 1 of the 2V contiguous ones
      float &x = 2 * i < V ? a[(2 * i) % V] : b[(2 * i) % V];
      float &y = 2 * i + 1 < V ? a[(2 * i + 1) % V] : b[(2 * i + 1) % V];
      const float x0 = x, y0 = y;
      x = fmaf(x0, c[i], -(y0 * s[i]));
      y = fmaf(y0, c[i], x0 * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x0 = a[i], y0 = b[i];
      a[i] = fmaf(x0, c[i], -(y0 * s[i]));
      b[i] = fmaf(y0, c[i], x0 * s[i]);
    }
  }
}

// Sequence of row r: the largest b with cu[b] <= r (empty sequences before it are passed over).
__device__ __forceinline__ int seq_of_row(const int32_t *cu, int B, int r) {
  int lo = 0, hi = B;  // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Place of one row: its position and, for a paged destination, its cache row of head 0
// (block * hkv * bs + row in block); -1 where it has none.
__device__ __forceinline__ void row_place(const Params &p, int row, bool cache, int &pos,
                                          long long &slot, bool report) {
  slot = -1;
  int b;
  if (p.pos != nullptr) {
    pos = p.pos[row];
    return;
  }
  int j;
  if (p.cu != nullptr) {
    b = seq_of_row(p.cu, p.B, row);
    j = row - p.cu[b];
    // rows in front of the first or behind the last sequence belong to none
    if (j < 0 || row >= p.cu[b + 1]) {
      pos = INT_MIN;
      return;
    }
  } else {
    b = row / p.per_seq;
    j = row - b * p.per_seq;
  }
  const int L = p.ctx_len[b];
  pos = L + j + p.q_offset;
  if (!cache) return;
  const int bi = pos / p.bs;
  const int blk = L >= 0 && pos >= 0 && bi < p.mbps ? p.table[(size_t)b * p.mbps + bi] : -1;
  if (blk < 0 || blk >= p.num_blocks) {
    if (report) record_status(p.status, SD_ERR_DEVICE);
    return;
  }
  slot = (long long)blk * p.hkv * p.bs + pos % p.bs;
}

// Rows [rows_per_cta * cta, ...) of head group hg: each thread one unit of one row, the heads of
// the group in runs of HEADS whose loads are issued together.
template <typename T, int V, int HEADS>
__device__ __forceinline__ void rows_body(const Params &p, int cta, int hg) {
  __shared__ int s_pos[kMaxThreads];
  __shared__ long long s_slot[kMaxThreads];
  const int tid = threadIdx.x;
  const bool cache = p.seg[1].heads > 0;
  for (int r = tid; r < p.rows_per_cta; r += blockDim.x) {
    const int row = cta * p.rows_per_cta + r;
    int pos = INT_MIN;
    long long slot = -1;
    if (row < p.rows) row_place(p, row, cache, pos, slot, hg == 0);
    s_pos[r] = pos;
    s_slot[r] = slot;
  }
  __syncthreads();
  const int h0 = hg * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.heads_total);
  const int total = p.rows_per_cta * p.units;
  for (int w = tid; w < total; w += blockDim.x) {
    const int r = w / p.units, u = w - r * p.units;
    const int row = cta * p.rows_per_cta + r;
    if (row >= p.rows || (p.pos == nullptr && s_pos[r] == INT_MIN)) continue;
    const Unit un = unit_of<V>(p, u);
    float c[V], s[V];
    bool have = false;
    for (int h = h0; h < h1; h += HEADS) {
      Vec<T, V> v0[HEADS], v1[HEADS];
      T *dst[HEADS];
      bool rot[HEADS];
#pragma unroll
      for (int e = 0; e < HEADS; ++e) {
        dst[e] = nullptr;
        rot[e] = false;
        int g = h + e;
        if (g >= h1) continue;
        int k = 0;
        while (g >= p.seg[k].heads) g -= p.seg[k++].heads;
        const Seg &sg = p.seg[k];
        if (sg.to_cache) {
          if (s_slot[r] < 0) continue;
          dst[e] = reinterpret_cast<T *>(sg.dst) + (s_slot[r] + (long long)g * p.bs) * p.D;
        } else {
          dst[e] = reinterpret_cast<T *>(sg.dst) + row * sg.ld_dst + (long long)g * p.D;
        }
        rot[e] = sg.rotate && un.rot;
        const T *src = reinterpret_cast<const T *>(sg.src) + row * sg.ld_src + (long long)g * p.D;
        v0[e] = *reinterpret_cast<const Vec<T, V> *>(src + un.p0);
        if (un.two) v1[e] = *reinterpret_cast<const Vec<T, V> *>(src + un.p1);
      }
      if (!have && un.rot) {  // after the first loads are on their way
        unit_turns<V>(p, u, s_pos[r], c, s);
        have = true;
      }
#pragma unroll
      for (int e = 0; e < HEADS; ++e) {
        if (dst[e] == nullptr) continue;
        if (rot[e]) {
          float a[V], b[V];
          v0[e].get(a);
          v1[e].get(b);
          unit_rotate<V>(p.rot.inter, c, s, a, b);
          v0[e].set(a);
          v1[e].set(b);
        }
        *reinterpret_cast<Vec<T, V> *>(dst[e] + un.p0) = v0[e];
        if (un.two) *reinterpret_cast<Vec<T, V> *>(dst[e] + un.p1) = v1[e];
      }
    }
  }
}

// At most 128 registers: 47 us for the rows of a prompt (16384 rows, 16 heads of 256, 64 of them turned;
// 5.7 TB/s), 50 with three CTAs on an SM, 62 with four.
template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads, 2) rows_kernel(const __grid_constant__ Params p) {
  pdl_trigger();
  pdl_wait();
  rows_body<T, V, 4>(p, blockIdx.x, blockIdx.y);
}

// ------------------------------------------------------------------------- e4m3 append

// Smallest e >= kMinExp with amax <= 448 * 2^e (448 = 1.75 * 2^8).
constexpr int kMinExp = -64;
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinExp);
}

__device__ __forceinline__ float pow2i(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four floats to e4m3 bytes, nearest even, beyond the range to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Two products in one instruction.
__device__ __forceinline__ void mul2(float &x, float &y, float f) {
  asm("{.reg .b64 v, w;\n\t"
      "mov.b64 v, {%0, %1};\n\t"
      "mov.b64 w, {%2, %2};\n\t"
      "mul.rn.f32x2 v, v, w;\n\t"
      "mov.b64 {%0, %1}, v;}"
      : "+f"(x), "+f"(y)
      : "f"(f));
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t *dst, const float (&x)[V], float inv) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    float a = x[4 * i], b = x[4 * i + 1], c = x[4 * i + 2], d = x[4 * i + 3];
    mul2(a, b, inv);
    mul2(c, d, inv);
    w[i] = e4m3x4(a, b, c, d);
  }
  if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t *>(dst) = w[0];
}

// Largest finite magnitude; what is not finite does not count.
constexpr float kFinite = 3.402823466e38f;
__device__ __forceinline__ float amax_of(float m, float x) {
  const float a = fabsf(x);
  return a <= kFinite ? fmaxf(m, a) : m;
}

// Item t: the t-th slot of the blocks that receive rows.  Sequence b has the slots from
// cu[b] / bs + 2 b on, at least as many as its rows can touch blocks, so the slot's sequence
// follows from cu alone: a 32-ary search by the warp.
__device__ __forceinline__ int seq_of_item(const Params &p, int t, int &first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.B;  // the sequence is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool le = lane * step < n && p.cu[b] / p.bs + 2 * b <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = max(__popc(m) - 1, 0);  // the starts rise with b
    n = min(step, n - k * step);
    lo += k * step;
  }
  first = p.cu[lo] / p.bs + 2 * lo;
  return lo;
}

// What one call adds to one cache block: rows of a sequence from source row `row` on, to the block's
// rows from off on.
struct Piece {
  int row, at, rows, off, blk;  // at: position of the first row; rows 0: nothing to do
};

__device__ __forceinline__ Piece piece_of(const Params &p, int item) {
  Piece x{};
  int b, i, row0, n;
  if (p.cu == nullptr) {
    const int per = (p.per_seq + p.bs - 2) / p.bs + 1;  // blocks that per_seq rows can touch
    b = item / per;
    i = item - b * per;
    row0 = b * p.per_seq;
    n = p.per_seq;
  } else {
    int first;
    b = seq_of_item(p, item, first);
    i = item - first;
    row0 = p.cu[b];
    n = p.cu[b + 1] - row0;
    if (row0 < 0 || n < 0 || row0 + n > p.rows) {
      record_status(p.status, SD_ERR_DEVICE);
      return x;
    }
    if (i < 0) return x;  // a slot before the first sequence's: cu[0] >= bs
  }
  if (n == 0) return x;
  const int L = p.ctx_len[b];
  if (L < 0) {
    record_status(p.status, SD_ERR_DEVICE);
    return x;
  }
  // in the block's own rows: the call's begin at L % bs of block L / bs
  const int l0 = L % p.bs, skip = i > 0 ? i * p.bs - l0 : 0;  // rows of the call before this block
  if (skip >= n) return x;
  const int bi = L / p.bs + i;
  x.blk = bi < p.mbps ? p.table[(size_t)b * p.mbps + bi] : -1;
  if (x.blk < 0 || x.blk >= p.num_blocks) {
    record_status(p.status, SD_ERR_DEVICE);
    return x;
  }
  x.off = i > 0 ? 0 : l0;
  x.row = row0 + skip;
  x.at = L + skip;
  x.rows = min(n - skip, p.bs - x.off);
  return x;
}

constexpr int kMaxHeads = 8;  // heads of a CTA

// One CTA: one piece, for up to heads_per_quant heads of K or V.  U units of a head stay in the
// thread's registers from the maximum to the rounding; U == 0 (more than 2 units a thread) goes over
// the rows twice.
template <typename T, int V, int U>
__device__ __forceinline__ void quant_body(const Params &p, int cta) {
  constexpr int Q = V / 4;  // float4 quads of a unit's cosines
  extern __shared__ float4 s_turns[];  // [unit of the thread][cosines, sines][Q][thread]
  __shared__ unsigned s_max[2][kQuantThreads / 32];
  __shared__ unsigned s_most[kMaxHeads];
  __shared__ float s_old[kMaxHeads];
  const int per_item = 2 * p.chunks;
  const int item = cta / per_item, part = cta % per_item;
  const bool is_v = part >= p.chunks;
  const int h0 = (is_v ? part - p.chunks : part) * p.heads_per_quant;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;

  const Piece pc = piece_of(p, item);
  const int rows = pc.rows, off = pc.off, at = pc.at;
  if (rows == 0) return;
  const int64_t ld = is_v ? p.ld_v : p.ld_k;
  const T *src = reinterpret_cast<const T *>(is_v ? p.v_new : p.k_new) +
                 pc.row * ld + (long long)h0 * p.D;
  uint8_t *codes = (is_v ? p.vc : p.kc) + ((size_t)pc.blk * p.hkv + h0) * p.bs * p.D;
  float *scale = (is_v ? p.vs : p.ks) + (size_t)pc.blk * p.hkv + h0;
  const int heads = min(p.heads_per_quant, p.hkv - h0);
  const bool rot = !is_v && p.rot.freqs != nullptr;

  const int lg = 31 - __clz(p.units);  // head sizes make units a power of two
  // place of unit w: source and destination of head 0, distance of its second vector
  struct Place {
    const T *src;
    uint8_t *dst;
    int second;
    bool rot;
  };
  // w's place; its cosines and sines go to slot k of the thread
  auto place = [&](int w, int k) {
    const int r = w >> lg, u = w & (p.units - 1);
    const Unit un = unit_of<V>(p, u);
    Place x;
    x.src = src + r * ld + un.p0;
    x.dst = codes + (size_t)(off + r) * p.D + un.p0;
    x.second = un.p1 - un.p0;
    x.rot = rot && un.rot;
    if (x.rot) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        float c[4], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          turn(p.rot.freqs[u * V + 4 * q + e], at + r, p.rot.amp, c[e], s[e]);
        float4 *to = s_turns + (2 * k * Q + q) * nt + tid;
        to[0] = make_float4(c[0], c[1], c[2], c[3]);
        to[Q * nt] = make_float4(s[0], s[1], s[2], s[3]);
      }
    }
    return x;
  };
  auto load = [&](const Place &x, int h, Vec<T, V> &v0, Vec<T, V> &v1) {
    const T *y = x.src + h * p.D;
    v0 = *reinterpret_cast<const Vec<T, V> *>(y);
    v1 = *reinterpret_cast<const Vec<T, V> *>(y + x.second);
  };
  // the unit's values, turned
  auto values = [&](const Place &x, int k, const Vec<T, V> &v0, const Vec<T, V> &v1, float (&a)[V],
                    float (&bb)[V]) {
    v0.get(a);
    v1.get(bb);
    if (x.rot) {
      float c[V], s[V];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 *from = s_turns + (2 * k * Q + q) * nt + tid;
        const float4 y = from[0], z = from[Q * nt];
        c[4 * q] = y.x, c[4 * q + 1] = y.y, c[4 * q + 2] = y.z, c[4 * q + 3] = y.w;
        s[4 * q] = z.x, s[4 * q + 1] = z.y, s[4 * q + 2] = z.z, s[4 * q + 3] = z.w;
      }
      unit_rotate<V>(p.rot.inter, c, s, a, bb);
    }
  };
  // largest finite magnitude: the plain maximum, and again with care where an infinity is in it
  auto largest = [&](const float (&a)[V], const float (&bb)[V]) {
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) mx = fmaxf(mx, fmaxf(fabsf(a[e]), fabsf(bb[e])));
    if (__builtin_expect(mx > kFinite, 0)) {
      mx = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) mx = amax_of(amax_of(mx, a[e]), bb[e]);
    }
    return mx;
  };
  auto put = [&](const Place &x, int h, float inv, const float (&a)[V], const float (&bb)[V]) {
    uint8_t *y = x.dst + (size_t)h * p.bs * p.D;
    store_codes<V>(y, a, inv);
    store_codes<V>(y + x.second, bb, inv);
  };
  // The CTA's maximum of head h; floats that are not negative rise with their bits.
  auto join = [&](int h, float m) {
    const unsigned mw = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (lane == 0) s_max[h & 1][warp] = mw;
    __syncthreads();
    const unsigned all = lane < nt / 32 ? s_max[h & 1][lane] : 0u;
    return __uint_as_float(__reduce_max_sync(0xffffffffu, all));
  };
  // Settles the scale of head h, whose new rows have the maximum m; returns its inverse.
  auto settle = [&](int h, float m) {
    float sc = pow2i(scale_exp(m));
    const float old = s_old[h];
    if (off > 0) {
      if (!(old > 0.f && old < INFINITY)) {
        if (tid == 0) record_status(p.status, SD_ERR_DEVICE);
      } else if (old >= sc) {
        sc = old;
      } else {
        // the block's live rows move to the larger scale: a power of two, so only codes that
        // become subnormal are rounded again
        const float f = old / sc;
        uint8_t *x = codes + (size_t)h * p.bs * p.D;
        for (int w = tid; w < off * p.D / 4; w += nt) {
          const uint32_t q = reinterpret_cast<const uint32_t *>(x)[w];
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_fp8_e4m3 z;
            z.__x = (__nv_fp8_storage_t)(q >> (8 * e));
            y[e] = (float)z;
          }
          reinterpret_cast<uint32_t *>(x)[w] = e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
        }
      }
    }
    if (tid == 0) scale[h] = sc;  // read by all before the first barrier
    // exact for the powers of two that this call chooses: 2^-e by its exponent
    return off == 0 ? __uint_as_float(0x7f000000u - __float_as_uint(sc)) : 1.f / sc;
  };

  // a block is begun by the call that writes its first row
  if (tid < heads) s_old[tid] = off > 0 ? scale[tid] : 0.f;
  const int total = rows * p.units;
  if constexpr (U > 0) {
    Place x[U];
    Vec<T, V> v0[U], v1[U];
    const int mine = total - tid;  // unit k is this thread's if k nt < mine
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (k * nt < mine) {
        x[k] = place(tid + k * nt, k);
        load(x[k], 0, v0[k], v1[k]);
      }
    __syncthreads();
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      float a[U][V], bb[U][V], m = 0.f;
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k * nt < mine) {
          values(x[k], k, v0[k], v1[k], a[k], bb[k]);
          m = fmaxf(m, largest(a[k], bb[k]));
          if (h + 1 < heads) load(x[k], h + 1, v0[k], v1[k]);
        }
      const float inv = settle(h, join(h, m));
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k * nt < mine) put(x[k], h, inv, a[k], bb[k]);
    }
  } else {
    if (tid < heads) s_most[tid] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
#pragma unroll 1
      for (int w = tid; w - lane < total; w += nt) {  // a warp stays together
        Place x{};
        if (w < total) x = place(w, 0);
#pragma unroll 1
        for (int h = 0; h < heads; ++h) {
          float a[V], bb[V], m = 0.f;
          if (w < total) {
            Vec<T, V> v0, v1;
            load(x, h, v0, v1);
            values(x, 0, v0, v1, a, bb);
            if (step == 0) m = largest(a, bb);
            else put(x, h, __uint_as_float(s_most[h]), a, bb);
          }
          if (step == 0) {
            const unsigned mw = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
            if (lane == 0) atomicMax(&s_most[h], mw);
          }
        }
      }
      if (step == 1) break;
#pragma unroll 1
      for (int h = 0; h < heads; ++h) {
        __syncthreads();
        const float inv = settle(h, __uint_as_float(s_most[h]));
        __syncthreads();
        if (tid == 0) s_most[h] = __float_as_uint(inv);  // from here on the inverse scale
      }
      __syncthreads();
    }
  }
}

// The first quant_ctas CTAs quantise K and V; the others turn the query rows.
// U <= 1 leaves two CTAs of 512 threads on an SM: 57 us for the prompts that two units a thread, 256
// threads and three CTAs took 59 for; two units a thread serve blocks of twice the size.
template <typename T, int V, int U>
__global__ void __launch_bounds__(kQuantThreads, U <= 1 ? 2 : 1)
    quant_kernel(const __grid_constant__ Params p) {
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < p.quant_ctas) {
    quant_body<T, V, U>(p, blockIdx.x);
  } else {
    const int groups = (p.heads_total + p.heads_per_cta - 1) / p.heads_per_cta;
    const int q = blockIdx.x - p.quant_ctas;
    rows_body<T, V, 2>(p, q / groups, q % groups);
  }
}

// Frequencies of the rotating pairs as 64-bit fractions of a turn.
__global__ void freqs_kernel(int half, double base, int scaling, double factor, double orig_ctx,
                             double beta_fast, double beta_slow, unsigned long long *out) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= half) return;
  double turns = pow(base, -(double)i / half) * 0.15915494309189533577;  // / (2 pi)
  if (scaling == SD_ROPE_LINEAR) {
    turns /= factor;
  } else if (scaling == SD_ROPE_BY_PARTS) {
    const double g = fmin(1.0, fmax(0.0, (orig_ctx * turns - beta_slow) / (beta_fast - beta_slow)));
    turns = turns * (g + (1.0 - g) / factor);
  }
  out[i] = __double2ull_rn(turns * 18446744073709551616.0);
}

// ------------------------------------------------------------------------------- host side

static bool rotary_ok(const sd_rotary *r, int head_dim) {
  return r->freqs != nullptr && r->rot_dim >= 2 && r->rot_dim % 2 == 0 &&
         r->rot_dim <= head_dim && (r->layout == SD_ROPE_HALF || r->layout == SD_ROPE_INTERLEAVED) &&
         r->amplitude == r->amplitude;
}

// 16-byte vectors fit the pairs and what lies behind them.
static bool vector_pairs(const Rot &rot, int D, int V) {
  if (D % V) return false;
  if (rot.freqs == nullptr) return true;
  return rot.inter ? (2 * rot.half) % (2 * V) == 0 : rot.half % V == 0;
}

static void set_units(Params &p, int V) {
  p.nrot = p.rot.freqs ? p.rot.half / V : 0;
  const int rest = p.D - (p.rot.freqs ? 2 * p.rot.half : 0);
  p.units = p.nrot + (rest + 2 * V - 1) / (2 * V);
}

// Threads, rows and heads of a CTA.  A thread takes up to 8 heads of its unit (the sines are
// shared, two runs of loads); with few rows the heads are spread over more CTAs until the threads
// fill the SMs once.
static void set_rows_grid(Params &p, int &threads, int &ctas, int &groups) {
  threads = std::min(kMaxThreads, ((p.units + 31) / 32) * 32);
  if (p.units < 128) threads = 128;
  p.rows_per_cta = std::max(1, std::min(threads / p.units, kMaxThreads));
  ctas = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
  int per = 8;
  const long long fill = (long long)std::max(sm_count(), 1) * 2;
  while (per > 1 && (long long)ctas * ((p.heads_total + per - 1) / per) < fill) per /= 2;
  p.heads_per_cta = per;
  groups = (p.heads_total + per - 1) / per;
}

template <typename T, int V>
static sd_status launch_rows(Params &p, cudaStream_t st) {
  set_units(p, V);
  int threads, ctas, groups;
  set_rows_grid(p, threads, ctas, groups);
  if (groups > 65535) return SD_ERR_UNSUPPORTED;
  return cuda_status(launch(rows_kernel<T, V>, dim3(ctas, groups), dim3(threads), 0, st, p));
}

static sd_status launch_rows_typed(Params &p, sd_dtype dt, bool vec, cudaStream_t st) {
  if (dt == SD_BF16)
    return vec ? launch_rows<__nv_bfloat16, 8>(p, st) : launch_rows<__nv_bfloat16, 1>(p, st);
  return vec ? launch_rows<float, 4>(p, st) : launch_rows<float, 1>(p, st);
}

template <typename T, int V, int U>
static sd_status launch_quant_units(const Params &p, int ctas, int threads, cudaStream_t st) {
  const int smem = std::max(U, 1) * threads * V * 8;  // 64 KB at most
  cudaError_t e = cudaSuccess;
  if (U > 1)  // above the 48 KB that every kernel has
    e = cudaFuncSetAttribute(quant_kernel<T, V, U>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             U * kQuantThreads * V * 8);
  if (e == cudaSuccess)
    e = launch(quant_kernel<T, V, U>, dim3(ctas), dim3(threads), smem, st, p);
  return cuda_status(e);
}

// A CTA takes up to eight heads of K or V (they share the turns), fewer where that leaves SMs idle.
template <typename T, int V>
static sd_status launch_quant(Params &p, int max_rows, cudaStream_t st) {
  set_units(p, V);
  const long long units = (long long)max_rows * p.units;
  int threads = (int)std::min<long long>(kQuantThreads, (units + 31) / 32 * 32);
  const int sms = std::max(sm_count(), 1);
  int per = std::min(p.hkv, kMaxHeads);
  while (per > 1 && (long long)p.items * 2 * ((p.hkv + per - 1) / per) < 2 * sms)
    per = (per + 1) / 2;
  p.heads_per_quant = per;
  p.chunks = (p.hkv + per - 1) / per;
  const long long quant = (long long)p.items * 2 * p.chunks;
  long long extra = 0;
  if (p.seg[0].heads > 0) {
    int rt, ctas, groups;
    set_rows_grid(p, rt, ctas, groups);
    threads = std::max(threads, rt);
    p.rows_per_cta = std::max(1, std::min(threads / p.units, kMaxThreads));
    ctas = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    extra = (long long)ctas * groups;
  }
  if (quant + extra > 0x7fffffffll) return SD_ERR_UNSUPPORTED;
  p.quant_ctas = (int)quant;
  const int ctas = (int)(quant + extra);
  if (units <= threads) return launch_quant_units<T, V, 1>(p, ctas, threads, st);
  if (units <= 2 * threads) return launch_quant_units<T, V, 2>(p, ctas, threads, st);
  return launch_quant_units<T, V, 0>(p, ctas, threads, st);
}

static Rot make_rot(const sd_rotary *r) {
  Rot x{};
  if (r != nullptr) {
    x.freqs = reinterpret_cast<const unsigned long long *>(r->freqs);
    x.half = r->rot_dim / 2;
    x.inter = r->layout == SD_ROPE_INTERLEAVED;
    x.amp = r->amplitude;
  }
  return x;
}

static size_t esize(sd_dtype t) { return t == SD_F32 ? 4 : t == SD_BF16 ? 2 : 1; }

static sd_status run_append(const sd_append_desc *d, const sd_rotary *rot, const void *k_new,
                            const void *v_new, const void *q, void *k_cache, void *v_cache,
                            float *k_scale, float *v_scale, const int32_t *table,
                            const int32_t *ctx_len, const int32_t *cu, void *q_out,
                            cudaStream_t st) {
  if (!d) return SD_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_rows < 0 || d->h_q < 0 || d->h_kv < 1 || d->head_dim < 1 ||
      d->block_size < 1 || d->max_blocks_per_seq < 1 || d->num_blocks < 1)
    return SD_ERR_INVALID_ARG;
  if (d->dtype != SD_F32 && d->dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (d->cache_dtype != d->dtype && d->cache_dtype != SD_E4M3) return SD_ERR_INVALID_ARG;
  if (cu == nullptr &&
      (d->n_new < 0 || (long long)d->n_new * d->batch != d->n_rows))
    return SD_ERR_INVALID_ARG;
  if (rot != nullptr && !rotary_ok(rot, d->head_dim)) return SD_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)d->h_kv * d->head_dim, q_row = (int64_t)d->h_q * d->head_dim;
  if (d->ld_k < kv_row || d->ld_v < kv_row) return SD_ERR_INVALID_ARG;
  if (d->h_q > 0 && (d->ld_q < q_row || d->ld_q_out < q_row)) return SD_ERR_INVALID_ARG;
  if ((long long)d->num_blocks * d->h_kv * d->block_size >= (1ll << 31)) return SD_ERR_UNSUPPORTED;
  const bool q8 = d->cache_dtype == SD_E4M3;
  const int V = d->dtype == SD_BF16 ? 8 : 4;
  Params p{};
  p.rot = make_rot(rot);
  p.D = d->head_dim;
  if (q8) {
    if (!(d->head_dim == 64 || d->head_dim == 128 || d->head_dim == 256 || d->head_dim == 512) ||
        d->block_size % 16 || (rot != nullptr && rot->rot_dim % 16))
      return SD_ERR_UNSUPPORTED;
    // a block's elements are counted in 32 bits
    if ((long long)d->block_size * d->head_dim >= (1ll << 31)) return SD_ERR_UNSUPPORTED;
  }
  if (d->n_rows > kMaxRows) return SD_ERR_UNSUPPORTED;
  if (d->n_rows == 0) return SD_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !table || !ctx_len) return SD_ERR_INVALID_ARG;
  if (d->h_q > 0 && (!q || !q_out)) return SD_ERR_INVALID_ARG;
  if (d->h_q > 0 && q == q_out && d->ld_q != d->ld_q_out) return SD_ERR_INVALID_ARG;
  bool vec = vector_pairs(p.rot, p.D, V) && d->ld_k % V == 0 && d->ld_v % V == 0 &&
             aligned16(k_new) && aligned16(v_new) && aligned16(k_cache) && aligned16(v_cache);
  if (d->h_q > 0)
    vec = vec && d->ld_q % V == 0 && d->ld_q_out % V == 0 && aligned16(q) && aligned16(q_out);
  const size_t e = esize(d->dtype);
  for (const void *x : {k_new, v_new, (const void *)(d->h_q > 0 ? q : nullptr),
                        (const void *)(d->h_q > 0 ? q_out : nullptr)})
    if (reinterpret_cast<uintptr_t>(x) % e) return SD_ERR_INVALID_ARG;
  if (!q8 && (reinterpret_cast<uintptr_t>(k_cache) % e || reinterpret_cast<uintptr_t>(v_cache) % e))
    return SD_ERR_INVALID_ARG;
  if (q8 && (!vec || !k_scale || !v_scale)) return SD_ERR_INVALID_ARG;
  p.rows = d->n_rows;
  p.B = d->batch;
  p.ctx_len = ctx_len;
  p.cu = cu;
  p.per_seq = d->n_new;
  p.table = table;
  p.hkv = d->h_kv;
  p.bs = d->block_size;
  p.mbps = d->max_blocks_per_seq;
  p.num_blocks = d->num_blocks;
  p.status = device_status_word();
  p.seg[0] = Seg{q, q_out, d->ld_q, d->ld_q_out, d->h_q, rot != nullptr, 0};
  if (!q8) {
    p.seg[1] = Seg{k_new, k_cache, d->ld_k, 0, d->h_kv, rot != nullptr, 1};
    p.seg[2] = Seg{v_new, v_cache, d->ld_v, 0, d->h_kv, 0, 1};
    p.heads_total = d->h_q + 2 * d->h_kv;
    return launch_rows_typed(p, d->dtype, vec, st);
  }
  p.heads_total = d->h_q;
  p.k_new = k_new;
  p.v_new = v_new;
  p.ld_k = d->ld_k;
  p.ld_v = d->ld_v;
  p.kc = reinterpret_cast<uint8_t *>(k_cache);
  p.vc = reinterpret_cast<uint8_t *>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  int max_rows = d->block_size;
  if (cu == nullptr) {
    const long long per = ((long long)d->n_new + d->block_size - 2) / d->block_size + 1;
    const long long items = d->batch * per;
    if (items > 0x7fffffffll) return SD_ERR_UNSUPPORTED;
    p.items = (int)items;
    max_rows = std::min(max_rows, d->n_new);
  } else {
    const long long items = (long long)d->n_rows / d->block_size + 2ll * d->batch;
    if (items > 0x7fffffffll) return SD_ERR_UNSUPPORTED;
    p.items = (int)items;
  }
  return d->dtype == SD_BF16 ? launch_quant<__nv_bfloat16, 8>(p, max_rows, st)
                             : launch_quant<float, 4>(p, max_rows, st);
}

}  // namespace app
}  // namespace sdv

extern "C" {

sd_status sd_rope_freqs(const sd_rope_freq_desc *d, uint64_t *freqs, float *amplitude,
                        sd_stream stream) {
  using namespace sdv;
  if (!d || !freqs) return SD_ERR_INVALID_ARG;
  if (d->rot_dim < 2 || d->rot_dim % 2 || !(d->base > 1.0) || d->base > 1e30)
    return SD_ERR_INVALID_ARG;
  if (d->scaling != SD_ROPE_PLAIN && d->scaling != SD_ROPE_LINEAR &&
      d->scaling != SD_ROPE_BY_PARTS)
    return SD_ERR_INVALID_ARG;
  if (d->scaling != SD_ROPE_PLAIN && !(d->factor >= 1.0 && d->factor <= 1e6))
    return SD_ERR_INVALID_ARG;
  if (d->scaling == SD_ROPE_BY_PARTS &&
      (d->orig_ctx < 1 || !(d->beta_slow >= 0.0) || !(d->beta_fast > d->beta_slow) ||
       d->beta_fast > 1e9))
    return SD_ERR_INVALID_ARG;
  if (amplitude) *amplitude = d->scaling == SD_ROPE_BY_PARTS ? (float)(0.1 * log(d->factor) + 1.0)
                                                             : 1.f;
  const int half = d->rot_dim / 2;
  return cuda_status(launch(app::freqs_kernel, dim3((half + 127) / 128), dim3(128), 0,
                            (cudaStream_t)stream, half, d->base, (int)d->scaling, d->factor,
                            (double)d->orig_ctx, d->beta_fast, d->beta_slow,
                            reinterpret_cast<unsigned long long *>(freqs)));
}

sd_status sd_rope(const sd_rope_desc *d, const sd_rotary *rot, const void *x, const int32_t *pos,
                  const int32_t *ctx_len, void *out, sd_stream stream) {
  using namespace sdv;
  if (!d || !rot) return SD_ERR_INVALID_ARG;
  if (d->rows < 0 || d->heads < 1 || d->head_dim < 1) return SD_ERR_INVALID_ARG;
  if (d->dtype != SD_F32 && d->dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (!app::rotary_ok(rot, d->head_dim)) return SD_ERR_INVALID_ARG;
  const int64_t row = (int64_t)d->heads * d->head_dim;
  if (d->ld_x < row || d->ld_out < row) return SD_ERR_INVALID_ARG;
  if (d->rows > app::kMaxRows) return SD_ERR_UNSUPPORTED;
  if (d->rows == 0) return SD_OK;
  if (!x || !out || (!pos && !ctx_len) || (!pos && d->rows_per_seq < 1)) return SD_ERR_INVALID_ARG;
  if (x == out && d->ld_x != d->ld_out) return SD_ERR_INVALID_ARG;
  const size_t e = app::esize(d->dtype);
  if (reinterpret_cast<uintptr_t>(x) % e || reinterpret_cast<uintptr_t>(out) % e)
    return SD_ERR_INVALID_ARG;
  const int V = d->dtype == SD_BF16 ? 8 : 4;
  app::Params p{};
  p.rot = app::make_rot(rot);
  p.D = d->head_dim;
  p.rows = d->rows;
  p.pos = pos;
  p.ctx_len = ctx_len;
  p.per_seq = d->rows_per_seq;
  p.q_offset = d->q_offset;
  p.seg[0] = app::Seg{x, out, d->ld_x, d->ld_out, d->heads, 1, 0};
  p.heads_total = d->heads;
  p.status = device_status_word();
  const bool vec = app::vector_pairs(p.rot, p.D, V) && d->ld_x % V == 0 && d->ld_out % V == 0 &&
                   aligned16(x) && aligned16(out);
  return app::launch_rows_typed(p, d->dtype, vec, (cudaStream_t)stream);
}

sd_status sd_append_kv(const sd_append_desc *desc, const sd_rotary *rot, const void *k_new,
                       const void *v_new, const void *q, void *k_cache, void *v_cache,
                       float *k_scale, float *v_scale, const int32_t *block_table,
                       const int32_t *ctx_len, const int32_t *cu_new, void *q_out,
                       sd_stream stream) {
  return sdv::app::run_append(desc, rot, k_new, v_new, q, k_cache, v_cache, k_scale, v_scale,
                              block_table, ctx_len, cu_new, q_out, (cudaStream_t)stream);
}

}  // extern "C"
