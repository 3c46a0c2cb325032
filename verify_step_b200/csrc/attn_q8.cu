// Verify attention and drafter cross-attention over a paged e4m3 KV cache (sm_100a).
//
// The calls of attention.cu over a cache of half the bytes (the pages: decoding is bound by the
// memory it reads, GeekNews summary of the Google blog, section "why speculative decoding"; the
// drafter shares the target's cache, section "MTP drafter internal optimisations").
//
// Mathematics.  Key p has codes k_p, v_p and scales a_p, c_p (one per cache block and kv head).
// Query q is split into two e4m3 parts, q = 2^e (q_hi + q_lo / 16): a bf16 has 8 significant bits,
// an e4m3 part 4, so the split is exact from 2^-13 of the row's largest element on (smaller ones are
// off by 2^-21 of it, half a step of the smallest low part).  So the scores
// s_p = scale 2^e a_p (k_p . q_hi + k_p . q_lo / 16) come from exact 8-bit products in float32.  The
// weight of v_p is 2^t, t = s_p log2(e) + log2(c_p); per tile of 128 keys and query row,
// w = 2^(t - max t + 8) is split the same way into w_hi + w_lo / 16: off by at most 2^-8 of it (half a
// step of each part; 2^-12 more from the f16 difference), or by 2^-22 of the tile's largest where
// that is more, which it is for weights below 2^-14 of the largest (the low part's fixed step).  A
// maximum of the tile, not a running one, keeps that range for every tile however large a weight
// another tile holds.  Tiles join in float32 registers, O <- O 2^(m - m') + O_tile 2^(max t - m').
// The denominator l sums 2^(s_p log2(e)), without c_p, so it has a maximum (a frame F) of its own,
// kept by thread: in the weights' frame a key of scale 0 would vanish from it, and scales far apart
// would leave float32's range.  The output is 2^(m - F) O / l.
//
// Bound by HBM: 2 D bytes a key and kv head are read once; 4 G n_q D flops.  Both products have
// the streamed operand as the tensor core's 128-row side, read from shared memory where TMA put
// it, so no code is ever converted or moved:
//   S^T[128 keys x 2R] = K[128 x D] Q^T     K-major A; the columns are R rows' hi and lo parts
//   O^T[D x 2R]        = V^T[D x 128] P^T   V as an MN-major A, one 128-column chunk at a time
// with tcgen05 (kind::f8f6f4) into tensor memory.  Roles of a persistent CTA, one on each SM: a warp
// for the copies (one ring of 128-key K and V tiles, TMA boxes of one cache block, and the tiles'
// scales), one that issues the scores' products, one that issues the outputs' and clears V rows that
// not every query attends to, one that splits the next item's queries; a softmax warpgroup for
// every eight rows (thread = key) and one to four that join the output tiles (thread = output
// column).  Scores run two tiles ahead of the outputs.  The flattened (sequence, kv head, tile) list is
// split evenly over the CTAs, so lengths need not be alike; shared items leave (o, m, F, l) partials
// that a second kernel joins in CTA order.
//
// Measured (floor at the copy rate of 6.54 TB/s): 8 sequences of 16384 keys, 4 kv heads of 512, one query
// row a head 87 us (82), three 94 us (82); 64 ragged sequences of up to 16384 keys at D 256 177 to 187
// us (146); one window of 514 keys, 2 kv heads of 256, 13.5 us, all latency.  At D 512 HBM bounds it.
// Below, the copy warp does: looking up and issuing the boxes of 128 keys takes it 1.4 us at pages of 16
// rows whatever D is (D 128 at 16 x 16384 keys: 2.7 to 3.0 TB/s).  Code is kept short in every role (eight
// rows a thread, loops): they share the instruction cache, and unrolling made them slower.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "host.cuh"

namespace sdv {
namespace q8 {

constexpr int kTile = 128;  // keys
constexpr int kScaleRing = 8;
// Score tiles computed ahead of the output products: V of a tile is then loaded when its weights
// are nearly done, so it does not hold a ring slot through the softmax.
constexpr int kAhead = 2;
constexpr float kNone = -1e30f;  // maximum of no scores

struct Params {
  int B, n_q, Hq, Hkv, G, D, bs, mbps, num_blocks, window, M;
  int is_draft, q_offset;
  int bk, box_bytes;  // keys and bytes of one TMA box
  int span;           // positions of a table's row, short of 2^31 by a tile and a query's rows
  int row_groups;     // 8-row groups of a cache
  int R, RG;          // row groups of an item, rows of a group
  int P;              // CTAs of one row group
  float scale_log2;
  const __nv_bfloat16 *q;
  const float *ks, *vs;
  const int32_t *table, *ctx_len, *q_pos;
  __nv_bfloat16 *out;
  float *ws_o;   // [slots][R * RG][D]
  float4 *ws_ml;  // [slots][R * RG]: frame of o, frame of l, l, -
  int4 *ws_rec;  // [P] items to join
  int *status;
};

// Keys [lo, hi] that some query of sequence b reads; tiles start at p0 (a multiple of bk).
struct Seq {
  int t0, lo, hi, p0, n;  // t0: position of query 0 (the drafter's one query)
};

__device__ __forceinline__ Seq seq_of(const Params &p, int b, bool report) {
  Seq s{0, 0, -1, 0, 0};
  const int L = p.ctx_len[b];
  s.t0 = p.is_draft ? (p.q_pos ? p.q_pos[b] : L + p.q_offset) : L;
  if (L < 0 || s.t0 < 0) {
    if (report) record_status(p.status, SD_ERR_DEVICE);
    return s;
  }
  const int last = p.is_draft ? min(s.t0, L - 1) : L;  // the verify rows' own keys follow it
  const int more = p.is_draft ? 0 : p.n_q - 1;
  const int lo = p.window > 0 ? max(0, s.t0 - p.window + 1) : 0;
  if (p.is_draft && last < lo) return s;
  if (last >= p.span - more) {
    if (report) record_status(p.status, SD_ERR_DEVICE);
    return s;
  }
  const int hi = last + more;
  s.lo = lo;
  s.hi = hi;
  s.p0 = lo / p.bk * p.bk;
  s.n = (hi - s.p0) / kTile + 1;
  return s;
}

// Last key of query j (row j * G + h) and its first one.
__device__ __forceinline__ int row_hi(const Params &p, const Seq &s, int j) {
  return p.is_draft ? s.hi : s.t0 + j;
}
__device__ __forceinline__ int row_lo(const Params &p, const Seq &s, int j) {
  const int t = s.t0 + j;
  return p.window > 0 ? max(0, t - p.window + 1) : 0;
}

// First tile of share c of P (P <= total): the shares differ by at most one tile.
__host__ __device__ __forceinline__ unsigned share(unsigned total, unsigned c, unsigned P) {
  return total / P * c + min(total % P, c);
}
// The share that holds tile x.
__device__ __forceinline__ unsigned share_of(unsigned total, unsigned x, unsigned P) {
  const unsigned q = total / P, r = total % P;
  return x < (q + 1) * r ? x / (q + 1) : r + (x - (q + 1) * r) / q;
}

// A CTA's share of the flattened list: where it begins.
struct Start {
  int b, g, tau;
  int left;  // tiles
};

// Tiles of all items (one warp).
__device__ __forceinline__ unsigned total_tiles(const Params &p, int lane, bool report) {
  unsigned total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const unsigned n = b0 + lane < p.B ? seq_of(p, b0 + lane, report).n : 0;
    total += __reduce_add_sync(0xffffffffu, n) * p.Hkv;
  }
  return total;
}
// Item and tile of place ``at`` of the flattened list (one warp; at < total).
__device__ __forceinline__ Start locate(const Params &p, unsigned at, int lane) {
  unsigned pre = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const unsigned n = b0 + lane < p.B ? seq_of(p, b0 + lane, false).n : 0;
    unsigned v = n * p.Hkv;
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const unsigned m = __ballot_sync(0xffffffffu, at < pre + v);
    if (m) {
      const int src = __ffs(m) - 1;
      const unsigned off = at - pre - __shfl_sync(0xffffffffu, v - n * p.Hkv, src);
      const unsigned nn = __shfl_sync(0xffffffffu, n, src);
      return Start{b0 + src, (int)(off / nn), (int)(off % nn), 0};
    }
    pre += __shfl_sync(0xffffffffu, v, 31);
  }
  return Start{0, 0, 0, 0};
}

// Walks the tiles of a CTA; every role walks the same ones.
struct Walk {
  int b, g, tau, left;
  Seq s;
  __device__ __forceinline__ void begin(const Params &p, const Start &st) {
    b = st.b;
    g = st.g;
    tau = st.tau;
    left = st.left;
    if (left > 0) s = seq_of(p, b, false);
  }
  __device__ __forceinline__ bool first(const Start &st) const {
    return tau == 0 || left == st.left;
  }
  __device__ __forceinline__ bool last() const { return left == 1 || tau == s.n - 1; }
  __device__ __forceinline__ int pos() const { return s.p0 + tau * kTile; }
  __device__ __forceinline__ void next(const Params &p) { advance(p, 1); }
  // k tiles on, at most to the end of the item
  __device__ __forceinline__ void advance(const Params &p, int k) {
    left -= k;
    tau += k;
    if (tau < s.n || left == 0) return;
    tau = 0;
    if (++g < p.Hkv) return;
    g = 0;
    do {
      s = seq_of(p, ++b, false);
    } while (s.n == 0);  // left > 0: a later sequence has tiles
  }
};

// The TMA boxes of a CTA's tiles, looked up a span of 32 boxes (of one item) at a time and one span
// ahead: with a lookup per tile the table's latency and the index arithmetic took 1.9 us a tile.
// Lane l holds box l: its row in the cache seen as a matrix of rows, -1 behind the last key, -2 where
// the table names no block.  Such boxes are loaded from behind the tensor's end, which fills them
// with zeros: their keys are masked, and 0 * V stays 0 whatever the slot held before.
struct Boxes {
  Walk w;
  int row, n, k;  // tiles of the span, and the current one
  int blk2, off2, g2, n2;  // the next span: block (the load is only waited for when the span
                           // comes up), row in it (-1: none), kv head
  int lb;         // log2 of a tile's boxes
  __device__ __forceinline__ int boxes() const { return 1 << lb; }
  __device__ __forceinline__ int box(int lane) const { return lane & (boxes() - 1); }
  __device__ __forceinline__ bool turn(int lane) const { return lane >> lb == k; }
  __device__ __forceinline__ void fetch(const Params &p, int lane) {
    n2 = 0;
    if (w.left == 0) return;
    n2 = min(min(32 >> lb, w.s.n - w.tau), w.left);
    const int pk = w.pos() + lane * p.bk;
    off2 = -1;
    g2 = w.g;
    if (lane < n2 << lb && pk <= w.s.hi) {
      const int bi = pk / p.bs;
      off2 = pk - bi * p.bs;
      blk2 = __ldg(p.table + (size_t)w.b * p.mbps + bi);
    }
    w.advance(p, n2);
  }
  __device__ __forceinline__ void begin(const Params &p, const Walk &at) {
    w = at;
    lb = 31 - __clz(kTile / p.bk);
    n = k = n2 = 0;
    off2 = -1;
  }
  // To the next tile; there is one.
  __device__ __forceinline__ void next(const Params &p, int lane) {
    if (++k < n) return;
    do {  // twice at the beginning
      row = off2 < 0 ? -1
            : blk2 >= 0 && blk2 < p.num_blocks ? (blk2 * p.Hkv + g2) * p.bs + off2 : -2;
      n = n2;
      k = 0;
      fetch(p, lane);
    } while (n == 0);
  }
};

template <int D_, int NR_>
struct Cfg {
  static constexpr int D = D_, NR = NR_, N2 = 2 * NR_;
  static constexpr int MT = D >= 128 ? D / 128 : 1;   // 128-column chunks of the output
  static constexpr int RB = D >= 128 ? 128 : 64;      // bytes of a swizzled row
  static constexpr int CH = D / RB;                   // chunks of a row
  // Eight rows a softmax warpgroup and at most 48 accumulators a joining thread: the code of a
  // role is short (the instruction cache of a GPC is shared by its SMs: with 16 rows a thread the
  // tile time differed by 1.3x between GPCs of 16 and 20 SMs).  With more threads than that leaves
  // registers for, some spill: at D 512 from 16 rows on (<512, 24>: 340 bytes stored), at D 256 from
  // 24, below with 32.
  static constexpr int SG = NR / 8;
  static constexpr int MJ = MT * NR <= 48 ? MT : MT / 2 * NR <= 48 ? MT / 2 : 1;
  static constexpr int JG = MT / MJ;                  // joining warpgroups, MJ chunks each
  static constexpr int THREADS = 128 * (1 + SG + JG);
  static constexpr int SLOT = kTile * D;
  static constexpr int NQ = D == 512 ? 1 : 2;         // query buffers
  static constexpr int NP = D == 512 && NR == 24 ? 1 : 2;  // weight buffers
  static constexpr int NO = D == 512 && NR == 24 ? 1 : 2;  // output tile buffers
  static constexpr int NS = kAhead + 1;               // score buffers
  static constexpr int QBYTES = N2 * D;
  static constexpr int PBYTES = N2 * kTile;
  static constexpr int S_COL = 0;
  static constexpr int O_COL = NS * N2;
  static constexpr int COLS = NS * N2 + NO * MT * N2;
  static constexpr uint32_t TMEM = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128
                                   : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512, "tensor memory");
  struct Small {
    alignas(16) float scales[kScaleRing][2][8];  // K's and V's of each box of a tile; -1: no such box
    alignas(16) float red[SG][2][4][8];
    alignas(16) float frame[SG][4][8];    // of the warps' l at an item's end
    alignas(16) float tm[4][NR];          // tile maxima for the joining warps
    alignas(16) float beta[4 * JG][NR];   // their factors of a tile, by warp
    float2 ml[2][NR];         // frame F and l of an item
    float qs[2][NR];          // 2^e scale of the query rows
    uint32_t nan_rows[2];     // of an item
    alignas(16) int rowj[NR];             // query position of a row (row / G)
    uint64_t kfull[8], vfull[8], empty[8];
    uint64_t sc_full[kScaleRing];
    uint64_t qfull[2], qempty[2], sfull[NS], sempty[NS], pfull[2], pempty[2], ofull[2], oempty[2],
        lfull[2], lempty[2], tmfull[4], drain[2];
    Start start;
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr int FIXED = 1024 + NQ * QBYTES + NP * PBYTES + (int)sizeof(Small);
  static constexpr int FIT = (232448 - FIXED) / SLOT;
  static constexpr int SLOTS = FIT < 8 ? FIT : 8;  // tiles of K or V in the ring
  static_assert(SLOTS >= 3, "shared memory");
  static constexpr size_t SMEM = FIXED + (size_t)SLOTS * SLOT;
};

// 4D box: row bytes, 8 rows, chunks, row groups.
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %3, %3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void cp_async_4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
// Arrives on bar when this thread's cp.async copies so far have landed (counted in its init).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// D[tmem] (+)= A B^T, 8-bit floats, float32 accumulator.  The whole warp calls it and one elected lane
// issues: with warp-uniform operands and control flow the descriptors stay in uniform registers
// (issued from inside a one-lane branch a product took 70 ns to issue, more than to compute).
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// umma_commit by the lane that issues for the warp.
__device__ __forceinline__ void warp_commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptor: rows of RB = 128 or 64 bytes with the swizzle of that width,
// 8-row groups sbo bytes apart.  K-major operands have one swizzled row per M/N index (the leading
// offset is unused); MN-major ones one per K index, RB bytes of M, and lbo bytes to the next RB.
// RB = 0, MN-major without swizzle: 16 bytes of M/N a K index, 8 K indexes in 128 bytes; the next 8
// lbo, the next 16 of M/N sbo bytes further.
template <int RB>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t sbo, uint32_t lbo16) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)lbo16 << 16) |
         ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)(RB == 128 ? 2 : RB == 64 ? 4 : 0) << 61);
}

// kind::f8f6f4, e4m3 x e4m3 -> float32; a_mn, b_mn: the operand is MN-major (bits 15 and 16).
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Two floats to two e4m3 bytes (first one low), nearest even, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// x and y (at most 448) as hi + lo / 16, both parts e4m3 (two bytes each).  What the high parts leave
// is taken in f16: its 11 bits round x by 2^-12 of it, far below the low part's step.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  uint16_t l;
  hi = e4m3x2(x, y);
  asm("{\n\t.reg .b32 a, h;\n\t"
      "cvt.rn.f16x2.f32 a, %3, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %1;\n\t"
      "sub.f16x2 a, a, h;\n\t"
      "mul.f16x2 a, a, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, a;\n\t}"
      : "=h"(l)
      : "h"((uint16_t)hi), "f"(x), "f"(y), "r"(0x4c004c00u));  // 16, 16
  lo = l;
}

// Maxima over the warp of eight values a lane: each step halves the rows a lane still holds, so
// nine shuffles do for eight rows; lane l returns row l / 4.
__device__ __forceinline__ float warp_max8(const float (&t)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool up = lane & 16;
    a[k] = fmaxf(up ? t[4 + k] : t[k], __shfl_xor_sync(0xffffffffu, up ? t[k] : t[4 + k], 16));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool up = lane & 8;
    b[k] = fmaxf(up ? a[2 + k] : a[k], __shfl_xor_sync(0xffffffffu, up ? a[k] : a[2 + k], 8));
  }
  const bool up = lane & 4;
  float c = fmaxf(up ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4));
  c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 2));
  return fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// Sums in the same way.
__device__ __forceinline__ float warp_sum8(const float (&t)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool up = lane & 16;
    a[k] = (up ? t[4 + k] : t[k]) + __shfl_xor_sync(0xffffffffu, up ? t[k] : t[4 + k], 16);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool up = lane & 8;
    b[k] = (up ? a[2 + k] : a[k]) + __shfl_xor_sync(0xffffffffu, up ? a[k] : a[2 + k], 8);
  }
  const bool up = lane & 4;
  float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// mbar_wait with a short way through: a try suspends in the hardware for about 4 us, so a few thousand
// of them in a loop of three instructions come before the abort flag and the 2 s limit are looked at.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort) {
  unsigned long long t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, 4096;\n\t"
        "@q bra TRY;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (__builtin_expect(ok, 1)) return true;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (*abort || now - t0 > kWaitLimitNs) return false;
  }
}

// wait_for of a whole warp with one answer.  Every lane waits itself: a single polling lane saves
// nothing and costs a divergent branch and a warp barrier per wait.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

// One arrival for the warp, once all its lanes are here (predicated, no branch).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// Barrier ``id`` of ``n`` threads that also tells whether any of them failed a wait.
__device__ __forceinline__ bool barrier_or(int id, int n, bool fail) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)fail), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// Byte of (row, col) in a K-major operand tile of `rows` rows stored chunk by chunk.
template <int RB>
__device__ __forceinline__ uint32_t tile_byte(int rows, int row, int col) {
  const int x = RB == 128 ? (row & 7) : ((row >> 1) & 3);
  const int chunk = col / RB, c = col % RB;
  return (uint32_t)(chunk * rows * RB + row * RB + (((c >> 4) ^ x) << 4) + (c & 15));
}

// Whether some row of the group (queries j_first .. j_last) does not attend to some key of the tile.
__device__ __forceinline__ bool is_edge(const Params &p, const Walk &w, int j_first, int j_last) {
  return w.pos() < row_lo(p, w.s, j_last) || w.pos() + kTile - 1 > row_hi(p, w.s, j_first);
}

// V rows that no query attends to may hold any codes, and 0 * NaN is NaN: they are cleared.  A NaN that
// not every row of the group attends to is cleared too, and the rows that see it are returned (their
// outputs become NaN as a whole; a NaN that every row of the group attends to takes its column).  One
// warp, a row (or the part of one that a lane's 16 bytes each cover) at a time.
template <int D, int NR>
__device__ __forceinline__ uint32_t clean_v(const Params &p, const Walk &w, uint8_t *tile,
                                            const int *rowj, int lane) {
  constexpr int RB = D >= 128 ? 128 : 64;
  const int p0 = w.pos(), j_first = rowj[0], j_last = rowj[NR - 1];
  uint32_t rows = 0;
  // keys [0, before) and [after, end): not every row attends to them; behind end are zeros already
  const int before = min(max(row_lo(p, w.s, j_last) - p0, 0), kTile);
  const int after = max(row_hi(p, w.s, j_first) + 1 - p0, before);
  const int end = min(w.s.p0 + ((w.s.hi - w.s.p0) / p.bk + 1) * p.bk - p0, kTile);
#pragma unroll 1
  for (int k = 0; k < before + max(end - after, 0); ++k) {
    const int key = k < before ? k : after + k - before, pos = p0 + key;
    const bool inside = pos >= w.s.lo && pos <= w.s.hi;
    uint8_t *v = tile + (key >> 3) * (8 * D) + (key & 7) * RB;
    bool any = false;
    for (int u = 16 * lane; u < D; u += 512) {
      uint4 *x = reinterpret_cast<uint4 *>(v + u / RB * (8 * RB) + u % RB);
      if (!inside) {
        *x = make_uint4(0, 0, 0, 0);
      } else {
        // bytes 0x7f and 0xff: bit 7 of each such byte
        auto nan = [](uint32_t z) { return ((z & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
        auto clear = [&](uint32_t z) { return z & ~((nan(z) >> 7) * 0xffu); };
        const uint4 y = *x;
        if (nan(y.x) | nan(y.y) | nan(y.z) | nan(y.w)) {
          any = true;
          *x = make_uint4(clear(y.x), clear(y.y), clear(y.z), clear(y.w));
        }
      }
    }
    if (__any_sync(0xffffffffu, any)) {
      const int j = lane < NR ? rowj[lane] : 0;
      rows |= __ballot_sync(0xffffffffu,
                            lane < NR && pos >= row_lo(p, w.s, j) && pos <= row_hi(p, w.s, j));
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  return rows;
}

// What an output sum in frame 2^m is multiplied by, its denominator l in frame 2^f: 2^(m - f) / l, in two
// factors that each stay in float32's range; 0 where there is no key.
__device__ __forceinline__ float joined_scale(float m, float f, float l) {
  const float h = ex2_approx(0.5f * (m - f));
  return l != 0.f ? h * (h / l) : 0.f;
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg<D, NR>::THREADS, 1)
    attn_q8_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
  using C = Cfg<D, NR>;
  constexpr int N2 = C::N2, MT = C::MT, RB = C::RB, SLOTS = C::SLOTS, NQ = C::NQ, NP = C::NP,
                NO = C::NO, NS = C::NS, SG = C::SG, MJ = C::MJ;
  extern __shared__ uint8_t smem_raw[];
  // aligned by pointer arithmetic, so that the compiler still knows it for shared memory (through an
  // integer cast every access becomes a generic one with 64-bit addresses: when this was found,
  // 64 sequences at D 256 took 252 us with them and 232 without)
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *slots = smem;
  uint8_t *qbuf = slots + (size_t)SLOTS * C::SLOT;
  uint8_t *pbuf = qbuf + NQ * C::QBYTES;
  typename C::Small &sm = *reinterpret_cast<typename C::Small *>(pbuf + NP * C::PBYTES);
  volatile int *abort_flag = &sm.abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x / p.R, rg = blockIdx.x % p.R;  // share of the list, row group
  const int row0 = rg * p.RG;
  const int rows = min(p.RG, p.M - row0);  // rows of this group
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sm.kfull[i], 1);
      mbar_init(&sm.vfull[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(&sm.sc_full[i], 8);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sempty[i], 4 * SG);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qfull[i], 1);
      mbar_init(&sm.qempty[i], 1 + 4 * SG);  // the item's last scores; its row scales are read
      mbar_init(&sm.pfull[i], 4 * SG);
      mbar_init(&sm.pempty[i], 1);
      mbar_init(&sm.ofull[i], 1);
      mbar_init(&sm.oempty[i], 4 * C::JG);
      mbar_init(&sm.lfull[i], 4 * SG + 1);
      mbar_init(&sm.lempty[i], 4 * C::JG);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.tmfull[i], SG);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem, C::TMEM);
    tmem_relinquish();
  }
  if (warp == 2 && lane < NR) sm.rowj[lane] = (row0 + min(lane, rows - 1)) / p.G;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    // where this CTA's share of the T tiles begins
    const unsigned total = total_tiles(p, lane, blockIdx.x == 0);
    const unsigned P = min((unsigned)p.P, total);
    Start st{0, 0, 0, 0};
    if ((unsigned)cta < P) {
      const unsigned at = share(total, cta, P);
      st = locate(p, at, lane);
      st.left = (int)(share(total, cta + 1, P) - at);
    }
    if (rg == 0) {  // the item whose first border inside is this share's begin
      int last = -1;
      if (st.tau > 0) {
        const unsigned first = share(total, cta, P) - st.tau;
        if (share_of(total, first, P) + 1 == (unsigned)cta)
          last = (int)share_of(total, first + seq_of(p, st.b, false).n - 1, P);
      }
      if (lane == 0) p.ws_rec[cta] = make_int4(st.b, st.g, last, 0);
    }
    if (lane == 0) sm.start = st;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const Start st = sm.start;
  auto fail = [&]() {
    record_status(p.status, SD_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  Walk w;
  w.begin(p, st);

  // The K and V tiles share one ring, in the order K0 .. K_ahead, V0, K, V1, ... in which the products
  // need them: K_i is entry i, from the first V on 2 i - ahead, V_i entry min(i + ahead + 1, tiles) + i.
  // One warp fills it in that order.  Two warps empty it, so each has its own barrier of a slot:
  // a wait never starts more than one phase early, and the parity says which phase it is.
  if (warp == 0) {
    // -------------------------------------------------------------------- TMA
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    const uint64_t policy = l2_policy_evict_first();
    Boxes x;
    x.begin(p, w);
    int slot = 0;
    uint32_t phase = 0, k_fills = 0, v_fills = 0;  // parities of each slot's fills
    bool ok = true;
    int zs[kAhead + 1] = {};  // group coordinates of the last tiles' boxes, V's turn being later
    bool turn[kAhead + 1] = {};
    for (int i = 0; i < st.left + kAhead && ok; ++i) {
#pragma unroll
      for (int u = kAhead; u > 0; --u) {
        zs[u] = zs[u - 1];
        turn[u] = turn[u - 1];
      }
      if (i < st.left) {
        x.next(p, lane);
        turn[0] = x.turn(lane);
        zs[0] = x.row >= 0 ? x.row >> 3 : p.row_groups;
      }
#pragma unroll 1
      for (int v = i < st.left ? 0 : 1; v <= (i >= kAhead ? 1 : 0); ++v) {
        ok = warp_wait(&sm.empty[slot], phase ^ 1, abort_flag);
        if (!ok) break;
        uint64_t *full = v ? &sm.vfull[slot] : &sm.kfull[slot];
        if (lane == 0) mbar_arrive_expect_tx(full, C::SLOT);
        __syncwarp();
        if (v ? turn[kAhead] : turn[0])
          tma_load_4d(slots + (size_t)slot * C::SLOT + x.box(lane) * p.box_bytes, v ? &vmap : &kmap,
                      full, v ? zs[kAhead] : zs[0], policy);
        (v ? v_fills : k_fills) ^= 1u << slot;
        if (++slot == SLOTS) {
          slot = 0;
          phase ^= 1;
        }
        if (v == 0) {
          // The tile's scales.  Their place is free: the slot's last entry was K_{i-4} or younger (or a
          // V younger than that), whose scores needed the buffer of tile i - 7, read after its scales.
          const int r = i % kScaleRing, box = x.box(lane);
          if (turn[0]) {
            if (x.row >= 0) {
              const int at = x.row / p.bs;
              cp_async_4(&sm.scales[r][0][box], p.ks + at);
              cp_async_4(&sm.scales[r][1][box], p.vs + at);
              cp_async_arrive(&sm.sc_full[r]);
            } else {
              sm.scales[r][0][box] = -1.f;  // its keys are masked
              mbar_arrive(&sm.sc_full[r]);
              if (x.row == -2) record_status(p.status, SD_ERR_DEVICE);
            }
          }
          if (lane < 8 - x.boxes()) mbar_arrive(&sm.sc_full[r]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {
      fail();
      // copies in flight land before the CTA ends
      for (int s = 0; s < SLOTS; ++s) {
        mbar_wait_timed(&sm.kfull[s], (k_fills >> s & 1) ^ 1);
        mbar_wait_timed(&sm.vfull[s], (v_fills >> s & 1) ^ 1);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------------- score products
    constexpr uint32_t id = idesc_f8(128, N2, false, false);
    int slot = 0, buf = 0;
    uint32_t filled = 0, bphase = 0, items = 0;  // filled: parity of each slot's K fills
    bool ok = true;
    for (int i = 0; w.left > 0; ++i) {
      if (w.first(st)) {
        ok = wait_for(&sm.qfull[items % NQ], (items / NQ) & 1, abort_flag);
        ++items;
      }
      ok &= wait_for(&sm.kfull[slot], filled >> slot & 1, abort_flag);
      ok &= wait_for(&sm.sempty[buf], bphase ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t a = smem_desc<RB>(smem_u32(slots) + slot * C::SLOT, D * 8, 1);
      const uint64_t b = smem_desc<RB>(smem_u32(qbuf) + ((items - 1) % NQ) * C::QBYTES, RB * 8, 1);
#pragma unroll 1
      for (int ch = 0; ch < C::CH; ++ch)
#pragma unroll
        for (int x = 0; x < RB / 32; ++x)  // addresses in 16-byte units
          umma_f8(tmem + C::S_COL + buf * N2, a + ch * (8 * RB / 16) + 2 * x,
                  b + ch * (N2 * RB / 16) + 2 * x, id, ch + x > 0);
      warp_commit(&sm.sfull[buf]);
      warp_commit(&sm.empty[slot]);
      if (w.last()) warp_commit(&sm.qempty[(items - 1) % NQ]);
      filled ^= 1u << slot;
      slot += i < kAhead ? 1 : 2;
      if (slot >= SLOTS) slot -= SLOTS;
      if (++buf == NS) {
        buf = 0;
        bphase ^= 1;
      }
      w.next(p);
    }
    if (lane == 0 && !ok) fail();
    warp_commit(&sm.drain[0]);
    if (lane == 0 && !mbar_wait_timed(&sm.drain[0], 0)) record_status(p.status, SD_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == 2) {
    // -------------------------------------------------------------------- output products
    constexpr uint32_t id = idesc_f8(128, N2, true, true);
    int slot = min(kAhead + 1, st.left) % SLOTS;
    uint32_t filled = 0;  // parity of each slot's V fills
    uint32_t items = 0, nan_rows = 0;
    const int j_first = sm.rowj[0], j_last = sm.rowj[NR - 1];
    bool ok = true;
    for (int i = 0; i < st.left; ++i) {
      const int ob = i % NO;
      ok &= wait_for(&sm.vfull[slot], filled >> slot & 1, abort_flag);
      ok &= wait_for(&sm.pfull[i % NP], (i / NP) & 1, abort_flag);
      ok &= wait_for(&sm.oempty[ob], ((i / NO) & 1) ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (w.first(st)) nan_rows = 0;
      if (is_edge(p, w, j_first, j_last))
        nan_rows |= clean_v<D, NR>(p, w, slots + (size_t)slot * C::SLOT, sm.rowj, lane);
      tc_fence_after();
      const uint64_t a = smem_desc<RB>(smem_u32(slots) + slot * C::SLOT, D * 8, 0);
      // weights: 16 columns x 8 keys in 128 bytes, key groups 128 and column groups 2048 bytes
      // apart, no swizzle
      const uint64_t b = smem_desc<0>(smem_u32(pbuf) + (i % NP) * C::PBYTES, 2048, 128 / 16);
#pragma unroll 1
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem + C::O_COL + (ob * MT + c) * N2, a + c * (8 * RB / 16) + k * (2 * D),
                  b + k * (4 * 128 / 16), id, k > 0);
      warp_commit(&sm.ofull[ob]);
      warp_commit(&sm.empty[slot]);
      warp_commit(&sm.pempty[i % NP]);
      filled ^= 1u << slot;
      slot += i + kAhead + 1 < st.left ? 2 : 1;
      if (slot >= SLOTS) slot -= SLOTS;
      if (w.last()) {  // rows with a NaN in a V row that only some queries attend to
        const int lb = items & 1;
        ok &= wait_for(&sm.lempty[lb], ((items >> 1) & 1) ^ 1, abort_flag);
        if (lane == 0) sm.nan_rows[lb] = nan_rows;
        warp_arrive(&sm.lfull[lb]);
        ++items;
      }
      w.next(p);
    }
    if (lane == 0 && !ok) fail();
    warp_commit(&sm.drain[1]);
    if (lane == 0 && !mbar_wait_timed(&sm.drain[1], 0)) record_status(p.status, SD_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == 3) {
    // -------------------------------------------------------------------- query splitter
    // Four rows at a time: scale to at most 256, split, store swizzled.  Row r has its high part in
    // column 16 (r / 8) + r % 8, its low part 8 further.
    uint32_t items = 0;
    constexpr int E = D / 64;  // pairs a lane holds of a row: elements 2 lane + 64 e
    bool ok = true;
    while (w.left > 0 && ok) {
      const int qb = items % NQ;
      uint8_t *dst = qbuf + qb * C::QBYTES;
#pragma unroll 1
      for (int r0 = 0; r0 < NR; r0 += 4) {
        uint32_t x[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u, row = row0 + r;
          const int j = row / p.G, h = w.g * p.G + row % p.G;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(
              p.q + (((size_t)w.b * p.n_q + j) * p.Hq + h) * D);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u][e] = r < rows ? src[lane + 32 * e] : 0u;
        }
        if (r0 == 0) {  // the first loads are on their way
          ok = warp_wait(&sm.qempty[qb], ((items / NQ) & 1) ^ 1, abort_flag);
          if (!ok) break;
        }
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u;
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float a = fabsf(__uint_as_float(x[0][e] << 16));
            const float b = fabsf(__uint_as_float(x[0][e] & 0xffff0000u));
            m = fmaxf(m, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
          }
          m = redux_max(m);
          // 2^ex with m <= 256 * 2^ex; from ex = -126 on down every bf16 is a whole number of e4m3 steps
          const int ex = max((int)(__float_as_uint(m) >> 23) - 127 + 1 - 8, -126);
          const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
          if (lane == 0) sm.qs[qb][r] = __uint_as_float((uint32_t)(127 + ex) << 23);
          const int n = 16 * (r >> 3) + (r & 7);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float a = __uint_as_float(x[0][e] << 16), b = __uint_as_float(x[0][e] & 0xffff0000u);
            // an infinity becomes NaN, and with it the row's output
            if (!(fabsf(a) < INFINITY)) a = __int_as_float(0x7fc00000);
            if (!(fabsf(b) < INFINITY)) b = __int_as_float(0x7fc00000);
            uint32_t hi, lo;
            split2(a * inv, b * inv, hi, lo);
            const int col = 2 * lane + 64 * e;
            *reinterpret_cast<uint16_t *>(dst + tile_byte<RB>(N2, n, col)) = (uint16_t)hi;
            *reinterpret_cast<uint16_t *>(dst + tile_byte<RB>(N2, n + 8, col)) = (uint16_t)lo;
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[0][e] = x[1][e];
            x[1][e] = x[2][e];
            x[2][e] = x[3][e];
          }
        }
      }
      if (!ok) {
        if (lane == 0) fail();
        break;
      }
      fence_proxy_async_smem();
      warp_arrive(&sm.qfull[qb]);
      ++items;
      bool end = false;
      while (!end) {  // to the next item
        end = w.last();
        w.next(p);
      }
    }
  } else if (warp < 4 + 4 * SG) {
    // -------------------------------------------------------------------- softmax
    // Thread = key, eight rows of the warpgroup.
    const int wg = (warp - 4) >> 2;
    const int wq = warp & 3, key = wq * 32 + lane, r0 = 8 * wg;
    const int box = key >> (31 - __clz(p.bk));
    const uint32_t s_at = tmem + C::S_COL + 2 * r0 + ((uint32_t)(wq * 32) << 16);
    bool bad = false;
    // l of this thread's keys in the frame 2^F: F follows the thread's largest score in steps of 2^20 and
    // more.  kNone stands for no key (or nothing but NaN) so far.
    float l[8], F[8], qsc[8];
    uint32_t items = 0;
    const int j_first = sm.rowj[0], j_last = sm.rowj[NR - 1];
    for (int i = 0; w.left > 0; ++i, w.next(p)) {
      const int buf = i % NS, ring = i % kScaleRing;
      if (__builtin_expect(w.first(st), 0)) {
        // the splitter wrote the rows' scales before the scores were computed
        bad |= !wait_for(&sm.qfull[items % NQ], (items / NQ) & 1, abort_flag);
        ++items;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          l[r] = 0.f;
          F[r] = kNone;
          qsc[r] = sm.qs[(items - 1) % NQ][r0 + r] * p.scale_log2;
        }
        warp_arrive(&sm.qempty[(items - 1) % NQ]);
      }
      const int p0 = w.pos();
      bad |= !wait_for(&sm.sc_full[ring], (i / kScaleRing) & 1, abort_flag);
      const float ks = sm.scales[ring][0][box];
      const bool edge = is_edge(p, w, j_first, j_last);
      // scale 0: no weight; a box that is not there: zeros for keys, no V scale, no term of l either
      const float lvs = ks < 0.f ? 0.f : __log2f(sm.scales[ring][1][box]);
      const float none = ks < 0.f ? -INFINITY : 0.f;
      bad |= !wait_for(&sm.sfull[buf], (i / NS) & 1, abort_flag);
      tc_fence_after();
      float s[8];  // log2 of a key's term of l; lvs more is its weight's
      {
        uint32_t v[16];
        tmem_ld16(s_at + buf * N2, v);
        tmem_ld_wait();
        tc_fence_before();
        warp_arrive(&sm.sempty[buf]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float x = fmaf(__uint_as_float(v[8 + r]), 0.0625f, __uint_as_float(v[r]));
          // the two scales first: a tiny and a large one meet before the sum leaves float32's range
          s[r] = fmaf(x, fminf(ks * qsc[r], 3.402823466e38f), none);
        }
      }
      if (__builtin_expect(edge, 0)) {
        // the key is for queries a <= j <= b; a window near 2^31 must not wrap around
        const int a = p0 + key - (p.is_draft ? w.s.hi : w.s.t0);
        const int rel = p0 + key - w.s.t0, far = p.window - 1;
        const int b = p.window > 0 && rel <= INT_MAX - far ? rel + far : INT_MAX;
        const int4 j0 = *reinterpret_cast<const int4 *>(&sm.rowj[r0]);
        const int4 j1 = *reinterpret_cast<const int4 *>(&sm.rowj[r0 + 4]);
        const int j[8] = {j0.x, j0.y, j0.z, j0.w, j1.x, j1.y, j1.z, j1.w};
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (j[r] < a || j[r] > b) s[r] = -INFINITY;
      }
      // maxima of the tile
      {
        float t[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) t[r] = s[r] + lvs;
        const float mx = warp_max8(t);
        if ((lane & 3) == 0) sm.red[wg][i & 1][wq][lane >> 2] = mx;
      }
      bad = barrier_or(1 + wg, 128, bad);
      if (bad) break;
      float tm[8];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(&sm.red[wg][i & 1][q][h]);
          tm[h] = q ? fmaxf(tm[h], x.x) : x.x;
          tm[h + 1] = q ? fmaxf(tm[h + 1], x.y) : x.y;
          tm[h + 2] = q ? fmaxf(tm[h + 2], x.z) : x.z;
          tm[h + 3] = q ? fmaxf(tm[h + 3], x.w) : x.w;
        }
      bool grow = false;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        tm[r] = fmaxf(tm[r], kNone);
        grow |= s[r] - F[r] > 20.f;
      }
      if (__builtin_expect(grow, 0)) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (s[r] - F[r] > 20.f) {
            l[r] *= ex2_approx(F[r] - s[r]);
            F[r] = s[r];
          }
      }
      bad |= !wait_for(&sm.pempty[i % NP], ((i / NP) & 1) ^ 1, abort_flag);
      if (wq == 0) {
        // tile i - 4's maxima are read: tile i - 2's output product, which this thread has seen
        // finish, waited for tile i - 4's output to be read
        if (lane == 0) {
          float4 *x = reinterpret_cast<float4 *>(&sm.tm[i & 3][r0]);
          x[0] = make_float4(tm[0], tm[1], tm[2], tm[3]);
          x[1] = make_float4(tm[4], tm[5], tm[6], tm[7]);
        }
        warp_arrive(&sm.tmfull[i & 3]);
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        float wt[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          wt[u] = ex2_approx(s[r + u] + lvs - (tm[r + u] - 8.f));
          l[r + u] += ex2_approx(s[r + u] - F[r + u]);
        }
        split2(wt[0], wt[1], hi[r / 2], lo[r / 2]);
      }
      *reinterpret_cast<uint4 *>(pbuf + (i % NP) * C::PBYTES + wg * 2048 + key * 16) =
          make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, lo[0] | lo[1] << 16,
                     lo[2] | lo[3] << 16);
      fence_proxy_async_smem();
      warp_arrive(&sm.pfull[i % NP]);
      if (__builtin_expect(w.last(), 0)) {
        // l over the 128 keys, brought to one frame; lane r of the warpgroup's first warp hands (F, l) of
        // row r over
        const int lb = (items - 1) & 1;
        bad |= !wait_for(&sm.lempty[lb], (((items - 1) >> 1) & 1) ^ 1, abort_flag);
        float (&red)[4][8] = sm.red[wg][(i & 1) ^ 1];
        float (&frame)[4][8] = sm.frame[wg];
        const float top = warp_max8(F);  // lane l: of row l / 4
#pragma unroll
        for (int r = 0; r < 8; ++r)
          l[r] *= ex2_approx(F[r] - __shfl_sync(0xffffffffu, top, 4 * r));
        const float sum = warp_sum8(l);
        if ((lane & 3) == 0) {
          red[wq][lane >> 2] = sum;
          frame[wq][lane >> 2] = top;
        }
        bad = barrier_or(1 + wg, 128, bad);
        if (wq == 0 && lane < 8) {
          float f = frame[0][lane], x = 0.f;
#pragma unroll
          for (int q = 1; q < 4; ++q) f = fmaxf(f, frame[q][lane]);
#pragma unroll
          for (int q = 0; q < 4; ++q) x = fmaf(red[q][lane], ex2_approx(frame[q][lane] - f), x);
          sm.ml[lb][r0 + lane] = make_float2(f, x);
        }
        // the next tile writes there again: not before the first warp has read it
        bad = barrier_or(1 + wg, 128, bad);
        warp_arrive(&sm.lfull[lb]);
        if (bad) break;
      }
    }
    if (bad && lane == 0) fail();
  } else {
    // -------------------------------------------------------------------- joining warps
    const int jg = (warp - 4 - 4 * SG) >> 2, wq = warp & 3, col = wq * 32 + lane;
    const int c0 = jg * MJ;  // first chunk of the warpgroup
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    // sequences with no key at all: zero rows
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
      if (seq_of(p, b, false).n == 0)
        for (int e = tid - 128 * (1 + SG); e < p.n_q * p.Hq * (D / 8); e += 128 * C::JG)
          reinterpret_cast<uint4 *>(p.out)[(size_t)b * p.n_q * p.Hq * (D / 8) + e] =
              make_uint4(0, 0, 0, 0);
    bool ok = true;
    float acc[MJ][NR];
    float m_run = kNone;  // of row `lane`
    uint32_t items = 0;
    bool whole = false;
    for (int i = 0; w.left > 0; ++i, w.next(p)) {
      const int buf = i % NO;
      if (w.first(st)) {
        whole = w.tau == 0 && w.left >= w.s.n;
        ++items;
        m_run = kNone;
#pragma unroll
        for (int c = 0; c < MJ; ++c)
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[c][r] = 0.f;
      }
      ok = warp_wait(&sm.tmfull[i & 3], (i >> 2) & 1, abort_flag) &&
           warp_wait(&sm.ofull[buf], (i / NO) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const float tm = lane < NR ? sm.tm[i & 3][lane] : kNone;
      const float m_new = fmaxf(m_run, tm);
      const float alpha = ex2_approx(m_run - m_new);
      float *const beta = sm.beta[warp - 4 - 4 * SG];
      if (lane < NR) beta[lane] = ex2_approx(tm - m_new) * 0x1p-8f;
      m_run = m_new;
      __syncwarp();
      if (D >= 128 || wq < 2) {
        const uint32_t o0 = tmem + C::O_COL + (buf * MT + c0) * N2 + lane_base;
        // only the first few tiles of an item raise a maximum
        if (__builtin_expect(__any_sync(0xffffffffu, alpha != 1.f), 0))
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float al = __shfl_sync(0xffffffffu, alpha, r);
#pragma unroll
            for (int c = 0; c < MJ; ++c) acc[c][r] *= al;
          }
#pragma unroll
        for (int r = 0; r < NR; r += 8) {
          float be[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) be[e] = beta[r + e];
#pragma unroll
          for (int c = 0; c < MJ; ++c) {
            uint32_t v[16];
            tmem_ld16(o0 + c * N2 + 2 * r, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              acc[c][r + e] = fmaf(
                  fmaf(__uint_as_float(v[8 + e]), 0.0625f, __uint_as_float(v[e])), be[e],
                  acc[c][r + e]);
          }
        }
      }
      tc_fence_before();
      warp_arrive(&sm.oempty[buf]);
      if (__builtin_expect(!w.last(), 1)) continue;
      const int lb = (items - 1) & 1;
      ok = warp_wait(&sm.lfull[lb], ((items - 1) >> 1) & 1, abort_flag);
      if (!ok) break;
      // frame and l of row `lane`
      float2 fl = make_float2(kNone, 0.f);
      if (lane < NR) fl = sm.ml[lb][lane];
      if (sm.nan_rows[lb] >> lane & 1) fl.y = __int_as_float(0x7fc00000);
      // lane r: where row r goes and its factor
      const int jr = sm.rowj[min(lane, NR - 1)], row = row0 + lane;
      const size_t item = (size_t)w.b * p.Hkv + w.g, at = (item + cta) * (size_t)(p.R * p.RG) + row;
      const float scale = whole ? joined_scale(m_run, fl.x, fl.y) : 1.f;
      const unsigned long long to =
          whole ? (unsigned long long)(p.out + (((size_t)w.b * p.n_q + jr) * p.Hq + w.g * p.G + row -
                                                (size_t)jr * p.G) * D)
                : (unsigned long long)(p.ws_o + at * D);
      if (!whole && jg == 0 && wq == 0 && lane < rows)
        p.ws_ml[at] = make_float4(m_run, fl.x, fl.y, 0.f);
      if (D >= 128 || wq < 2) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float f = __shfl_sync(0xffffffffu, scale, r);
          const unsigned long long dst = __shfl_sync(0xffffffffu, to, r);
          if (r >= rows) continue;
#pragma unroll
          for (int c = 0; c < MJ; ++c) {
            const float v = acc[c][r] * f;
            const int d = (c0 + c) * 128 + col;
            if (whole) reinterpret_cast<__nv_bfloat16 *>(dst)[d] = __float2bfloat16_rn(v);
            else reinterpret_cast<float *>(dst)[d] = v;
          }
        }
      }
      warp_arrive(&sm.lempty[lb]);
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM);
}

// Joins the partials of items that several CTAs shared, in CTA order.  One CTA per (border between two
// shares, row), 4 columns a thread; the attention kernel left a record of the item whose first border
// it is.
__global__ void __launch_bounds__(128, 6) combine_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int4 rec = p.ws_rec[blockIdx.x + 1];  // sequence, kv head, last share; -1: nothing here
  if (rec.z < 0) return;
  const int b = rec.x, g = rec.y, c0 = blockIdx.x, c1 = rec.z, row = blockIdx.y;
  const int item = b * p.Hkv + g;
  __nv_bfloat16 *dst =
      p.out + (((size_t)b * p.n_q + row / p.G) * p.Hq + g * p.G + row % p.G) * p.D;
  const int d = threadIdx.x * 4;
  const size_t pitch = (size_t)p.R * p.RG;
  float m = kNone, f = kNone, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // runs of 8 partials: their loads are on their way together
  for (int c = c0; c <= c1; c += 8) {
    float4 ml[8];
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int x = c + u;
      const bool held = x <= c1;
      const size_t at = ((size_t)item + x) * pitch + row;
      ml[u] = held ? p.ws_ml[at] : make_float4(kNone, kNone, 0.f, 0.f);
      o[u] = held && d < p.D ? __ldcg(reinterpret_cast<const float4 *>(p.ws_o + at * p.D + d))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = m, fx = f;
#pragma unroll
    for (int u = 0; u < 8; ++u) mx = fmaxf(mx, ml[u].x), fx = fmaxf(fx, ml[u].y);
    const float a = ex2_approx(m - mx);
    den *= ex2_approx(f - fx);
    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
    m = mx;
    f = fx;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float b = ex2_approx(ml[u].x - mx);
      den = fmaf(ex2_approx(ml[u].y - fx), ml[u].z, den);
      acc.x = fmaf(b, o[u].x, acc.x), acc.y = fmaf(b, o[u].y, acc.y);
      acc.z = fmaf(b, o[u].z, acc.z), acc.w = fmaf(b, o[u].w, acc.w);
    }
  }
  const float inv = joined_scale(m, f, den);
  if (d < p.D)
    *reinterpret_cast<uint2 *>(dst + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------------------- host side

// Rows of a group: what tensor memory (2 N2 (1 + chunks) columns), shared memory and the joining
// warps' registers hold: 24 at D 512, 32 below.  Larger items take groups of equal size, one CTA
// each over the same tiles (the second reads them from L2).
struct Rows {
  int R, RG, NR;
};
static Rows rows_of(int M, int D) {
  const int most = D == 512 ? 24 : 32;
  Rows r;
  r.R = (M + most - 1) / most;
  r.RG = (M + r.R - 1) / r.R;
  r.NR = (r.RG + 7) / 8 * 8;
  return r;
}

template <int D, int NR>
static sd_status launch_one(const CUtensorMap &km, const CUtensorMap &vm, const Params &p,
                            cudaStream_t st) {
  using C = Cfg<D, NR>;
  static int ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SD_ERR_CUDA;
  if (dev >= 64 || !ready[dev]) {
    if (cudaFuncSetAttribute(attn_q8_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::SMEM) != cudaSuccess)
      return SD_ERR_CUDA;
    if (dev < 64) ready[dev] = 1;
  }
  return cuda_status(launch(attn_q8_kernel<D, NR>, dim3(p.P * p.R), dim3(C::THREADS), C::SMEM, st,
                            km, vm, p));
}

static sd_status validate(const sd_attn_desc *d, bool draft) {
  if (!d) return SD_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_q < 1 || d->h_q < 1 || d->h_kv < 1 || d->h_q % d->h_kv)
    return SD_ERR_INVALID_ARG;
  if (draft && d->n_q != 1) return SD_ERR_INVALID_ARG;
  if (d->block_size < 1 || d->max_blocks_per_seq < 1 || d->num_blocks < 1)
    return SD_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) || d->dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (!(d->head_dim == 64 || d->head_dim == 128 || d->head_dim == 256 || d->head_dim == 512) ||
      d->block_size % 16)
    return SD_ERR_UNSUPPORTED;
  if ((long long)d->num_blocks * d->h_kv * d->block_size >= (1ll << 31)) return SD_ERR_UNSUPPORTED;
  if ((long long)(d->h_q / d->h_kv) * d->n_q > 64) return SD_ERR_UNSUPPORTED;
  if ((long long)d->batch * d->h_kv >= (1ll << 31)) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

// CTAs of one row group: one per SM over all groups.
static int ctas(const Rows &r) { return std::max(1, sm_count() / r.R); }

static size_t ws_o_bytes(const sd_attn_desc *d, const Rows &r) {
  const size_t slots = (size_t)d->batch * d->h_kv + ctas(r);
  return round_up(slots * r.R * r.RG * d->head_dim * 4, 256);
}
static size_t ws_size(const sd_attn_desc *d) {
  const Rows r = rows_of(d->h_q / d->h_kv * d->n_q, d->head_dim);
  const size_t slots = (size_t)d->batch * d->h_kv + ctas(r);
  return ws_o_bytes(d, r) + round_up(slots * r.R * r.RG * sizeof(float4), 256) + ctas(r) * sizeof(int4);
}

static sd_status run(const sd_attn_desc *d, bool draft, const void *q, const void *kc,
                     const void *vc, const float *ks, const float *vs, const int32_t *table,
                     const int32_t *ctx_len, const int32_t *q_pos, void *out, void *ws,
                     size_t ws_bytes, cudaStream_t st) {
  const sd_status s = validate(d, draft);
  if (s != SD_OK) return s;
  if (!q || !kc || !vc || !ks || !vs || !table || !ctx_len || !out) return SD_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kc) || !aligned16(vc) || !aligned16(out))
    return SD_ERR_INVALID_ARG;
  if (!ws || ws_bytes < ws_size(d)) return SD_ERR_WORKSPACE;
  if (!aligned16(ws)) return SD_ERR_INVALID_ARG;
  const int M = d->h_q / d->h_kv * d->n_q;
  const Rows r = rows_of(M, d->head_dim);
  Params p{};
  p.B = d->batch;
  p.n_q = d->n_q;
  p.Hq = d->h_q;
  p.Hkv = d->h_kv;
  p.G = d->h_q / d->h_kv;
  p.D = d->head_dim;
  p.bs = d->block_size;
  p.mbps = d->max_blocks_per_seq;
  p.num_blocks = d->num_blocks;
  p.window = d->window > 0 ? d->window : 0;
  p.M = M;
  p.is_draft = draft ? 1 : 0;
  p.q_offset = d->q_offset;
  p.bk = p.bs % 128 == 0 ? 128 : p.bs % 64 == 0 ? 64 : p.bs % 32 == 0 ? 32 : 16;
  p.box_bytes = p.bk * p.D;
  p.row_groups = (int)((long long)p.num_blocks * p.Hkv * p.bs / 8);
  p.R = r.R;
  p.RG = r.RG;
  // no more CTAs than there can be tiles (the table and a window bound a sequence's): one window on 12
  // CTAs 14.3 us, on 148 14.8
  const long long span = (long long)p.mbps * p.bs;
  const long long keys = p.window ? std::min(span, (long long)p.window + p.n_q + p.bk - 2) : span;
  p.span = (int)std::min<long long>(span, INT_MAX - kTile - 64);
  p.P = (int)std::min<long long>(ctas(r), (long long)p.B * p.Hkv * ((keys - 1) / kTile + 1));
  p.scale_log2 = d->scale * 1.4426950408889634f;
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  p.ks = ks;
  p.vs = vs;
  p.table = table;
  p.ctx_len = ctx_len;
  p.q_pos = q_pos;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float4 *>(reinterpret_cast<uint8_t *>(ws) + ws_o_bytes(d, r));
  p.ws_rec = reinterpret_cast<int4 *>(
      reinterpret_cast<uint8_t *>(ws) + ws_size(d) - (size_t)p.P * sizeof(int4));
  p.status = device_status_word();
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)p.num_blocks * p.Hkv * p.bs;
  if (!encode_tmap_kv_bytes(&km, kc, p.D, rows, p.bk) ||
      !encode_tmap_kv_bytes(&vm, vc, p.D, rows, p.bk))
    return SD_ERR_CUDA;
  sd_status e = SD_ERR_UNSUPPORTED;
#define SDV_CASE(DD, NN) \
  if (p.D == DD && r.NR == NN) e = launch_one<DD, NN>(km, vm, p, st); else
  SDV_CASE(64, 8) SDV_CASE(64, 16) SDV_CASE(64, 24) SDV_CASE(64, 32)
  SDV_CASE(128, 8) SDV_CASE(128, 16) SDV_CASE(128, 24) SDV_CASE(128, 32)
  SDV_CASE(256, 8) SDV_CASE(256, 16) SDV_CASE(256, 24) SDV_CASE(256, 32)
  SDV_CASE(512, 8) SDV_CASE(512, 16) SDV_CASE(512, 24) return SD_ERR_UNSUPPORTED;
#undef SDV_CASE
  if (e != SD_OK) return e;
  if (p.P == 1) return SD_OK;
  return cuda_status(launch(combine_kernel, dim3(p.P - 1, p.M), dim3(128), 0, st, p));
}

}  // namespace q8
}  // namespace sdv

extern "C" {

size_t sd_verify_attn_q8_workspace_size(const sd_attn_desc *desc) {
  if (sdv::q8::validate(desc, false) != SD_OK) return 0;
  return sdv::q8::ws_size(desc);
}

sd_status sd_verify_attn_q8(const sd_attn_desc *desc, const void *q, const void *k_cache,
                            const void *v_cache, const float *k_scale, const float *v_scale,
                            const int32_t *block_table, const int32_t *ctx_len, void *out,
                            void *ws, size_t ws_bytes, sd_stream stream) {
  return sdv::q8::run(desc, false, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_len,
                      nullptr, out, ws, ws_bytes, (cudaStream_t)stream);
}

size_t sd_draft_xattn_q8_workspace_size(const sd_attn_desc *desc) {
  if (sdv::q8::validate(desc, true) != SD_OK) return 0;
  return sdv::q8::ws_size(desc);
}

sd_status sd_draft_xattn_q8(const sd_attn_desc *desc, const void *q, const void *k_cache,
                            const void *v_cache, const float *k_scale, const float *v_scale,
                            const int32_t *block_table, const int32_t *ctx_len,
                            const int32_t *q_pos, void *out, void *ws, size_t ws_bytes,
                            sd_stream stream) {
  return sdv::q8::run(desc, true, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_len,
                      q_pos, out, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
