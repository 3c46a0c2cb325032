// Verify attention and drafter cross-attention over a paged e4m3 KV cache (sm_100a).
//
// The calls of attention.cu over a cache of half the bytes (the pages: decoding is bound by the
// memory it reads, GeekNews summary of the Google blog, section "why speculative decoding"; the
// drafter shares the target's cache, section "MTP drafter internal optimisations").
//
// Mathematics.  Key p has codes k_p, v_p and scales a_p, c_p (one per cache block and kv head).
// Query q is split exactly into two e4m3 parts, q = 2^e (q_hi + q_lo / 16): a bf16 has 8
// significant bits, an e4m3 part 4.  So the scores s_p = scale 2^e a_p (k_p . q_hi + k_p . q_lo /
// 16) come from exact 8-bit products in float32.  The weight of v_p is 2^t, t = s_p log2(e) +
// log2(c_p); per tile of 128 keys and query row, w = 2^(t - max t + 8) is split the same way into
// w_hi + w_lo / 16 (relative error at most 2^-8, half a step of each part; w down to 2^-21 of the
// tile's largest is kept).  A maximum of the tile, not a running one, keeps that range for every
// tile however large a weight another tile holds.  Tiles join in float32 registers,
// O <- O 2^(m - m') + O_tile 2^(max t - m'), l likewise from the unrounded w / c_p.
//
// Bound by HBM: 2 D bytes a key and kv head are read once; 4 G n_q D flops.  Both products have
// the streamed operand as the tensor core's 128-row side, read from shared memory where TMA put
// it, so no code is ever converted or moved:
//   S^T[128 keys x 2R] = K[128 x D] Q^T     K-major A; the columns are R rows' hi and lo parts
//   O^T[D x 2R]        = V^T[D x 128] P^T   V as an MN-major A, one 128-column chunk at a time
// with tcgen05 (kind::f8f6f4) into tensor memory.  Roles of a persistent CTA: a TMA warp (ring
// of 128-key K and V tiles, boxes of one cache block), an MMA thread, two warps that split the
// next item's queries, four softmax warps (thread = key), four warps that join the output tiles
// (thread = output column).  S of tile i + 1 is computed while tile i is in the softmax, and its
// output tile while tile i + 1 is.  The flattened (sequence, kv head, tile) list is split evenly
// over the CTAs; shared items leave (o, m, l) partials that a second kernel joins in CTA order.
#include <algorithm>

#include "common.cuh"
#include "host.cuh"

namespace sdv {
namespace q8 {

constexpr int kTile = 128;  // keys
constexpr int kScaleRing = 4;
// Score tiles computed ahead of the output products: V of a tile is then loaded when its weights
// are nearly done, so it does not hold a ring slot through the softmax.
constexpr int kAhead = 2;

struct Params {
  int B, n_q, Hq, Hkv, G, D, bs, mbps, num_blocks, window, M;
  int is_draft, q_offset;
  int bk, box_bytes;  // keys and bytes of one TMA box
  int R, RG;          // row groups of an item, rows of a group
  int P;              // CTAs of one row group
  float scale_log2;
  const __nv_bfloat16 *q;
  const float *ks, *vs;
  const int32_t *table, *ctx_len, *q_pos;
  __nv_bfloat16 *out;
  float *ws_o;   // [slots][R * RG][D]
  float *ws_ml;  // [slots][R * RG][2]
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
  const int hi = p.is_draft ? min(s.t0, L - 1) : L + p.n_q - 1;
  const int lo = p.window > 0 ? max(0, s.t0 - p.window + 1) : 0;
  if (hi < lo) return s;
  if ((long long)hi >= (long long)p.mbps * p.bs) {
    if (report) record_status(p.status, SD_ERR_DEVICE);
    return s;
  }
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
  __device__ __forceinline__ void next(const Params &p) {
    --left;
    if (++tau < s.n || left == 0) return;
    tau = 0;
    if (++g < p.Hkv) return;
    g = 0;
    do {
      s = seq_of(p, ++b, false);
    } while (s.n == 0);  // left > 0: a later sequence has tiles
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
  // tile time differed by 1.3x between GPCs of 16 and 20 SMs) and no register spills.
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
    float scales[kScaleRing][2][8];
    float red[SG][2][4][8];
    float row[4 * SG][3][8];  // per softmax warp: tile max - 8, alpha, beta
    float2 ab[4][NR];         // alpha, beta for the joining warps
    float2 ml[2][NR];         // m, l of an item
    float qs[2][NR];          // 2^e scale of the query rows
    int rowj[NR];             // query position of a row (row / G)
    uint64_t full[8], empty[8];
    uint64_t sc_full[kScaleRing], sc_empty[kScaleRing];
    uint64_t qfull[2], qempty[2], sfull[NS], sempty[NS], pfull[2], pempty[2], ofull[2], oempty[2],
        lfull[2], lempty[2], abfull[4], drain;
    Start start;
    uint32_t tmem;
    int hole[kScaleRing];     // a block of the tile does not exist
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

// D[tmem] (+)= A B^T, 8-bit floats, float32 accumulator.
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Shared-memory matrix descriptor: rows of RB = 128 or 64 bytes with the swizzle of that width,
// 8-row groups sbo bytes apart.  K-major operands have one swizzled row per M/N index (the leading
// offset is unused); MN-major ones one per K index, RB bytes of M, and lbo bytes to the next RB.
template <int RB>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t sbo, uint32_t lbo16) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)lbo16 << 16) |
         ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)(RB == 128 ? 2 : 4) << 61);
}

// kind::f8f6f4, e4m3 x e4m3 -> float32; a_mn: A is MN-major (bit 15).
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Two floats to two e4m3 bytes (first one low), nearest even, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_float(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, "
      "b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// x and y as hi + lo / 16, both parts e4m3 (two bytes each).
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = e4m3x2(x, y);
  const float2 h = e4m3x2_float(hi);
  lo = e4m3x2((x - h.x) * 16.f, (y - h.y) * 16.f);
}

// 32 lanes x 8 columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// mbar_wait that sleeps in the hardware between tries: a spinning warp takes issue slots from the
// warps that compute (B 8 verify at D 512: 157 us spinning).
__device__ __forceinline__ bool try_wait_hint(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort) {
  unsigned long long t0 = 0;
  while (!try_wait_hint(bar, parity)) {
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (*abort || now - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// One arrival for the warp, once all its lanes are here (32 arrivals on one address serialise).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
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

template <int D, int NR>
__global__ void __launch_bounds__(Cfg<D, NR>::THREADS, 1)
    attn_q8_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
  using C = Cfg<D, NR>;
  constexpr int N2 = C::N2, MT = C::MT, RB = C::RB, SLOTS = C::SLOTS, NQ = C::NQ, NP = C::NP,
                NO = C::NO, NS = C::NS, SG = C::SG, JG = C::JG, MJ = C::MJ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&sm.sc_full[i], 16 + 1);
      mbar_init(&sm.sc_empty[i], 4 * SG);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sempty[i], 4 * SG);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qfull[i], 2);
      mbar_init(&sm.qempty[i], 1 + 4 * SG);  // the item's last scores; its row scales are read
      mbar_init(&sm.pfull[i], 4 * SG);
      mbar_init(&sm.pempty[i], 1);
      mbar_init(&sm.ofull[i], 1);
      mbar_init(&sm.oempty[i], 4 * JG);
      mbar_init(&sm.lfull[i], 4 * SG);
      mbar_init(&sm.lempty[i], 4 * JG);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.abfull[i], SG);
    mbar_init(&sm.drain, 1);
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
    unsigned total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const unsigned n = b < p.B ? seq_of(p, b, blockIdx.x == 0).n : 0;
      total += __reduce_add_sync(0xffffffffu, n) * p.Hkv;
    }
    const unsigned P = min((unsigned)p.P, total);
    Start st{0, 0, 0, 0};
    unsigned at = 0;
    if ((unsigned)cta < P) {
      at = share(total, cta, P);
      st.left = (int)(share(total, cta + 1, P) - at);
    }
    unsigned pre = 0;
    for (int b0 = 0; b0 < p.B && st.left > 0; b0 += 32) {
      const int b = b0 + lane;
      const unsigned n = b < p.B ? seq_of(p, b, false).n : 0;
      unsigned v = n * p.Hkv;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      const unsigned m = __ballot_sync(0xffffffffu, at < pre + v);
      if (m) {
        const int src = __ffs(m) - 1;
        const unsigned before = pre + __shfl_sync(0xffffffffu, v - n * p.Hkv, src);
        const unsigned nn = __shfl_sync(0xffffffffu, n, src);
        st.b = b0 + src;
        st.g = (int)((at - before) / nn);
        st.tau = (int)((at - before) % nn);
        break;
      }
      pre += __shfl_sync(0xffffffffu, v, 31);
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

  if (warp == 0) {
    // -------------------------------------------------------------------- TMA producer
    // Ring order K0 .. K_ahead, V0, K, V1, ...: the order in which the products need the tiles.
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    const uint64_t policy = l2_policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    const int boxes = kTile / p.bk, per_blk = p.bs / p.bk;
    int v_row[kAhead + 1], v_boxes[kAhead + 1];  // boxes of the last tiles: lane i holds its i-th
    auto load_slot = [&](const CUtensorMap *map, int row, uint32_t bytes) {
      const int slot = it % SLOTS;
      const bool free = wait_for(&sm.empty[slot], ((it / SLOTS) & 1) ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, free)) {
        if (lane == 0) fail();
        return false;
      }
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], bytes);
      __syncwarp();
      if (row >= 0)
        tma_load_4d(slots + (size_t)slot * C::SLOT + lane * p.box_bytes, map, &sm.full[slot],
                    row >> 3, policy);
      ++it;
      return true;
    };
    for (int i = 0; i < st.left + kAhead; ++i) {
      int row = -1, nb = 0;
      if (i < st.left) {
        const int pk = w.pos() + lane * p.bk;  // lane's box
        bool hole = false;
        if (lane < boxes && pk <= w.s.hi) {
          const int blk = p.table[(size_t)w.b * p.mbps + pk / p.bs];
          if (blk >= 0 && blk < p.num_blocks)
            row = (blk * p.Hkv + w.g) * p.bs + (pk / p.bk % per_blk) * p.bk;
          else
            hole = true;
        }
        nb = __popc(__ballot_sync(0xffffffffu, row >= 0));
        hole = __any_sync(0xffffffffu, hole);
        const int r = i % kScaleRing;
        ok = wait_for(&sm.sc_empty[r], ((i / kScaleRing) & 1) ^ 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        if (lane == 0) {
          if (hole) record_status(p.status, SD_ERR_DEVICE);
          sm.hole[r] = hole;
          mbar_arrive(&sm.sc_full[r]);
        }
        // scales of the 16-key group lane & 7
        const int grp = lane & 7;
        const int srow = __shfl_sync(0xffffffffu, row, grp * 16 / p.bk);
        if (lane < 16) {
          float *dst = &sm.scales[r][lane >> 3][grp];
          if (srow >= 0) {
            cp_async_4(dst, (lane < 8 ? p.ks : p.vs) + srow / p.bs);
            cp_async_arrive(&sm.sc_full[r]);
          } else {
            *dst = -1.f;  // no such block: its keys are masked
            mbar_arrive(&sm.sc_full[r]);
          }
        }
        ok = load_slot(&kmap, row, nb * p.box_bytes);
        if (!ok) break;
        w.next(p);
      }
#pragma unroll
      for (int k = kAhead; k > 0; --k) {
        v_row[k] = v_row[k - 1];
        v_boxes[k] = v_boxes[k - 1];
      }
      v_row[0] = row;
      v_boxes[0] = nb;
      if (i >= kAhead) {
        ok = load_slot(&vmap, v_row[kAhead], v_boxes[kAhead] * p.box_bytes);
        if (!ok) break;
      }
    }
    if (!ok && lane == 0)
      for (uint32_t j = it > (uint32_t)SLOTS ? it - SLOTS : 0; j < it; ++j)
        mbar_wait_timed(&sm.full[j % SLOTS], (j / SLOTS) & 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1) {
    // -------------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f8(128, N2, false), id_o = idesc_f8(128, N2, true);
      const uint32_t s0 = smem_u32(slots), q0 = smem_u32(qbuf), pb0 = smem_u32(pbuf);
      uint32_t it = 0, items = 0;
      const int n = st.left;
      bool ok = true;
      for (int i = 0; i < n + kAhead; ++i) {
        if (i < n) {  // scores of tile i
          const int slot = it % SLOTS, buf = i % NS;
          if (w.first(st)) {
            ok = wait_for(&sm.qfull[items % NQ], (items / NQ) & 1, abort_flag);
            if (!ok) break;
            ++items;
          }
          ok = wait_for(&sm.full[slot], (it / SLOTS) & 1, abort_flag) &&
               wait_for(&sm.sempty[buf], ((i / NS) & 1) ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = smem_desc<RB>(s0 + slot * C::SLOT, D * 8, 1);
          const uint64_t b = smem_desc<RB>(q0 + ((items - 1) % NQ) * C::QBYTES, RB * 8, 1);
#pragma unroll 1
          for (int ch = 0; ch < C::CH; ++ch)
#pragma unroll
            for (int x = 0; x < RB / 32; ++x)  // addresses in 16-byte units
              umma_f8(tmem + C::S_COL + buf * N2, a + ch * (8 * RB / 16) + 2 * x,
                      b + ch * (N2 * RB / 16) + 2 * x, id_s, ch + x > 0);
          umma_commit(&sm.sfull[buf]);
          umma_commit(&sm.empty[slot]);
          if (w.last()) umma_commit(&sm.qempty[(items - 1) % NQ]);
          ++it;
          w.next(p);
        }
        if (i >= kAhead) {  // output tile
          const int o = i - kAhead, slot = it % SLOTS, buf = o % NO;
          ok = wait_for(&sm.full[slot], (it / SLOTS) & 1, abort_flag) &&
               wait_for(&sm.pfull[o % NP], (o / NP) & 1, abort_flag) &&
               wait_for(&sm.oempty[buf], ((o / NO) & 1) ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = smem_desc<RB>(s0 + slot * C::SLOT, D * 8, 0);
          const uint64_t b = smem_desc<128>(pb0 + (o % NP) * C::PBYTES, 1024, 1);
#pragma unroll 1
          for (int c = 0; c < MT; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8(tmem + C::O_COL + (buf * MT + c) * N2, a + c * (8 * RB / 16) + k * (2 * D),
                      b + 2 * k, id_o, k > 0);
          umma_commit(&sm.ofull[buf]);
          umma_commit(&sm.empty[slot]);
          umma_commit(&sm.pempty[o % NP]);
          ++it;
        }
      }
      if (!ok) fail();
      umma_commit(&sm.drain);
      if (!mbar_wait_timed(&sm.drain, 0)) record_status(p.status, SD_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 4) {
    // -------------------------------------------------------------------- query splitter
    // Rows in turn over the two warps, four at a time: scale to at most 256, split, store
    // swizzled.
    uint32_t items = 0;
    const int half = warp - 2;
    constexpr int E = D / 64;  // pairs a lane holds of a row: elements 2 lane + 64 e
    while (w.left > 0) {
      const int qb = items % NQ;
      uint8_t *dst = qbuf + qb * C::QBYTES;
#pragma unroll 1
      for (int r0 = half; r0 < NR; r0 += 8) {
        uint32_t x[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + 2 * u, row = row0 + r;
          const int j = row / p.G, h = w.g * p.G + row % p.G;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(
              p.q + (((size_t)w.b * p.n_q + j) * p.Hq + h) * D);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u][e] = r < rows ? src[lane + 32 * e] : 0u;
        }
        if (r0 == half) {  // the loads are on their way
          const bool free = wait_for(&sm.qempty[qb], ((items / NQ) & 1) ^ 1, abort_flag);
          if (!__all_sync(0xffffffffu, free)) {
            if (lane == 0) fail();
            goto splitter_done;
          }
        }
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + 2 * u;
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float a = fabsf(__uint_as_float(x[0][e] << 16));
            const float b = fabsf(__uint_as_float(x[0][e] & 0xffff0000u));
            m = fmaxf(m, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
          }
          m = redux_max(m);
          // 2^ex with m <= 256 * 2^ex, ex >= -100
          const int ex = max((int)(__float_as_uint(m) >> 23) - 127 + 1 - 8, -100);
          const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
          if (lane == 0) sm.qs[qb][r] = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float a = __uint_as_float(x[0][e] << 16), b = __uint_as_float(x[0][e] & 0xffff0000u);
            // an infinity becomes NaN, and with it the row's output
            if (!(fabsf(a) < INFINITY)) a = __int_as_float(0x7fc00000);
            if (!(fabsf(b) < INFINITY)) b = __int_as_float(0x7fc00000);
            uint32_t hi, lo;
            split2(a * inv, b * inv, hi, lo);
            const int col = 2 * lane + 64 * e;
            *reinterpret_cast<uint16_t *>(dst + tile_byte<RB>(N2, r, col)) = (uint16_t)hi;
            *reinterpret_cast<uint16_t *>(dst + tile_byte<RB>(N2, NR + r, col)) = (uint16_t)lo;
          }
#pragma unroll
          for (int v = 0; v < 3; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) x[v][e] = x[v + 1][e];
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&sm.qfull[qb]);
      ++items;
      do {  // to the next item
        const bool end = w.last();
        w.next(p);
        if (end) break;
      } while (true);
    }
  splitter_done:;
  } else if (warp < 4 + 4 * SG) {
    // -------------------------------------------------------------------- softmax
    // Thread = key, eight rows of the warpgroup.
    const int wg = (warp - 4) >> 2, wq = warp & 3, key = wq * 32 + lane, wr = warp - 4;
    const int r0 = 8 * wg;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    bool bad = false;
    float m_run = -INFINITY;  // of row r0 + lane
    float l[8], qsc[8];
    uint32_t items = 0;
    const int j_first = sm.rowj[0], j_last = sm.rowj[NR - 1];
    for (int i = 0; w.left > 0; ++i, w.next(p)) {
      const int buf = i % NS;
      const int p0 = w.pos(), pos = p0 + key;
      if (w.first(st)) {
        // the splitter wrote the rows' scales before the scores were computed
        bad |= !wait_for(&sm.qfull[items % NQ], (items / NQ) & 1, abort_flag);
        ++items;
        m_run = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          l[r] = 0.f;
          qsc[r] = sm.qs[(items - 1) % NQ][r0 + r] * p.scale_log2;
        }
        warp_arrive(&sm.qempty[(items - 1) % NQ]);
      }
      const int ring = i % kScaleRing;
      bad |= !wait_for(&sm.sc_full[ring], (i / kScaleRing) & 1, abort_flag);
      const float ks = sm.scales[ring][0][key >> 4];
      const float vs = fmaxf(sm.scales[ring][1][key >> 4], 0x1p-100f);
      const bool hole = sm.hole[ring] != 0;
      warp_arrive(&sm.sc_empty[ring]);
      const float lvs = log2f(vs), rvs = 1.f / vs;
      // a tile at a range's end, where not every row attends to every key
      const bool edge = hole || p0 < row_lo(p, w.s, j_last) ||
                        p0 + kTile - 1 > row_hi(p, w.s, j_first);
      bad |= !wait_for(&sm.sfull[buf], (i / NS) & 1, abort_flag);
      tc_fence_after();
      float t[8];
      {
        uint32_t hi[8], lo[8];
        tmem_ld8(tmem + C::S_COL + buf * N2 + r0 + lane_base, hi);
        tmem_ld8(tmem + C::S_COL + buf * N2 + NR + r0 + lane_base, lo);
        tmem_ld_wait();
        tc_fence_before();
        warp_arrive(&sm.sempty[buf]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float s = fmaf(__uint_as_float(lo[r]), 0.0625f, __uint_as_float(hi[r]));
          t[r] = fmaf(s * ks, qsc[r], lvs);
        }
      }
      bool nan_v = false;
      if (edge) {
        const bool inside = pos >= w.s.lo && pos <= w.s.hi && ks >= 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int j = sm.rowj[r0 + r];
          if (!inside || pos < row_lo(p, w.s, j) || pos > row_hi(p, w.s, j)) t[r] = -INFINITY;
        }
        // V rows that no query attends to may hold any codes, and 0 * NaN is NaN: they are
        // cleared; a NaN that only some queries attend to is cleared and goes into their l
        const bool part =
            inside && (pos < row_lo(p, w.s, j_last) || pos > row_hi(p, w.s, j_first));
        const uint32_t vit = min(i + kAhead + 1, st.left) + i;  // V_i in the ring's order
        bad |= !wait_for(&sm.full[vit % SLOTS], (vit / SLOTS) & 1, abort_flag);
        uint8_t *v = slots + (size_t)(vit % SLOTS) * C::SLOT + (key >> 3) * (8 * D) + (key & 7) * RB;
        // bytes 0x7f and 0xff: bit 7 of each such byte
        auto nan = [](uint32_t z) { return ((z & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
        if (part)
#pragma unroll 1
          for (int u = 0; u < D; u += 16) {
            const uint4 y = *reinterpret_cast<const uint4 *>(v + u / RB * (8 * RB) +
                                                             ((u + 16 * lane) & (RB - 1)));
            nan_v |= (nan(y.x) | nan(y.y) | nan(y.z) | nan(y.w)) != 0;
          }
        // every warpgroup has seen the codes before the first one clears them
        bad = barrier_or(1, 128 * SG, bad);
        if (wg == 0 && !bad && (!inside || (part && nan_v)))
#pragma unroll 1
          for (int u = 0; u < D; u += 16) {
            uint4 *x = reinterpret_cast<uint4 *>(v + u / RB * (8 * RB) +
                                                 ((u + 16 * lane) & (RB - 1)));
            uint4 y = make_uint4(0, 0, 0, 0);
            if (inside) {
              auto clear = [&](uint32_t z) { return z & ~((nan(z) >> 7) * 0xffu); };
              y = *x;
              y = make_uint4(clear(y.x), clear(y.y), clear(y.z), clear(y.w));
            }
            *x = y;
          }
      }
      // maxima of the tile: lane r ends up with row r's
      {
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float v = redux_max(t[r]);
          if (lane == r) mx = v;
        }
        if (lane < 8) sm.red[wg][i & 1][wq][lane] = mx;
      }
      bad = barrier_or(2 + wg, 128, bad);
      if (bad) break;
      if (lane < 8) {
        float tm = sm.red[wg][i & 1][0][lane];
#pragma unroll
        for (int q = 1; q < 4; ++q) tm = fmaxf(tm, sm.red[wg][i & 1][q][lane]);
        if (tm != tm) tm = 0.f;  // nothing but NaN: the weights are, and l and O become NaN
        const float m_new = fmaxf(m_run, tm);
        const float alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
        const float beta = tm == -INFINITY ? 0.f : ex2_approx(tm - m_new) * 0x1p-8f;
        m_run = m_new;
        sm.row[wr][0][lane] = tm == -INFINITY ? 0.f : tm - 8.f;
        sm.row[wr][1][lane] = alpha;
        sm.row[wr][2][lane] = beta;
      }
      __syncwarp();
      bad |= !wait_for(&sm.pempty[i % NP], ((i / NP) & 1) ^ 1, abort_flag);
      if (wq == 0) {
        // tile i - 4's pair is read: tile i - 2's output product, which this thread has seen
        // finish, waited for tile i - 4's output to be read
        if (lane < 8)
          sm.ab[i & 3][r0 + lane] = make_float2(sm.row[wr][1][lane], sm.row[wr][2][lane]);
        warp_arrive(&sm.abfull[i & 3]);
      }
      uint8_t *pd = pbuf + (i % NP) * C::PBYTES;
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        const float2 mx = *reinterpret_cast<const float2 *>(&sm.row[wr][0][r]);
        const float2 al = *reinterpret_cast<const float2 *>(&sm.row[wr][1][r]);
        const float2 be = *reinterpret_cast<const float2 *>(&sm.row[wr][2][r]);
        const float w0 = ex2_approx(t[r] - mx.x), w1 = ex2_approx(t[r + 1] - mx.y);
        float f0 = rvs, f1 = rvs;
        if (nan_v) {
          if (t[r] != -INFINITY) f0 = __int_as_float(0x7fc00000);
          if (t[r + 1] != -INFINITY) f1 = __int_as_float(0x7fc00000);
        }
        l[r] = fmaf(l[r], al.x, w0 * f0 * be.x);
        l[r + 1] = fmaf(l[r + 1], al.y, w1 * f1 * be.y);
        uint32_t hi, lo;
        split2(w0, w1, hi, lo);
        pd[tile_byte<128>(N2, r0 + r, key)] = (uint8_t)hi;
        pd[tile_byte<128>(N2, r0 + r + 1, key)] = (uint8_t)(hi >> 8);
        pd[tile_byte<128>(N2, NR + r0 + r, key)] = (uint8_t)lo;
        pd[tile_byte<128>(N2, NR + r0 + r + 1, key)] = (uint8_t)(lo >> 8);
      }
      fence_proxy_async_smem();
      warp_arrive(&sm.pfull[i % NP]);
      if (w.last()) {
        // l over the 128 keys; lane r of the warpgroup's first warp hands (m, l) of row r over
        const int lb = (items - 1) & 1;
        bad |= !wait_for(&sm.lempty[lb], (((items - 1) >> 1) & 1) ^ 1, abort_flag);
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          float v = l[r];
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == r) mine = v;
        }
        float (&red)[4][8] = sm.red[wg][(i & 1) ^ 1];
        if (lane < 8) red[wq][lane] = mine;
        bad = barrier_or(2 + wg, 128, bad);
        if (bad) break;
        if (wq == 0 && lane < 8)
          sm.ml[lb][r0 + lane] =
              make_float2(m_run, red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane]);
        // the next tile writes there again: not before the first warp has read it
        bad = barrier_or(2 + wg, 128, bad);
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
    bool ok = true;
    float acc[MJ][NR];
    uint32_t items = 0;
    bool whole = false;
    for (int i = 0; w.left > 0; ++i, w.next(p)) {
      const int buf = i % NO;
      if (w.first(st)) {
        whole = w.tau == 0 && w.left >= w.s.n;
        ++items;
#pragma unroll
        for (int c = 0; c < MJ; ++c)
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[c][r] = 0.f;
      }
      ok = wait_for(&sm.abfull[i & 3], (i >> 2) & 1, abort_flag) &&
           wait_for(&sm.ofull[buf], (i / NO) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (D >= 128 || wq < 2) {
        const uint32_t o0 = tmem + C::O_COL + (buf * MT + c0) * N2 + lane_base;
#pragma unroll
        for (int c = 0; c < MJ; ++c)
#pragma unroll
          for (int r = 0; r < NR; r += 8) {
            uint32_t hi[8], lo[8];
            tmem_ld8(o0 + c * N2 + r, hi);
            tmem_ld8(o0 + c * N2 + NR + r, lo);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 ab = sm.ab[i & 3][r + e];
              const float o = fmaf(__uint_as_float(lo[e]), 0.0625f, __uint_as_float(hi[e]));
              acc[c][r + e] = fmaf(acc[c][r + e], ab.x, o * ab.y);
            }
          }
      }
      tc_fence_before();
      warp_arrive(&sm.oempty[buf]);
      if (!w.last()) continue;
      const int lb = (items - 1) & 1;
      ok = wait_for(&sm.lfull[lb], ((items - 1) >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const size_t item = (size_t)w.b * p.Hkv + w.g;
      if (D >= 128 || wq < 2) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (r >= rows) continue;
          const float2 ml = sm.ml[lb][r];
          const int row = row0 + r, j = sm.rowj[r];
          if (whole) {
            const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;  // no key: a zero row
            __nv_bfloat16 *dst =
                p.out + (((size_t)w.b * p.n_q + j) * p.Hq + w.g * p.G + row - j * p.G) * D;
#pragma unroll
            for (int c = 0; c < MJ; ++c)
              dst[(c0 + c) * 128 + col] = __float2bfloat16_rn(acc[c][r] * inv);
          } else {
            const size_t at = (item + cta) * (size_t)(p.R * p.RG) + row;
#pragma unroll
            for (int c = 0; c < MJ; ++c) p.ws_o[at * D + (c0 + c) * 128 + col] = acc[c][r];
            if (jg == 0 && wq == 0 && lane == 0)
              *reinterpret_cast<float2 *>(p.ws_ml + at * 2) = ml;
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

// Joins the partials of items that several CTAs shared, in CTA order; zero rows for sequences
// with no keys.  One CTA per (item, row), 4 columns a thread.
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int item = blockIdx.x, row = blockIdx.y;
  const int b = item / p.Hkv, g = item % p.Hkv;
  __shared__ unsigned s_pre, s_total;
  if (threadIdx.x < 32) {
    unsigned pre = 0, total = 0;
    for (int i = threadIdx.x; i < p.B; i += 32) {
      const unsigned n = seq_of(p, i, false).n * p.Hkv;
      total += n;
      if (i < b) pre += n;
    }
    pre = __reduce_add_sync(0xffffffffu, pre);
    total = __reduce_add_sync(0xffffffffu, total);
    if (threadIdx.x == 0) {
      s_pre = pre;
      s_total = total;
    }
  }
  const unsigned n = seq_of(p, b, false).n;
  __syncthreads();
  __nv_bfloat16 *dst =
      p.out + (((size_t)b * p.n_q + row / p.G) * p.Hq + g * p.G + row % p.G) * p.D;
  const int d = threadIdx.x * 4;
  if (n == 0) {
    if (d < p.D) *reinterpret_cast<uint2 *>(dst + d) = make_uint2(0, 0);
    return;
  }
  const unsigned total = s_total, P = min((unsigned)p.P, total), first = s_pre + g * n;
  const int c0 = (int)share_of(total, first, P), c1 = (int)share_of(total, first + n - 1, P);
  if (c0 == c1) return;  // written by its only CTA
  const size_t pitch = (size_t)p.R * p.RG;
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // runs of 8 partials: their loads are on their way together
  for (int c = c0; c <= c1; c += 8) {
    float2 ml[8];
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int x = c + u;
      const bool held = x <= c1;
      const size_t at = ((size_t)item + x) * pitch + row;
      ml[u] = held ? *reinterpret_cast<const float2 *>(p.ws_ml + at * 2)
                   : make_float2(-INFINITY, 0.f);
      o[u] = held && d < p.D ? __ldcg(reinterpret_cast<const float4 *>(p.ws_o + at * p.D + d))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < 8; ++u) mx = fmaxf(mx, ml[u].x);
    if (mx == -INFINITY) continue;
    const float a = ex2_approx(m - mx);  // 0 from -inf
    den *= a;
    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
    m = mx;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = ex2_approx(ml[u].x - mx);
      den = fmaf(f, ml[u].y, den);
      acc.x = fmaf(f, o[u].x, acc.x), acc.y = fmaf(f, o[u].y, acc.y);
      acc.z = fmaf(f, o[u].z, acc.z), acc.w = fmaf(f, o[u].w, acc.w);
    }
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;
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
  return ws_o_bytes(d, r) + round_up(slots * r.R * r.RG * 8, 256);
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
  p.R = r.R;
  p.RG = r.RG;
  p.P = ctas(r);
  p.scale_log2 = d->scale * 1.4426950408889634f;
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  p.ks = ks;
  p.vs = vs;
  p.table = table;
  p.ctx_len = ctx_len;
  p.q_pos = q_pos;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(ws) + ws_o_bytes(d, r));
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
  return cuda_status(launch(combine_kernel, dim3(p.B * p.Hkv, p.M), dim3(128), 0, st, p));
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
