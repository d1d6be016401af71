// tree_attention.cuh — attention of every request's drafted tree (or chain, or
// single token) over its paged KV cache, on the tensor cores.
//
//   s_p = scale * q . K_p,  out = sum_p e^{s_p} V_p / sum_p e^{s_p}
// over p < ctx, and p = ctx + j for the nodes j in the row's ancestor mask.
//
// A round has few query rows for each KV head (nodes x query heads per KV head)
// and long contexts, so the product is bound by reading K and V once.  Both
// products therefore take the cache as the 128-row operand and the query rows as
// the narrow one (N = NT columns):
//   S^T [128 tokens x NT] = K_tile . Q^T       O^T [D x NT] += V_tile^T . P^T
// With the rows on the 128-row side instead, a chain of 6 nodes x 4 heads would
// leave 104 of 128 accumulator rows empty and one warp to do every exponential.
// Here a thread owns one token (TMEM lane) and the rows run along registers.  Its
// price is the maximum over tokens, which lies across lanes; it is paid only when
// it matters: the exponent's reference is kept from tile to tile and raised (with
// O rescaled) only when some weight would exceed 2^RAISE.
//
// A bf16 cache's weight meets V as the sum of two bf16 numbers, its rounding and
// what that left out (columns j and NT + j of P, and two parts of O added at the
// end): rounded to one, a row's error would be of the output's own rounding's size,
// and below 64 rows the wider product costs nothing, as reading V's tile bounds it.
//
// An 8-bit cache's tiles are widened to f16, which holds every e4m3 value and takes
// one conversion for two of them (bf16 takes four), and meet Q and P in f16: Q's
// tile is scaled by the power of two that brings its largest value to 2^14 (f16
// then keeps all 8 bits of what lies within 2^28 of it; a row beside one that is larger
// by more keeps fewer), and a weight has 11 bits.  Weights are at most 2^14 there and
// count down to 2^-24, with fewer bits below 2^-14.
//
// Work is cut into units of (request, KV head, row tile, 128-token tile), listed
// in that order, and every CTA takes an equal share of the list: ragged contexts
// balance, and a long context is split over as many CTAs as there are.  A CTA's
// first and last item may be cut; those leave (O, maximum, sum) in the workspace
// and tree_attention_join adds the pieces in order (no atomics: the same bits
// from call to call).
//
// One CTA per SM: warp 0 loads K and V (TMA, one copy per page and 64 columns), warp
// 1 issues the MMAs, warp 2 loads Q, two groups of four warps do the softmax (a warp for
// each 32 tokens, CH chunks of 16 or 32 columns one after the other), and for an 8-bit
// cache four more widen the tiles to f16 between two rings.
//
// What it measured, and what bounds it (D = 128, 32 query heads over 8 KV heads):
//   256 chains of 1..6 rows over contexts of 64 to 8192 tokens, bf16: 1.77 GB in
//     264 to 273 us in a graph (boxes differ; 271 to 281 by calls), 6.5 to 6.7 TB/s;
//     eight chains over 65536 tokens 6.6 to 6.8: reading K and V.
//     The copies then are late often enough that the softmax's own time is hidden.
//   1024 chains over 400 tokens 4.8 TB/s: items begin and end every four tiles.
//   64 trees of 64 rows over 512 to 4096 tokens, bf16 (two tiles of 128 rows):
//     120 GFLOP in 296 to 303 us.  A tile takes 4200 cycles, of which the softmax's chain is
//     3650 (scores read and masked 1350, exponentials 1050, which is their unit's
//     rate, waiting for P's place 400, P written 850); shared memory alone would
//     take 2300.
//   Four chains of 9 rows over 33 to 131 thousand tokens, 8 bits: 0.58 GB in 179 us,
//     3.2 TB/s.  1530 ns a tile: the tile is copied in, read, written as f16 and read
//     by the products, 224 KB of shared-memory traffic or 1750 cycles, beside the
//     conversions and the exponentials.
//   One row over 1000 tokens: 12.1 us in a graph, launches and latencies.
// Every wait is bounded; on expiry the CTA raises DSPARK_ERR_TIMEOUT, drains its
// own copies and MMAs, frees TMEM and exits.
#pragma once
#include <cuda_fp8.h>

#include "kv_cache.cuh"
#include "tcgen05_attn.cuh"

namespace attn {

constexpr int BT = 128;                 // tokens of a tile
constexpr int SMEM_LIMIT = 232448;      // 227 KB
constexpr int CTL_BYTES = 3072;
constexpr int MAX_SLOTS = 12;           // tiles in a ring
constexpr int SEGS = 8;                 // segments published ahead
// What beginning and ending an item costs a CTA, in tiles; counted so that short
// contexts balance too.  The number is not critical (256 ragged chains: 282 us with one,
// 279 with two, 282 with three, where boxes differ by as much).
constexpr int ITEM_UNITS = 2;
// log2: how far scores may pass the reference, and where a raised reference puts the
// largest.  Beside a bf16 cache weights, their sum and O are floating-point numbers
// of f32's range, so nothing is lost by weights up to 2^32 (O of fewer than 2^31 tokens
// stays finite for |V| < 2^64); f16 weights start high, for the sake of the small ones.
template <bool FP8>
struct Range {
  static constexpr float RAISE = FP8 ? 14.0f : 32.0f, PEAK = FP8 ? 6.0f : 0.0f;
};
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Args {
  int R, heads, group, nodes_tile, max_nodes, n_rows, max_pages, page_shift, n_pages;
  const int *ctx, *row_start, *block_table;
  const uint64_t *anc;
  const float *k_scale, *v_scale;
  const uint8_t *v;                     // for non-finite values only
  int64_t page_bytes, token_bytes, head_bytes;
  float scale;
  bf16 *out;
  int64_t out_row, out_head;
  float *lse;
  float *part_o;                        // [ctas][2][NT][D]
  float *part_ml;                       // [ctas][2][2][NT]
  int *desc;                            // [ctas][8]: the item each CTA leaves to its successors
};

template <int TYPE, int D, int NT>
struct Geo {
  static constexpr bool FP8 = TYPE == DSPARK_KV_E4M3;
  static constexpr int PARTS = FP8 ? 1 : 2;          // of a weight, and of O
  // Up to 64 columns two sets of softmax warps take a segment's tiles in turn, each
  // with its S, P, references, sums and O: what one waits for (S, the tensor
  // memory, the group's barrier, P's place) the other's work covers.  128 columns
  // leave no room for a second P and O: one set of two groups, each with half the
  // columns.
  static constexpr int SETS = NT <= 64 ? 2 : 1;
  // Columns of a softmax thread's chunk: 32 where they divide the tile (128 rows in
  // chunks of 16: 558 against 299 us for 64 trees; 64 rows beside an 8-bit cache: 443
  // against 172 us for eight contexts of 32768).
  static constexpr int CW = NT % 32 ? 16 : 32;
  // Whether a segment's description is read again at its end, and what a tile needs of
  // it alone kept in registers: for wide tiles and beside an 8-bit cache, where they are
  // short (four contexts in 8 bits: 183 against 186 us; 64 trees: 299 against 303); 1024
  // chains of 400 tokens in tiles of 32 columns took 380 with it, 376 without.
  static constexpr bool REREAD = FP8 || NT > 32;
  static constexpr int CG = SETS == 2 ? 1 : 2;       // groups of four warps in a set
  static constexpr int CH = NT / (CW * CG);          // chunks of a thread
  static constexpr int SW = 4 * CG * SETS;
  static constexpr int CV = FP8 ? 4 : 0;
  // Warps 0..3 copy and issue (one of them rests), the softmax's follow, then those
  // that widen.  The softmax keeps a column's sums and scores in registers, more of
  // them than a thread's share: the others give theirs up.
  static constexpr int THREADS = 32 * (4 + SW + CV);
  static constexpr int REGS_FEW = 40, REGS_SOFTMAX = FP8 ? 208 : 232, REGS_WIDEN = 56;
  static_assert(SW == 8 && (CV == 0 || CV == 4), "warps 4..11: the softmax");
  static_assert(REGS_FEW + 2 * REGS_SOFTMAX + (FP8 ? REGS_WIDEN : 0) <=
                    65536 / THREADS / 8 * 8 * (THREADS / 128),
                "a block's registers");
  static constexpr int SLOT = BT * D * 2;
  // Q of the next segment beside the present one's, where two sets leave room
  static constexpr int QS = FP8 && NT > 32 ? 1 : SETS;
  static constexpr int Q_ONE = NT * D * 2, Q_BYTES = QS * Q_ONE;
  static constexpr int P_SET = BT * 128 * ((PARTS * NT + 63) / 64);
  static constexpr int P_BYTES = SETS * P_SET;
  static constexpr int ROOM = SMEM_LIMIT - CTL_BYTES - Q_BYTES - P_BYTES;
  static constexpr int RAW = FP8 ? BT * D : 0;
  // 8-bit: four widened tiles where they leave room for three of the copies in flight
  // (two read by the products, two being written), else three
  static constexpr int SLOTS = FP8 ? (4 * SLOT + 3 * RAW <= ROOM ? 4 : 3)
                                   : (ROOM / SLOT < MAX_SLOTS ? ROOM / SLOT : MAX_SLOTS);
  static constexpr int RAWS_FIT = FP8 ? (ROOM - SLOTS * SLOT) / (RAW + !FP8) : 0;
  static constexpr int RAWS = RAWS_FIT < MAX_SLOTS ? RAWS_FIT : MAX_SLOTS;
  static constexpr int SMEM_BYTES = SLOTS * SLOT + RAWS * RAW + Q_BYTES + P_BYTES + CTL_BYTES;
  // two tiles of S, and each set's O in its parts
  static constexpr uint32_t TMEM_USED = 2 * NT + SETS * PARTS * NT;
  static constexpr uint32_t TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  static_assert(SLOTS >= 3 && (!FP8 || RAWS >= 3) && SMEM_BYTES <= SMEM_LIMIT, "shared memory");
};

// f32 as an int of the same order (-0 below +0; NaN outside the numbers).
__device__ __forceinline__ int order_key(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float order_value(int k) {
  return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff);
}

// A request as the kernel takes it: every later index is in bounds by this.
struct Request {
  int row0, n, ctx, total, tiles, row_tiles;
  __device__ __forceinline__ bool set(const Args &a, int c, int start, int end) {
    bool ok = true;
    row0 = min(max(start, 0), a.n_rows);
    n = min(max(end, row0), a.n_rows) - row0;
    if (n > a.max_nodes) {
      n = a.max_nodes;
      ok = false;
    }
    ctx = max(c, 0);
    const long long cap = min((long long)a.max_pages << a.page_shift, 0x7fffff00ll);
    if ((long long)ctx + n > cap) {
      total = (int)cap;
      ctx = min(ctx, total);
      ok = false;
    } else {
      total = ctx + n;
    }
    tiles = n ? (total + BT - 1) / BT : 0;
    row_tiles = (n + a.nodes_tile - 1) / a.nodes_tile;
    return ok || n == 0;
  }
  __device__ __forceinline__ long long units(const Args &a) const {
    return n ? (long long)(tiles + ITEM_UNITS) * row_tiles * a.heads : 0;
  }
};

// One CTA's consecutive tiles of one item; none (tb == te): the end of its share.
struct Segment {
  int r, row0, n, ctx, total, tiles, h, node0, nodes, tb, te;
  float c;  // log2(e) * scale (* the head's K scale)
};

// Where the copying warp stands in its CTA's share of the list of units.
struct Walker {
  int r, h, rt, tile, over, next_ctx, next_end, end;  // over: own units of the item left
  long long pos, last;  // the next unit, and the end of the share
  Request q;
  float scale;            // of K in head h
  // What the next request and head need, read before it is needed.
  __device__ __forceinline__ void ahead(const Args &a) {
    if (r + 1 < a.R) {
      next_ctx = a.ctx[r + 1];
      next_end = a.row_start[r + 2];
    }
  }
  __device__ __forceinline__ void ahead_head(const Args &a) {
    scale = a.k_scale ? a.k_scale[h == a.heads ? 0 : h] : 1.0f;
  }
};

__device__ __forceinline__ bool next_segment(Walker &w, Segment &s, const Args &a) {
  w.pos += w.over;
  w.over = 0;
  if (w.pos >= w.last) return false;
  if (w.h == a.heads) {
    w.h = 0;
    do {
      if (++w.r >= a.R) {
        w.pos = w.last;
        return false;
      }
      const int start = w.end;
      w.end = w.next_end;
      w.q.set(a, w.next_ctx, start, w.end);
      w.ahead(a);
    } while (w.q.n == 0);
  }
  s.r = w.r;
  s.row0 = w.q.row0;
  s.n = w.q.n;
  s.ctx = w.q.ctx;
  s.total = w.q.total;
  s.tiles = w.q.tiles;
  s.h = w.h;
  s.node0 = w.rt * a.nodes_tile;
  s.nodes = min(a.nodes_tile, w.q.n - s.node0);
  s.c = a.scale * LOG2E * w.scale;
  s.tb = w.tile;
  s.te = (int)min((long long)w.q.tiles, w.tile + (w.last - w.pos));
  w.pos += s.te - s.tb;
  w.tile = s.te;
  if (s.te == w.q.tiles) {
    w.tile = 0;
    w.over = ITEM_UNITS;
    if (++w.rt == w.q.row_tiles) {
      w.rt = 0;
      ++w.h;
      w.ahead_head(a);
    }
  }
  return true;
}

// 2^k in two factors, as 2^k alone may pass f32's range (|k| <= 252).
__device__ __forceinline__ float times_power(float x, int k) {
  const int half = k / 2;
  return x * __int_as_float((127 + half) << 23) * __int_as_float((127 + k - half) << 23);
}

// Quotients of non-negative 64-bit numbers without the long division's code, which is
// a call: by a divisor below 2^16, digit by digit; and a quotient below 2^20, by an
// estimate that is at most one off.
__device__ __forceinline__ long long divide_small(long long x, uint32_t d) {
  uint32_t rest = 0;
  long long q = 0;
#pragma unroll 1
  for (int i = 48; i >= 0; i -= 16) {
    const uint32_t now = rest << 16 | ((uint32_t)(x >> i) & 0xffffu);
    q = q << 16 | now / d;
    rest = now % d;
  }
  return q;
}
__device__ __forceinline__ int quotient(long long x, long long y) {
  int q = (int)__fdividef((float)x, (float)y);
  if (q * y > x) --q;
  if ((q + 1) * y <= x) ++q;
  return q;
}

struct Ctl {
  uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], rfull[MAX_SLOTS], rempty[MAX_SLOTS];
  uint64_t q_full[2], q_empty[2], s_full[2], s_empty[2], drain;
  // by set: P written, its product done, O read by the segment's last set, and the
  // other's sums ready for it
  uint64_t p_full[2], pv_done[2], o_free[2], half[2];
  // by set and column (one set: 128 columns)
  alignas(16) float nm[128];  // minus the column's reference exponent (log2)
  // how far a tile's scores pass it, as an ordered key; at a segment's end where the
  // column's row of the output lies from the tile's first one
  alignas(16) int top[128];
  alignas(16) float other[2][64];  // a set's references and sums, for the other
  // of the warps before the shares are known; the shares' size, how many are a unit
  // longer, and where this CTA's ends, for an item that goes on in others
  long long sums[16], share, longer, end;
  Walker walk;
  // The share's segments as the copying warp comes to them, for the other roles.
  alignas(16) Segment seg[SEGS];
  uint64_t seg_full[SEGS], seg_empty[SEGS];
  // 8-bit: Q of a place is in f16, by which power of two it was multiplied (by segment
  // mod 4: S of three segments before is read), the warps' largest values on the way
  uint64_t q_ready[2];
  int q_exp[4], q_top[4];
  unsigned long long odd[4];  // nodes with non-finite V, by segment mod 4
  int tail;               // the CTA leaves an item to its successors
  int abort;
  uint32_t tmem;
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block");

// The library's bounded wait in few instructions, as many places have one; the
// clock, which is slow to read, is looked at once in 64 tries.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  uint64_t t0 = 0;
  for (uint32_t tries = 1; !tc::mbar_try_wait_sleep(bar, parity); ++tries) {
    if (tries & 63) continue;
    const uint64_t now = tc::globaltimer();
    if (t0 == 0) t0 = now;
    if (*abort) return false;
    if (now - t0 > tc::WAIT_LIMIT_NS) *abort = 1;
  }
  return true;
}
// By every lane of a warp; one answer for all.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

__device__ __forceinline__ void group_sync(int id) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

// A warpgroup's registers, given up or taken.
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Two 8-bit floats as two f16 (exact).
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.y << 16 | h.x;
}

// The maximum of v[j] over the warp's lanes, left in lane j (lanes j and j + 16 of
// 16 columns): 31 exchanges for 32 columns.  A NaN counts for nothing.
template <int CW>
__device__ __forceinline__ float column_max(float (&v)[CW], int lane) {
  if constexpr (CW == 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = fmaxf(v[j], __shfl_xor_sync(0xffffffffu, v[j], 16));
  }
#pragma unroll
  for (int o = CW / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float send = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
      v[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(Geo<TYPE, D, NT>::THREADS, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tma_k,
                          const __grid_constant__ CUtensorMap tma_v,
                          const __grid_constant__ CUtensorMap tma_q,
                          const __grid_constant__ Args a) {
  using G = Geo<TYPE, D, NT>;
  constexpr int CW = G::CW, CG = G::CG, SLOTS = G::SLOTS, RAWS = G::RAWS;
  constexpr int HALVES = D / 64;            // 64-column halves of a head
  constexpr int HALF_BYTES = BT * 128;      // one half of a tile
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *slots = smem;
  uint8_t *raws = slots + SLOTS * G::SLOT;
  uint8_t *sq = raws + RAWS * G::RAW;
  uint8_t *sp = sq + G::Q_BYTES;
  Ctl *ctl = reinterpret_cast<Ctl *>(sp + G::P_BYTES);
  volatile int *abort = &ctl->abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(&ctl->full[s], G::FP8 ? G::CV : 1);
      tc::mbar_init(&ctl->empty[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < RAWS; ++s) {
      tc::mbar_init(&ctl->rfull[s], 1);
      tc::mbar_init(&ctl->rempty[s], G::CV);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&ctl->q_full[b], 1);
      tc::mbar_init(&ctl->q_empty[b], 1);
      tc::mbar_init(&ctl->q_ready[b], 4);
      tc::mbar_init(&ctl->s_full[b], 1);
      tc::mbar_init(&ctl->s_empty[b], 4 * CG);
      tc::mbar_init(&ctl->p_full[b], 4 * CG);
      tc::mbar_init(&ctl->pv_done[b], 1);
      tc::mbar_init(&ctl->o_free[b], 4);
      tc::mbar_init(&ctl->half[b], 1);
    }
    tc::mbar_init(&ctl->drain, 1);
    for (int i = 0; i < 4; ++i) ctl->odd[i] = 0;
    ctl->tail = 0;
    ctl->abort = 0;
#pragma unroll 1
    for (int i = 0; i < SEGS; ++i) {
      tc::mbar_init(&ctl->seg_full[i], 1);
      // the MMA issuer, the warp that copies Q, each group, those that widen
      tc::mbar_init(&ctl->seg_empty[i], 2 + G::SETS * CG + (G::FP8 ? 1 : 0));
    }
    tc::fence_barrier_init();
    tc::tma_prefetch_desc(&tma_k);
    tc::tma_prefetch_desc(&tma_v);
    tc::tma_prefetch_desc(&tma_q);
  }
  if (warp == 1) tc::tmem_alloc(&ctl->tmem, G::TMEM_COLS);
  pdl_trigger();
  pdl_wait();

  // the list's length, and where this CTA's share of it begins
  const int per = (a.R + G::THREADS - 1) / G::THREADS;
  const int r_lo = min((int)threadIdx.x * per, a.R), r_hi = min(r_lo + per, a.R);
  long long mine = 0;
  Request own;  // the thread's only request, where it has one
#pragma unroll 1
  for (int r = r_lo; r < r_hi; ++r) {
    if (!own.set(a, a.ctx[r], a.row_start[r], a.row_start[r + 1]) && cta == 0)
      dspark_set_status(DSPARK_ERR_LENGTH);
    mine += own.units(a);
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) ctl->sums[warp] = upto;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  static_assert(G::THREADS / 32 <= 16, "a sum for each warp");
  long long units = lane < G::THREADS / 32 ? ctl->sums[lane] : 0;  // of warps up to the lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, units, o);
    if (lane >= o) units += t;
  }
  const long long before = __shfl_sync(0xffffffffu, units, max(warp - 1, 0));
  const long long first = (warp ? before : 0) + upto - mine;  // of requests before the thread's
  units = __shfl_sync(0xffffffffu, units, 31);                // of all requests
  // equal shares, the first ones a unit longer; with fewer units than CTAs the
  // first take one each, so that an item's pieces lie in consecutive CTAs
  const int shares = (int)min((long long)gridDim.x, max(units, 1ll));
  const long long share = divide_small(units, (uint32_t)shares), longer = units - share * shares;
  const long long u0 = cta < shares ? cta * share + min((long long)cta, longer) : units;
  const long long u1 = cta < shares ? u0 + share + (cta < longer) : units;
  if (threadIdx.x == 0) {
    ctl->share = share;
    ctl->longer = longer;
    ctl->end = u1;
  }
  Walker *walk0 = &ctl->walk;
  if (u0 == u1) {
    if (threadIdx.x == 0) {
      walk0->pos = walk0->last = units;
      walk0->over = 0;
    }
  } else if (mine > 0 && first <= u0 && u0 < first + mine) {
    long long off = u0 - first;
    int r = r_lo;
    Request q = own;
    if (per > 1) {
#pragma unroll 1
      for (;; ++r) {
        q.set(a, a.ctx[r], a.row_start[r], a.row_start[r + 1]);
        const long long m = q.units(a);
        if (off < m) break;
        off -= m;
      }
    }
    const int each = q.tiles + ITEM_UNITS;
    const int item = quotient(off, each), rest = (int)(off - (long long)item * each);
    walk0->over = max(ITEM_UNITS - rest, 0);
    walk0->tile = max(rest - ITEM_UNITS, 0);
    walk0->h = item / q.row_tiles;
    walk0->rt = item % q.row_tiles;
    walk0->r = r;
    walk0->q = q;
    walk0->end = a.row_start[r + 1];
    walk0->pos = u0;
    walk0->last = u1;
    walk0->ahead(a);
    walk0->ahead_head(a);
  }
  __syncthreads();
  const uint32_t tmem = ctl->tmem, tmem_o = tmem + 2 * NT;

  if (warp < 4) fewer_registers<G::REGS_FEW>();
  if (warp == 0) {
    // -------------------------------------------------- copies of K and V ----
    // Row tiles of one item read the same K and V: keep them in L2 for the next.
    const uint64_t pol =
        a.max_nodes > a.nodes_tile ? tc::policy_evict_normal() : tc::policy_evict_first();
    constexpr int RING = G::FP8 ? RAWS : SLOTS;
    uint64_t *full = G::FP8 ? ctl->rfull : ctl->full, *empty = G::FP8 ? ctl->rempty : ctl->empty;
    uint8_t *ring = G::FP8 ? raws : slots;
    constexpr int RING_BYTES = G::FP8 ? G::RAW : G::SLOT;
    const int rows = min(1 << a.page_shift, BT), boxes = BT / rows;
    const uint32_t box_bytes = (uint32_t)(rows * D * (G::FP8 ? 1 : 2));
    int slot = 0;
    uint32_t phase = 0, used = 0;
    bool ok = true;
    // Segments are published ahead of the copies, so that a role that needs a later
    // one never waits for room in the ring.
    constexpr int AHEAD = 2;
    Walker walk = ctl->walk;  // by every lane alike: what it reads ahead stays in flight
    int published = 0;
    auto publish = [&]() {
      const int i = published % SEGS;
      ok = ok && warp_wait(&ctl->seg_empty[i], ((published / SEGS) & 1) ^ 1, abort);
      Segment n;
      if (!next_segment(walk, n, a)) n.tb = n.te = n.r = n.total = 0;
      if (ok && lane == 0) {
        ctl->seg[i] = n;
        tc::mbar_arrive(&ctl->seg_full[i]);
      }
      __syncwarp();
      ++published;
    };
    // the page of box `lane` of a segment's tile; none past the request's end
    auto page_of = [&](const Segment &s, int tile) {
      const int p = tile * BT + lane * rows;
      return lane < boxes && p < s.total
                 ? a.block_table[(size_t)s.r * a.max_pages + (p >> a.page_shift)]
                 : 0;
    };
    int page = 0, next_page = 0;  // of this tile; of the next segment's first one
    int here = 0;                 // the segment
    while (ok) {
      if (published == 0) publish();
      const Segment s = ctl->seg[here % SEGS];
      if (s.tb == s.te) break;
      page = here == 0 ? page_of(s, s.tb) : next_page;
      bool asked = false;  // for the next segment's first page
      for (int tile = s.tb; ok && tile < s.te; ++tile) {
        const int id = page, p = tile * BT + lane * rows;
        const bool mine = lane < boxes && p < s.total;
        if (tile + 1 < s.te) page = page_of(s, tile + 1);
        const int n_boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const bool in = id >= 0 && id < a.n_pages;
        if (mine && !in) dspark_set_status(DSPARK_ERR_PAGES);
        const int z = in ? id : -1;  // outside the map: zeros
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (!warp_wait(&empty[slot], phase ^ 1, abort)) {
            ok = false;
            break;
          }
          if (lane == 0) tc::mbar_expect_tx(&full[slot], n_boxes * box_bytes);
          __syncwarp();
          if (mine) {
            const CUtensorMap *map = kv ? &tma_v : &tma_k;
            uint8_t *dst = ring + slot * RING_BYTES;
            const int y = p & ((1 << a.page_shift) - 1);
            if constexpr (G::FP8) {
              tc::tma_load_4d(dst + lane * rows * D, map, 0, y, s.h, z, &full[slot], pol);
            } else {
#pragma unroll
              for (int c = 0; c < HALVES; ++c)
                tc::tma_load_4d(dst + c * HALF_BYTES + lane * rows * 128, map, c * 64, y, s.h, z,
                                &full[slot], pol);
            }
          }
          used |= 1u << slot;
          if (++slot == RING) {
            slot = 0;
            phase ^= 1;
          }
        }
        // under the first tile's copies, what the next segments need
#pragma unroll 1
        while (ok && published <= here + AHEAD) publish();
        if (ok && !asked) {
          const Segment &n = ctl->seg[(here + 1) % SEGS];
          next_page = page_of(n, n.tb);
          asked = true;
        }
      }
      ++here;
    }
    // drain: every copy issued has landed (a slot's last fill is of this pass of
    // the ring before `slot`, of the last pass from it on)
    volatile int never = 0;
#pragma unroll 1
    for (int i = 0; i < RING; ++i)
      if (used >> i & 1) warp_wait(&full[i], i < slot ? phase : phase ^ 1, &never);
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer ----
    {
      constexpr uint32_t idesc_s = G::FP8 ? tc::idesc_f16(BT, NT) : tc::idesc_bf16(BT, NT);
      constexpr uint32_t idesc_o =
          (G::FP8 ? tc::idesc_f16(128, G::PARTS * NT) : tc::idesc_bf16(128, G::PARTS * NT)) |
          tc::IDESC_A_MN | tc::IDESC_B_MN;
      int k_slot = 0, v_slot = 1;
      uint32_t k_phase = 0, v_phase = 0;
      auto advance = [&](int &slot, uint32_t &phase) {
        slot += 2;
        if (slot >= SLOTS) {
          slot -= SLOTS;
          phase ^= 1;
        }
      };
      auto ready = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::mbar_test(bar, parity)) != 0;
      };
      // The products in the order in which their operands come: a tile's S as soon as
      // there are K, Q and a place for it, at most two tiles ahead of the O's, which
      // follow in turn.  Neither then waits behind the other: O's product frees V's
      // and P's places, S keeps the softmax fed.
      uint32_t t = 0, pv = 0, seg = 0;  // S and O products issued, segments begun
      bool more = true, have = false, first = true;
      int tile = 0, te = 0, total = 0, place = 0;  // place: of the tile in its segment
      // of the tiles between S and O, by turns: whether the tile adds to what its set
      // has, and the tokens from it on
      bool acc0 = false, acc1 = false;
      int tokens0 = 0, tokens1 = 0;
      uint32_t uses0 = 0, uses1 = 0;  // segments that each set had a part in
      uint32_t idle = 0;
      uint64_t since = 0;
      for (;;) {
        bool did = false;
        if (more && !have) {
          const int i = seg % SEGS;
          if (ready(&ctl->seg_full[i], (seg / SEGS) & 1)) {
            tile = ctl->seg[i].tb;
            te = ctl->seg[i].te;
            total = ctl->seg[i].total;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[i]);
            more = have = tile < te;
            first = true;
            place = 0;
          }
        }
        if (have && t - pv < 2) {
          const uint32_t b = t & 1;
          uint64_t *const q = G::FP8 ? &ctl->q_ready[seg % G::QS] : &ctl->q_full[seg % G::QS];
          if (ready(&ctl->full[k_slot], k_phase) && ready(&ctl->s_empty[b], ((t >> 1) & 1) ^ 1) &&
              (!first || ready(q, (seg / G::QS) & 1))) {
            did = true;
            tc::fence_after_sync();
            const uint64_t kd = tc::smem_desc_sw128(slots + k_slot * G::SLOT);
            const uint64_t qd = tc::smem_desc_sw128(sq + seg % G::QS * G::Q_ONE);
#pragma unroll 1
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::umma_warp(tmem + b * NT, kd + h * (HALF_BYTES / 16) + 2 * k,
                              qd + h * (NT * 128 / 16) + 2 * k, idesc_s, (h | k) != 0);
            tc::umma_commit_warp(&ctl->empty[k_slot]);
            tc::umma_commit_warp(&ctl->s_full[b]);
            advance(k_slot, k_phase);
            if (b) {
              acc1 = place >= G::SETS;
              tokens1 = total - tile * BT;
            } else {
              acc0 = place >= G::SETS;
              tokens0 = total - tile * BT;
            }
            ++place;
            ++t;
            first = false;
            if (++tile == te) {
              tc::umma_commit_warp(&ctl->q_empty[seg % G::QS]);
              ++seg;
              have = false;
            }
          }
        }
        if (!did && pv < t) {
          const int x = G::SETS == 2 ? pv & 1 : 0;
          const bool acc = pv & 1 ? acc1 : acc0;
          const int tokens = pv & 1 ? tokens1 : tokens0;
          const uint32_t uses = x ? uses1 : uses0;
          // a segment's first: the set's last O is read
          if (ready(&ctl->p_full[x], (pv / G::SETS) & 1) && ready(&ctl->full[v_slot], v_phase) &&
              (G::SETS == 1 || acc || uses == 0 || ready(&ctl->o_free[x], (uses - 1) & 1))) {
            did = true;
            uses0 += !acc && x == 0;
            uses1 += !acc && x == 1;
            tc::fence_after_sync();
            // D = 64: the 128-row operand's second 64 rows are the first again, and
            // accumulator lanes 64..127 are not read
            const uint64_t vd = tc::smem_desc_sw128_mn(slots + v_slot * G::SLOT,
                                                       D == 128 ? HALF_BYTES : 0);
            const uint64_t pd = tc::smem_desc_sw128_mn(sp + x * G::P_SET, HALF_BYTES);
            const uint32_t to = tmem_o + x * G::PARTS * NT;
            if (tokens >= BT) {
#pragma unroll
              for (int k = 0; k < BT / 16; ++k)
                tc::umma_warp(to, vd + 128 * k, pd + 128 * k, idesc_o, acc | (k != 0));
            } else {  // the steps that hold tokens; in the last some may be past the end
#pragma unroll 1
              for (int k = 0; k * 16 < tokens; ++k)
                tc::umma_warp(to, vd + 128 * k, pd + 128 * k, idesc_o, acc | (k != 0));
            }
            tc::umma_commit_warp(&ctl->empty[v_slot]);
            tc::umma_commit_warp(&ctl->pv_done[x]);
            advance(v_slot, v_phase);
            ++pv;
          }
        }
        if (did) {
          idle = 0;
          since = 0;
        } else {
          if (!more && !have && pv == t) break;
          if ((++idle & 63) == 0) {
            const uint64_t now = tc::globaltimer();
            if (since == 0) since = now;
            if (__any_sync(0xffffffffu, *abort != 0)) break;
            if (now - since > tc::WAIT_LIMIT_NS) *abort = 1;
          }
        }
      }
      tc::umma_commit_warp(&ctl->drain);  // all MMAs issued have finished
      volatile int never = 0;
      warp_wait(&ctl->drain, 0, &never);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------ copies of Q ----
    // A segment's tile of Q, as soon as the last product with what lay in its place
    // is done: rows node0.. of the request, the heads of one KV head.
    uint32_t i = 0;
    bool ok = true;
    for (;; ++i) {
      ok = warp_wait(&ctl->seg_full[i % SEGS], (i / SEGS) & 1, abort);
      if (!ok) break;
      const Segment *n = &ctl->seg[i % SEGS];
      if (n->tb == n->te) break;
      const int head = n->h * a.group, row = n->row0 + n->node0;
      if (i >= G::QS) ok = warp_wait(&ctl->q_empty[i % G::QS], (i / G::QS - 1) & 1, abort);
      if (!ok) break;
      if (lane == 0) {
        tc::mbar_arrive(&ctl->seg_empty[i % SEGS]);
        uint64_t *full = &ctl->q_full[i % G::QS];
        tc::mbar_expect_tx(full, HALVES * a.nodes_tile * a.group * 128);
        for (int c = 0; c < HALVES; ++c)
          tc::tma_load_3d(sq + i % G::QS * G::Q_ONE + c * NT * 128, &tma_q, c * 64, head, row, full,
                          tc::policy_evict_normal());
      }
      __syncwarp();
    }
    // drain: the last copies have landed (no later one took their place)
    volatile int never = 0;
    for (uint32_t k = i > G::QS ? i - G::QS : 0; k < i; ++k)
      warp_wait(&ctl->q_full[k % G::QS], (k / G::QS) & 1, &never);
  } else if (warp >= 4 && warp < 4 + G::SW) {
    more_registers<G::REGS_SOFTMAX>();
    // ----------------------------------------------------------- softmax ----
    const int quarter = warp & 3, group = (warp - 4) >> 2, bar = 1 + group;
    const int set = G::SETS == 2 ? group : 0, cg = G::SETS == 2 ? 0 : group;
    const int token = quarter * 32 + lane, c_group = cg * G::CH * CW;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const bool leader = quarter == 0 && lane == 0;  // of the group
    using R = Range<G::FP8>;
    uint8_t *const sp_set = sp + set * G::P_SET;
    float *const nm = ctl->nm + set * 64;
    int *const top = ctl->top + set * 64;
    const uint32_t tmem_set = tmem_o + set * G::PARTS * NT;
    // P[token][column]: 64-column halves; 16-byte chunk c of a row lies at
    // c ^ (token & 7)
    auto p_at = [&](int col) -> uint4 * {
      return reinterpret_cast<uint4 *>(sp_set + (col / 64) * HALF_BYTES + token * 128 +
                                       (((col % 64) / 8) ^ (token & 7)) * 16);
    };
    // At a segment's end the group's 64 columns of P take a chunk's f32 numbers, one
    // for each token and column.
    auto f32_at = [&](int row, int j) -> float * {
      return reinterpret_cast<float *>(sp_set + (c_group / 64) * HALF_BYTES + row * 128 +
                                       ((j / 4) ^ (row & 7)) * 16) + j % 4;
    };
    uint32_t t0 = 0, seg = 0;   // the segment's first tile, of all of the share's
    uint32_t mine = 0;          // tiles that this set has taken
    uint32_t uses = 0, helped = 0;  // segments that this set had a part in; that the other helped
    bool ok = true, gone = false;
    auto segment_here = [&](uint32_t i) {
      return wait(&ctl->seg_full[i % SEGS], (i / SEGS) & 1, abort);
    };
    for (;;) {
      ok = ok && __all_sync(0xffffffffu, segment_here(seg));
      if (group_any(bar, !ok)) break;
      const Segment *const now = &ctl->seg[seg % SEGS];
      Segment s;
      if constexpr (!G::REREAD) s = *now;
      const int tb = now->tb, n_tiles = now->te - tb, seg_ctx = now->ctx, total = now->total;
      if (n_tiles == 0) break;
      float c = now->c;
      const int rows = now->nodes * a.group;  // columns in use
      const int first = G::SETS == 2 ? (set ^ t0) & 1 : 0;  // this set's tiles: every SETS-th
      const bool part = first < n_tiles;
      // lane j: the ancestor mask of each chunk's column j
      unsigned long long word[G::CH];
#pragma unroll
      for (int ch = 0; ch < G::CH; ++ch) {
        const int col = c_group + ch * CW + lane;
        word[ch] = 0;
        if (lane < CW && col < rows) {
          const int node = now->node0 + col / a.group;
          word[ch] = a.anc ? a.anc[now->row0 + node] : (2ull << node) - 1;
        }
        if (quarter == 0 && lane < CW) {
          // a column that no row uses has no weight and calls for nothing
          nm[col] = col < rows ? 0.0f : -INFINITY;
          top[col] = order_key(-INFINITY);
        }
      }
      group_sync(bar);
      float l[G::CH][CW];
#pragma unroll
      for (int ch = 0; ch < G::CH; ++ch)
#pragma unroll
        for (int j = 0; j < CW; ++j) l[ch][j] = 0.0f;
      // bit j: column j of the chunk has no reference yet (its rows have seen nothing)
      uint32_t unset[G::CH];
#pragma unroll
      for (int ch = 0; ch < G::CH; ++ch) {
        const int n = min(max(rows - c_group - ch * CW, 0), CW);
        unset[ch] = n == 32 ? ~0u : (1u << n) - 1;
      }

      for (int k = first; k < n_tiles; k += G::SETS, ++mine) {
        const int tile = tb + k;
        const uint32_t t = t0 + k, b = t & 1;
        ok = ok && warp_wait(&ctl->s_full[b], (t >> 1) & 1, abort);
        // Q's power of two out of its scores: known since the product is done
        if (G::FP8 && k == first) c = times_power(now->c, -ctl->q_exp[seg & 3]);
        const int pos = tile * BT + token;
        const bool edge = tile * BT + BT > seg_ctx;  // some token is a node or past the end
        bool waited = mine == 0;
        tc::fence_after_sync();
        // which of each chunk's columns see this thread's token
        uint32_t seen[G::CH];
#pragma unroll
        for (int ch = 0; ch < G::CH; ++ch) seen[ch] = 0xffffffffu;
        if (edge) {
          const int node0 = tile * BT + quarter * 32 - seg_ctx;  // lane 0's node
          const int stop = min(total - seg_ctx, node0 + 32);
#pragma unroll
          for (int ch = 0; ch < G::CH; ++ch) {
            if (node0 + lane >= 0) seen[ch] = 0;
#pragma unroll 1
            for (int j = max(node0, 0); j < stop; ++j) {
              const uint32_t by = __ballot_sync(0xffffffffu, word[ch] >> j & 1);
              if (lane == j - node0) seen[ch] = by;
            }
          }
        }
        // e = c * S - reference, masked; again where the references are raised
        float e[G::CH][CW];
        auto used = [&](int ch) { return ch == 0 || c_group + ch * CW < rows; };
        int again;  // a zero that the compiler does not see: one copy of the loop's body
        asm volatile("mov.u32 %0, 0;" : "=r"(again));
        for (;; again = 1) {
          float most = -INFINITY;
          if (ok) {
            uint32_t sr[G::CH][CW];
#pragma unroll
            for (int ch = 0; ch < G::CH; ++ch)
              if (used(ch)) tc::tmem_ld(tmem + lanes + b * NT + c_group + ch * CW, sr[ch]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int ch = 0; ch < G::CH; ++ch) {
              if (!used(ch)) break;
              tc::reg_fence(sr[ch]);
#pragma unroll
              for (int j = 0; j < CW; j += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&nm[c_group + ch * CW + j]);
                e[ch][j] = fmaf(__uint_as_float(sr[ch][j]), c, m.x);
                e[ch][j + 1] = fmaf(__uint_as_float(sr[ch][j + 1]), c, m.y);
                e[ch][j + 2] = fmaf(__uint_as_float(sr[ch][j + 2]), c, m.z);
                e[ch][j + 3] = fmaf(__uint_as_float(sr[ch][j + 3]), c, m.w);
              }
              if (edge) {
#pragma unroll
                for (int j = 0; j < CW; ++j) e[ch][j] = seen[ch] >> j & 1 ? e[ch][j] : -INFINITY;
              }
            }
          }
          if (k == first && !again && tile * BT < seg_ctx) {
            // The first references: the scores of the tile's first token, which every
            // row sees, so that no column's maximum lies below its reference; one
            // that lies far above raises it.  No number: by the longer way.
            group_sync(bar);  // the references so far are read
#pragma unroll
            for (int ch = 0; ch < G::CH; ++ch) {
              const int c0 = c_group + ch * CW;
              if (quarter == 0 && used(ch)) {
                if (lane == 0) {
#pragma unroll
                  for (int j = 0; j < CW; j += 4)
                    *reinterpret_cast<float4 *>(&nm[c0 + j]) =
                        make_float4(e[ch][j], e[ch][j + 1], e[ch][j + 2], e[ch][j + 3]);
                }
                __syncwarp();
                const float x = nm[c0 + lane % CW];
                __syncwarp();
                if (lane < CW)
                  nm[c0 + lane] = c0 + lane >= rows
                                      ? -INFINITY
                                      : (fabsf(x) < INFINITY ? R::PEAK - x : INFINITY);
              }
            }
            group_sync(bar);
#pragma unroll
            for (int ch = 0; ch < G::CH; ++ch) {
              if (!used(ch)) break;
#pragma unroll
              for (int j = 0; j < CW; j += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&nm[c_group + ch * CW + j]);
                e[ch][j] += m.x;
                e[ch][j + 1] += m.y;
                e[ch][j + 2] += m.z;
                e[ch][j + 3] += m.w;
              }
              const int c0 = c_group + ch * CW;
              unset[ch] = __ballot_sync(0xffffffffu, lane < CW && nm[c0 + lane % CW] == INFINITY);
            }
          }
          uint32_t fresh_any = 0;
#pragma unroll
          for (int ch = 0; ch < G::CH; ++ch) {
            if (!used(ch)) break;
            fresh_any |= unset[ch];
#pragma unroll
            for (int j = 0; j < CW; ++j) most = fmaxf(most, e[ch][j]);
          }
          if (again || !group_any(bar, fresh_any != 0 || most > R::RAISE || !ok)) break;
          if (group_any(bar, !ok)) {
            gone = true;
            break;
          }
          if (!waited) ok = warp_wait(&ctl->pv_done[set], (mine - 1) & 1, abort);
          waited = true;
#pragma unroll
          for (int ch = 0; ch < G::CH; ++ch) {
            const int c0 = c_group + ch * CW;
            if (!used(ch)) break;
            // a first reference that was no number: as if there were none
            const uint32_t none =
                __ballot_sync(0xffffffffu, lane < CW && nm[c0 + lane % CW] == INFINITY);
            if (none) {
              unset[ch] |= none;
              group_sync(bar);
              if (quarter == 0 && lane < CW && (none >> lane & 1)) nm[c0 + lane] = 0.0f;
              group_sync(bar);
              uint32_t sr[CW];
              tc::tmem_ld(tmem + lanes + b * NT + c0, sr);
              tc::tmem_wait_ld();
              tc::reg_fence(sr);
#pragma unroll
              for (int j = 0; j < CW; ++j)
                e[ch][j] = seen[ch] >> j & 1 ? fmaf(__uint_as_float(sr[j]), c, nm[c0 + j])
                                             : -INFINITY;
            }
            // by how much the tile passes each reference: lane j for column j
            const float peak = column_max<CW>(e[ch], lane);
            if (lane < CW) atomicMax(&top[c0 + lane], order_key(peak));
            group_sync(bar);
            float raise = order_value(top[c0 + lane % CW]);
            const bool fresh = unset[ch] >> (lane % CW) & 1;
            raise -= R::PEAK;
            if (!(raise > -INFINITY) || (!fresh && raise < 0.0f)) raise = 0.0f;
            unset[ch] &= __ballot_sync(0xffffffffu, lane < CW && top[c0 + lane % CW] ==
                                                                     order_key(-INFINITY));
            if (k != first && ok) {  // what is summed so far, to the new references
              tc::fence_after_sync();
              const float keep = fresh ? 1.0f : ex2_fast(-raise);
#pragma unroll
              for (int j = 0; j < CW; ++j) l[ch][j] *= __shfl_sync(0xffffffffu, keep, j);
#pragma unroll 1
              for (int h = 0; h < G::PARTS * CW; h += 16) {
                const uint32_t at = tmem_set + lanes + (h < CW ? 0 : NT - CW) + c0 + h;
                uint32_t o[16];
                tc::tmem_ld16(at, o);
                tc::tmem_wait_ld();
                tc::reg_fence(o);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) *
                                         __shfl_sync(0xffffffffu, keep, (h + i) % CW));
                tc::tmem_st16(at, o);
              }
              tc::tmem_wait_st();
            }
            group_sync(bar);
            if (quarter == 0 && lane < CW) {
              nm[c0 + lane] -= raise;
              top[c0 + lane] = order_key(-INFINITY);
            }
            group_sync(bar);
          }
        }
        if (gone) break;
        tc::fence_before_sync();  // the tile's scores are read
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->s_empty[b]);
        // e's place is taken by the weights, as P has them: two bf16 roundings below
        // and their rests above, or two f16 ones
#pragma unroll
        for (int ch = 0; ch < G::CH; ++ch) {
          if (!used(ch)) break;
#pragma unroll
          for (int j = 0; j < CW; j += 2) {
            const float x = ex2_fast(e[ch][j]), y = ex2_fast(e[ch][j + 1]);
            l[ch][j] += x;
            l[ch][j + 1] += y;
            if constexpr (G::FP8) {
              const __half2 hi = __floats2half2_rn(x, y);
              e[ch][j] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&hi));
            } else {
              const uint32_t hi = pack_bf16(x, y);
              e[ch][j] = __uint_as_float(hi);
              e[ch][j + 1] = __uint_as_float(pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi)));
            }
          }
        }
        if (!waited) ok = warp_wait(&ctl->pv_done[set], (mine - 1) & 1, abort);  // P is free
#pragma unroll
        for (int ch = 0; ch < G::CH; ++ch) {
          if (!used(ch)) break;
#pragma unroll
          for (int j = 0; j < CW; j += 8) {
#pragma unroll
            for (int part = 0; part < G::PARTS; ++part)
              *p_at(part * NT + c_group + ch * CW + j) =
                  make_uint4(__float_as_uint(e[ch][j + part]), __float_as_uint(e[ch][j + 2 + part]),
                             __float_as_uint(e[ch][j + 4 + part]),
                             __float_as_uint(e[ch][j + 6 + part]));
          }
        }
        const int stop16 = (total + 15) & ~15;  // the products take 16 tokens a step
        const int warp_pos = tile * BT + quarter * 32;
        if (warp_pos + 31 >= seg_ctx && warp_pos < stop16) {
          // What a row does not see must not meet its zero weight as infinity or
          // NaN: V past the end is cleared, and so are the nodes' non-finite
          // values, which the epilogue gives to the rows that do see them.
          const uint32_t fill = 2 * t + 1;
          ok = ok && warp_wait(&ctl->full[fill % SLOTS], (fill / SLOTS) & 1, abort);
          uint8_t *row = slots + fill % SLOTS * G::SLOT + token * 128;
          if (ok && pos >= seg_ctx && pos < stop16) {
            // sign bit of a half of odd: its exponent is all ones
            constexpr uint32_t EXP = G::FP8 ? 0x7c00u : 0x7f80u, ONE = 0x8000u - EXP;
            constexpr uint32_t EXPS = EXP << 16 | EXP, ONES = ONE << 16 | ONE;
            uint32_t odd = 0;
#pragma unroll 1
            for (int i = cg * 4; i < HALVES * 8; i += CG * 4) {
              // four chunks of the row; which ones, by the token: no bank conflicts
              uint4 *const x = reinterpret_cast<uint4 *>(row + (i / 8) * HALF_BYTES);
              const int at = (i & 4) ^ (token & 7);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 y = x[at ^ q];
                odd |= ((y.x & EXPS) + ONES) | ((y.y & EXPS) + ONES) | ((y.z & EXPS) + ONES) |
                       ((y.w & EXPS) + ONES);
                if (pos >= total) x[at ^ q] = make_uint4(0, 0, 0, 0);
              }
            }
            if (pos < total && (odd & 0x80008000u)) {
              atomicOr(&ctl->odd[seg & 3], 1ull << (pos - seg_ctx));
#pragma unroll 1
              for (int i = cg * 4; i < HALVES * 8; i += CG * 4)
#pragma unroll 1
                for (int q = 0; q < 16; ++q) {
                  uint32_t *const w =
                      reinterpret_cast<uint32_t *>(row + (i / 8) * HALF_BYTES) +
                      ((((i & 4) ^ (token & 7)) ^ (q / 4)) * 4 + q % 4);
                  if ((*w & EXP) == EXP) *w &= 0xffff0000u;
                  if ((*w & EXP << 16) == EXP << 16) *w &= 0xffffu;
                }
            }
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->p_full[set]);
      }
      if (gone) break;

      // ------------------------------------------------- end of a segment ----
      // The set with the segment's last tile takes both sets' sums and O together.
      if constexpr (G::REREAD) s = *now;
      const int other = set ^ 1;
      const bool last = ((t0 + n_tiles - 1 - set) & (G::SETS - 1)) == 0;
      const bool both = G::SETS == 2 && n_tiles > 1;
      if (part) {
        ok = ok && warp_wait(&ctl->pv_done[set], (mine - 1) & 1, abort);
        // A column's sum over the tokens: in the warp by way of shared memory (lane j
        // adds column j), in a fixed order; then over the four warps.
        if (ok) {
          float sums[G::CH];
#pragma unroll
          for (int ch = 0; ch < G::CH; ++ch) {
#pragma unroll
            for (int j = 0; j < CW; j += 4)
              *reinterpret_cast<float4 *>(f32_at(token, j)) =
                  make_float4(l[ch][j], l[ch][j + 1], l[ch][j + 2], l[ch][j + 3]);
            __syncwarp();
            sums[ch] = 0.0f;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) sums[ch] += *f32_at(quarter * 32 + i, lane % CW);
            __syncwarp();
          }
#pragma unroll
          for (int ch = 0; ch < G::CH; ++ch)
            if (lane < CW) *f32_at(quarter * 32 + ch, lane) = sums[ch];
        }
        // `other` is free once its last reader has given this set's O back
        if (!last && uses) ok = ok && warp_wait(&ctl->o_free[set], (uses - 1) & 1, abort);
        if (last && both) {
          const uint32_t theirs = (t0 + n_tiles + (other ^ 1)) / 2;  // tiles of the other set
          ok = ok && warp_wait(&ctl->half[other], helped & 1, abort) &&
               warp_wait(&ctl->pv_done[other], (theirs - 1) & 1, abort);
        }
        if (group_any(bar, !ok)) {
          gone = true;
          break;
        }
        tc::fence_after_sync();
      }
      const bool whole = s.tb == 0 && s.te == s.tiles;
      const int piece = s.tb == 0 ? 1 : 0;
      if (part && quarter == 0 && lane < CW) {
        const float vs = a.v_scale ? a.v_scale[s.h] : 1.0f;
#pragma unroll
        for (int ch = 0; ch < G::CH; ++ch) {
          const int c0 = c_group + ch * CW, col = c0 + lane;
          if (col >= rows) continue;
          float sum = (*f32_at(ch, lane) + *f32_at(32 + ch, lane)) +
                      (*f32_at(64 + ch, lane) + *f32_at(96 + ch, lane));
          float ref = unset[ch] >> lane & 1 ? -INFINITY : -nm[col];
          if (!last) {
            ctl->other[0][col] = ref;
            ctl->other[1][col] = sum;
            continue;
          }
          float mine_w = 1.0f, their_w = 0.0f;
          if (both) {
            const float their_ref = ctl->other[0][col], to = fmaxf(ref, their_ref);
            mine_w = ref == -INFINITY ? 0.0f : ex2_fast(ref - to);
            their_w = their_ref == -INFINITY ? 0.0f : ex2_fast(their_ref - to);
            sum = mine_w * sum + their_w * ctl->other[1][col];
            ref = to;
          }
          const bool sees = s.ctx > 0 || (word[ch] & (~0ull >> (64 - s.n))) != 0;
          const int node = col / a.group, g = col - node * a.group;
          float f = 1.0f;
          if (!whole) {
            float *ml = a.part_ml + (size_t)(cta * 2 + piece) * 2 * NT + col;
            ml[0] = ref;
            ml[NT] = sum;
          } else {
            f = sees ? __fdividef(vs, sum) : 0.0f;
            if (a.lse) {
              a.lse[(size_t)(s.row0 + s.node0 + node) * a.heads * a.group + s.h * a.group + g] =
                  sees ? (ref + log2f(sum)) * LN2 : -INFINITY;
            }
          }
          top[col] = node * (int)a.out_row + g * (int)a.out_head;  // where the column's row lies
          // The factors of both O.  Without the other set's part `other` is not this set's
          // to write: the other may be at a later segment's end already, and its sums there.
          nm[col] = mine_w * f;
          if (both) ctl->other[1][col] = their_w * f;
        }
      }
      if (part && !last) {
        __syncwarp();
        if (quarter == 0 && lane == 0) tc::mbar_arrive(&ctl->half[set]);
      }
      const unsigned long long odd = last ? ctl->odd[seg & 3] : 0;
      if (last) {
        group_sync(bar);
        if (G::SETS == 2 ? leader : leader && group == 0) ctl->odd[(seg + (G::SETS == 2 ? 0 : 2)) & 3] = 0;
      }
      if (last && quarter * 32 < D) {
        const int d = token;  // accumulator lane = column of the head
#pragma unroll 1
        for (int c0 = c_group; c0 < min(rows, c_group + G::CH * CW); c0 += 16) {
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll 1
          for (int y = 0; y < (both ? 2 : 1); ++y) {  // this set's O, and the other's
            const uint32_t from = tmem_o + (y ? other : set) * G::PARTS * NT + lanes + c0;
            const float4 *f = reinterpret_cast<const float4 *>((y ? ctl->other[1] : nm) + c0);
            uint32_t o[16], o_lo[16] = {};
            tc::tmem_ld16(from, o);
            if constexpr (G::PARTS == 2) tc::tmem_ld16(from + NT, o_lo);
            tc::tmem_wait_ld();
            tc::reg_fence(o);
            if constexpr (G::PARTS == 2) tc::reg_fence(o_lo);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 g = f[i / 4];
              const float h[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                // an infinite V met both parts of a weight, of which the second may be
                // zero or below: the first part's product alone has its sign
                float both_parts = __uint_as_float(o[i + q]);
                if (G::PARTS == 2 && fabsf(both_parts) < INFINITY)
                  both_parts += __uint_as_float(o_lo[i + q]);
                x[i + q] = fmaf(both_parts, h[q], x[i + q]);
              }
            }
          }
          const int j0 = (c0 - c_group) % CW;  // of the chunk's columns
#pragma unroll 1
          for (unsigned long long m = odd; m; m &= m - 1) {
            const int at = __ffsll((long long)m) - 1, pos = s.ctx + at;
            const int page = a.block_table[(size_t)s.r * a.max_pages + (pos >> a.page_shift)];
            float v = 0.0f;
            if (page >= 0 && page < a.n_pages) {
              const uint8_t *src = a.v + page * a.page_bytes +
                                   (pos & ((1 << a.page_shift) - 1)) * a.token_bytes +
                                   s.h * a.head_bytes;
              if constexpr (G::FP8)
                v = __half2float(__ushort_as_half((unsigned short)widen_e4m3x2(src[d])));
              else
                v = __bfloat162float(reinterpret_cast<const bf16 *>(src)[d]);
            }
            const bool finite = fabsf(v) < INFINITY;
            uint32_t by = 0;
#pragma unroll
            for (int ch = 0; ch < G::CH; ++ch) {
              const uint32_t all = __ballot_sync(0xffffffffu, word[ch] >> at & 1);
              if ((c0 - c_group) / CW == ch) by = all >> j0;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!finite && (by >> i & 1)) x[i] += v;
          }
          const int count = min(rows - c0, 16);
          if (whole) {
            bf16 *const dst = a.out + (s.row0 + s.node0) * a.out_row +
                              (int64_t)s.h * a.group * a.out_head + d;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const int4 to = *reinterpret_cast<const int4 *>(&top[c0 + j]);
              if (j < count) dst[to.x] = __float2bfloat16_rn(x[j]);
              if (j + 1 < count) dst[to.y] = __float2bfloat16_rn(x[j + 1]);
              if (j + 2 < count) dst[to.z] = __float2bfloat16_rn(x[j + 2]);
              if (j + 3 < count) dst[to.w] = __float2bfloat16_rn(x[j + 3]);
            }
          } else {
            float *po = a.part_o + ((size_t)(cta * 2 + piece) * NT + c0) * D + d;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (j < count) po[j * D] = x[j];
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (G::SETS == 2 && last && lane == 0) {  // both O are read
        tc::mbar_arrive(&ctl->o_free[set]);
        if (both) tc::mbar_arrive(&ctl->o_free[other]);
      }
      if (last && leader && group == set && !whole && piece == 1) {
        // the item goes on in the CTAs up to the one that holds its last unit
        const long long end = ctl->end + (s.tiles - s.te), share = ctl->share, longer = ctl->longer;
        int *desc = a.desc + cta * 8;
        desc[1] = s.row0;
        desc[2] = s.node0;
        desc[3] = s.nodes;
        desc[4] = s.h;
        const long long u = end - 1, split = longer * (share + 1);
        desc[0] = (u < split ? quotient(u, share + 1) : (int)longer + quotient(u - split, share)) -
                  cta + 1;
        *(volatile int *)&ctl->tail = 1;
      }
      // the group's warps have read the segment's place (with a part in it they have met)
      if (G::REREAD && !part) group_sync(bar);
      __syncwarp();
      if (quarter == 0 && lane == 0) tc::mbar_arrive(&ctl->seg_empty[seg % SEGS]);
      uses += part;
      helped += last && both;
      t0 += n_tiles;
      ++seg;
    }
    __syncwarp();
  } else if (warp >= 4 + G::SW) {
    if constexpr (G::FP8) {
    fewer_registers<G::REGS_WIDEN>();
      // ------------------------- 8-bit tiles, and Q, made f16 -------------
      const int w = warp - 4 - G::SW, token = w * 32 + lane;
      int slot = 0, raw = 0;
      uint32_t phase = 0, raw_phase = 0;
      bool ok = true;
      for (uint32_t seg = 0; ok; ++seg) {
        ok = warp_wait(&ctl->seg_full[seg % SEGS], (seg / SEGS) & 1, abort);
        if (!ok) break;
        const int tiles = ctl->seg[seg % SEGS].te - ctl->seg[seg % SEGS].tb;
        const int rows = ctl->seg[seg % SEGS].nodes * a.group;
        if (tiles == 0) break;
        // Q's tile in place, times the power of two that brings its largest finite
        // value to 2^14; rows that nothing uses stay as they are
        ok = warp_wait(&ctl->q_full[seg % G::QS], (seg / G::QS) & 1, abort);
        if (!ok) break;
        uint8_t *q = sq + seg % G::QS * G::Q_ONE;
        int most = 0;  // bf16 bits without the sign: ordered as numbers
#pragma unroll 1
        for (int i = token; i < rows * HALVES * 8; i += 128) {
          const int row = i / (HALVES * 8), part = i % (HALVES * 8);
          const uint4 x = *reinterpret_cast<const uint4 *>(
              q + (part / 8) * NT * 128 + row * 128 + part % 8 * 16);
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int lo = v[k] & 0x7fff, hi = v[k] >> 16 & 0x7fff;
            most = max(most, max(lo < 0x7f80 ? lo : 0, hi < 0x7f80 ? hi : 0));
          }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) ctl->q_top[w] = most;
        group_sync(5);
        most = max(max(ctl->q_top[0], ctl->q_top[1]), max(ctl->q_top[2], ctl->q_top[3]));
        // its exponent is (most >> 7) - 127; a subnormal's is taken as the least
        const int up = most ? 14 + 127 - max(most >> 7, 1) : 0;
#pragma unroll 1
        for (int i = token; i < rows * HALVES * 8; i += 128) {
          const int row = i / (HALVES * 8), part = i % (HALVES * 8);
          uint4 *at = reinterpret_cast<uint4 *>(q + (part / 8) * NT * 128 + row * 128 +
                                                part % 8 * 16);
          const uint4 x = *at;
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(times_power(bf16_lo(v[k]), up),
                                                times_power(bf16_hi(v[k]), up));
            o[k] = *reinterpret_cast<const uint32_t *>(&h);
          }
          *at = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (w == 0 && lane == 0) ctl->q_exp[seg & 3] = up;
        tc::fence_async_smem();
        group_sync(5);  // q_top is read
        if (lane == 0) tc::mbar_arrive(&ctl->q_ready[seg % G::QS]);
        if (w == 0 && lane == 0) tc::mbar_arrive(&ctl->seg_empty[seg % SEGS]);
#pragma unroll 1
        for (int fill = 0; fill < 2 * tiles; ++fill) {
          ok = warp_wait(&ctl->rfull[raw], raw_phase, abort) &&
               warp_wait(&ctl->empty[slot], phase ^ 1, abort);
          if (!ok) break;
          const uint8_t *src = raws + raw * G::RAW;
          uint8_t *dst = slots + slot * G::SLOT;
          // eight lanes take eight tokens: the swizzles spread both sides over all
          // banks (raw rows of 128 bytes by token & 7, of 64 bytes by (token >> 1) & 3)
          const int raw_x = D == 128 ? token & 7 : (token >> 1) & 3;
          uint4 x[D / 16];  // all read before the first is written: they might overlap
#pragma unroll
          for (int p = 0; p < D / 16; ++p)
            x[p] = *reinterpret_cast<const uint4 *>(src + token * D + ((p ^ raw_x) * 16));
#pragma unroll
          for (int p = 0; p < D / 16; ++p) {
            const uint32_t v[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[2 * i] = widen_e4m3x2(v[i] & 0xffffu);
              o[2 * i + 1] = widen_e4m3x2(v[i] >> 16);
            }
            uint8_t *row = dst + (p / 4) * HALF_BYTES + token * 128;
            const int c = (2 * p) % 8;
            *reinterpret_cast<uint4 *>(row + ((c ^ (token & 7)) * 16)) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(row + (((c + 1) ^ (token & 7)) * 16)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&ctl->full[slot]);
            tc::mbar_arrive(&ctl->rempty[raw]);
          }
          if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1;
          }
          if (++raw == RAWS) {
            raw = 0;
            raw_phase ^= 1;
          }
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (ctl->abort) dspark_set_status(DSPARK_ERR_TIMEOUT);
    if (!ctl->tail) a.desc[cta * 8] = 0;
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, G::TMEM_COLS);
  }
}

// The cut items: block (c, y) joins the pieces of the item that CTA c began and
// could not finish, a warp taking one row, its own pieces in order:
//   out = sum_k e^{m_k - m} O_k / sum_k e^{m_k - m} l_k,  m the largest m_k.
// At most two pieces a CTA, a few MB from L2: bound by its launch, which the
// attention's end overlaps (some 3 us of the 12.1 of a single row).
template <int D>
__global__ void __launch_bounds__(128) tree_attention_join(const __grid_constant__ Args a, int nt) {
  constexpr int E = D / 32;
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int *desc = a.desc + c * 8;
  const int pieces = desc[0], col = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (pieces == 0 || col >= desc[3] * a.group) return;
  // piece 0 is CTA c's last one, piece k > 0 CTA (c + k)'s first
  auto at = [&](int k) -> size_t { return (size_t)(k ? 2 * (c + k) : 2 * c + 1) * nt; };
  float top = -INFINITY;
#pragma unroll 1
  for (int k = lane; k < pieces; k += 32) top = fmaxf(top, a.part_ml[2 * at(k) + col]);
  top = warp_max(top);
  float sum = 0.0f, o[E] = {};
#pragma unroll 4
  for (int k = 0; k < pieces; ++k) {
    const float m = a.part_ml[2 * at(k) + col], w = m == -INFINITY ? 0.0f : ex2_fast(m - top);
    const float *src = a.part_o + (at(k) + col) * D + lane;
    sum = fmaf(w, a.part_ml[2 * at(k) + nt + col], sum);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(w, src[32 * i], o[i]);
  }
  const int row = desc[1] + desc[2] + col / a.group, h = desc[4];
  const int head = h * a.group + col % a.group;
  const float f = (a.v_scale ? a.v_scale[h] : 1.0f) / sum;
  bf16 *dst = a.out + row * a.out_row + head * a.out_head + lane;
#pragma unroll
  for (int i = 0; i < E; ++i) dst[32 * i] = __float2bfloat16_rn(o[i] * f);
  if (a.lse && lane == 0)
    a.lse[(size_t)row * a.heads * a.group + head] = (top + log2f(sum)) * LN2;
}

}  // namespace attn
