// chunk_attention.cuh — attention of any number of new rows of each request over its
// paged KV cache, each row over the tokens up to its own position, on the tensor cores.
//
//   s_p = scale * q . K_p,  out = sum_p e^{s_p} V_p / sum_p e^{s_p},  p <= ctx + i
//
// Many rows meet every token here, so the products bound it, and the rows are the
// 128-row operand: a CTA takes an item, two tiles of 128 rows (nodes x query heads of one
// KV head) of one request and KV head, over the item's tokens in tiles of 128:
//   S_x [128 rows x 128 tokens] = Q_x . K^T       O_x [128 x D] += P_x . V     x = 0, 1
// A thread owns a row (a TMEM lane): maximum, sum and reference of its softmax lie in
// its registers, with no exchange between threads.  P takes the place of S in tensor
// memory, as bf16, and is the second product's operand from there: no weight passes
// through shared memory.  While one tile's softmax runs, the other's products do.
//
// The reference of a row's exponents is kept from tile to tile and raised (with O
// rescaled) only where a weight would exceed 2^RAISE.  f32 sums lose nothing by that, but
// weights of up to 2^32 beside a bf16 cache take that much of O's range: values below 2^64,
// of up to 2^31 tokens, overflow nowhere, as the header promises; larger ones may.
//
// Work is counted in tokens: an item costs its tokens and OVERHEAD more, the list of all
// items is cut into equal shares, one for each CTA, at tile boundaries, and the pieces of
// cut items are joined in order by chunk_attention_join (no atomics: the same bits from
// call to call).  Ragged batches balance so, and few rows over a long context are split
// over the GPU.
//
// One CTA per SM: warp 0 copies K and V (TMA, one copy for a page and 64 columns), warp 1
// issues the products, warp 2 copies Q, warp 3 clears what no row of the item may meet
// out of V's last tiles, two groups of four warps do the softmax of a tile each.
//
// Beside an 8-bit cache four more warps widen the tiles to f16, which holds every e4m3
// value and takes one conversion for two of them, in the place where they were copied
// to, so that as many are in flight as beside a bf16 cache.  They meet
// Q and P in f16: each row of Q is scaled by the power of two that brings its largest
// value to 2^14, weights are at most 2^14 and count down to 2^-24.
//
// What bounds it: a pair of tiles takes the tensor pipe 2048 cycles and about 2900 in
// all, as S's product reads shared memory at its full rate while P.V, the copies and the
// widening read and write it too.  32 query heads over 8 KV heads of 128: one prompt of 8192
// rows 331 to 343 us (1600 to 1660 TFLOP/s) for the first milliseconds; again and again for
// seconds, in a graph as by calls, the board's power limit takes the clock to 1810-1840 MHz,
// and it is 361 to 367 (1500 to 1520).  So eight chunks of 4096 over 4096: 2190 to 2220 us at
// first, 2500 (1320) for seconds, at 1430 MHz; and two chunks of 512 over 40 and 50 thousand
// tokens in 8 bits: 507 to 525 at first, 537 (1390) for seconds, at 1940 MHz.
// What an item's beginning and end cost counts in batches of short requests: 12 of 1 to
// 1500 rows 57 us, 705 TFLOP/s; there code that is seldom run counts too, as it comes through
// the instruction cache at about five cycles an instruction.  And an item whose rows fit
// one tile leaves the second stream of products empty: 64 next tokens over 512 to 4096
// beside a chunk of 512 rows over 2048 take 127 us, in 8 bits 160, where the bytes take 92
// and 47; without the chunk 109 and 131 here, 101 and 89 by the tree attention.
// Every wait is bounded; on expiry the CTA raises DSPARK_ERR_TIMEOUT, drains its own
// copies and MMAs, frees TMEM and exits.
#pragma once
#include "tree_attention.cuh"

namespace chunk {

using attn::fewer_registers;
using attn::more_registers;
using attn::pack_bf16;

constexpr int BT = 128;             // tokens of a tile
constexpr int BM = 128;             // rows of a tile of Q
constexpr int SMEM_LIMIT = 232448;  // 227 KB
constexpr int CTL_BYTES = 3 * 1024;
// Places for tiles of K and of V, each; more of them gain nothing (of V, three with 128 or
// four with 64 columns: one prompt of 8192 rows 342 us instead of 339, eight chunks of 4096
// over 4096 with 64 columns in 8 bits 2152 instead of 2036).
constexpr int SLOTS = 2;
constexpr int SEGS = 4;             // segments published ahead
// What beginning and ending an item costs, in tokens (a batch of 12 requests 57 us, by 256
// 58, by 384 63); the least share worth a CTA of its own, below any item's cost, so that no
// CTA takes two items while others are free (by 320, 100 rows 9.5 us instead of 7.5); and
// the least piece, in tiles, that an item is cut into.
constexpr int OVERHEAD = 192, MIN_SHARE = 192, MIN_PIECE = 2;
// log2: how far scores may pass the reference, and where a new reference puts the largest.
template <bool FP8>
struct Range {
  static constexpr float RAISE = FP8 ? 14.0f : 32.0f, PEAK = FP8 ? 6.0f : 0.0f;
};
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Args {
  int R, heads, group, nodes_tile, max_rows, n_rows, max_pages, page_shift, n_pages;
  const int *ctx, *row_start, *block_table;
  const float *k_scale, *v_scale;
  const uint8_t *v;                     // for non-finite values only
  int64_t page_bytes, token_bytes, head_bytes;
  float scale;
  bf16 *out;
  int64_t out_row, out_head;
  int wide;                             // every row of out begins at a multiple of 32 bytes
  float *lse;
  float4 *part_o;                       // [ctas][2][D / 4][2 BM]
  float *part_ml;                       // [ctas][2][2][2 BM]
  int *desc;                            // [ctas][8]: the item each CTA leaves, see below
};
// desc: 0 whether the CTA leaves an item to its successors, then its row0, node0, nodes,
// head; 5 whether the CTA's first item began before it: 1 and goes on after it, 2 and ends.

// Until the barrier's phase is complete; by every lane of a warp, one answer for all.  As
// short as can be: all roles' code shares the instruction cache (attn::warp_wait in its
// place: eight prompts of 1024 rows 83 us instead of 80, 32 of 256 49 instead of 47, eight
// chunks of 4096 rows of 64 columns in 8 bits 1874 instead of 1808).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait_sleep(bar, parity))) return true;
  uint32_t since = 0;
#pragma unroll 1
  do {
    uint32_t now;  // wraps after 4 s, and is asked at every hint's end
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
    if (since == 0) since = now | 1;
    if ((int)(now - since) > (int)tc::WAIT_LIMIT_NS) *abort = 1;
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
  } while (!__all_sync(0xffffffffu, tc::mbar_try_wait_sleep(bar, parity)));
  return true;
}

template <int TYPE, int D>
struct Geo {
  static constexpr bool FP8 = TYPE == DSPARK_KV_E4M3;
  static constexpr int CV = FP8 ? 4 : 0;
  static constexpr int THREADS = 32 * (12 + CV);
  static constexpr int REGS_FEW = FP8 ? 56 : 64, REGS_SOFTMAX = FP8 ? 184 : 216, REGS_WIDEN = 88;
  static_assert(REGS_FEW + 2 * REGS_SOFTMAX + (FP8 ? REGS_WIDEN : 0) <=
                    65536 / THREADS / 8 * 8 * (THREADS / 128),
                "a block's registers");
  // A tile's place.  An 8-bit tile of 128 columns is copied to its second half, where the
  // row of a token then holds the last 64 of them: a thread that has read its row may
  // write it.  One of 64 columns is copied behind it.
  static constexpr int SLOT = BT * D * 2, RAW_AT = D == 128 ? SLOT / 2 : SLOT;
  static constexpr int PLACE = SLOT + (FP8 && D == 64 ? BT * D : 0);
  static constexpr int Q_ONE = BM * D * 2, Q_BYTES = 2 * Q_ONE;
  static constexpr int SMEM_BYTES = 2 * SLOTS * PLACE + Q_BYTES + CTL_BYTES;
  static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;  // S_0, S_1, O_0, O_1
};

// A request as the kernel takes it: every later index is in bounds by this.
struct Request {
  int row0, n, ctx, total, items;  // items: of one KV head
  __device__ __forceinline__ bool set(const Args &a, int c, int start, int end) {
    bool ok = true;
    row0 = min(max(start, 0), a.n_rows);
    n = min(max(end, row0), a.n_rows) - row0;
    if (n > a.max_rows) {
      n = a.max_rows;
      ok = false;
    }
    ctx = max(c, 0);
    const long long cap = min((long long)a.max_pages << a.page_shift, 0x7fffff00ll);
    if ((long long)ctx + n > cap) {
      total = (int)cap;
      ok = false;
    } else {
      total = ctx + n;
    }
    items = (int)(((uint32_t)n + 2 * a.nodes_tile - 1) / (uint32_t)(2 * a.nodes_tile));
    return ok || n == 0;
  }
  // the cost of a KV head's first x items
  __device__ __forceinline__ long long upto(const Args &a, int x) const {
    const long long each = 2 * a.nodes_tile;
    long long s = x * ((long long)OVERHEAD + ctx) + each * x * (x + 1) / 2;
    if (x == items) s -= each * x - n;  // the last item's rows
    return s;
  }
  // an item's tokens, in tiles
  __device__ __forceinline__ int tiles(const Args &a, int item) const {
    const long long rows = min((long long)n, (long long)(item + 1) * 2 * a.nodes_tile);
    return (int)((min((long long)total, ctx + rows) + BT - 1) >> 7);
  }
};

// A place in the list of all work: tile `tile` of item `item` of (request, head).
struct Place {
  int r, h, item, tile;
};
__device__ __forceinline__ bool same_item(const Place &a, const Place &b) {
  return a.r == b.r && a.h == b.h && a.item == b.item;
}
__device__ __forceinline__ bool before(const Place &a, const Place &b) {
  if (a.r != b.r) return a.r < b.r;
  if (a.h != b.h) return a.h < b.h;
  return a.item != b.item ? a.item < b.item : a.tile < b.tile;
}

// Where cost `off` of request r's own lies: both CTAs beside a cut find the same place.
// By a warp.
__device__ __forceinline__ Place locate(const Args &a, const Request &q, int r, long long off) {
  const int lane = threadIdx.x & 31;
  Place p;
  p.r = r;
  const long long each = q.upto(a, q.items);
  p.h = attn::quotient(off, each);
  off -= p.h * each;
  int lo = 0;  // the last item that begins at or before off, 32 candidates at a time
  for (int n = q.items; n > 1;) {
    const int step = (int)(((uint32_t)n + 31) >> 5), at = lane * step;
    const uint32_t by =
        __ballot_sync(0xffffffffu, (long long)lane * step < n && q.upto(a, lo + at) <= off);
    const int k = 31 - __clz(by);  // the first one always does
    lo += k * step;
    n = min(step, n - k * step);
  }
  p.item = lo;
  const long long in = off - q.upto(a, lo) - OVERHEAD;
  const int tiles = q.tiles(a, lo);
  p.tile = in <= 0 ? 0 : (int)min((in + BT / 2) >> 7, (long long)tiles);
  if (p.tile < MIN_PIECE) p.tile = 0;
  if (p.tile && tiles - p.tile < MIN_PIECE) {  // the next item's beginning
    p.tile = 0;
    if (++p.item == q.items) {
      p.item = 0;
      if (++p.h == a.heads) {
        p.h = 0;
        ++p.r;
      }
    }
  }
  return p;
}

// One CTA's consecutive tiles [tb, te) of one item; none: the end of its share.
struct Segment {
  int r, row0, ctx, total, h, node0, nodes, tb, te, tiles;
  int count[2];     // of these tiles, those that each tile of Q meets
  float c;          // log2(e) * scale (* the head's K scale)
  unsigned odd[8];  // the item's nodes with non-finite V
};

struct Ctl {
  uint64_t k_full[SLOTS], k_empty[SLOTS], v_full[SLOTS], v_empty[SLOTS];
  uint64_t v_ready[SLOTS];          // and nothing in V that must not be met
  uint64_t kr_full[SLOTS], vr_full[SLOTS];  // 8-bit tiles as they were copied
  // by tile of Q: copied; in f16 (8 bits); its last S issued; S, P and the item's O complete
  uint64_t q_full[2], q_ready[2], q_empty[2], s_full[2], p_full[2], o_full[2], drain;
  uint64_t seg_full[SEGS], seg_empty[SEGS];
  long long sums[16];
  // the share's first place and the one behind its last: their request, and the cost in it
  Request cut_q[2];
  long long cut_off[2];
  int cut_r[2];
  Place first, last;
  alignas(16) Segment seg[SEGS];
  int tail[5], head;
  int abort;
  uint32_t tmem;
  // 8 bits: of each row of Q the largest exponent, by turns of items
  uint8_t q_exp[2][2][BM];
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block");

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Of two pairs of halves (f16 or bf16) the larger magnitudes, NaN before all; a is none
// below zero.
template <bool F16>
__device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("{\n .reg .b32 t;\n abs.f16x2 t, %2;\n max.NaN.f16x2 %0, %1, t;\n}\n"
        : "=r"(d)
        : "r"(a), "r"(b));
  else
    asm("{\n .reg .b32 t;\n abs.bf16x2 t, %2;\n max.NaN.bf16x2 %0, %1, t;\n}\n"
        : "=r"(d)
        : "r"(a), "r"(b));
  return d;
}

// D += A . B with A in tensor memory (bf16, two values in a column), by a warp in step.
__device__ __forceinline__ void umma_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Registers into 32 lanes x 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 32 bytes, aligned to as many.
__device__ __forceinline__ void store32(bf16 *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                        uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b),
               "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}
// Of a row of Q beside an 8-bit cache: the power of two that it was multiplied by, from
// its largest value's exponent (0 for a row of zeros).
__device__ __forceinline__ int row_exponent(int e) { return e ? 14 + 127 - e : 0; }

template <int TYPE, int D>
__global__ void __launch_bounds__(Geo<TYPE, D>::THREADS, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tma_k,
                           const __grid_constant__ CUtensorMap tma_v,
                           const __grid_constant__ CUtensorMap tma_q,
                           const __grid_constant__ Args a) {
  using G = Geo<TYPE, D>;
  constexpr int HALVES = D / 64;        // 64-column halves of a head
  constexpr int HALF_BYTES = BT * 128;  // one half of a tile
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *const sk = smem, *const sv = sk + SLOTS * G::PLACE;
  uint8_t *const sq = sv + SLOTS * G::PLACE;
  Ctl *ctl = reinterpret_cast<Ctl *>(sq + G::Q_BYTES);
  volatile int *abort = &ctl->abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(&ctl->k_full[s], G::FP8 ? G::CV : 1);
      tc::mbar_init(&ctl->v_full[s], G::FP8 ? G::CV : 1);
      tc::mbar_init(&ctl->k_empty[s], 2);  // each tile of Q is done with it
      tc::mbar_init(&ctl->v_empty[s], 2);
      tc::mbar_init(&ctl->v_ready[s], 1);
      tc::mbar_init(&ctl->kr_full[s], 1);
      tc::mbar_init(&ctl->vr_full[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(&ctl->q_full[x], 1);
      tc::mbar_init(&ctl->q_ready[x], 4);
      tc::mbar_init(&ctl->q_empty[x], 1);
      tc::mbar_init(&ctl->s_full[x], 1);
      tc::mbar_init(&ctl->p_full[x], 4);
      tc::mbar_init(&ctl->o_full[x], 1);
    }
    tc::mbar_init(&ctl->drain, 1);
    for (int i = 0; i < SEGS; ++i) {
      tc::mbar_init(&ctl->seg_full[i], 1);
      // both streams of the issuer, the copies of Q, the warp at V, the softmax's warps,
      // those that widen
      tc::mbar_init(&ctl->seg_empty[i], 12 + G::CV);
    }
    for (int i = 0; i < 5; ++i) ctl->tail[i] = 0;
    ctl->head = 0;
    ctl->abort = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch_desc(&tma_k);
    tc::tma_prefetch_desc(&tma_v);
    tc::tma_prefetch_desc(&tma_q);
  }
  if (warp == 1) tc::tmem_alloc(&ctl->tmem, G::TMEM_COLS);
  pdl_trigger();
  pdl_wait();

  // the list's cost, and where this CTA's share of it begins and ends
  {
    const int per = (a.R + G::THREADS - 1) / G::THREADS;
    const int r_lo = min((int)threadIdx.x * per, a.R), r_hi = min(r_lo + per, a.R);
    long long mine = 0;
    Request q;
#pragma unroll 1
    for (int r = r_lo; r < r_hi; ++r) {
      if (!q.set(a, a.ctx[r], a.row_start[r], a.row_start[r + 1]) && cta == 0)
        dspark_set_status(DSPARK_ERR_LENGTH);
      mine += q.upto(a, q.items) * a.heads;
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
    // of all warps, and of those before this one
    long long all = lane < G::THREADS / 32 ? ctl->sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += t;
    }
    const long long warps_before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
    const long long below = (warp ? warps_before : 0) + upto - mine;
    all = __shfl_sync(0xffffffffu, all, 31);
    const int shares = all >= (long long)MIN_SHARE * gridDim.x ? gridDim.x
                                                                : max((int)all / MIN_SHARE, 1);
    const long long share = all >> 32 ? attn::divide_small(all, (uint32_t)shares)
                                      : (uint32_t)all / (uint32_t)shares;
    const long long longer = all - share * shares;
    // the thread whose requests a cut lies in says which one; the last cut is the end
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int cut = cta + side;
      const long long u = cut * share + min((long long)cut, longer);
      if (threadIdx.x == 0 && (cut >= shares || u >= all)) ctl->cut_r[side] = -1;
      if (cut < shares && mine > 0 && below <= u && u < below + mine) {
        long long off = u - below;
        int r = r_lo;
        if (per > 1) {
#pragma unroll 1
          for (;; ++r) {
            q.set(a, a.ctx[r], a.row_start[r], a.row_start[r + 1]);
            const long long m = q.upto(a, q.items) * a.heads;
            if (off < m) break;
            off -= m;
          }
        }
        ctl->cut_r[side] = r;
        ctl->cut_off[side] = off;
        ctl->cut_q[side] = q;
      }
    }
    __syncthreads();
    if (warp < 2) {
      const int r = ctl->cut_r[warp];
      Place p = {a.R, 0, 0, 0};
      if (r >= 0) p = locate(a, ctl->cut_q[warp], r, ctl->cut_off[warp]);
      if (lane == 0) (warp ? ctl->last : ctl->first) = p;
    }
    __syncthreads();
  }
  const uint32_t tmem = ctl->tmem, tmem_o = tmem + 2 * BT;

  if (warp < 4) fewer_registers<G::REGS_FEW>();
  if (warp == 0) {
    // -------------------------------------------------- copies of K and V ----
    const uint64_t pol = tc::policy_evict_normal();
    const int rows = min(1 << a.page_shift, BT), boxes = BT / rows;
    const uint32_t box_bytes = (uint32_t)(rows * D * (G::FP8 ? 1 : 2));
    int k_slot = 0, v_slot = 0;
    uint32_t k_phase = 0, v_phase = 0, fills = 0;
    bool ok = true;
    Place p = ctl->first;
    const Place last = ctl->last;
    Request q = ctl->cut_q[0];
    int known = ctl->cut_r[0];
    for (int published = 0; ok; ++published) {
      while (before(p, last) && known != p.r) {
        q.set(a, a.ctx[p.r], a.row_start[p.r], a.row_start[p.r + 1]);
        known = p.r;
        if (q.n == 0) p = {p.r + 1, 0, 0, 0};
      }
      Segment s;
      s.tb = s.te = 0;
      const bool none = !before(p, last);
      if (!none) {
        s.r = p.r;
        s.row0 = q.row0;
        s.ctx = q.ctx;
        s.total = q.total;
        s.h = p.h;
        s.node0 = p.item * 2 * a.nodes_tile;
        s.nodes = min(2 * a.nodes_tile, q.n - s.node0);
        s.tiles = q.tiles(a, p.item);
        s.tb = p.tile;
        s.te = same_item(p, last) ? last.tile : s.tiles;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rows_x = min(s.nodes - x * a.nodes_tile, a.nodes_tile);
          const long long sees = min((long long)q.total,
                                     (long long)q.ctx + s.node0 + x * a.nodes_tile + rows_x);
          const int tiles_x = rows_x > 0 ? (int)((sees + BT - 1) >> 7) : 0;
          s.count[x] = max(0, min(s.te, tiles_x) - s.tb);
        }
        s.c = a.scale * LOG2E * (a.k_scale ? a.k_scale[p.h] : 1.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s.odd[i] = 0;
        p.tile = 0;
        if (++p.item == q.items) {
          p.item = 0;
          if (++p.h == a.heads) p = {p.r + 1, 0, 0, 0};
        }
      }
      const int i = published % SEGS;
      ok = warp_wait(&ctl->seg_empty[i], ((published / SEGS) & 1) ^ 1, abort);
      if (ok && lane == 0) {
        ctl->seg[i] = s;
        tc::mbar_arrive(&ctl->seg_full[i]);
      }
      __syncwarp();
      if (none) break;
      for (int tile = s.tb; ok && tile < s.te; ++tile) {
        const long long t0 = (long long)tile * BT + lane * rows;
        const bool mine = lane < boxes && t0 < s.total;
        const int id = mine ? a.block_table[(size_t)s.r * a.max_pages + (t0 >> a.page_shift)] : 0;
        const int n_boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const bool in = id >= 0 && id < a.n_pages;
        if (mine && !in) dspark_set_status(DSPARK_ERR_PAGES);
        const int z = in ? id : -1;  // outside the map: zeros
        const int y = (int)(t0 & ((1 << a.page_shift) - 1));
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int place = kv ? v_slot : k_slot;
          if (!warp_wait(kv ? &ctl->v_empty[place] : &ctl->k_empty[place],
                         (kv ? v_phase : k_phase) ^ 1, abort)) {
            ok = false;
            break;
          }
          uint64_t *bar = G::FP8 ? (kv ? &ctl->vr_full[place] : &ctl->kr_full[place])
                                 : (kv ? &ctl->v_full[place] : &ctl->k_full[place]);
          if (lane == 0) tc::mbar_expect_tx(bar, n_boxes * box_bytes);
          __syncwarp();
          if (mine) {
            const CUtensorMap *map = kv ? &tma_v : &tma_k;
            uint8_t *dst = (kv ? sv : sk) + place * G::PLACE;
            if constexpr (G::FP8) {
              tc::tma_load_4d(dst + G::RAW_AT + lane * rows * D, map, 0, y, s.h, z, bar, pol);
            } else {
#pragma unroll
              for (int c = 0; c < HALVES; ++c)
                tc::tma_load_4d(dst + c * HALF_BYTES + lane * rows * 128, map, c * 64, y, s.h, z,
                                bar, pol);
            }
          }
          ++fills;
          if (kv) {
            if (++v_slot == SLOTS) {
              v_slot = 0;
              v_phase ^= 1;
            }
          } else if (++k_slot == SLOTS) {
            k_slot = 0;
            k_phase ^= 1;
          }
        }
      }
    }
    // drain: every copy issued has landed
    volatile int never = 0;
    for (int i = 0; i < SLOTS; ++i)
      if ((uint32_t)i < (fills + 1) / 2)
        warp_wait(G::FP8 ? &ctl->kr_full[i] : &ctl->k_full[i], i < k_slot ? k_phase : k_phase ^ 1,
                  &never);
    for (int i = 0; i < SLOTS; ++i)
      if ((uint32_t)i < fills / 2)
        warp_wait(G::FP8 ? &ctl->vr_full[i] : &ctl->v_full[i], i < v_slot ? v_phase : v_phase ^ 1,
                  &never);
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer ----
    // Each tile of Q is a stream of products S, O, S, O, ..; a stream's next S follows
    // its last O at once, as P's place is S's.  K and V are polled, the streams taking turns
    // as their tiles come: a stream that held the other up there could wait for a place
    // which only the other gives back.  P hangs on its own stream alone, so that the warp
    // stays with it until it is there: the tensor pipe holds the other's products meanwhile,
    // and the next are issued sooner than by a round of polls.  A prompt of 8192 rows takes
    // 371 -> 341 us by that, eight chunks of 4096 over 4096 with 64 columns 1808 -> 1600, two
    // of 512 over 40 and 50 thousand tokens in 8 bits 562 -> 551.
    constexpr uint32_t idesc_s = G::FP8 ? tc::idesc_f16(BM, BT) : tc::idesc_bf16(BM, BT);
    constexpr uint32_t idesc_o =
        (G::FP8 ? tc::idesc_f16(BM, D) : tc::idesc_bf16(BM, D)) | tc::IDESC_B_MN;
    struct Stream {
      uint32_t seg, done, items;  // segments begun, O products and last S's issued, all in all
      int k, count, tiles;        // tiles of the segment taken; that this stream meets; all
      int k_slot, v_slot;
      uint32_t k_phase, v_phase;
      bool s_out, open, over;     // s_out: S is issued, its O is next
    } st[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) st[x] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, false, false, false};
    auto ready = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, tc::mbar_test(bar, parity)) != 0;
    };
    // Asked again and again, without sleep and with few looks at the clock.
    auto stay = [&](uint64_t *bar, uint32_t parity) {
      uint64_t t0 = 0;
      bool there = true;
      for (uint32_t tries = 1; !tc::mbar_try_wait(bar, parity); ++tries) {
        if (tries & 1023) continue;
        const uint64_t now = tc::globaltimer();
        if (t0 == 0) t0 = now;
        if (now - t0 > tc::WAIT_LIMIT_NS) *abort = 1;
        if (*abort) {
          there = false;
          break;
        }
      }
      return __all_sync(0xffffffffu, there) != 0;
    };
    auto next_k = [&](Stream &s) {
      if (++s.k_slot == SLOTS) {
        s.k_slot = 0;
        s.k_phase ^= 1;
      }
    };
    auto next_v = [&](Stream &s) {
      if (++s.v_slot == SLOTS) {
        s.v_slot = 0;
        s.v_phase ^= 1;
      }
    };
    uint32_t idle = 0;
    uint64_t since = 0;
    bool ok = true;
    while (ok && !(st[0].over && st[1].over)) {
      bool did = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Stream &s = st[x];
        if (s.over) continue;
        if (!s.open) {
          const int i = s.seg % SEGS;
          if (!ready(&ctl->seg_full[i], (s.seg / SEGS) & 1)) continue;
          s.tiles = ctl->seg[i].te - ctl->seg[i].tb;
          s.count = ctl->seg[i].count[x];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[i]);
          ++s.seg;
          s.k = 0;
          s.s_out = false;
          did = true;
          if (s.tiles == 0) {
            s.over = true;
            continue;
          }
          s.open = true;
        }
        if (s.s_out) {
          // O of tile k
          if (!ready(&ctl->v_ready[s.v_slot], s.v_phase)) continue;
          ok = stay(&ctl->p_full[x], s.done & 1);
          if (!ok) break;
          did = true;
          tc::fence_after_sync();
          const uint64_t vd =
              tc::smem_desc_sw128_mn(sv + s.v_slot * G::PLACE, D == 128 ? HALF_BYTES : 0);
#pragma unroll
          for (int k = 0; k < BT / 16; ++k)
            umma_ts_warp(tmem_o + x * D, tmem + x * BT + 8 * k, vd + 128 * k, idesc_o,
                         s.k > 0 || k != 0);
          tc::umma_commit_warp(&ctl->v_empty[s.v_slot]);
          if (s.k + 1 == s.count) tc::umma_commit_warp(&ctl->o_full[x]);
          next_v(s);
          ++s.done;
          ++s.k;
          s.s_out = false;
        }
        if (s.k < s.count) {
          // S of tile k
          if (!ready(&ctl->k_full[s.k_slot], s.k_phase) ||
              (s.k == 0 && !ready(G::FP8 ? &ctl->q_ready[x] : &ctl->q_full[x], s.items & 1)))
            continue;
          did = true;
          tc::fence_after_sync();
          const uint64_t kd = tc::smem_desc_sw128(sk + s.k_slot * G::PLACE);
          const uint64_t qd = tc::smem_desc_sw128(sq + x * G::Q_ONE);
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::umma_warp(tmem + x * BT, qd + h * (BM * 128 / 16) + 2 * k,
                            kd + h * (HALF_BYTES / 16) + 2 * k, idesc_s, (h | k) != 0);
          tc::umma_commit_warp(&ctl->s_full[x]);
          tc::umma_commit_warp(&ctl->k_empty[s.k_slot]);
          if (s.k + 1 == s.count) {
            tc::umma_commit_warp(&ctl->q_empty[x]);
            ++s.items;
          }
          next_k(s);
          s.s_out = true;
        } else if (s.k < s.tiles) {
          // a tile that no row of this stream sees: given back once it is there
          if (!ready(&ctl->k_full[s.k_slot], s.k_phase) ||
              !ready(&ctl->v_ready[s.v_slot], s.v_phase))
            continue;
          did = true;
          if (lane == 0) {
            tc::mbar_arrive(&ctl->k_empty[s.k_slot]);
            tc::mbar_arrive(&ctl->v_empty[s.v_slot]);
          }
          __syncwarp();
          next_k(s);
          next_v(s);
          ++s.k;
        }
        if (s.k == s.tiles) s.open = false;
      }
      if (did) {
        idle = 0;
        since = 0;
      } else if ((++idle & 63) == 0) {
        const uint64_t now = tc::globaltimer();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort != 0)) break;
        if (now - since > tc::WAIT_LIMIT_NS) *abort = 1;
      }
    }
    tc::umma_commit_warp(&ctl->drain);  // all MMAs issued have finished
    volatile int never = 0;
    warp_wait(&ctl->drain, 0, &never);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------ copies of Q ----
    uint32_t uses[2] = {0, 0};
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = warp_wait(&ctl->seg_full[i % SEGS], (i / SEGS) & 1, abort);
      if (!ok) break;
      const Segment *n = &ctl->seg[i % SEGS];
      if (n->tb == n->te) break;
      const int head = n->h * a.group, row = n->row0 + n->node0;
      const int count[2] = {n->count[0], n->count[1]};
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[i % SEGS]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (count[x] == 0 || !ok) continue;
        ok = warp_wait(&ctl->q_empty[x], (uses[x] & 1) ^ 1, abort);
        if (!ok) continue;
        if (lane == 0) {
          tc::mbar_expect_tx(&ctl->q_full[x], HALVES * a.nodes_tile * a.group * 128);
          for (int c = 0; c < HALVES; ++c)
            tc::tma_load_3d(sq + x * G::Q_ONE + c * BM * 128, &tma_q, c * 64, head,
                            row + x * a.nodes_tile, &ctl->q_full[x], tc::policy_evict_normal());
        }
        __syncwarp();
        ++uses[x];
      }
    }
    volatile int never = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x)  // drain
      if (uses[x]) warp_wait(&ctl->q_full[x], (uses[x] - 1) & 1, &never);
  } else if (warp == 3) {
    // ------------------------------------------------- V's last tiles ----
    // A weight of zero must not meet an infinity or NaN of a token that its row does not
    // see.  Rows of V past the item's last token are cleared; the non-finite values of
    // the tokens after its first row's are too, and the epilogue gives them to the rows
    // that do see them.
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = warp_wait(&ctl->seg_full[i % SEGS], (i / SEGS) & 1, abort);
      if (!ok) break;
      Segment *n = &ctl->seg[i % SEGS];
      const int tb = n->tb, te = n->te;
      if (tb == te) break;
      const long long first = (long long)n->ctx + n->node0;  // the first row's own token
      const long long end = min((long long)n->total, first + n->nodes);
      // what comes before it every row sees; rows may lie past a table that is too short
      const long long seen = min((long long)n->total, first + 1);
      for (int tile = tb; ok && tile < te; ++tile) {
        ok = warp_wait(&ctl->v_full[slot], phase, abort);
        if (ok && (long long)tile * BT + BT > seen) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int token = q * 32 + lane;
            const long long pos = (long long)tile * BT + token;
            uint8_t *row = sv + slot * G::PLACE + token * 128;
            if (pos >= end) {
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4 *>(row + h * HALF_BYTES + ((c ^ (token & 7)) * 16)) =
                      make_uint4(0, 0, 0, 0);
            } else if (pos > first) {
              // The largest magnitudes of the row's halves: no number, if the exponent is all
              // ones.  (A test of every half's exponent held up items of few tiles: 32 prompts
              // of 256 rows 51 us instead of 49, eight of 1024 86 instead of 83.)
              constexpr uint32_t EXP = G::FP8 ? 0x7c00u : 0x7f80u, ONE = 0x8000u - EXP;
              constexpr uint32_t EXPS = EXP << 16 | EXP, ONES = ONE << 16 | ONE;
              uint32_t odd = 0;
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const uint4 y = *reinterpret_cast<const uint4 *>(row + h * HALF_BYTES +
                                                                   ((c ^ (token & 7)) * 16));
                  odd = largest<G::FP8>(odd, y.x);
                  odd = largest<G::FP8>(odd, y.y);
                  odd = largest<G::FP8>(odd, y.z);
                  odd = largest<G::FP8>(odd, y.w);
                }
              if (((odd & EXPS) + ONES) & 0x80008000u) {
                const int node = (int)(pos - first);
                atomicOr(&n->odd[node >> 5], 1u << (node & 31));
#pragma unroll 1
                for (int w = 0; w < HALVES * 32; ++w) {
                  uint32_t *at = reinterpret_cast<uint32_t *>(row + (w / 32) * HALF_BYTES) + w % 32;
                  if ((*at & EXP) == EXP) *at &= 0xffff0000u;
                  if ((*at & EXP << 16) == EXP << 16) *at &= 0xffffu;
                }
              }
            }
          }
          tc::fence_async_smem();
          __threadfence_block();
        }
        __syncwarp();
        if (ok && lane == 0) tc::mbar_arrive(&ctl->v_ready[slot]);
        if (++slot == SLOTS) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[i % SEGS]);
    }
  } else if (warp < 12) {
    more_registers<G::REGS_SOFTMAX>();
    using R = Range<G::FP8>;
    // ----------------------------------------------------------- softmax ----
    const int x = (warp - 4) >> 2, quarter = warp & 3, m = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + x * BT, to = tmem_o + lanes + x * D;
    const int my_node = m / a.group, g = m - my_node * a.group;
    uint32_t tiles_done = 0, items_done = 0;
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      ok = warp_wait(&ctl->seg_full[seg % SEGS], (seg / SEGS) & 1, abort);
      if (!ok) break;
      const Segment *const n = &ctl->seg[seg % SEGS];
      const int tb = n->tb, count = n->count[x];
      if (tb == n->te) break;
      const int node = n->node0 + x * a.nodes_tile + my_node;  // of the request
      const bool mine = my_node < a.nodes_tile && x * a.nodes_tile + my_node < n->nodes;
      // tokens that this row sees, and that the tile's first row does
      const int sees = (int)min((long long)n->total, (long long)n->ctx + node + 1);
      const int all_see =
          (int)min((long long)n->total, (long long)n->ctx + n->node0 + x * a.nodes_tile + 1);
      // a row that is none has weights of 1 and calls for nothing
      float c = mine ? n->c : 0.0f;
      float nm = 0.0f;  // minus the reference (log2)
      bool unset = mine;
      float2 l0 = {0.0f, 0.0f}, l1 = {0.0f, 0.0f};
      for (int k = 0; k < count; ++k, ++tiles_done) {
        ok = warp_wait(&ctl->s_full[x], tiles_done & 1, abort);
        if (!ok) break;
        tc::fence_after_sync();
        // the row's power of two out of its scores: known since the product is done
        if (G::FP8 && k == 0)
          c = attn::times_power(c, -row_exponent(ctl->q_exp[items_done & 1][x][m]));
        float2 e[64];
        {
          uint32_t s[4][32];
          tc::tmem_ld32(ts, s[0]);
          tc::tmem_ld32(ts + 32, s[1]);
          tc::tmem_wait_ld();
          tc::reg_fence(s[0]);
          tc::reg_fence(s[1]);
          tc::tmem_ld32(ts + 64, s[2]);  // under the first half's work
          tc::tmem_ld32(ts + 96, s[3]);
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            if (j == 32) {
              tc::tmem_wait_ld();
              tc::reg_fence(s[2]);
              tc::reg_fence(s[3]);
            }
            e[j] = fma2(make_float2(__uint_as_float(s[j / 16][2 * j % 32]),
                                    __uint_as_float(s[j / 16][2 * j % 32 + 1])),
                        make_float2(c, c), make_float2(nm, nm));
          }
        }
        const int t0 = (tb + k) * BT;
        if (t0 + BT > all_see) {
          // by bits, which take half the instructions (32 prompts of 256 rows 53 -> 51 us);
          // beside 8 bits by comparisons (eight chunks of 4096 over 4096 2430 us, by bits 2510)
          const int lim = sees - t0;
          if constexpr (G::FP8) {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              e[j].x = 2 * j < lim ? e[j].x : -INFINITY;
              e[j].y = 2 * j + 1 < lim ? e[j].y : -INFINITY;
            }
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t hide = __funnelshift_lc(0u, ~0u, min(max(lim - 32 * h, 0), 32));
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (hide & 1u << (2 * j)) e[16 * h + j].x = -INFINITY;
                if (hide & 2u << (2 * j)) e[16 * h + j].y = -INFINITY;
              }
            }
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; ++j) top[j & 3] = max3(top[j & 3], e[j].x, e[j].y);
        const float most = max3(fmaxf(top[0], top[1]), top[2], top[3]);
        if (__any_sync(0xffffffffu, unset || most > R::RAISE)) {  // the first tile, and rarely
          const bool fresh = unset, number = fabsf(most) < INFINITY;
          const float raise = number && (fresh || most > R::RAISE) ? most - R::PEAK : 0.0f;
          if (number) unset = false;
          const float keep = fresh ? 1.0f : ex2_fast(-raise);
          if (k > 0 && __any_sync(0xffffffffu, keep != 1.0f)) {
            // O of the tiles so far is complete: its product came before this S
            l0.x *= keep;
            l0.y *= keep;
            l1.x *= keep;
            l1.y *= keep;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              uint32_t o[16];
              tc::tmem_ld16(to + d, o);
              tc::tmem_wait_ld();
              tc::reg_fence(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
              tc::tmem_st16(to + d, o);
            }
          }
          nm -= raise;
#pragma unroll
          for (int j = 0; j < 64; ++j) e[j] = add2(e[j], make_float2(-raise, -raise));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 v = make_float2(ex2_fast(e[8 * j + i].x), ex2_fast(e[8 * j + i].y));
            if (i & 1) l1 = add2(l1, v);
            else l0 = add2(l0, v);
            if constexpr (G::FP8) {
              const __half2 h = __floats2half2_rn(v.x, v.y);
              pk[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
              pk[i] = pack_bf16(v.x, v.y);
            }
          }
          tmem_st8(ts + 8 * j, pk);  // two weights a column
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->p_full[x]);
      }
      if (!ok) break;

      // ---------------------------------------------------- end of an item ----
      const bool whole = tb == 0 && n->te == n->tiles;
      const int piece = tb == 0 ? 1 : 0;
      const float sum = (l0.x + l0.y) + (l1.x + l1.y);
      const size_t slot = (size_t)cta * 2 + piece;
      if (!whole) {
        float *ml = a.part_ml + slot * 4 * BM + x * BM + m;
        ml[0] = unset && sum == 0.0f ? -INFINITY : -nm;
        ml[2 * BM] = sum;
        if (x == 0 && m == 0) {
          if (piece) {
            ctl->tail[0] = 1;
            ctl->tail[1] = n->row0;
            ctl->tail[2] = n->node0;
            ctl->tail[3] = n->nodes;
            ctl->tail[4] = n->h;
          } else {
            ctl->head = n->te == n->tiles ? 2 : 1;
          }
        }
      }
      if (count > 0) {
        ok = warp_wait(&ctl->o_full[x], items_done & 1, abort);
        if (!ok) break;
        ++items_done;
        tc::fence_after_sync();
        const float vs = a.v_scale ? a.v_scale[n->h] : 1.0f;
        const float f = whole ? __fdividef(vs, sum) : 1.0f;
        const int64_t row = (int64_t)n->row0 + node;
        const int head = n->h * a.group + g;
        if (whole && mine && a.lse)
          a.lse[row * a.heads * a.group + head] = (log2f(sum) - nm) * LN2;
        bf16 *const dst = a.out + row * a.out_row + head * a.out_head;
        // Two lanes write 64 bytes of one row together, of the even lane's and then of the
        // odd lane's: an SM writes a line's sectors one line at a time (a lane 16 bytes
        // of its own row: 32 prompts of 256 rows 56 us, a batch of 12 requests 69; 32
        // bytes: 51 and 63).
        const bool odd_lane = lane & 1;
        const unsigned there = __ballot_sync(0xffffffffu, mine) >> (lane & 30);
        bf16 *const even =
            reinterpret_cast<bf16 *>(__shfl_sync(
                0xffffffffu, reinterpret_cast<unsigned long long>(dst), lane & 30)) + 16 * odd_lane;
        bf16 *const odd =
            reinterpret_cast<bf16 *>(__shfl_sync(
                0xffffffffu, reinterpret_cast<unsigned long long>(dst), lane | 1)) + 16 * odd_lane;
        // rolled: it is fetched anew at every item's end
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          tc::tmem_ld32(to + d, o);
          tc::tmem_wait_ld();
          tc::reg_fence(o);
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = pack_bf16(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
            if (a.wide) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint32_t got =
                    __shfl_xor_sync(0xffffffffu, odd_lane ? o[j] : o[8 + j], 1);
                if (odd_lane) o[j] = got;
                else o[8 + j] = got;
              }
              if (there & 1) store32(even + d, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
              if (there & 2) store32(odd + d, o[8], o[9], o[10], o[11], o[12], o[13], o[14], o[15]);
            } else if (mine) {
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<uint4 *>(dst + d + 2 * j) =
                    make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          } else if (mine) {
            float4 *po = a.part_o + (slot * (D / 4) + d / 4) * 2 * BM + x * BM + m;
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              po[(j / 4) * 2 * BM] =
                  make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                              __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
          }
        }
        unsigned any = 0;
        for (int i = 0; i < 8; ++i) any |= n->odd[i];
        // Infinities and NaN, to the rows that see them.  Asked by the warp: bits of later
        // tokens may still come in.
        if (__any_sync(0xffffffffu, any != 0)) {
          __syncwarp();  // the row is written, by two lanes
          if (mine) {
            float *po = reinterpret_cast<float *>(a.part_o + slot * (D / 4) * 2 * BM + x * BM + m);
#pragma unroll 1
            for (int at = 1; at <= node - n->node0 && at < n->nodes; ++at) {
              if (!(n->odd[at >> 5] >> (at & 31) & 1)) continue;
              const long long pos = (long long)n->ctx + n->node0 + at;
              const int page = a.block_table[(size_t)n->r * a.max_pages + (pos >> a.page_shift)];
              if (page < 0 || page >= a.n_pages) continue;
              const uint8_t *src = a.v + page * a.page_bytes +
                                   (pos & ((1 << a.page_shift) - 1)) * a.token_bytes +
                                   n->h * a.head_bytes;
#pragma unroll 1
              for (int d = 0; d < D; ++d) {
                float y;
                if constexpr (G::FP8)
                  y = (src[d] & 0x7f) == 0x7f ? NAN : 0.0f;
                else
                  y = __bfloat162float(reinterpret_cast<const bf16 *>(src)[d]);
                if (fabsf(y) < INFINITY) continue;
                if (whole)
                  dst[d] = __float2bfloat16_rn(__bfloat162float(dst[d]) + y);
                else
                  po[(d / 4) * 8 * BM + d % 4] += y;
              }
            }
          }
        }
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[seg % SEGS]);
    }
    __syncwarp();
  } else {
    if constexpr (G::FP8) {
      fewer_registers<G::REGS_WIDEN>();
      // ------------------------------- 8-bit tiles, and Q, made f16 ----
      const int w = warp - 12, token = w * 32 + lane;
      int slot = 0;
      uint32_t phase = 0, uses[2] = {0, 0};
      bool ok = true;
      // A tile in its place, a thread a token: its row is read before it is written.  One
      // copy of this code for K and V: the roles together overrun the instruction cache (with
      // two, two chunks of 512 over 40 and 50 thousand tokens took 535 us instead of 507,
      // eight of 4096 over 4096 2750 instead of 2460).
      auto widen = [&](uint8_t *slot, uint64_t *raw, uint64_t *full, uint32_t phase) {
        ok = warp_wait(raw, phase, abort);
        // eight lanes take eight tokens: the swizzles spread both sides over all banks
        const int raw_x = D == 128 ? token & 7 : (token >> 1) & 3;
        uint4 v[D / 16];
#pragma unroll
        for (int p = 0; p < D / 16; ++p)
          v[p] = *reinterpret_cast<const uint4 *>(slot + G::RAW_AT + token * D +
                                                  ((p ^ raw_x) * 16));
#pragma unroll
        for (int p = 0; p < D / 16; ++p) {
          const uint32_t in[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[2 * i] = attn::widen_e4m3x2(in[i] & 0xffffu);
            o[2 * i + 1] = attn::widen_e4m3x2(in[i] >> 16);
          }
          uint8_t *row = slot + (p / 4) * HALF_BYTES + token * 128;
          const int cc = (2 * p) % 8;
          *reinterpret_cast<uint4 *>(row + ((cc ^ (token & 7)) * 16)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(row + (((cc + 1) ^ (token & 7)) * 16)) =
              make_uint4(o[4], o[5], o[6], o[7]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (ok && lane == 0) tc::mbar_arrive(full);
      };
      for (uint32_t seg = 0; ok; ++seg) {
        ok = warp_wait(&ctl->seg_full[seg % SEGS], (seg / SEGS) & 1, abort);
        if (!ok) break;
        const Segment *n = &ctl->seg[seg % SEGS];
        const int tiles = n->te - n->tb, count[2] = {n->count[0], n->count[1]};
        if (tiles == 0) break;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            widen((kv ? sv : sk) + slot * G::PLACE, kv ? &ctl->vr_full[slot] : &ctl->kr_full[slot],
                  kv ? &ctl->v_full[slot] : &ctl->k_full[slot], phase);
            if (kv || t != 0) continue;
            // Q's tiles in place, a thread a row: times the power of two that brings its
            // largest finite value to 2^14
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              const uint32_t use = x ? uses[1] : uses[0];
              if ((x ? count[1] : count[0]) == 0) continue;
              ok = ok && warp_wait(&ctl->q_full[x], use & 1, abort);
              uint8_t *row = sq + x * G::Q_ONE + token * 128;
              int most = 0;  // bf16 bits without the sign: ordered as numbers
#pragma unroll
              for (int p = 0; p < HALVES * 8; ++p) {
                const uint4 y = *reinterpret_cast<const uint4 *>(row + (p / 8) * BM * 128 +
                                                                 ((p % 8) ^ (token & 7)) * 16);
                const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int lo = v[i] & 0x7fff, hi = v[i] >> 16 & 0x7fff;
                  most = max(most, max(lo < 0x7f80 ? lo : 0, hi < 0x7f80 ? hi : 0));
                }
              }
              // its exponent is (most >> 7) - 127; a subnormal's is taken as the least
              const int top = most ? max(most >> 7, 1) : 0, up = row_exponent(top);
#pragma unroll
              for (int p = 0; p < HALVES * 8; ++p) {
                uint4 *at = reinterpret_cast<uint4 *>(row + (p / 8) * BM * 128 +
                                                      ((p % 8) ^ (token & 7)) * 16);
                const uint4 y = *at;
                const uint32_t v[4] = {y.x, y.y, y.z, y.w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __half2 h = __floats2half2_rn(attn::times_power(bf16_lo(v[i]), up),
                                                      attn::times_power(bf16_hi(v[i]), up));
                  o[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *at = make_uint4(o[0], o[1], o[2], o[3]);
              }
              ctl->q_exp[use & 1][x][token] = (uint8_t)top;
              tc::fence_async_smem();
              __syncwarp();
              if (ok && lane == 0) tc::mbar_arrive(&ctl->q_ready[x]);
              if (x) ++uses[1];
              else ++uses[0];
            }
          }
          if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1;
          }
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->seg_empty[seg % SEGS]);
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (ctl->abort) dspark_set_status(DSPARK_ERR_TIMEOUT);
    int *desc = a.desc + cta * 8;
    for (int i = 0; i < 5; ++i) desc[i] = ctl->tail[i];
    desc[5] = ctl->head;
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, G::TMEM_COLS);
  }
}

// The cut items: block (c, x, y) joins 16 columns of tile x of the item that CTA c began
// and could not finish, a thread taking one row, its own pieces in order:
//   out = sum_k e^{m_k - m} O_k / sum_k e^{m_k - m} l_k,  m the largest m_k.
template <int D>
__global__ void __launch_bounds__(BM) chunk_attention_join(const __grid_constant__ Args a) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x, x = blockIdx.y, d0 = blockIdx.z * 16, m = threadIdx.x;
  const int *desc = a.desc + c * 8;
  const int lane = m & 31;
  // piece 0 is CTA c's last one, piece k > 0 CTA (c + k)'s first: up to the first CTA whose
  // piece ends the item
  int heads_here = c + 1 + lane < (int)gridDim.x ? a.desc[(c + 1 + lane) * 8 + 5] : 2;
  if (desc[0] == 0) return;
  int pieces = 1;
  for (int k = 0;; k += 32) {
    const uint32_t ends = __ballot_sync(0xffffffffu, heads_here != 1);
    if (ends) {
      pieces += k + __ffs((int)ends);
      break;
    }
    heads_here = c + 33 + k + lane < (int)gridDim.x ? a.desc[(c + 33 + k + lane) * 8 + 5] : 2;
  }
  const int node = m / a.group, g = m - node * a.group;
  const int in_item = x * a.nodes_tile + node;
  if (node >= a.nodes_tile || in_item >= desc[3]) return;
  // Piece by piece, two at a time and all of their values asked for at once, as reads that
  // wait for one another bound it; the sums so far follow the largest m.  (One after the
  // other, m first, by 32 columns: a batch of 12 requests 60.5 us instead of 58.7, 65 rows
  // over 60 thousand tokens 104 instead of 98.)
  float top = -INFINITY, sum = 0.0f, o[16] = {};
  for (int k = 0; k < pieces; k += 2) {
    float m_k[2], l_k[2];
    float4 v[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int j = min(k + p, pieces - 1);
      const size_t slot = j ? 2 * (size_t)(c + j) : 2 * (size_t)c + 1;
      const float *ml = a.part_ml + slot * 4 * BM + x * BM + m;
      const float4 *src = a.part_o + (slot * (D / 4) + d0 / 4) * 2 * BM + x * BM + m;
      m_k[p] = ml[0];
      l_k[p] = ml[2 * BM];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[p][i] = src[i * 2 * BM];
    }
    if (k + 1 == pieces) m_k[1] = -INFINITY;
    const float now = fmaxf(top, fmaxf(m_k[0], m_k[1]));
    if (now == -INFINITY) continue;  // the row saw nothing there
    const float keep = ex2_fast(top - now);
    top = now;
    sum *= keep;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= keep;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (m_k[p] == -INFINITY) continue;
      const float w = ex2_fast(m_k[p] - now);
      sum = fmaf(w, l_k[p], sum);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[4 * i] = fmaf(w, v[p][i].x, o[4 * i]);
        o[4 * i + 1] = fmaf(w, v[p][i].y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(w, v[p][i].z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(w, v[p][i].w, o[4 * i + 3]);
      }
    }
  }
  const int h = desc[4], head = h * a.group + g;
  const int64_t row = (int64_t)desc[1] + desc[2] + in_item;
  const float f = __fdividef(a.v_scale ? a.v_scale[h] : 1.0f, sum);
  bf16 *dst = a.out + row * a.out_row + head * a.out_head + d0;
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    *reinterpret_cast<uint4 *>(dst + i) =
        make_uint4(pack_bf16(o[i] * f, o[i + 1] * f), pack_bf16(o[i + 2] * f, o[i + 3] * f),
                   pack_bf16(o[i + 4] * f, o[i + 5] * f), pack_bf16(o[i + 6] * f, o[i + 7] * f));
  if (a.lse && d0 == 0) a.lse[row * a.heads * a.group + head] = (top + log2f(sum)) * LN2;
}

}  // namespace chunk
