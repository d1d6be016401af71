// kv_cache.cu — the bookkeeping of a round over the target's paged KV cache:
// rows, pages, slots and masks (plan), writing the rows (append), the confirmed
// path of a drafted tree (accept) and moving it together (compact).
#include "kv_cache.cuh"

DSPARK_DECLARE_STATUS(s_status_kv)

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_CLUSTER = 8;
constexpr int MAX_R = 16384;

struct PlanArgs {
  int R, gamma, extra, n_rows, page_shift, n_pages, max_pages;
  const int *ctx, *len, *parent, *held, *n_free;
  int *free_pages, *block_table, *held_out, *n_free_out, *row_start, *position;
  int64_t *slot;
  uint64_t *anc;
};

__device__ __forceinline__ void cluster_or_block_sync(bool cluster) {
  if (cluster)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
  else
    __syncthreads();
}

// Exclusive sums over the block's threads of three values; totals in `sum`.
__device__ __forceinline__ void block_scan3(int64_t (&v)[3], int64_t (&sum)[3],
                                            int64_t (*warp_sums)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    inc[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, inc[i], o);
      if (lane >= o) inc[i] += t;
    }
    if (lane == 31) warp_sums[warp][i] = inc[i];
  }
  __syncthreads();
  // every warp scans the 32 warps' sums itself: no second barrier
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int64_t w = warp_sums[lane][i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    sum[i] = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    v[i] = before + inc[i] - v[i];
  }
}

// One round's plan.  Every CTA of the cluster takes the same sums over the
// requests (rows, pages needed, pages returned; a few KB from L2), so that none
// waits for another's; the work over pages and rows is then spread over all of
// them.  One barrier separates the pages pushed by requests that left from the
// pages popped.  Sums in 64 bits: no input overflows them.
// 0.4 MB for 1024 trees of 31 drafts: bound by the chain of dependent reads, sums and
// barriers.  12.1 us there with the cluster, 3.9 us for four requests (one CTA), in a graph.
__global__ void __launch_bounds__(PLAN_THREADS, 1) kv_plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  __shared__ int64_t warp_sums[32][3];
  int *row_off = smem;                   // [R + 1] first row, at most n_rows
  int *need_off = row_off + a.R + 1;     // [R + 1] pages needed before request r
  int *held = need_off + a.R + 1;        // [R] held_out may be held: read once
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int warps = ctas * (PLAN_THREADS / 32), warp = cta * (PLAN_THREADS / 32) + (tid >> 5);
  const int ps = 1 << a.page_shift;
  pdl_trigger();
  pdl_wait();

  int top = a.n_free[0];
  if (top < 0 || top > a.n_pages) {
    dspark_set_status(DSPARK_ERR_PAGES);
    top = top < 0 ? 0 : a.n_pages;
  }
  const int n_free = top;
  const int most = a.parent ? a.gamma + a.extra : (a.anc ? DSPARK_MAX_NODES : 0x7fffffff);

  // rows, pages needed and pages returned of request r
  auto request = [&](int r, int &h, int64_t &rows, int64_t &need, int64_t &back) {
    const int c = a.ctx[r], l = a.len[r];
    h = a.held[r];
    if (h < 0 || h > a.max_pages) {
      dspark_set_status(DSPARK_ERR_PAGES);
      h = h < 0 ? 0 : a.max_pages;
    }
    rows = need = back = 0;
    if (c < 0) {
      back = h;
      return;
    }
    if (l >= 0) rows = (int64_t)l + a.extra;
    if (l < 0 || rows > most) dspark_set_status(DSPARK_ERR_LENGTH);
    if (rows > most) rows = most;
    const int64_t pages = (c + rows + ps - 1) >> a.page_shift;
    if (pages > a.max_pages)
      dspark_set_status(DSPARK_ERR_LENGTH);
    else if (pages > h)
      need = pages - h;
  };
  const int per = (a.R + PLAN_THREADS - 1) / PLAN_THREADS;
  const int r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
  int64_t mine[3] = {0, 0, 0}, sum[3];
  for (int r = r0; r < r1; ++r) {
    int64_t rows, need, back;
    int h;
    request(r, h, rows, need, back);
    held[r] = h;
    row_off[r] = (int)min(rows, (int64_t)0x7fffffff);
    need_off[r] = (int)(need ? need : -back);
    mine[0] += rows;
    mine[1] += need;
    mine[2] += back;
  }
  block_scan3(mine, sum, warp_sums);
  int64_t rows_at = mine[0], need_at = mine[1], back_at = mine[2];
  if (sum[0] > a.n_rows && tid == 0) dspark_set_status(DSPARK_ERR_LENGTH);
  const int64_t pushed = min(sum[2], (int64_t)(a.n_pages - n_free));
  if (pushed < sum[2] && tid == 0) dspark_set_status(DSPARK_ERR_PAGES);
  top = n_free + (int)pushed;
  for (int i = 0; i < per; ++i) {
    const int r = r0 + i;
    int back = 0;
    int64_t to = 0;
    if (r < r1) {
      const int rows = row_off[r], need = need_off[r];
      row_off[r] = (int)min(rows_at, (int64_t)a.n_rows);
      need_off[r] = (int)min(need_at, (int64_t)0x7fffffff);
      if (cta == 0) a.row_start[r] = row_off[r];
      rows_at += rows;
      if (need >= 0) {
        need_at += need;
      } else {
        back = -need;
        to = n_free + back_at;
        back_at += back;
      }
    }
    // requests that left: their pages onto the stack, by the whole warp of the
    // CTA whose turn it is
    uint32_t left = __ballot_sync(0xffffffffu, back > 0 && r % ctas == cta);
    for (; left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      const int rr = __shfl_sync(0xffffffffu, r, from), n = __shfl_sync(0xffffffffu, back, from);
      const int64_t at = __shfl_sync(0xffffffffu, to, from);
      const int *table = a.block_table + (size_t)rr * a.max_pages;
      for (int j = lane; j < n; j += 32)
        if (at + j < a.n_pages) a.free_pages[at + j] = table[j];
    }
  }
  const int total = (int)min(sum[0], (int64_t)a.n_rows);
  if (tid == 0) {
    row_off[a.R] = total;
    need_off[a.R] = (int)min(sum[1], (int64_t)0x7fffffff);
    if (cta == 0) a.row_start[a.R] = total;
  }
  __syncwarp();
  cluster_or_block_sync(ctas > 1);

  // A warp takes a request: its new pages, what it then holds, and in a tree its
  // rows.  The lanes read 32 of the warp's requests' lengths at once.
  for (int at = warp; at < a.R; at += 32 * warps) {
    const int mine_r = at + lane * warps;
    const int mine_ctx = mine_r < a.R ? a.ctx[mine_r] : -1;
    for (int k = 0; k < 32 && at + k * warps < a.R; ++k) {
      const int r = at + k * warps, c = __shfl_sync(0xffffffffu, mine_ctx, k);
      const int h = held[r], first = need_off[r], need = need_off[r + 1] - first;
      // the requests that the stack covers come first, so what is left of it is
      // known from the first one without
      const bool granted = need_off[r + 1] <= top;
      int *table = a.block_table + (size_t)r * a.max_pages;
      const int row0 = row_off[r], n = a.parent ? row_off[r + 1] - row0 : 0;
      // what the tree needs is asked for before anything is waited for: a node's
      // parent, and the page of its place
      int up[2] = {0, 0}, page[2] = {-1, -1};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int node = lane + 32 * q;
        if (node < n) {
          if (node > 0) up[q] = a.parent[(size_t)r * a.gamma + node - 1];
          const int64_t p = ((int64_t)c + node) >> a.page_shift;
          if (p < h) page[q] = table[p];
          else if (p - h < need && granted) page[q] = a.free_pages[top - 1 - first - (int)(p - h)];
        }
      }
      for (int j = lane; j < need; j += 32)
        table[h + j] = granted ? a.free_pages[top - 1 - first - j] : -1;
      if (lane == 0) {
        a.held_out[r] = c < 0 ? 0 : h + (granted ? need : 0);
        if (!granted && need) dspark_set_status(DSPARK_ERR_PAGES);
        // the one request whose need crosses the stack's end, or the last of all
        if (granted ? r == a.R - 1 : first <= top)
          a.n_free_out[0] = top - (granted ? need_off[r + 1] : first);
      }
      if (n == 0) continue;
      // ancestor masks by doubling: after i rounds a node knows 2^i levels up
      unsigned long long bits[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int node = lane + 32 * q;
        if (up[q] < 0 || (node > 0 && up[q] >= node)) {
          dspark_set_status(DSPARK_ERR_ARG);
          up[q] = 0;
        }
        bits[q] = 1ull << node;
      }
      for (int levels = 1; levels < n; levels *= 2) {
        // a parent comes before its node: the low half only looks at the low half
        const unsigned long long lo0 = __shfl_sync(0xffffffffu, bits[0], up[0]);
        const int u0 = __shfl_sync(0xffffffffu, up[0], up[0]);
        if (n > 32) {
          const unsigned long long lo1 = __shfl_sync(0xffffffffu, bits[0], up[1] & 31);
          const unsigned long long hi1 = __shfl_sync(0xffffffffu, bits[1], up[1] & 31);
          const int ulo = __shfl_sync(0xffffffffu, up[0], up[1] & 31);
          const int uhi = __shfl_sync(0xffffffffu, up[1], up[1] & 31);
          bits[1] |= up[1] < 32 ? lo1 : hi1;
          up[1] = up[1] < 32 ? ulo : uhi;
        }
        bits[0] |= lo0;
        up[0] = u0;
        if (!__any_sync(0xffffffffu, up[0] | up[1])) {  // every chain has reached the anchor
          bits[0] |= 1;
          bits[1] |= 1;
          break;
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int node = lane + 32 * q;
        if (node < n) {
          const int64_t pos = (int64_t)c + node;
          a.position[row0 + node] = c + __popcll(bits[q]) - 1;
          a.slot[row0 + node] = page[q] < 0 || page[q] >= a.n_pages
                                    ? -1
                                    : ((int64_t)page[q] << a.page_shift) + (pos & (ps - 1));
          if (a.anc) a.anc[row0 + node] = bits[q];
        }
      }
    }
  }
  // slot of request r's position: a held page from the table, a new one from the
  // stack (the table's entry may not be written yet)
  auto slot_of = [&](int r, int64_t pos) -> int64_t {
    const int64_t p = pos >> a.page_shift;
    const int h = held[r], first = need_off[r], need = need_off[r + 1] - first;
    int page = -1;
    if (p < h)
      page = a.block_table[(size_t)r * a.max_pages + p];
    else if (p - h < need && need_off[r + 1] <= top)
      page = a.free_pages[top - 1 - first - (int)(p - h)];
    if (page < 0 || page >= a.n_pages) return -1;
    return ((int64_t)page << a.page_shift) + (pos & (ps - 1));
  };
  // chains: a thread takes a row, its request by search; then the padding
  for (int i = (a.parent ? total : 0) + cta * PLAN_THREADS + tid; i < a.n_rows;
       i += ctas * PLAN_THREADS) {
    if (i >= total) {
      a.position[i] = -1;
      a.slot[i] = -1;
      if (a.anc) a.anc[i] = 0;
      continue;
    }
    int lo = 0, hi = a.R - 1;  // the last request whose first row is <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (row_off[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int node = i - row_off[lo];
    const int64_t pos = (int64_t)a.ctx[lo] + node;
    a.position[i] = (int)pos;
    a.slot[i] = slot_of(lo, pos);
    if (a.anc) a.anc[i] = (2ull << node) - 1;
  }
}

// ------------------------------------------------------------------ append ----

// Four bf16 over a scale as e4m3 (out of line: it is seldom called).
__device__ __noinline__ uint32_t divide_four(uint32_t a, uint32_t b, float scale) {
  return pack_e4m3x2(bf16_lo(a) / scale, bf16_hi(a) / scale) |
         pack_e4m3x2(bf16_lo(b) / scale, bf16_hi(b) / scale) << 16;
}

// The same by the scale's reciprocal `inv`, for a scale in [2^-96, 2^96].  The product
// is within two units of its last place of the quotient.  e4m3 rounds at values
// whose 19 last bits are zero, so only a product within four units of such a value
// can round to another side, and those are divided.  Where `exact`, the scale is a
// power of two, and the product is the quotient.  (16384 rows of 2 x 1024 values: the
// divisions took 4 of 29 us.)
__device__ __forceinline__ uint32_t scale_four(uint32_t a, uint32_t b, float scale, float inv,
                                               bool exact) {
  const float q[4] = {bf16_lo(a) * inv, bf16_hi(a) * inv, bf16_lo(b) * inv, bf16_hi(b) * inv};
  uint32_t least = 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) least = min(least, (__float_as_uint(q[i]) + 4) & 0x7ffff);
  if (least < 8 && !exact) return divide_four(a, b, scale);
  return pack_e4m3x2(q[0], q[1]) | pack_e4m3x2(q[2], q[3]) << 16;
}

// A thread moves 16 values of one head (two 16-byte loads; two 16-byte stores, or
// one of 8-bit values) of every so many rows: its place in a row is found once.
// Places of one row are neighbours, so a warp's accesses are whole lines.  Blocks
// stay (a grid of many more, of a pass or two each, took 33 us for the prompts
// above, this one 25, both behind a write of all of L2; one row at a time 27, four
// 31).  Bound by its 101 MB: 20.4 us, 4.9 TB/s; a round of 256 chains 2.9 us in a graph.
constexpr int APPEND_THREADS = 256, APPEND_ROWS = 2, APPEND_BLOCKS_SM = 8;

template <bool FP8>
__global__ void __launch_bounds__(APPEND_THREADS)
    kv_append_kernel(const CacheView c, int n_rows, const bf16 *__restrict__ k,
                     const bf16 *__restrict__ v, int64_t row_stride, int64_t head_stride,
                     const int64_t *__restrict__ slot) {
  pdl_trigger();
  pdl_wait();
  const int per_head = c.dim / 16, units = 2 * c.heads * per_head;
  const int at_once = max(1, APPEND_THREADS / units);  // rows of a block's pass
  const int64_t n_slots = (int64_t)c.n_pages << c.page_shift;
  const int64_t rows_pass = (int64_t)gridDim.x * at_once;
  const int unit0 = threadIdx.x % units, sub = threadIdx.x / units;
  if (sub >= at_once && units <= APPEND_THREADS) return;
  for (int unit = units <= APPEND_THREADS ? unit0 : threadIdx.x; unit < units;
       unit += APPEND_THREADS) {
    const bool is_v = unit >= units / 2;
    const int e = is_v ? unit - units / 2 : unit, head = e / per_head, part = e - head * per_head;
    const bf16 *src = (is_v ? v : k) + head * head_stride + part * 16;
    uint8_t *dst = (is_v ? c.v : c.k) + head * c.head_bytes + part * (FP8 ? 16 : 32);
    const float *scales = is_v ? c.v_scale : c.k_scale;
    const float scale = FP8 && scales ? scales[head] : 1.0f, inv = 1.0f / scale;
    const bool near_one = scale >= 0x1p-96f && scale <= 0x1p96f;
    const bool exact = (__float_as_uint(scale) & 0x7fffff) == 0;
    const int64_t row0 = (int64_t)blockIdx.x * at_once + (units <= APPEND_THREADS ? sub : 0);
    for (int64_t row = row0; row < n_rows; row += APPEND_ROWS * rows_pass) {
      uint4 x[APPEND_ROWS], y[APPEND_ROWS];
      int64_t s[APPEND_ROWS];
#pragma unroll
      for (int i = 0; i < APPEND_ROWS; ++i) {  // every row's loads before the first's stores
        const int64_t m = row + i * rows_pass;
        s[i] = m < n_rows ? slot[m] : -1;
        if (m < n_rows) {
          const uint4 *p = reinterpret_cast<const uint4 *>(src + m * row_stride);
          x[i] = p[0];
          y[i] = p[1];
        }
      }
#pragma unroll
      for (int i = 0; i < APPEND_ROWS; ++i) {
        if (s[i] < 0) continue;
        if (s[i] >= n_slots) {
          dspark_set_status(DSPARK_ERR_PAGES);
          continue;
        }
        uint4 *to = reinterpret_cast<uint4 *>(dst + (s[i] >> c.page_shift) * c.page_bytes +
                                              (s[i] & ((1 << c.page_shift) - 1)) * c.token_bytes);
        if constexpr (FP8) {
          const uint32_t w[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = near_one ? scale_four(w[2 * j], w[2 * j + 1], scale, inv, exact)
                            : divide_four(w[2 * j], w[2 * j + 1], scale);
          *to = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          to[0] = x[i];
          to[1] = y[i];
        }
      }
    }
  }
}

// ------------------------------------------------------------------ accept ----

// A warp takes a request, a lane drafts l + 1 and l + 33.  Whether a node's
// token is its parent's choice is known for all nodes at once; the walk from the
// anchor then only asks, once per level, which matching node has the present one
// as its parent.  Under 1 MB: bound by its launch and the walk's ballots, 1.5 us in a
// graph for one chain, 2.9 for 1024 trees of 64 nodes.
__global__ void __launch_bounds__(128)
    tree_accept_kernel(int R, int gamma, int n_rows, const int *__restrict__ row_start,
                       const int *__restrict__ parent, const int *__restrict__ tokens,
                       const int *__restrict__ choice, const int *ctx, int *accepted, int *bonus,
                       int *path, int *ctx_out) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= R) return;
  int row0 = row_start[r], n = row_start[r + 1] - row0;
  const int c = ctx[r];
  if (row0 < 0 || n < 0 || n > gamma + 1 || row0 > n_rows - n) {
    dspark_set_status(DSPARK_ERR_LENGTH);
    n = 0;
  }
  int up[2];
  bool hit[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int node = lane + 32 * q + 1;
    up[q] = -1;
    hit[q] = false;
    if (node < n) {
      const int p = parent ? parent[(size_t)r * gamma + node - 1] : node - 1;
      if (p < 0 || p >= node) {
        dspark_set_status(DSPARK_ERR_ARG);
      } else {
        up[q] = p;
        hit[q] = tokens[(size_t)r * gamma + node - 1] == choice[row0 + p];
      }
    }
  }
  int cur = 0, count = 0, step[2] = {-1, -1};  // step[q]: node at path entry lane + 32 q
  while (count < n) {  // a child comes after its node: at most n - 1 steps
    const uint32_t lo = __ballot_sync(0xffffffffu, hit[0] && up[0] == cur);
    const uint32_t hi = __ballot_sync(0xffffffffu, hit[1] && up[1] == cur);
    if (!(lo | hi)) break;
    cur = lo ? __ffs(lo) : 32 + __ffs(hi);
    if (lane == (count & 31)) step[count >> 5] = cur;
    ++count;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (lane + 32 * q < gamma) path[(size_t)r * gamma + lane + 32 * q] = step[q];
  if (lane == 0) {
    accepted[r] = count;
    bonus[r] = n > 0 ? choice[row0 + cur] : -1;
    ctx_out[r] = n > 0 ? c + 1 + count : c;
  }
}

// ----------------------------------------------------------------- compact ----

// Block (x, r): 128 of request r's 16-byte columns (K or V, head, part), each
// moved down the path by one thread.  Every source lies at or past its
// destination and both ascend, so a batch of sources read before its
// destinations are written is never overwritten too early, and columns are
// independent: no barrier.  78 MB of a batch's cache in 14.4 us in a
// graph, 5.4 TB/s.
__global__ void __launch_bounds__(128)
    kv_compact_kernel(const CacheView c, int size, int gamma, int max_pages,
                      const int *__restrict__ ctx, const int *__restrict__ accepted,
                      const int *__restrict__ path, const int *__restrict__ block_table) {
  constexpr int BATCH = 8;
  __shared__ int64_t from[64], to[64];  // byte offsets of the path's tokens
  __shared__ int bad;
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.y, tid = threadIdx.x;
  const int n = accepted[r], base = ctx[r];
  if (n <= 0) return;
  if (n > gamma || base < 0) {
    if (tid == 0) dspark_set_status(n > gamma ? DSPARK_ERR_LENGTH : DSPARK_ERR_ARG);
    return;
  }
  if (tid == 0) bad = 0;
  __syncthreads();
  auto place = [&](int64_t pos) -> int64_t {
    const int64_t p = pos >> c.page_shift;
    const int page = p < max_pages ? block_table[(size_t)r * max_pages + p] : -1;
    if (page < 0 || page >= c.n_pages) {
      bad = DSPARK_ERR_PAGES;
      return 0;
    }
    return page * c.page_bytes + (pos & ((1 << c.page_shift) - 1)) * c.token_bytes;
  };
  if (tid < n) {
    const int node = path[(size_t)r * gamma + tid];
    const int before = tid ? path[(size_t)r * gamma + tid - 1] : 0;
    if (node <= before || node > 63) {
      bad = DSPARK_ERR_ARG;
    } else {
      from[tid] = place((int64_t)base + node);
      to[tid] = place((int64_t)base + 1 + tid);
    }
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) dspark_set_status(bad);
    return;
  }
  const int parts = c.dim * size / 16;
  const int col = blockIdx.x * 128 + tid;
  if (col >= 2 * c.heads * parts) return;
  const int head = col / parts;  // heads of K, then heads of V
  uint8_t *base_col = (head < c.heads ? c.k + head * c.head_bytes
                                      : c.v + (head - c.heads) * c.head_bytes) +
                      (col - head * parts) * 16;
  for (int j = 0; j < n; j += BATCH) {
    uint4 x[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (j + i < n && from[j + i] != to[j + i])
        x[i] = *reinterpret_cast<const uint4 *>(base_col + from[j + i]);
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (j + i < n && from[j + i] != to[j + i])
        *reinterpret_cast<uint4 *>(base_col + to[j + i]) = x[i];
  }
}

}  // namespace

extern "C" int dspark_kv_plan(int32_t R, int32_t gamma, int32_t extra, int32_t n_rows,
                              int32_t page_size, int32_t n_pages, int32_t max_pages,
                              const int32_t *ctx, const int32_t *len, const int32_t *parent,
                              const int32_t *held, const int32_t *n_free, int32_t *free_pages,
                              int32_t *block_table, int32_t *held_out, int32_t *n_free_out,
                              int32_t *row_start, int32_t *position, int64_t *slot, uint64_t *anc,
                              dspark_stream_t stream) {
  if (R < 1 || n_rows < 1 || n_pages < 1 || max_pages < 1 || extra < 0 || extra > 1)
    return DSPARK_ERR_ARG;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return DSPARK_ERR_ARG;
  if (!ctx || !len || !held || !n_free || !free_pages || !block_table || !held_out ||
      !n_free_out || !row_start || !position || !slot)
    return DSPARK_ERR_ARG;
  if (parent && (extra != 1 || gamma < 1 || gamma >= DSPARK_MAX_NODES)) return DSPARK_ERR_ARG;
  if (R > MAX_R) return DSPARK_ERR_TOO_LARGE;
  PlanArgs a;
  a.R = R;
  a.gamma = gamma;
  a.extra = extra;
  a.n_rows = n_rows;
  a.page_shift = 31 - __builtin_clz((unsigned)page_size);
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.ctx = ctx;
  a.len = len;
  a.parent = parent;
  a.held = held;
  a.n_free = n_free;
  a.free_pages = free_pages;
  a.block_table = block_table;
  a.held_out = held_out;
  a.n_free_out = n_free_out;
  a.row_start = row_start;
  a.position = position;
  a.slot = slot;
  a.anc = anc;
  static DsparkPerDevice attr;
  if (dspark_per_device(attr, [] {
        return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (3 * MAX_R + 2) * (int)sizeof(int)) == cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return DSPARK_ERR_CUDA;
  // One CTA while a request takes a warp and a row a thread of it; else a cluster.
  const int ctas = R <= PLAN_THREADS / 32 && n_rows <= PLAN_THREADS ? 1 : PLAN_CLUSTER;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.dynamicSmemBytes = (size_t)(3 * R + 2) * sizeof(int);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kv_plan_kernel, a) != cudaSuccess) return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

extern "C" int dspark_kv_append(const dspark_kv_cache *cache, int32_t n_rows, const void *k,
                                const void *v, int64_t row_stride, int64_t head_stride,
                                const int64_t *slot, dspark_stream_t stream) {
  if (!dspark_kv_cache_ok(cache) || n_rows < 0) return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  if (!k || !v || !slot) return DSPARK_ERR_ARG;
  if (((uintptr_t)k | (uintptr_t)v) & 15 || row_stride <= 0 || head_stride <= 0 ||
      row_stride % 8 || head_stride % 8)
    return DSPARK_ERR_ARG;
  const int units = 2 * cache->heads * (cache->dim / 16);
  const int64_t at_once = units < APPEND_THREADS ? APPEND_THREADS / units : 1;
  const int64_t blocks = (n_rows + at_once - 1) / at_once;
  const int64_t most = (int64_t)dspark_sm_count() * APPEND_BLOCKS_SM;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  const CacheView c = view_of(cache);
  const cudaError_t e =
      cache->type == DSPARK_KV_E4M3
          ? dspark_launch_pdl(kv_append_kernel<true>, grid, dim3(256), 0, stream, c, n_rows,
                              (const bf16 *)k, (const bf16 *)v, row_stride, head_stride, slot)
          : dspark_launch_pdl(kv_append_kernel<false>, grid, dim3(256), 0, stream, c, n_rows,
                              (const bf16 *)k, (const bf16 *)v, row_stride, head_stride, slot);
  if (e != cudaSuccess) return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

extern "C" int dspark_tree_accept(int32_t R, int32_t gamma, int32_t n_rows,
                                  const int32_t *row_start, const int32_t *parent,
                                  const int32_t *tokens, const int32_t *choice, const int32_t *ctx,
                                  int32_t *accepted, int32_t *bonus, int32_t *path,
                                  int32_t *ctx_out, dspark_stream_t stream) {
  if (R < 1 || gamma < 1 || gamma >= DSPARK_MAX_NODES || n_rows < 1 || !row_start || !tokens ||
      !choice || !ctx || !accepted || !bonus || !path || !ctx_out)
    return DSPARK_ERR_ARG;
  if (dspark_launch_pdl(tree_accept_kernel, dim3((R + 3) / 4), dim3(128), 0, stream, R, gamma,
                        n_rows, row_start, parent, tokens, choice, ctx, accepted, bonus, path,
                        ctx_out) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

extern "C" int dspark_kv_compact(const dspark_kv_cache *cache, int32_t R, int32_t gamma,
                                 int32_t max_pages, const int32_t *ctx, const int32_t *accepted,
                                 const int32_t *path, const int32_t *block_table,
                                 dspark_stream_t stream) {
  if (!dspark_kv_cache_ok(cache) || R < 1 || gamma < 1 || gamma >= DSPARK_MAX_NODES ||
      max_pages < 1 || !ctx || !accepted || !path || !block_table)
    return DSPARK_ERR_ARG;
  if (R > 65535) return DSPARK_ERR_TOO_LARGE;
  const int size = dspark_kv_bytes(cache->type);
  const int cols = 2 * cache->heads * (cache->dim * size / 16);
  if (dspark_launch_pdl(kv_compact_kernel, dim3((cols + 127) / 128, R), dim3(128), 0, stream,
                        view_of(cache), size, gamma, max_pages, ctx, accepted, path,
                        block_table) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

int dspark_status_kv(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_kv, sizeof(int)) != cudaSuccess) return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_kv, &zero, sizeof(int));
  }
  return v;
}
