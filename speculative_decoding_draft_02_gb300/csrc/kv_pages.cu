// kv_pages.cu — pages with several holders: continuations of a request (fork), pages
// given back (release), the pages in use moved together (squeeze), and the copies of K
// and V that these leave to be done (copy).
#include <cooperative_groups.h>

#include "kv_cache.cuh"

DSPARK_DECLARE_STATUS(s_status_pages)

namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 1024, WARPS = THREADS / 32, CLUSTER = 8, MAX_R = 16384;

// The tables' kernels are one CTA for small calls and a cluster for others.  What one CTA
// writes to global memory, another reads behind this barrier, past L1.
__device__ __forceinline__ void sync_all(int ctas) {
  __syncwarp();  // the cluster's barrier wants whole warps
  if (ctas > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
  else
    __syncthreads();
}

// Exclusive sum over the block's threads; the total in `sum`.
__device__ __forceinline__ long long block_scan(long long v, long long &sum, long long *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();  // the last scan's sums are read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  sum = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp ? before : 0) + inc - v;
}

// -------------------------------------------------------------------- fork ----

struct ForkArgs {
  int n, R, page_shift, n_pages, max_pages;
  const int *source, *target, *free_pages;
  int *ctx, *held, *n_free, *block_table, *refs, *copy_from, *copy_to, *copy_tokens;
};

// Every CTA settles all forks for itself (which are sound, which page of the stack each
// takes: a few KB from L2); behind one barrier the warps of all of them write.  Under a
// MB: bound by its launch, dependent reads and the barrier (three forks 3.2 us in a graph,
// one CTA; 480 forks of 32 prompts, 9660 holds, with their release 23 us).
__global__ void __launch_bounds__(THREADS, 1) kv_fork_kernel(const ForkArgs a) {
  extern __shared__ int smem[];
  __shared__ long long warp_sums[WARPS];
  int *first = smem;          // [R] the first fork to each place
  int *tokens = first + a.R;  // [n] a sound fork's, or -1
  int *taken = tokens + a.n;  // [n] pages taken up to and with this fork
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int ps = 1 << a.page_shift;
  pdl_trigger();
  pdl_wait();

  int top = a.n_free[0];
  if (top < 0 || top > a.n_pages) {
    dspark_set_status(DSPARK_ERR_PAGES);
    top = top < 0 ? 0 : a.n_pages;
  }
  for (int r = tid; r < a.R; r += THREADS) first[r] = 0x7fffffff;
  __syncthreads();
  for (int i = tid; i < a.n; i += THREADS) {
    const int dst = a.target[i];
    if (a.source[i] >= 0 && dst >= 0 && dst < a.R) atomicMin(&first[dst], i);
  }
  __syncthreads();
  const int per = (a.n + THREADS - 1) / THREADS;
  const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
  long long mine = 0, all;
  for (int i = i0; i < i1; ++i) {
    const int src = a.source[i], dst = a.target[i];
    int t = -1;
    if (src >= 0) {
      bool ok = src < a.R && dst >= 0 && dst < a.R;
      if (ok) {
        t = a.ctx[src];
        const long long pages = ((long long)t + ps - 1) >> a.page_shift;
        ok = t >= 0 && pages <= a.held[src] && pages <= a.max_pages && a.ctx[dst] < 0 &&
             a.held[dst] == 0 && first[dst] == i;
      }
      if (!ok) {
        dspark_set_status(DSPARK_ERR_ARG);
        t = -1;
      }
    }
    tokens[i] = t;
    mine += t > 0 && (t & (ps - 1));
  }
  long long at = block_scan(mine, all, warp_sums);
  for (int i = i0; i < i1; ++i) {
    at += tokens[i] > 0 && (tokens[i] & (ps - 1));
    taken[i] = (int)at;
  }
  __syncthreads();
  sync_all(ctas);  // every CTA has read the places

  for (int i = cta * WARPS + (tid >> 5); i < a.n; i += ctas * WARPS) {
    const int t = tokens[i], tail = t & (ps - 1);
    const bool need = t > 0 && tail, granted = t >= 0 && (!need || taken[i] <= top);
    int from = -1, to = -1;
    if (granted) {
      const int src = a.source[i], dst = a.target[i], full = t >> a.page_shift;
      const int *theirs = a.block_table + (size_t)src * a.max_pages;
      int *ours = a.block_table + (size_t)dst * a.max_pages;
      for (int j = lane; j < full; j += 32) {
        const int page = theirs[j];
        ours[j] = page;
        if (page >= 0 && page < a.n_pages)
          atomicAdd(&a.refs[page], 1);
        else
          dspark_set_status(DSPARK_ERR_PAGES);
      }
      if (lane == 0) {
        if (need) {
          from = theirs[full];
          to = a.free_pages[top - taken[i]];
          ours[full] = to;
        }
        a.ctx[dst] = t;
        a.held[dst] = full + need;
      }
    } else if (t >= 0) {
      dspark_set_status(DSPARK_ERR_PAGES);
    }
    if (lane == 0) {
      a.copy_from[i] = from;
      a.copy_to[i] = to;
      a.copy_tokens[i] = granted && need ? tail : 0;
    }
  }
  // the pages taken: once one fork in need goes without, so do all after it
  if (cta == 0 && tid == 0) a.n_free[0] = top - (int)min(all, (long long)top);
}

// ----------------------------------------------------------------- release ----

struct ReleaseArgs {
  int R, n_pages, max_pages;
  const int *ctx, *block_table;
  int *held, *n_free, *free_pages, *refs;
};

// Holds are numbered request by request and in block order, and every thread takes some
// consecutive ones.  Every hold takes one off its page's count, which a page that nobody
// holds any more then shows as -1; those pages keep, as -(number + 2), the last of their
// holds, whose place on the stack they take.  Barriers lie between; orders of atomics
// never matter.  Bound by these steps of dependent reads: 2 us where nobody has left; the
// first KEPT pages of a thread are read once (a fork and a release of 480 requests 33 -> 24 us,
// against reading the table at each of four steps).
__global__ void __launch_bounds__(THREADS, 1) kv_release_kernel(const ReleaseArgs a) {
  constexpr int KEPT = 4;  // pages of a thread's holds that are read once
  extern __shared__ int first[];  // [R + 1] number of a request's first hold
  __shared__ long long warp_sums[WARPS];
  __shared__ int counts[CLUSTER];  // pages that each CTA gives back
  const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x;
  pdl_trigger();
  pdl_wait();

  int top = a.n_free[0];
  if (top < 0 || top > a.n_pages) {
    dspark_set_status(DSPARK_ERR_PAGES);
    top = top < 0 ? 0 : a.n_pages;
  }
  const int per_r = (a.R + THREADS - 1) / THREADS;
  const int r0 = min(tid * per_r, a.R), r1 = min(r0 + per_r, a.R);
  long long mine = 0, all;
  for (int r = r0; r < r1; ++r) {
    int h = a.ctx[r] < 0 ? a.held[r] : 0;
    if (h < 0 || h > a.max_pages) {
      dspark_set_status(DSPARK_ERR_PAGES);
      h = h < 0 ? 0 : a.max_pages;
    }
    first[r] = h;
    mine += h;
  }
  long long at = block_scan(mine, all, warp_sums);
  if (all == 0) return;  // nobody has left (the same answer in every CTA)
  if (all > 0x7ffffff0ll) {
    if (tid == 0) dspark_set_status(DSPARK_ERR_LENGTH);
    return;
  }
  for (int r = r0; r < r1; ++r) {
    const int h = first[r];
    first[r] = (int)at;
    at += h;
  }
  if (tid == 0) first[a.R] = (int)all;
  __syncthreads();

  // the page of hold e; -1 outside the cache
  auto page_of = [&](int e) {
    int lo = 0, hi = a.R - 1;  // the last request whose first hold is at or before e
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    const int page = a.block_table[(size_t)lo * a.max_pages + (e - first[lo])];
    return page >= 0 && page < a.n_pages ? page : -1;
  };
  const int threads = ctas * THREADS, thread = cta * THREADS + tid;
  const int per = (int)((all + threads - 1) / threads);
  const int e0 = (int)min((long long)thread * per, all), n = (int)min((long long)per, all - e0);
  int kept[KEPT];
#pragma unroll
  for (int i = 0; i < KEPT; ++i) kept[i] = i < n ? page_of(e0 + i) : -1;
  auto each = [&](auto &&f) {
#pragma unroll
    for (int i = 0; i < KEPT; ++i)
      if (i < n) f(e0 + i, kept[i]);
    for (int i = KEPT; i < n; ++i) f(e0 + i, page_of(e0 + i));
  };

  each([&](int, int page) {
    if (page < 0) {
      dspark_set_status(DSPARK_ERR_PAGES);
    } else if (atomicSub(&a.refs[page], 1) < 0) {  // more holds than were counted
      atomicAdd(&a.refs[page], 1);
      dspark_set_status(DSPARK_ERR_PAGES);
    }
  });
  __threadfence();
  sync_all(ctas);
  each([&](int e, int page) {
    if (page >= 0 && __ldcg(&a.refs[page]) < 0) atomicMin(&a.refs[page], -e - 2);
  });
  for (int r = thread; r < a.R; r += threads)  // every CTA has read held
    if (first[r + 1] > first[r]) a.held[r] = 0;
  __threadfence();
  sync_all(ctas);
  mine = 0;
  each([&](int e, int page) { mine += page >= 0 && __ldcg(&a.refs[page]) == -e - 2; });
  at = top + block_scan(mine, all, warp_sums);
  if (ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (tid < ctas) *cluster.map_shared_rank(&counts[cta], tid) = (int)all;
    cluster.sync();
    all = 0;
    for (int i = 0; i < ctas; ++i) {
      if (i < cta) at += counts[i];
      all += counts[i];
    }
  }
  each([&](int e, int page) {
    if (page >= 0 && __ldcg(&a.refs[page]) == -e - 2) {
      __stcg(&a.refs[page], 0);
      if (at < a.n_pages) a.free_pages[at] = page;
      ++at;
    }
  });
  if (thread == 0) {
    if (top + all > a.n_pages) dspark_set_status(DSPARK_ERR_PAGES);
    a.n_free[0] = (int)min(top + all, (long long)a.n_pages);
  }
}

// ----------------------------------------------------------------- squeeze ----

struct SqueezeArgs {
  int R, n_pages, max_pages;
  const int *held, *n_free, *free_pages, *block_table, *refs;
  int *free_out, *table_out, *refs_out, *new_page, *move_from, *move_to, *n_moves;
};

// Free pages are marked in new_page; every warp then counts, in a stretch of pages of its
// own, those that go (in use, U or higher) and those that take them (free, below U), and
// by the counts of all warps before it knows their ranks.  Bound by its five barriers: 96
// pages 6 us, 8000 pages 12 us in a graph.
__global__ void __launch_bounds__(THREADS, 1) kv_squeeze_kernel(const SqueezeArgs a) {
  __shared__ int counts[2][CLUSTER * WARPS];  // of every warp of the cluster
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int warps = ctas * WARPS, warp = cta * WARPS + (tid >> 5);
  const int threads = ctas * THREADS, thread = cta * THREADS + tid;
  pdl_trigger();
  pdl_wait();

  int n_free = a.n_free[0];
  if (n_free < 0 || n_free > a.n_pages) {
    dspark_set_status(DSPARK_ERR_PAGES);
    n_free = n_free < 0 ? 0 : a.n_pages;
  }
  const int used = a.n_pages - n_free, half = a.n_pages / 2;
  for (int p = thread; p < a.n_pages; p += threads) __stcg(&a.new_page[p], p);
  for (int i = thread; i < half; i += threads) {
    __stcg(&a.move_from[i], -1);
    __stcg(&a.move_to[i], -1);
  }
  __threadfence();
  sync_all(ctas);
  for (int i = thread; i < n_free; i += threads) {
    const int p = a.free_pages[i];
    if (p < 0 || p >= a.n_pages || atomicExch(&a.new_page[p], -1) < 0)
      dspark_set_status(DSPARK_ERR_PAGES);
  }
  __threadfence();
  sync_all(ctas);
  const int stretch = (int)(((long long)a.n_pages + 32 * warps - 1) / (32 * warps)) * 32;
  const int p0 = (int)min((long long)warp * stretch, (long long)a.n_pages);
  const int p1 = (int)min((long long)p0 + stretch, (long long)a.n_pages);
  int go = 0, take = 0;
  for (int b = p0; b < p1; b += 32) {
    const int p = b + lane;
    const bool in = p < p1, free = in && __ldcg(&a.new_page[p]) < 0;
    go += __popc(__ballot_sync(0xffffffffu, in && !free && p >= used));
    take += __popc(__ballot_sync(0xffffffffu, free && p < used));
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (lane < ctas) {
    cluster.map_shared_rank(&counts[0][0], lane)[warp] = go;
    cluster.map_shared_rank(&counts[1][0], lane)[warp] = take;
  }
  cluster.sync();
  int goes = 0, takes = 0, moves = 0, takers = 0;  // before this warp, and in all
  for (int w = lane; w < warps; w += 32) {
    goes += w < warp ? counts[0][w] : 0;
    takes += w < warp ? counts[1][w] : 0;
    moves += counts[0][w];
    takers += counts[1][w];
  }
  goes = __reduce_add_sync(0xffffffffu, goes);
  takes = __reduce_add_sync(0xffffffffu, takes);
  moves = __reduce_add_sync(0xffffffffu, moves);
  takers = __reduce_add_sync(0xffffffffu, takers);
  // as many go as take them, unless the stack is not what it should be; at most half of all
  moves = min(min(moves, takers), half);
  for (int b = p0; b < p1; b += 32) {
    const int p = b + lane;
    const bool in = p < p1, free = in && __ldcg(&a.new_page[p]) < 0;
    const uint32_t by_go = __ballot_sync(0xffffffffu, in && !free && p >= used);
    const uint32_t by_take = __ballot_sync(0xffffffffu, free && p < used);
    const uint32_t below = (1u << lane) - 1;
    const int g = goes + __popc(by_go & below), t = takes + __popc(by_take & below);
    if ((by_go >> lane & 1) && g < moves) __stcg(&a.move_from[g], p);
    if ((by_take >> lane & 1) && t < moves) __stcg(&a.move_to[t], p);
    goes += __popc(by_go);
    takes += __popc(by_take);
  }
  __threadfence();
  sync_all(ctas);
  // refs_out may be refs: the counts of pages that go are read before they are cleared
  for (int k = thread; k < moves; k += threads) {
    const int from = __ldcg(&a.move_from[k]), to = __ldcg(&a.move_to[k]);
    __stcg(&a.new_page[from], to);
    a.refs_out[to] = a.refs[from];
  }
  __threadfence();
  sync_all(ctas);
  for (int p = thread; p < a.n_pages; p += threads) {
    const int to = __ldcg(&a.new_page[p]);
    if (to == p)
      a.refs_out[p] = a.refs[p];
    else if (p >= used)
      a.refs_out[p] = 0;
  }
  for (int i = thread; i < a.n_pages; i += threads)
    a.free_out[i] = i < n_free ? a.n_pages - 1 - i : a.free_pages[i];
  for (int r = warp; r < a.R; r += warps) {
    int h = a.held[r];
    if (h < 0 || h > a.max_pages) {
      if (lane == 0) dspark_set_status(DSPARK_ERR_PAGES);
      h = h < 0 ? 0 : a.max_pages;
    }
    const size_t row = (size_t)r * a.max_pages;
    for (int j = lane; j < a.max_pages; j += 32) {
      int page = a.block_table[row + j];
      if (j < h) {
        if (page < 0 || page >= a.n_pages)
          dspark_set_status(DSPARK_ERR_PAGES);
        else
          page = __ldcg(&a.new_page[page]);
      }
      a.table_out[row + j] = page;
    }
  }
  if (thread == 0) a.n_moves[0] = moves;
}

// -------------------------------------------------------------------- copy ----

// A block takes some tokens of one page, a thread one 16-byte column (head, part) of
// every so many of them, K and V together: eight loads before the first store.
// Neighbouring columns are neighbours in memory where heads are.  Bound by its bytes: 2010
// pages of 32 tokens, 8 heads of 128, bf16, read and written in 83 us, 6.4 TB/s.
constexpr int COPY_THREADS = 256, COPY_TOKENS = 4, COPY_BLOCKS_SM = 8;

__global__ void __launch_bounds__(COPY_THREADS)
    kv_copy_kernel(const CacheView c, int size, int n, int splits, const int *__restrict__ from,
                   const int *__restrict__ to, const int *__restrict__ tokens) {
  pdl_trigger();
  pdl_wait();
  const int parts = c.dim * size / 16, cols = c.heads * parts, ps = 1 << c.page_shift;
  const int at_once = max(1, COPY_THREADS / cols);  // tokens of a block's pass
  const int sub = cols <= COPY_THREADS ? threadIdx.x / cols : 0;
  const int col0 = cols <= COPY_THREADS ? threadIdx.x % cols : threadIdx.x;
  if (sub >= at_once) return;
  for (int64_t unit = blockIdx.x; unit < (int64_t)n * splits; unit += gridDim.x) {
    const int i = (int)(unit / splits), split = (int)(unit - (int64_t)i * splits);
    const int src = from[i];
    if (src < 0) continue;
    const int dst = to[i], count = tokens ? tokens[i] : ps;
    if (src >= c.n_pages || dst < 0 || dst >= c.n_pages || count < 0 || count > ps) {
      if (threadIdx.x == 0)
        dspark_set_status(count < 0 || count > ps ? DSPARK_ERR_LENGTH : DSPARK_ERR_PAGES);
      continue;
    }
    const int t0 = split * at_once * COPY_TOKENS + sub;
    for (int col = col0; col < cols; col += COPY_THREADS) {
      const int head = col / parts;
      const int64_t in = head * c.head_bytes + (col - head * parts) * 16;
      const int64_t off_from = src * c.page_bytes + in, off_to = dst * c.page_bytes + in;
      uint4 x[2][COPY_TOKENS];
#pragma unroll
      for (int u = 0; u < COPY_TOKENS; ++u) {
        const int t = t0 + u * at_once;
        if (t < count) {
          x[0][u] = *reinterpret_cast<const uint4 *>(c.k + off_from + t * c.token_bytes);
          x[1][u] = *reinterpret_cast<const uint4 *>(c.v + off_from + t * c.token_bytes);
        }
      }
#pragma unroll
      for (int u = 0; u < COPY_TOKENS; ++u) {
        const int t = t0 + u * at_once;
        if (t < count) {
          *reinterpret_cast<uint4 *>(c.k + off_to + t * c.token_bytes) = x[0][u];
          *reinterpret_cast<uint4 *>(c.v + off_to + t * c.token_bytes) = x[1][u];
        }
      }
    }
  }
}

// One CTA for small calls, else a cluster.
template <class K, class A>
int launch_tables(K kernel, const A &a, bool small, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = small ? 1 : CLUSTER;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(small ? 1 : CLUSTER);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

template <class K>
bool allow_smem(DsparkPerDevice &once, K kernel, int bytes) {
  return dspark_per_device(once, [&] {
           return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       bytes) == cudaSuccess
                      ? 1
                      : -1;
         }) >= 0;
}

}  // namespace

extern "C" int dspark_kv_fork(int32_t n, const int32_t *source, const int32_t *target, int32_t R,
                              int32_t page_size, int32_t n_pages, int32_t max_pages, int32_t *ctx,
                              int32_t *held, int32_t *n_free, const int32_t *free_pages,
                              int32_t *block_table, int32_t *refs, int32_t *copy_from,
                              int32_t *copy_to, int32_t *copy_tokens, dspark_stream_t stream) {
  if (n < 0 || R < 1 || n_pages < 1 || max_pages < 1 || page_size < 16 || page_size > 256 ||
      (page_size & (page_size - 1)))
    return DSPARK_ERR_ARG;
  if (R > MAX_R || n > R) return DSPARK_ERR_TOO_LARGE;
  if (n == 0) return DSPARK_OK;
  if (!source || !target || !ctx || !held || !n_free || !free_pages || !block_table || !refs ||
      !copy_from || !copy_to || !copy_tokens)
    return DSPARK_ERR_ARG;
  ForkArgs a;
  a.n = n;
  a.R = R;
  a.page_shift = 31 - __builtin_clz((unsigned)page_size);
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.source = source;
  a.target = target;
  a.free_pages = free_pages;
  a.ctx = ctx;
  a.held = held;
  a.n_free = n_free;
  a.block_table = block_table;
  a.refs = refs;
  a.copy_from = copy_from;
  a.copy_to = copy_to;
  a.copy_tokens = copy_tokens;
  static DsparkPerDevice once;
  if (!allow_smem(once, kv_fork_kernel, 3 * MAX_R * (int)sizeof(int))) return DSPARK_ERR_CUDA;
  return launch_tables(kv_fork_kernel, a, n <= WARPS,
                       ((size_t)R + 2 * (size_t)n) * sizeof(int), stream);
}

extern "C" int dspark_kv_release(int32_t R, int32_t n_pages, int32_t max_pages, const int32_t *ctx,
                                 int32_t *held, int32_t *n_free, int32_t *free_pages,
                                 const int32_t *block_table, int32_t *refs,
                                 dspark_stream_t stream) {
  if (R < 1 || n_pages < 1 || max_pages < 1 || !ctx || !held || !n_free || !free_pages ||
      !block_table || !refs)
    return DSPARK_ERR_ARG;
  if (R > MAX_R) return DSPARK_ERR_TOO_LARGE;
  ReleaseArgs a;
  a.R = R;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.ctx = ctx;
  a.block_table = block_table;
  a.held = held;
  a.n_free = n_free;
  a.free_pages = free_pages;
  a.refs = refs;
  static DsparkPerDevice once;
  if (!allow_smem(once, kv_release_kernel, (MAX_R + 1) * (int)sizeof(int)))
    return DSPARK_ERR_CUDA;
  return launch_tables(kv_release_kernel, a, R <= WARPS, ((size_t)R + 1) * sizeof(int), stream);
}

extern "C" int dspark_kv_squeeze(int32_t R, int32_t n_pages, int32_t max_pages,
                                 const int32_t *held, const int32_t *n_free,
                                 const int32_t *free_pages, const int32_t *block_table,
                                 const int32_t *refs, int32_t *free_pages_out,
                                 int32_t *block_table_out, int32_t *refs_out, int32_t *new_page,
                                 int32_t *move_from, int32_t *move_to, int32_t *n_moves,
                                 dspark_stream_t stream) {
  if (R < 1 || n_pages < 2 || max_pages < 1 || !held || !n_free || !free_pages || !block_table ||
      !refs || !free_pages_out || !block_table_out || !refs_out || !new_page || !move_from ||
      !move_to || !n_moves)
    return DSPARK_ERR_ARG;
  if (R > MAX_R) return DSPARK_ERR_TOO_LARGE;
  SqueezeArgs a;
  a.R = R;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.held = held;
  a.n_free = n_free;
  a.free_pages = free_pages;
  a.block_table = block_table;
  a.refs = refs;
  a.free_out = free_pages_out;
  a.table_out = block_table_out;
  a.refs_out = refs_out;
  a.new_page = new_page;
  a.move_from = move_from;
  a.move_to = move_to;
  a.n_moves = n_moves;
  return launch_tables(kv_squeeze_kernel, a, n_pages <= THREADS && R <= WARPS, 0, stream);
}

extern "C" int dspark_kv_copy(const dspark_kv_cache *cache, int32_t n, const int32_t *from,
                              const int32_t *to, const int32_t *tokens, dspark_stream_t stream) {
  if (!dspark_kv_cache_ok(cache) || n < 0) return DSPARK_ERR_ARG;
  if (n == 0) return DSPARK_OK;
  if (!from || !to) return DSPARK_ERR_ARG;
  const int size = dspark_kv_bytes(cache->type);
  const int64_t cols = (int64_t)cache->heads * (cache->dim * size / 16);
  if (cols > 0x7fffffff) return DSPARK_ERR_TOO_LARGE;
  const int at_once = cols < COPY_THREADS ? (int)(COPY_THREADS / cols) : 1;
  const int splits = (cache->page_size + at_once * COPY_TOKENS - 1) / (at_once * COPY_TOKENS);
  const int64_t units = (int64_t)n * splits;
  const int64_t most = (int64_t)dspark_sm_count() * COPY_BLOCKS_SM;
  if (dspark_launch_pdl(kv_copy_kernel, dim3((unsigned)(units < most ? units : most)),
                        dim3(COPY_THREADS), 0, stream, view_of(cache), size, n, splits, from, to,
                        tokens) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

int dspark_status_pages(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_pages, sizeof(int)) != cudaSuccess) return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_pages, &zero, sizeof(int));
  }
  return v;
}
