// chunk_attention.cu — dspark_chunk_attention: attention of any number of new rows of each
// request over its paged cache, each row over the tokens up to its own position.
//
//   s_p = scale * q . K_p,  out = sum_p e^{s_p} V_p / sum_p e^{s_p},  p <= ctx + i
#include "kv_cache.cuh"

DSPARK_DECLARE_STATUS(s_status_chunk)

namespace {

struct Args {
  CacheView c;
  int R, heads_q, max_rows, n_rows, max_pages;
  const bf16 *q;
  int64_t q_row, q_head;
  const int *ctx, *row_start, *block_table;
  float scale;
  bf16 *out;
  int64_t out_row, out_head;
  float *lse;
};

// A warp takes a row and a query head, 32 tokens at a time: a lane a token for the scores,
// D / 32 columns for the sums.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) chunk_attention_kernel(const Args a) {
  constexpr int E = D / 32;
  __shared__ float qs[4][D];
  const CacheView &c = a.c;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = a.heads_q / c.heads;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + w; unit < (int64_t)a.n_rows * a.heads_q;
       unit += (int64_t)gridDim.x * 4) {
    const int row = (int)(unit / a.heads_q), h = (int)(unit - (int64_t)row * a.heads_q);
    int lo = 0, hi = a.R - 1;  // the last request whose first row is <= row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.row_start[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    const int i = row - a.row_start[lo];
    if (i < 0 || row >= a.row_start[lo + 1]) continue;
    if (i >= a.max_rows) {
      dspark_set_status(DSPARK_ERR_LENGTH);
      continue;
    }
    const long long cap = (long long)a.max_pages << c.page_shift;
    long long total = (long long)max(a.ctx[lo], 0) + i + 1;
    if (total > cap) {
      dspark_set_status(DSPARK_ERR_LENGTH);
      total = cap;
    }
    const int g = h / group;
    const float ks = FP8 && c.k_scale ? c.k_scale[g] : 1.0f;
    const float vs = FP8 && c.v_scale ? c.v_scale[g] : 1.0f;
    __syncwarp();
    for (int d = lane; d < D; d += 32)
      qs[w][d] = __bfloat162float(a.q[row * a.q_row + h * a.q_head + d]);
    __syncwarp();
    float m = -INFINITY, sum = 0.0f, o[E] = {};
    for (long long p0 = 0; p0 < total; p0 += 32) {
      const long long p = p0 + lane;
      int page = -1;
      int64_t at = 0;
      float s = -INFINITY;
      if (p < total) {
        page = a.block_table[(size_t)lo * a.max_pages + (p >> c.page_shift)];
        if (page < 0 || page >= c.n_pages) {
          dspark_set_status(DSPARK_ERR_PAGES);
          page = -1;
        }
        at = page * c.page_bytes + (p & ((1 << c.page_shift) - 1)) * c.token_bytes + g * c.head_bytes;
        float dot = 0.0f;
        if (page >= 0)
          for (int d = 0; d < D; ++d) {
            float k;
            if (FP8) {
              __half_raw r = __nv_cvt_fp8_to_halfraw(c.k[at + d], __NV_E4M3);
              k = __half2float(__half(r));
            } else {
              k = __bfloat162float(reinterpret_cast<const bf16 *>(c.k + at)[d]);
            }
            dot = fmaf(qs[w][d], k, dot);
          }
        s = dot * (a.scale * ks);
      }
      const float top = warp_max(s);
      const float to = fmaxf(m, top);
      const float keep = m == -INFINITY ? 0.0f : expf(m - to);
      const float e = p < total ? (to == -INFINITY ? 0.0f : expf(s - to)) : 0.0f;
      sum = sum * keep + warp_sum(e);
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] *= keep;
      for (int j = 0; j < 32 && p0 + j < total; ++j) {
        const float pj = __shfl_sync(0xffffffffu, e, j);
        const int64_t aj = __shfl_sync(0xffffffffu, at, j);
        if (__shfl_sync(0xffffffffu, page, j) < 0) continue;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const int d = lane + 32 * k;
          float v;
          if (FP8) {
            __half_raw r = __nv_cvt_fp8_to_halfraw(c.v[aj + d], __NV_E4M3);
            v = __half2float(__half(r));
          } else {
            v = __bfloat162float(reinterpret_cast<const bf16 *>(c.v + aj)[d]);
          }
          o[k] = fmaf(pj, v, o[k]);
        }
      }
      m = to;
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
      a.out[row * a.out_row + h * a.out_head + lane + 32 * k] = __float2bfloat16_rn(o[k] * vs / sum);
    if (a.lse && lane == 0) a.lse[(size_t)row * a.heads_q + h] = m + logf(sum);
  }
}

}  // namespace

extern "C" size_t dspark_chunk_attention_workspace_bytes(const dspark_kv_cache *cache, int32_t R,
                                                         int32_t heads_q, int32_t max_rows) {
  if (!dspark_kv_cache_ok(cache) || R < 1 || heads_q < 1 || heads_q % cache->heads ||
      heads_q / cache->heads > 64 || max_rows < 1)
    return 0;
  return 256;
}

extern "C" int dspark_chunk_attention(const dspark_kv_cache *cache, int32_t R, int32_t heads_q,
                                      int32_t max_rows, int32_t n_rows, int32_t max_pages,
                                      const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                      const int32_t *ctx, const int32_t *row_start,
                                      const int32_t *block_table, float scale, void *out,
                                      int64_t out_row_stride, int64_t out_head_stride, float *lse,
                                      void *workspace, size_t workspace_bytes,
                                      dspark_stream_t stream) {
  const size_t need = dspark_chunk_attention_workspace_bytes(cache, R, heads_q, max_rows);
  if (need == 0 || n_rows < 0 || max_pages < 1) return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  const int64_t most = (int64_t)1 << 39;
  if (!q || !ctx || !row_start || !block_table || !out ||
      (((uintptr_t)q | (uintptr_t)out) & 15) || q_row_stride <= 0 || q_head_stride <= 0 ||
      q_row_stride >= most || q_head_stride >= most || q_row_stride % 8 || q_head_stride % 8 ||
      out_row_stride <= 0 || out_head_stride <= 0 || out_row_stride >= most ||
      out_head_stride >= most || out_row_stride % 8 || out_head_stride % 8)
    return DSPARK_ERR_ARG;
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)
    return DSPARK_ERR_WORKSPACE;
  Args a;
  a.c = view_of(cache);
  a.R = R;
  a.heads_q = heads_q;
  a.max_rows = max_rows;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.q = (const bf16 *)q;
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.ctx = ctx;
  a.row_start = row_start;
  a.block_table = block_table;
  a.scale = scale;
  a.out = (bf16 *)out;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.lse = lse;
  const bool fp8 = cache->type == DSPARK_KV_E4M3;
  const int64_t blocks = ((int64_t)n_rows * heads_q + 3) / 4, cap = (int64_t)dspark_sm_count() * 64;
  const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
  if (cache->dim == 64) {
    if (fp8) chunk_attention_kernel<64, true><<<grid, 128, 0, stream>>>(a);
    else chunk_attention_kernel<64, false><<<grid, 128, 0, stream>>>(a);
  } else {
    if (fp8) chunk_attention_kernel<128, true><<<grid, 128, 0, stream>>>(a);
    else chunk_attention_kernel<128, false><<<grid, 128, 0, stream>>>(a);
  }
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

int dspark_status_chunk(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_chunk, sizeof(int)) != cudaSuccess) return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_chunk, &zero, sizeof(int));
  }
  return v;
}
