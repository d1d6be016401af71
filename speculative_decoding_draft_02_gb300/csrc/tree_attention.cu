// tree_attention.cu — dspark_tree_attention: checks, the choice of the row tile,
// and the launches of tree_attention.cuh.
#include "kv_cache.cuh"
#include "tcgen05_attn.cuh"
#include "tensor_map.cuh"

DSPARK_DECLARE_STATUS(s_status_attention)

#include "tree_attention.cuh"

namespace {

using attn::Args;

// Query rows of a tile: the narrowest that takes a request's rows, so that no
// product, exponential or byte of shared memory is spent on empty columns; at
// most 128 (two tiles of scores and O in tensor memory, and Q and P in shared memory,
// beside the tiles in flight).  Beside an 8-bit cache the widening warps leave room for
// 64 (eight contexts of 32768, 64 rows: 172 us, 272 in tiles of 32; 128 rows: 324 and
// 519; 64 trees of 64 nodes over 512 to 4096 tokens, where the masked tiles weigh more:
// 742 and 692), and take 33 to 48 rows so too (36 rows: 307 us, 311 in tiles of 48).
int row_tile(const dspark_kv_cache *c, int heads_q, int max_nodes) {
  const int group = heads_q / c->heads, rows = max_nodes * group;
  if (rows <= 16) return 16;
  if (rows <= 32) return 32;
  if (c->type == DSPARK_KV_E4M3) return 64;
  if (rows <= 48) return 48;
  return rows <= 64 ? 64 : 128;
}

struct Layout {
  size_t ml, desc, bytes;
};
Layout layout_of(int ctas, int nt, int dim) {
  Layout l;
  l.ml = dspark_align_up((size_t)ctas * 2 * nt * dim * sizeof(float), 256);
  l.desc = l.ml + dspark_align_up((size_t)ctas * 4 * nt * sizeof(float), 256);
  l.bytes = l.desc + dspark_align_up((size_t)ctas * 8 * sizeof(int), 256);
  return l;
}

struct Launch {
  const dspark_kv_cache *cache;
  Args a;
  const void *q;
  int64_t q_row, q_head;
  int ctas;
  cudaStream_t stream;
};

template <int TYPE, int D, int NT>
int launch(const Launch &l) {
  using G = attn::Geo<TYPE, D, NT>;
  const dspark_kv_cache *c = l.cache;
  Args a = l.a;
  a.nodes_tile = NT / a.group;
  const uint64_t size = G::FP8 ? 1 : 2;
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)c->page_size, (uint64_t)c->heads,
                            (uint64_t)c->n_pages};
  const uint64_t strides[3] = {c->token_stride * size, c->head_stride * size,
                               c->page_stride * size};
  const uint32_t rows = c->page_size < attn::BT ? c->page_size : attn::BT;
  const uint32_t box[4] = {G::FP8 ? (uint32_t)D : 64u, rows, 1, 1};
  const CUtensorMapDataType type =
      G::FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle swizzle =
      G::FP8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t q_dims[3] = {(uint64_t)D, (uint64_t)(a.heads * a.group), (uint64_t)a.n_rows};
  const uint64_t q_strides[2] = {(uint64_t)l.q_head * 2, (uint64_t)l.q_row * 2};
  const uint32_t q_box[3] = {64, (uint32_t)a.group, (uint32_t)a.nodes_tile};
  CUtensorMap tk, tv, tq;
  if (!make_map(&tk, type, c->k, dims, strides, box, swizzle) ||
      !make_map(&tv, type, c->v, dims, strides, box, swizzle) ||
      !make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.q, q_dims, q_strides, q_box,
                CU_TENSOR_MAP_SWIZZLE_128B))
    return DSPARK_ERR_CUDA;
  auto kernel = attn::tree_attention_kernel<TYPE, D, NT>;
  static DsparkPerDevice attr;
  if (dspark_per_device(attr, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    G::SMEM_BYTES) == cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return DSPARK_ERR_CUDA;
  if (dspark_launch_pdl(kernel, dim3(l.ctas), dim3(G::THREADS), G::SMEM_BYTES, l.stream, tk, tv,
                        tq, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  if (dspark_launch_pdl(attn::tree_attention_join<D>, dim3(l.ctas, NT / 4), dim3(128), 0,
                        l.stream, a, NT) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(2);
  return DSPARK_OK;
}

template <int TYPE, int D>
int launch_tile(const Launch &l, int nt) {
  if (nt == 16) return launch<TYPE, D, 16>(l);
  if (nt == 32) return launch<TYPE, D, 32>(l);
  if constexpr (TYPE == DSPARK_KV_BF16) {
    if (nt == 48) return launch<TYPE, D, 48>(l);
    if (nt == 128) return launch<TYPE, D, 128>(l);
  }
  return launch<TYPE, D, 64>(l);
}

}  // namespace

extern "C" size_t dspark_tree_attention_workspace_bytes(const dspark_kv_cache *cache, int32_t R,
                                                        int32_t heads_q, int32_t max_nodes) {
  if (!dspark_kv_cache_ok(cache) || R < 1 || heads_q < 1 || heads_q % cache->heads ||
      heads_q / cache->heads > 64 || max_nodes < 1 || max_nodes > DSPARK_MAX_NODES)
    return 0;
  return layout_of(dspark_sm_count(), row_tile(cache, heads_q, max_nodes), cache->dim).bytes;
}

extern "C" int dspark_tree_attention(const dspark_kv_cache *cache, int32_t R, int32_t heads_q,
                                     int32_t max_nodes, int32_t n_rows, int32_t max_pages,
                                     const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                     const int32_t *ctx, const int32_t *row_start,
                                     const uint64_t *anc, const int32_t *block_table, float scale,
                                     void *out, int64_t out_row_stride, int64_t out_head_stride,
                                     float *lse, void *workspace, size_t workspace_bytes,
                                     dspark_stream_t stream) {
  const size_t need = dspark_tree_attention_workspace_bytes(cache, R, heads_q, max_nodes);
  if (need == 0 || n_rows < 0 || max_pages < 1) return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  const int64_t most = (int64_t)1 << 39;  // elements: a tensor map's strides are below 2^40 bytes
  const int64_t out_most = (int64_t)1 << 24;  // a tile's rows lie within 2^31 elements
  if (!q || !ctx || !row_start || !block_table || !out || ((uintptr_t)q & 15) ||
      ((uintptr_t)out & 1) || q_row_stride <= 0 || q_head_stride <= 0 || q_row_stride >= most ||
      q_head_stride >= most || q_row_stride % 8 || q_head_stride % 8 || out_row_stride <= 0 ||
      out_head_stride <= 0 || out_row_stride > out_most || out_head_stride > out_most)
    return DSPARK_ERR_ARG;
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)
    return DSPARK_ERR_WORKSPACE;
  Launch l;
  l.cache = cache;
  l.q = q;
  l.q_row = q_row_stride;
  l.q_head = q_head_stride;
  l.ctas = dspark_sm_count();
  l.stream = stream;
  const bool fp8 = cache->type == DSPARK_KV_E4M3;
  const int nt = row_tile(cache, heads_q, max_nodes);
  const Layout at = layout_of(l.ctas, nt, cache->dim);
  const int64_t size = dspark_kv_bytes(cache->type);
  Args &a = l.a;
  a.R = R;
  a.heads = cache->heads;
  a.group = heads_q / cache->heads;
  a.max_nodes = max_nodes;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
  a.n_pages = cache->n_pages;
  a.ctx = ctx;
  a.row_start = row_start;
  a.block_table = block_table;
  a.anc = anc;
  a.k_scale = fp8 ? cache->k_scale : nullptr;
  a.v_scale = fp8 ? cache->v_scale : nullptr;
  a.v = (const uint8_t *)cache->v;
  a.page_bytes = cache->page_stride * size;
  a.token_bytes = cache->token_stride * size;
  a.head_bytes = cache->head_stride * size;
  a.scale = scale;
  a.out = (bf16 *)out;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.lse = lse;
  a.part_o = (float *)workspace;
  a.part_ml = (float *)((uint8_t *)workspace + at.ml);
  a.desc = (int *)((uint8_t *)workspace + at.desc);
  if (fp8)
    return cache->dim == 64 ? launch_tile<DSPARK_KV_E4M3, 64>(l, nt)
                            : launch_tile<DSPARK_KV_E4M3, 128>(l, nt);
  return cache->dim == 64 ? launch_tile<DSPARK_KV_BF16, 64>(l, nt)
                          : launch_tile<DSPARK_KV_BF16, 128>(l, nt);
}

int dspark_status_attention(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_attention, sizeof(int)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_attention, &zero, sizeof(int));
  }
  return v;
}
