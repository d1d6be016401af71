// rope_append.cu — dspark_rope_append: norm of every head of the queries and keys, the
// rotation by position, and the keys and values into their slots, in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// Each value is read once and written once; everything else (statistics, angles, the
// other half of a pair) stays in a warp's registers.  Bound by those bytes.
//
// Angles.  t = 2 pi frac(p turns / 2^64): the product modulo 2^64 is the fraction of a
// turn, exact but for the rounding of `turns` itself, so no wide floating-point
// product and no range reduction is needed.  Its upper 32 bits, as a signed number of
// 2^-31 half turns, go to sincospi: off by at most 2^-25 of half a turn.
#include "kv_cache.cuh"

DSPARK_DECLARE_STATUS(s_status_rope)

namespace {

struct RopeArgs {
  CacheView c;
  int n_rows, heads_q, rot, parts;
  const bf16 *q, *k, *v, *q_weight, *k_weight;
  bf16 *out;
  int64_t q_row, q_head, kv_row, kv_head, out_row, out_head;
  float eps;
  const uint64_t *turns;
  const int *position;
  const int64_t *slot;
};

constexpr int THREADS = 256, BLOCKS_SM = 4;
constexpr int AT_ONCE = 4;  // heads of a lane whose loads are in flight together

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t *>(&two);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __noinline__ uint2 divided_e4m3(const float (&x)[8], float scale) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = pack_e4m3x2(x[4 * i] / scale, x[4 * i + 1] / scale) |
           pack_e4m3x2(x[4 * i + 2] / scale, x[4 * i + 3] / scale) << 16;
  return make_uint2(o[0], o[1]);
}

// Eight values over a scale as e4m3, by the scale's reciprocal where the quotient rounds
// the same: for a scale in [2^-96, 2^96] the product is within two units of its last
// place of the quotient, and e4m3 rounds at values whose 19 last bits are zero, so only a
// product within four units of such a value is divided.
__device__ __forceinline__ uint2 scaled_e4m3(const float (&x)[8], float scale, float inv,
                                             bool near_one) {
  float q[8];
  uint32_t least = 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x[i] * inv;
    least = min(least, (__float_as_uint(q[i]) + 4) & 0x7ffff);
  }
  if (!near_one || (least < 8 && (__float_as_uint(scale) & 0x7fffff) != 0))
    return divided_e4m3(x, scale);
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = pack_e4m3x2(q[4 * i], q[4 * i + 1]) | pack_e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
  return make_uint2(o[0], o[1]);
}

// A lane holds 16 values of a head, two chunks of 8: D / 16 lanes a head, 32 * 16 / D
// heads a warp and step.  Chunks are dealt so that both values of a pair lie in one
// lane: in halves chunk t and its partner rot / 2 values on, in pairs chunks 2 t and
// 2 t + 1; lanes past the rotated values take two chunks of the rest.  All lanes with
// one t turn by the same eight angles, which the warp computes once a row, one or two a
// lane.  A warp takes a row, or with few rows a part of its heads (`parts` warps a row).
template <int D, bool FP8, bool PAIRS>
__global__ void __launch_bounds__(THREADS) rope_append_kernel(const RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, FREQS = D / 64;
  pdl_trigger();
  pdl_wait();
  const CacheView &c = a.c;
  const int lane = threadIdx.x & 31, t = lane % LPH, sub = lane / LPH;
  const bool turns = 16 * t < a.rot;
  const int rest = a.rot / 8 + 2 * (t - a.rot / 16);
  const int lo = 8 * (PAIRS ? 2 * t : (turns ? t : rest));
  const int hi = PAIRS ? lo + 8 : (turns ? lo + a.rot / 2 : lo + 8);
  uint64_t turn[FREQS];
#pragma unroll
  for (int f = 0; f < FREQS; ++f) {
    const int i = 8 * t + sub * FREQS + f;  // the pair that this lane computes for lanes t
    turn[f] = 2 * i < a.rot ? a.turns[i] : 0;
  }
  uint4 wq[2] = {}, wk[2] = {};
  if (a.q_weight) {
    wq[0] = *reinterpret_cast<const uint4 *>(a.q_weight + lo);
    wq[1] = *reinterpret_cast<const uint4 *>(a.q_weight + hi);
  }
  if (a.k_weight) {
    wk[0] = *reinterpret_cast<const uint4 *>(a.k_weight + lo);
    wk[1] = *reinterpret_cast<const uint4 *>(a.k_weight + hi);
  }
  const int heads = a.heads_q + 2 * c.heads, steps = (heads + HPW - 1) / HPW;
  const int64_t n_slots = (int64_t)c.n_pages << c.page_shift;
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  for (int64_t unit = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
       unit < (int64_t)a.n_rows * a.parts; unit += warps) {
    const int row = (int)(unit / a.parts), part = (int)(unit - (int64_t)row * a.parts);
    const int pos = a.position[row];
    if (pos < 0) continue;
    const int64_t slot = a.slot[row];
    const bool stored = slot >= 0 && slot < n_slots;
    if (slot >= n_slots && lane == 0) dspark_set_status(DSPARK_ERR_PAGES);
    const int64_t place = stored ? (slot >> c.page_shift) * c.page_bytes +
                                       (slot & ((1 << c.page_shift) - 1)) * c.token_bytes
                                 : 0;
    const int s0 = (int)((int64_t)steps * part / a.parts);
    const int s1 = (int)((int64_t)steps * (part + 1) / a.parts);
    float cs[8], sn[8];
    bool known = false;
#pragma unroll 1
    for (int s = s0; s < s1; s += AT_ONCE) {
      uint4 x[AT_ONCE][2];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int h = (s + u) * HPW + sub;
        if (s + u >= s1 || h >= heads) continue;
        const int g = h - a.heads_q;
        const bf16 *src = g < 0 ? a.q + row * a.q_row + h * a.q_head
                                : (g < c.heads ? a.k + row * a.kv_row + g * a.kv_head
                                               : a.v + row * a.kv_row + (g - c.heads) * a.kv_head);
        x[u][0] = *reinterpret_cast<const uint4 *>(src + lo);
        x[u][1] = *reinterpret_cast<const uint4 *>(src + hi);
      }
      if (!known) {  // under the first loads
        known = true;
        float my_c[FREQS], my_s[FREQS];
#pragma unroll
        for (int f = 0; f < FREQS; ++f) {
          const int32_t half_turns = (int32_t)(((uint64_t)pos * turn[f]) >> 32);
          sincospif((float)half_turns * 0x1p-31f, &my_s[f], &my_c[f]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cs[j] = __shfl_sync(0xffffffffu, my_c[j % FREQS], t + LPH * (j / FREQS));
          sn[j] = __shfl_sync(0xffffffffu, my_s[j % FREQS], t + LPH * (j / FREQS));
        }
      }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int h = (s + u) * HPW + sub, g = h - a.heads_q;
        if (s + u >= s1) continue;  // a warp's lanes alike
        const bool there = h < heads, is_q = g < 0, is_v = g >= c.heads;
        float p[8] = {}, q[8] = {};
        if (there) {
          unpack8(x[u][0], p);
          unpack8(x[u][1], q);
        }
        if (a.q_weight || a.k_weight) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(p[i], p[i], fmaf(q[i], q[i], sum));
#pragma unroll
          for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (!is_v && (is_q ? a.q_weight : a.k_weight)) {
            const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
            float w[8];
            unpack8(is_q ? wq[0] : wk[0], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = p[i] * inv * w[i];
            unpack8(is_q ? wq[1] : wk[1], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = q[i] * inv * w[i];
          }
        }
        if (!there) continue;
        if (turns && !is_v) {
          if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a0 = p[2 * i], b0 = p[2 * i + 1], a1 = q[2 * i], b1 = q[2 * i + 1];
              p[2 * i] = a0 * cs[i] - b0 * sn[i];
              p[2 * i + 1] = b0 * cs[i] + a0 * sn[i];
              q[2 * i] = a1 * cs[4 + i] - b1 * sn[4 + i];
              q[2 * i + 1] = b1 * cs[4 + i] + a1 * sn[4 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a0 = p[i], b0 = q[i];
              p[i] = a0 * cs[i] - b0 * sn[i];
              q[i] = b0 * cs[i] + a0 * sn[i];
            }
          }
        }
        if (is_q) {
          bf16 *dst = a.out + row * a.out_row + h * a.out_head;
          *reinterpret_cast<uint4 *>(dst + lo) = pack8(p);
          *reinterpret_cast<uint4 *>(dst + hi) = pack8(q);
          continue;
        }
        if (!stored) continue;
        const int kv = is_v ? g - c.heads : g;
        uint8_t *dst = (is_v ? c.v : c.k) + place + kv * c.head_bytes;
        if constexpr (FP8) {
          const float *scales = is_v ? c.v_scale : c.k_scale;
          const float scale = scales ? scales[kv] : 1.0f, inv = 1.0f / scale;
          const bool near_one = scale >= 0x1p-96f && scale <= 0x1p96f;
          *reinterpret_cast<uint2 *>(dst + lo) = scaled_e4m3(p, scale, inv, near_one);
          *reinterpret_cast<uint2 *>(dst + hi) = scaled_e4m3(q, scale, inv, near_one);
        } else {
          // V's bits as they are
          *reinterpret_cast<uint4 *>(dst + 2 * lo) = is_v ? x[u][0] : pack8(p);
          *reinterpret_cast<uint4 *>(dst + 2 * hi) = is_v ? x[u][1] : pack8(q);
        }
      }
    }
  }
}

template <int D, bool FP8>
cudaError_t launch(const RopeArgs &a, bool pairs, dim3 grid, cudaStream_t stream) {
  return pairs ? dspark_launch_pdl(rope_append_kernel<D, FP8, true>, grid, dim3(THREADS), 0,
                                   stream, a)
               : dspark_launch_pdl(rope_append_kernel<D, FP8, false>, grid, dim3(THREADS), 0,
                                   stream, a);
}

bool rows_ok(const void *p, int64_t row, int64_t head) {
  const int64_t most = (int64_t)1 << 39;
  return p && !((uintptr_t)p & 15) && row > 0 && head > 0 && row < most && head < most &&
         row % 8 == 0 && head % 8 == 0;
}

}  // namespace

extern "C" int dspark_rope_append(const dspark_kv_cache *cache, int32_t n_rows, int32_t heads_q,
                                  const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                  const void *k, const void *v, int64_t kv_row_stride,
                                  int64_t kv_head_stride, const void *q_weight,
                                  const void *k_weight, float eps, const dspark_rope *rope,
                                  const int32_t *position, const int64_t *slot, void *q_out,
                                  int64_t out_row_stride, int64_t out_head_stride,
                                  dspark_stream_t stream) {
  if (!dspark_kv_cache_ok(cache) || n_rows < 0 || heads_q < 1 || heads_q > 65535 ||
      cache->heads > 65535 || !rope || rope->dims < 0 || rope->dims > cache->dim ||
      rope->dims % 16 || (rope->style != DSPARK_ROPE_HALVES && rope->style != DSPARK_ROPE_PAIRS) ||
      !(eps >= 0.0f))
    return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  if (!rows_ok(q, q_row_stride, q_head_stride) || !rows_ok(k, kv_row_stride, kv_head_stride) ||
      !rows_ok(v, kv_row_stride, kv_head_stride) ||
      !rows_ok(q_out, out_row_stride, out_head_stride) || !position || !slot ||
      (rope->dims && (!rope->turns || ((uintptr_t)rope->turns & 7))) ||
      (((uintptr_t)q_weight | (uintptr_t)k_weight) & 15))
    return DSPARK_ERR_ARG;
  RopeArgs a;
  a.c = view_of(cache);
  a.n_rows = n_rows;
  a.heads_q = heads_q;
  a.rot = rope->dims;
  a.q = (const bf16 *)q;
  a.k = (const bf16 *)k;
  a.v = (const bf16 *)v;
  a.q_weight = (const bf16 *)q_weight;
  a.k_weight = (const bf16 *)k_weight;
  a.out = (bf16 *)q_out;
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.kv_row = kv_row_stride;
  a.kv_head = kv_head_stride;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.eps = eps;
  a.turns = rope->turns;
  a.position = position;
  a.slot = slot;
  // Rows are split over warps while that fills the GPU: half of its resident warps.
  const int64_t resident = (int64_t)dspark_sm_count() * BLOCKS_SM * (THREADS / 32);
  const int steps = (heads_q + 2 * cache->heads + 512 / cache->dim - 1) / (512 / cache->dim);
  const int64_t want = resident / 2 / n_rows;
  a.parts = (int)(want < 1 ? 1 : want < steps ? want : steps);
  const int64_t blocks = ((int64_t)n_rows * a.parts + THREADS / 32 - 1) / (THREADS / 32);
  const int64_t most = resident / (THREADS / 32);
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  const bool pairs = rope->style == DSPARK_ROPE_PAIRS, fp8 = cache->type == DSPARK_KV_E4M3;
  const cudaError_t e = cache->dim == 64 ? (fp8 ? launch<64, true>(a, pairs, grid, stream)
                                                : launch<64, false>(a, pairs, grid, stream))
                                         : (fp8 ? launch<128, true>(a, pairs, grid, stream)
                                                : launch<128, false>(a, pairs, grid, stream));
  if (e != cudaSuccess) return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

int dspark_status_rope(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_rope, sizeof(int)) != cudaSuccess) return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_rope, &zero, sizeof(int));
  }
  return v;
}
