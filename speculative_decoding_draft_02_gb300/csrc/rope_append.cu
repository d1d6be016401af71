// rope_append.cu — dspark_rope_append: norm of every head of the queries and keys, the
// rotation by position, and the keys and values into their slots, in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// Each value is read once and written once; everything else (statistics, angles, the
// other half of a pair) stays in a warp's registers.  Bound by those bytes: eight prompts
// of 2048 rows (32 + 8 + 8 heads of 128, bf16) take 66 us in a graph, 6.1 TB/s; 3510 ragged
// rows in pairs into e4m3 pages 14 us, where latencies and instructions count beside
// them; four single tokens 3 us, the launch.  Into e4m3 pages instructions bound long ones
// too: the eight prompts' rows 83 us, 4.5 TB/s.  So they do beside few KV heads, as a step
// takes 512 / dim heads of one kind and lanes without a head idle: 16384 rows of 8 + 1 + 1
// heads of 128 26 us (e4m3 34) where the bytes take 12, of 64 21 (29) where they take 6.
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

constexpr int THREADS = 256, BLOCKS_SM = 2;
constexpr int BATCH = 4;          // steps of a warp whose loads are asked for together
constexpr int STEP_BYTES = 1024;  // 32 bytes a lane
constexpr int SMEM_BYTES = THREADS / 32 * 2 * BATCH * STEP_BYTES;
enum { Q_HEADS, K_HEADS, V_HEADS };

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// A lane's 16 values of a head, two chunks of 8, as the first and the second values of
// eight pairs, two of them in a float2.
template <bool PAIRS>
__device__ __forceinline__ void unpack(const uint4 (&x)[2], float2 (&a)[4], float2 (&b)[4]) {
  const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PAIRS) {
      a[i] = make_float2(bf16_lo(v[2 * i]), bf16_lo(v[2 * i + 1]));
      b[i] = make_float2(bf16_hi(v[2 * i]), bf16_hi(v[2 * i + 1]));
    } else {
      a[i] = make_float2(bf16_lo(v[i]), bf16_hi(v[i]));
      b[i] = make_float2(bf16_lo(v[4 + i]), bf16_hi(v[4 + i]));
    }
  }
}
// Back in the chunks' order.
template <bool PAIRS>
__device__ __forceinline__ void in_order(const float2 (&a)[4], const float2 (&b)[4],
                                         float (&lo)[8], float (&hi)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PAIRS) {
      float *to = i < 2 ? lo + 4 * i : hi + 4 * (i - 2);
      to[0] = a[i].x;
      to[1] = b[i].x;
      to[2] = a[i].y;
      to[3] = b[i].y;
    } else {
      lo[2 * i] = a[i].x;
      lo[2 * i + 1] = a[i].y;
      hi[2 * i] = b[i].x;
      hi[2 * i + 1] = b[i].y;
    }
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

// (out of line: it is seldom called)
__device__ __noinline__ uint32_t divided_e4m3(float a, float b, float c, float d, float scale) {
  return pack_e4m3x2(a / scale, b / scale) | pack_e4m3x2(c / scale, d / scale) << 16;
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
    return make_uint2(divided_e4m3(x[0], x[1], x[2], x[3], scale),
                      divided_e4m3(x[4], x[5], x[6], x[7], scale));
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = pack_e4m3x2(q[4 * i], q[4 * i + 1]) | pack_e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
  return make_uint2(o[0], o[1]);
}

// A lane holds 16 values of a head, two chunks of 8: D / 16 lanes a head, 32 * 16 / D
// heads a warp and step.  Chunks are dealt so that both values of a pair lie in one
// lane: in halves chunk t and its partner rot / 2 values on (lanes past the rotated
// values take two chunks of the rest), in pairs chunks t and t + D / 16.  All lanes with
// one t turn by the same eight angles, which the warp computes once a row, one or two a
// lane, and multiplies by the weights: a head then takes four products a pair, and one
// factor for its norm.
//
// A warp takes a row, or with few rows a part of its steps (`parts` warps a row), the
// queries' heads first, then the keys', then the values'.  Its loads run one batch of
// steps ahead, into the lanes' own places in shared memory (no barrier): 128 KB are then
// in flight on an SM, which registers have no room for (with the loads in registers the
// eight prompts took 80 us).
template <int D, bool FP8, bool PAIRS>
__global__ void __launch_bounds__(THREADS, BLOCKS_SM) rope_append_kernel(const RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, FREQS = D / 64;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();
  pdl_wait();
  const CacheView &c = a.c;
  const int lane = threadIdx.x & 31, t = lane % LPH, sub = lane / LPH;
  uint8_t *const mine = smem + (threadIdx.x >> 5) * 2 * BATCH * STEP_BYTES + lane * 16;
  // whether the lane's first four pairs turn, and its last four
  const bool turns[2] = {(PAIRS ? 8 : 16) * t < a.rot, (PAIRS ? 8 * t + D / 2 : 16 * t) < a.rot};
  const int rest = a.rot / 8 + 2 * (t - a.rot / 16);
  const int lo = 8 * (PAIRS || turns[0] ? t : rest);
  const int hi = lo + (PAIRS ? D / 2 : turns[0] ? a.rot / 2 : 8);
  const int steps_q = (a.heads_q + HPW - 1) / HPW, steps_k = (c.heads + HPW - 1) / HPW;
  const int steps = steps_q + 2 * steps_k;
  const int64_t n_slots = (int64_t)c.n_pages << c.page_shift;
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  const int64_t units = (int64_t)a.n_rows * a.parts;

  struct Unit {
    int row, s, end, pos;
    int64_t slot;
  };
  int64_t at = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  auto read_unit = [&](Unit &u) {
    if (at >= units) {
      u.row = -1;
      return;
    }
    u.row = (int)(at / a.parts);
    const int part = (int)(at - (int64_t)u.row * a.parts);
    u.s = (int)((int64_t)steps * part / a.parts);
    u.end = (int)((int64_t)steps * (part + 1) / a.parts);
    u.pos = a.position[u.row];
    u.slot = a.slot[u.row];
    at += warps;
  };
  // the next row that is no padding
  auto next_unit = [&](Unit &u, Unit &ahead) {
    do {
      u = ahead;
      if (u.row < 0) return;
      read_unit(ahead);
    } while (u.pos < 0);
  };
  // a batch of steps from u.s on, into one half of the warp's place
  auto issue = [&](const Unit &u, int half) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int s = u.s + i;
      if (s >= u.end) break;
      const bool is_q = s < steps_q, is_k = s < steps_q + steps_k;
      const int h = (s - (is_q ? 0 : is_k ? steps_q : steps_q + steps_k)) * HPW + sub;
      if (h >= (is_q ? a.heads_q : c.heads)) continue;
      const bf16 *src = is_q ? a.q + u.row * a.q_row + h * a.q_head
                             : (is_k ? a.k : a.v) + u.row * a.kv_row + h * a.kv_head;
      const uint32_t to =
          (uint32_t)__cvta_generic_to_shared(mine + (half * BATCH + i) * STEP_BYTES);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + lo) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + STEP_BYTES / 2),
                   "l"(src + hi)
                   : "memory");
    }
  };

  uint64_t turn[FREQS];
#pragma unroll
  for (int f = 0; f < FREQS; ++f) {
    // the pair that this lane computes for lanes t, the j-th of their eight
    const int j = sub * FREQS + f;
    const int i = PAIRS ? 4 * t + j + (j < 4 ? 0 : D / 4 - 4) : 8 * t + j;
    turn[f] = 2 * i < a.rot ? a.turns[i] : 0;
  }
  Unit u, ahead;
  read_unit(ahead);
  next_unit(u, ahead);
  if (u.row < 0) return;
  issue(u, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  float my_c[FREQS], my_s[FREQS];
  float2 ca[4], sa[4], cb[4], sb[4];  // by value: weight times cosine, times sine
  int turned = -1, kind_made = -1;    // what they are for: a row, its queries or keys
#pragma unroll 1
  for (int half = 0;; half ^= 1) {
    Unit next = u;
    next.s += BATCH;
    if (next.s >= u.end) next_unit(next, ahead);
    if (next.row >= 0) issue(next, half ^ 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (turned != u.row) {  // under the loads
      turned = u.row;
      kind_made = -1;
#pragma unroll
      for (int f = 0; f < FREQS; ++f) {
        const int32_t half_turns = (int32_t)(((uint64_t)u.pos * turn[f]) >> 32);
        sincospif((float)half_turns * 0x1p-31f, &my_s[f], &my_c[f]);
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const bool stored = u.slot >= 0 && u.slot < n_slots;
    if (u.slot >= n_slots && lane == 0) dspark_set_status(DSPARK_ERR_PAGES);
    const int64_t place = stored ? (u.slot >> c.page_shift) * c.page_bytes +
                                       (u.slot & ((1 << c.page_shift) - 1)) * c.token_bytes
                                 : 0;
    const int end = min(u.s + BATCH, u.end);
#pragma unroll 1
    for (int s = u.s; s < end; ++s) {  // a warp's lanes alike
      const int kind = s < steps_q ? Q_HEADS : s < steps_q + steps_k ? K_HEADS : V_HEADS;
      const int h =
          (s - (kind == Q_HEADS ? 0 : kind == K_HEADS ? steps_q : steps_q + steps_k)) * HPW + sub;
      const bool there = h < (kind == Q_HEADS ? a.heads_q : c.heads);
      const uint8_t *from = mine + (half * BATCH + s - u.s) * STEP_BYTES;
      const uint4 x[2] = {*reinterpret_cast<const uint4 *>(from),
                          *reinterpret_cast<const uint4 *>(from + STEP_BYTES / 2)};
      if (kind == V_HEADS && !FP8) {  // V's bits as they are
        if (there && stored) {
          uint8_t *dst = c.v + place + h * c.head_bytes;
          *reinterpret_cast<uint4 *>(dst + 2 * lo) = x[0];
          *reinterpret_cast<uint4 *>(dst + 2 * hi) = x[1];
        }
        continue;
      }
      float2 p[4], q[4];
      unpack<PAIRS>(x, p, q);
      if (kind != V_HEADS) {
        const bf16 *weight = kind == Q_HEADS ? a.q_weight : a.k_weight;
        if (kind_made != kind) {
          kind_made = kind;
          uint4 w[2];
          w[0] = w[1] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
          if (weight) {
            w[0] = *reinterpret_cast<const uint4 *>(weight + lo);
            w[1] = *reinterpret_cast<const uint4 *>(weight + hi);
          }
          unpack<PAIRS>(w, ca, cb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float cs[2], sn[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int f = 2 * i + j;
              cs[j] = __shfl_sync(0xffffffffu, my_c[f % FREQS], t + LPH * (f / FREQS));
              sn[j] = __shfl_sync(0xffffffffu, my_s[f % FREQS], t + LPH * (f / FREQS));
            }
            sa[i] = make_float2(ca[i].x * sn[0], ca[i].y * sn[1]);
            sb[i] = make_float2(-cb[i].x * sn[0], -cb[i].y * sn[1]);
            ca[i] = make_float2(ca[i].x * cs[0], ca[i].y * cs[1]);  // 1 where nothing turns
            cb[i] = make_float2(cb[i].x * cs[0], cb[i].y * cs[1]);
          }
        }
        float inv = 1.0f;
        if (weight) {
          float2 sum = mul2(p[0], p[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) sum = fma2(p[i], p[i], sum);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fma2(q[i], q[i], sum);
          float all = sum.x + sum.y;
#pragma unroll
          for (int o = 1; o < LPH; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
          inv = rsqrtf(all * (1.0f / D) + a.eps);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 pc[2] = {mul2(p[i], ca[i]), mul2(p[i + 1], ca[i + 1])};
          const float2 qc[2] = {mul2(q[i], cb[i]), mul2(q[i + 1], cb[i + 1])};
          if (turns[i / 2]) {
            const float2 ps[2] = {p[i], p[i + 1]};
            p[i] = fma2(q[i], sb[i], pc[0]);
            p[i + 1] = fma2(q[i + 1], sb[i + 1], pc[1]);
            q[i] = fma2(ps[0], sa[i], qc[0]);
            q[i + 1] = fma2(ps[1], sa[i + 1], qc[1]);
          } else {  // what does not turn meets nothing else
            p[i] = pc[0];
            p[i + 1] = pc[1];
            q[i] = qc[0];
            q[i + 1] = qc[1];
          }
        }
        if (weight) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = mul2(p[i], make_float2(inv, inv));
            q[i] = mul2(q[i], make_float2(inv, inv));
          }
        }
      }
      if (!there) continue;
      float y0[8], y1[8];
      in_order<PAIRS>(p, q, y0, y1);
      if (kind == Q_HEADS) {
        bf16 *dst = a.out + u.row * a.out_row + h * a.out_head;
        *reinterpret_cast<uint4 *>(dst + lo) = pack8(y0);
        *reinterpret_cast<uint4 *>(dst + hi) = pack8(y1);
      } else if (stored) {
        uint8_t *dst = (kind == V_HEADS ? c.v : c.k) + place + h * c.head_bytes;
        if constexpr (FP8) {
          const float *scales = kind == V_HEADS ? c.v_scale : c.k_scale;
          const float scale = scales ? scales[h] : 1.0f, inv = 1.0f / scale;
          const bool near_one = scale >= 0x1p-96f && scale <= 0x1p96f;
          *reinterpret_cast<uint2 *>(dst + lo) = scaled_e4m3(y0, scale, inv, near_one);
          *reinterpret_cast<uint2 *>(dst + hi) = scaled_e4m3(y1, scale, inv, near_one);
        } else {
          *reinterpret_cast<uint4 *>(dst + 2 * lo) = pack8(y0);
          *reinterpret_cast<uint4 *>(dst + 2 * hi) = pack8(y1);
        }
      }
    }
    if (next.row < 0) break;
    u = next;
  }
}

template <int D, bool FP8, bool PAIRS>
cudaError_t launch(const RopeArgs &a, dim3 grid, cudaStream_t stream) {
  auto kernel = rope_append_kernel<D, FP8, PAIRS>;
  static DsparkPerDevice attr;
  if (dspark_per_device(attr, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    SMEM_BYTES) == cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return cudaErrorInvalidValue;
  return dspark_launch_pdl(kernel, grid, dim3(THREADS), SMEM_BYTES, stream, a);
}
template <int D>
cudaError_t launch(const RopeArgs &a, bool fp8, bool pairs, dim3 grid, cudaStream_t stream) {
  if (fp8) return pairs ? launch<D, true, true>(a, grid, stream) : launch<D, true, false>(a, grid, stream);
  return pairs ? launch<D, false, true>(a, grid, stream) : launch<D, false, false>(a, grid, stream);
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
  const int at_once = 512 / cache->dim;
  const int steps = (heads_q + at_once - 1) / at_once + 2 * ((cache->heads + at_once - 1) / at_once);
  const int64_t resident = (int64_t)dspark_sm_count() * BLOCKS_SM * (THREADS / 32);
  // Into how many parts a row is split: what leaves the busiest warp the least work, a
  // part's angles and weights counted as two steps.
  a.parts = 1;
  int64_t least = INT64_MAX;
  for (int parts = 1; parts <= steps && parts <= 64; ++parts) {
    const int64_t turns = ((int64_t)n_rows * parts + resident - 1) / resident;
    const int64_t work = turns * ((steps + parts - 1) / parts + 2);
    if (work < least) {
      least = work;
      a.parts = parts;
    }
    if (turns > 64) break;
  }
  const int64_t blocks = ((int64_t)n_rows * a.parts + THREADS / 32 - 1) / (THREADS / 32);
  const int64_t most = resident / (THREADS / 32);
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  const bool pairs = rope->style == DSPARK_ROPE_PAIRS, fp8 = cache->type == DSPARK_KV_E4M3;
  const cudaError_t e = cache->dim == 64 ? launch<64>(a, fp8, pairs, grid, stream)
                                         : launch<128>(a, fp8, pairs, grid, stream);
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
