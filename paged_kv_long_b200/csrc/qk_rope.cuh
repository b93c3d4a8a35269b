// qk_rope.cuh — the step between the projections and attention, in one pass: the norm of each
// query and key head, the rotation by position, and the write of keys and values into their
// pool slots. Included by pa_kernels.cu.
//
// For a head row x of D values at position p (q and k heads; v heads are copied):
//   y = x * rsqrt(mean(x^2) + eps) * w             (where the weight w is given)
//   pair (a, b) = (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) interleaved, i < rot/2:
//   (a, b) -> (a cos - b sin, b cos + a sin), cos and sin from row p of the rotation table;
//   values past rot stay. All in fp32, rounded once to the 16-bit type at the end.
// q rows go to q_out, k and v rows to slot slots[t] of the pools.
//
// HBM-bound: each 16-bit value is read once and written once. D / 8 lanes hold a head, eight
// values (16 bytes) each, so a warp covers 1, 2 or 4 heads at once; it takes NU such sets of one
// token's heads, all loads issued before the first is used, and shares the token's cosines and
// sines (held with the weight folded in: out_j = inv * (x_j * (w_j cos_j) +- x_i * (w_i sin_j)),
// i the partner) over its heads. A warp's sets are either query heads or key/value heads.

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

struct RopeArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t *positions, *slots;
  const float* rope;                     // [max_pos][rot_dim]: cosines, then sines
  const void *q_weight, *k_weight;       // D values, fp32 or the 16-bit type; null: no norm
  uint16_t *q_out, *k_pool, *v_pool;
  int64_t max_pos, n_slots;
  float eps;
  int32_t rows, Hq, Hkv, rot_dim, weight_f32;
  int32_t q_warps, kv_warps;             // warps of a token over its query and key/value heads
};

// Eight weights from element e0 on.
template <bool BF16>
__device__ __forceinline__ void load_weight8(const void* w, bool f32, int e0, float (&x)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + e0);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + e0)), x);
  }
}

template <int D, bool BF16, bool INTER, int NU>
__global__ void __launch_bounds__(256) qk_rope_append_kernel(const RopeArgs a) {
  constexpr int LPH = D / 8;    // lanes of a head
  constexpr int HPW = 32 / LPH; // heads of a set
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH, e0 = 8 * l;
  const int per_token = a.q_warps + a.kv_warps;
  const int64_t wg = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t tok = wg / per_token;
  if (tok >= a.rows) return;
  const int w = (int)(wg - tok * per_token);
  const bool is_q = w < a.q_warps;
  const int n_heads = is_q ? a.Hq : 2 * a.Hkv;
  const int h0 = (is_q ? w : w - a.q_warps) * NU * HPW + sub;

  const int32_t slot = __ldg(a.slots + tok);
  const int32_t pos = __ldg(a.positions + tok);
  uint4 raw[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int h = h0 + u * HPW;
    if (h < n_heads) {
      const uint16_t* src = is_q ? a.q + tok * a.q_stride + (int64_t)h * D
                            : h < a.Hkv ? a.k + tok * a.k_stride + (int64_t)h * D
                                        : a.v + tok * a.v_stride + (int64_t)(h - a.Hkv) * D;
      raw[u] = *reinterpret_cast<const uint4*>(src + e0);
    } else {
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (slot < 0) return;  // a padded row: nothing of it is written
  if (slot >= a.n_slots || pos < 0 || pos >= a.max_pos) {
    if (w == 0 && lane == 0) atomicOr(&g_pa_error_flags, kFlagPage);
    return;
  }

  // Factors of the eight values: own and partner's, the norm's weight included.
  const void* wt = is_q ? a.q_weight : a.k_weight;
  const int half = a.rot_dim >> 1;
  const bool rotated = e0 < a.rot_dim;
  int peer = lane;  // lane that holds the partners (half-split pairs)
  float fc[8], fs[8];
  {
    float wx[8], wp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wx[i] = wp[i] = 1.f;
    const bool upper = !INTER && rotated && e0 >= half;
    const int ep = INTER || !rotated ? e0 : upper ? e0 - half : e0 + half;
    peer = sub * LPH + ep / 8;
    if (wt) {
      load_weight8<BF16>(wt, a.weight_f32, e0, wx);
      if (!INTER) load_weight8<BF16>(wt, a.weight_f32, ep, wp);
    }
    const float* row = a.rope + (int64_t)pos * a.rot_dim;
    if (!rotated) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        fc[i] = wx[i];
        fs[i] = 0.f;
      }
    } else if constexpr (INTER) {  // pair (2i, 2i + 1) of this lane: angle e0 / 2 + i
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + e0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + e0 / 2));
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fc[2 * i] = wx[2 * i] * c[i];
        fc[2 * i + 1] = wx[2 * i + 1] * c[i];
        fs[2 * i] = -wx[2 * i + 1] * s[i];
        fs[2 * i + 1] = wx[2 * i] * s[i];
      }
    } else {
      const int c0 = upper ? e0 - half : e0;
      const float4* cp = reinterpret_cast<const float4*>(row + c0);
      const float4* sp = reinterpret_cast<const float4*>(row + half + c0);
      const float4 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
      const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
      const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        fc[i] = wx[i] * c[i];
        fs[i] = wp[i] * (upper ? s[i] : -s[i]);
      }
    }
  }

#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int h = h0 + u * HPW;
    // Every lane takes part in the shuffles; sets without a head hold zeros.
    float x[8];
    unpack8<BF16>(raw[u], x);
    float inv = 1.f;
    if (wt) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
    }
    float xp[8];
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
    } else {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw[u].x, peer);
      o.y = __shfl_sync(0xffffffffu, raw[u].y, peer);
      o.z = __shfl_sync(0xffffffffu, raw[u].z, peer);
      o.w = __shfl_sync(0xffffffffu, raw[u].w, peer);
      unpack8<BF16>(o, xp);
    }
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int e = 2 * i + j;
        // past rot the partner's factor is 0: kept out of the sum, it may be infinite
        r[j] = inv * (rotated ? fmaf(x[e], fc[e], xp[e] * fs[e]) : x[e] * fc[e]);
      }
      y[i] = pack2<BF16>(r[0], r[1]);
    }
    if (h >= n_heads) continue;
    const uint4 out = make_uint4(y[0], y[1], y[2], y[3]);
    if (is_q)
      *reinterpret_cast<uint4*>(a.q_out + (tok * a.Hq + h) * (int64_t)D + e0) = out;
    else if (h < a.Hkv)
      *reinterpret_cast<uint4*>(a.k_pool + ((int64_t)slot * a.Hkv + h) * D + e0) = out;
    else
      *reinterpret_cast<uint4*>(a.v_pool + ((int64_t)slot * a.Hkv + h - a.Hkv) * D + e0) = raw[u];
  }
}
