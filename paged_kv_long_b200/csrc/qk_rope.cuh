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
// HBM-bound: each 16-bit value is read once and written once. D / 8 lanes hold a head, a lane
// both members of four pairs: eight values side by side (interleaved pairs), or four and their
// four partners (half-split; past rot the remaining values pair up the same way, unturned), so
// the rotation needs no shuffle. A warp covers a set of 1, 2 or 4 heads at once and walks its
// share of one token's query sets, or of its key and value sets, with the loads of the next
// kRopeAhead sets out before it works on the current ones. The token's cosines and sines (times
// the weights) stay in registers. A block is one warp: query warps walk up to Hq sets and
// key/value warps few, and in blocks of eight warps the short ones left a quarter of the SM's
// warps idle (32,768 rows of 16 + 2 x 2 heads of 256: 133 us, 120 us as it is, 5.9 TB/s).

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
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
  int32_t q_warps, kv_warps;             // warps of a token over its query and key/value sets
};

// Four weights from element e on.
template <bool BF16>
__device__ __forceinline__ void load_weight4(const void* w, bool f32, int e, float (&x)[4]) {
  if (f32) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + e));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + e));
    const float2 a = unpack2<BF16>(v.x), b = unpack2<BF16>(v.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

constexpr int kRopeAhead = 2;

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(32, 32) qk_rope_append_kernel(const RopeArgs a) {
  constexpr int LPH = D / 8;    // lanes of a head
  constexpr int HPW = 32 / LPH; // heads of a set
  constexpr int NU = kRopeAhead;
  const int lane = threadIdx.x;
  const int sub = lane / LPH, l = lane % LPH;
  const uint32_t per_token = a.q_warps + a.kv_warps;
  const uint32_t tok = blockIdx.x / per_token;
  const uint32_t w = blockIdx.x - tok * per_token;
  const bool is_q = w < (uint32_t)a.q_warps;
  const int32_t slot = __ldg(a.slots + tok);
  const int32_t pos = __ldg(a.positions + tok);

  // The lane's values: e .. e + 3 and f .. f + 3 of a head. Interleaved: f = e + 4, the pairs
  // side by side. Half-split: the pairs (e + i, f + i); rot is a multiple of 16, so four pairs
  // are all turned or all past rot.
  const int half = a.rot_dim >> 1;
  int e = 8 * l, f = 8 * l + 4;
  bool turned = e < a.rot_dim;
  if constexpr (!INTER) {
    turned = 4 * l < half;
    e = turned ? 4 * l : half + 4 * l;             // past rot: rot + (4 l - half)
    f = turned ? half + 4 * l : D / 2 + 4 * l;     // that plus (D - rot) / 2
  }
  // this warp's share of its token's query sets, or key and value sets (32 bits: the host keeps
  // parts <= sets < 2^16)
  const int n_heads = is_q ? a.Hq : 2 * a.Hkv;
  const uint32_t sets = (n_heads + HPW - 1) / HPW;
  const uint32_t part = is_q ? w : w - a.q_warps, parts = is_q ? a.q_warps : a.kv_warps;
  const int s0 = (int)(part * sets / parts), s1 = (int)((part + 1) * sets / parts);
  const uint16_t* src0 = is_q ? a.q + tok * a.q_stride : a.k + tok * a.k_stride;
  const uint16_t* srcv = a.v + tok * a.v_stride - (int64_t)a.Hkv * D;
  uint16_t* dst0 = is_q ? a.q_out + (int64_t)tok * a.Hq * D : a.k_pool + (int64_t)slot * a.Hkv * D;
  uint16_t* dstv = a.v_pool + ((int64_t)slot - 1) * a.Hkv * D;
  uint2 raw[NU][2], next[NU][2];
  auto load = [&](int set, uint2 (&r)[NU][2]) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int h = (set + u) * HPW + sub;
      r[u][0] = r[u][1] = make_uint2(0u, 0u);
      if (set + u < s1 && h < n_heads) {
        const uint16_t* src = (is_q || h < a.Hkv ? src0 : srcv) + h * D;
        if constexpr (INTER) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + e);
          r[u][0] = make_uint2(x.x, x.y);
          r[u][1] = make_uint2(x.z, x.w);
        } else {
          r[u][0] = *reinterpret_cast<const uint2*>(src + e);
          r[u][1] = *reinterpret_cast<const uint2*>(src + f);
        }
      }
    }
  };
  load(s0, raw);  // does not wait for the slot
  if (slot < 0) return;  // a padded row: nothing of it is written
  if (slot >= a.n_slots || pos < 0 || pos >= a.max_pos) {
    if (lane == 0) atomicOr(&g_pa_error_flags, kFlagPage);
    return;
  }
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turned) {
    const float* row = a.rope + (int64_t)pos * a.rot_dim + 4 * l;
    c = __ldg(reinterpret_cast<const float4*>(row));
    s = __ldg(reinterpret_cast<const float4*>(row + half));
  }

  // Pair i of the lane is (x_i, z_i): out x' = inv (x xc + z xs), z' = inv (z zc + x zs).
  float2 xc[2], xs[2], zc[2], zs[2];
  const void* wt = is_q ? a.q_weight : a.k_weight;
  {
    float we[4] = {1.f, 1.f, 1.f, 1.f}, wf[4] = {1.f, 1.f, 1.f, 1.f};
    if (wt) {
      load_weight4<BF16>(wt, a.weight_f32, e, we);
      load_weight4<BF16>(wt, a.weight_f32, f, wf);
    }
    float wx[4], wz[4];  // weights of the pairs' members
    if constexpr (INTER) {
      wx[0] = we[0]; wz[0] = we[1]; wx[1] = we[2]; wz[1] = we[3];
      wx[2] = wf[0]; wz[2] = wf[1]; wx[3] = wf[2]; wz[3] = wf[3];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wx[i] = we[i];
        wz[i] = wf[i];
      }
    }
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = 2 * i, q = 2 * i + 1;
      xc[i] = make_float2(wx[p] * cc[p], wx[q] * cc[q]);
      xs[i] = make_float2(-wz[p] * ss[p], -wz[q] * ss[q]);
      zc[i] = make_float2(wz[p] * cc[p], wz[q] * cc[q]);
      zs[i] = make_float2(wx[p] * ss[p], wx[q] * ss[q]);
    }
  }

  for (int set = s0; set < s1; set += NU) {
    if (set + NU < s1) load(set + NU, next);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int h = (set + u) * HPW + sub;
      // Every lane takes part in the shuffles; lanes without a head hold zeros.
      const float2 r0 = unpack2<BF16>(raw[u][0].x), r1 = unpack2<BF16>(raw[u][0].y);
      const float2 r2 = unpack2<BF16>(raw[u][1].x), r3 = unpack2<BF16>(raw[u][1].y);
      float2 x[2], z[2];
      if constexpr (INTER) {
        x[0] = make_float2(r0.x, r1.x);
        z[0] = make_float2(r0.y, r1.y);
        x[1] = make_float2(r2.x, r3.x);
        z[1] = make_float2(r2.y, r3.y);
      } else {
        x[0] = r0;
        x[1] = r1;
        z[0] = r2;
        z[1] = r3;
      }
      float2 inv = make_float2(1.f, 1.f);
      if (wt) {
        float2 s2 = fmul2(x[0], x[0]);
        s2 = ffma2(x[1], x[1], s2);
        s2 = ffma2(z[0], z[0], s2);
        s2 = ffma2(z[1], z[1], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv.x = inv.y = rsqrtf(ss * (1.f / D) + a.eps);
      }
      if (set + u >= s1 || h >= n_heads) continue;
      float2 ox[2], oz[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ox[i] = fmul2(x[i], xc[i]);
        oz[i] = fmul2(z[i], zc[i]);
        if (turned) {  // past rot the partner stays out of the sum: it may be infinite
          ox[i] = ffma2(z[i], xs[i], ox[i]);
          oz[i] = ffma2(x[i], zs[i], oz[i]);
        }
        ox[i] = fmul2(ox[i], inv);
        oz[i] = fmul2(oz[i], inv);
      }
      uint2 y0, y1;
      if constexpr (INTER) {
        y0 = make_uint2(pack2<BF16>(ox[0].x, oz[0].x), pack2<BF16>(ox[0].y, oz[0].y));
        y1 = make_uint2(pack2<BF16>(ox[1].x, oz[1].x), pack2<BF16>(ox[1].y, oz[1].y));
      } else {
        y0 = make_uint2(pack2<BF16>(ox[0].x, ox[0].y), pack2<BF16>(ox[1].x, ox[1].y));
        y1 = make_uint2(pack2<BF16>(oz[0].x, oz[0].y), pack2<BF16>(oz[1].x, oz[1].y));
      }
      uint16_t* dst = dst0 + h * D;
      if (!is_q && h >= a.Hkv) {  // a value head: its bits
        dst = dstv + h * D;
        y0 = raw[u][0];
        y1 = raw[u][1];
      }
      if constexpr (INTER) {
        *reinterpret_cast<uint4*>(dst + e) = make_uint4(y0.x, y0.y, y1.x, y1.y);
      } else {
        *reinterpret_cast<uint2*>(dst + e) = y0;
        *reinterpret_cast<uint2*>(dst + f) = y1;
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      raw[u][0] = next[u][0];
      raw[u][1] = next[u][1];
    }
  }
}
