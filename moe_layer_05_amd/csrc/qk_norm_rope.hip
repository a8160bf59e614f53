// RMS norm of every query and key head and its rotary embedding, in one pass.
//
// Per token t and head h (D features, the first R rotated), with the norm's
// weight w (none: r = 1 and w = 1, the rotation alone):
//   r = 1 / sqrt(mean(x^2) + eps),   z = x * r * w,
//   pairs (i, i + R/2) ("half" layout) or (2i, 2i + 1) ("interleaved"),
//   c = table[p][i], s = table[p][R/2 + i], p = positions[t]:
//     y1 = z1 * c - z2 * s,  y2 = z2 * c + z1 * s      (rotation by +theta)
// and features from R on pass through as z.  All in float32, rounded once to
// bfloat16: rounding z first, as two separate passes would, doubles the error.
//
// Layout of the work: one wave takes a unit of up to `iters` steps of one
// token's query heads or key heads; a head takes G lanes, G the power of two
// >= D / 8, so a step covers 64 / G heads.  Lane j of a head holds features
// 8j .. 8j + 7 (one 16-byte load and store).  The token's cosines and sines
// and the norm's weights do not depend on the head: a wave reads them once
// per unit into registers, where a row-per-lane-group form reads as many
// table bytes per head as head bytes.  Half layout: the partner of feature
// f < R/2 is R/16 lanes further on, fetched by one shuffle of four words.
// Every head is read whole before it is written, so a head may be written
// onto itself.
//
// HBM-bound (latency-bound below some hundred tokens): every head read and
// written once, the table's rows of the call's positions read once.  Measured:
// 4096 tokens, 72 heads of 128: 31 us = 4.9 TB/s; 1023 tokens, 32 heads of 192,
// 64 features rotated, no norm: 5.9 us = 4.3 TB/s; 16 tokens, 18 heads: 3.2 us.
// Outputs go past the L2 (through it 34 and 6.6 us); inputs do not (7.1 us for
// the second).
#include "device_common.hpp"
#include "internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / kWave;
constexpr int kMostSteps = 6;              // of a wave

// Heads that a wave takes in one step: 64 lanes, D / 8 of them (rounded up to
// a power of two) a head.
int heads_of_step(int D) {
  int lanes = 1;
  while (lanes < D / 8) lanes *= 2;
  return kWave / lanes;
}

struct HeadsArgs {
  const uint4* x;      // bf16, 8 per uint4
  uint4* y;
  int64_t x_stride8;   // token strides in uint4 units
  int64_t y_stride8;
  const void* w;       // [D] or null
  int heads;
  int units;           // units of a token
};

struct NormRopeArgs {
  HeadsArgs side[2];   // queries, keys
  const int64_t* positions;
  const float* table;
  int64_t max_pos;
  int64_t units;       // T * (units of a token over both sides)
  int D, R, gshift, iters;
  int w_f32;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
  v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
}

// Eight weights from feature f0 on, as float32.
__device__ __forceinline__ void load_weights(const void* w, bool f32, int f0, float (&out)[8]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = static_cast<const float*>(w)[f0 + i];
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + f0), out);
  }
}

template <bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(NormRopeArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t unit = (int64_t)blockIdx.x * kWavesPerBlock +
                       __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (unit >= a.units) return;
  const int G = 1 << a.gshift;
  const int j = lane & (G - 1);
  const int d8 = a.D >> 3;
  const bool holds = j < d8;
  const int f0 = 8 * j;
  const int half = a.R >> 1;
  const int per_token = a.side[0].units + a.side[1].units;
  const int64_t t = unit / per_token;
  const int u = (int)(unit - t * per_token);
  const bool key = u >= a.side[0].units;
  const HeadsArgs& s = a.side[key ? 1 : 0];
  const int step = kWave >> a.gshift;                  // heads of a step
  const int h0 = (key ? u - a.side[0].units : u) * step * a.iters + (lane >> a.gshift);
  const uint4* x = s.x + t * s.x_stride8;
  uint4* y = s.y + t * s.y_stride8;
  uint4 q = make_uint4(0, 0, 0, 0);
  if (holds && h0 < s.heads) q = x[(int64_t)h0 * d8 + j];   // the first head, while the table loads

  // lanes between partners; srcl is this lane's partner (half layout)
  const int off = a.R >> 4;
  const bool rot = holds && f0 < a.R;
  const bool first = f0 < half;
  const int srcl = (!INTERLEAVED && rot) ? (first ? lane + off : lane - off) : lane;
  float w[8], wp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = wp[i] = 1.0f;
  if (s.w && holds) {
    load_weights(s.w, a.w_f32, f0, w);
    if (!INTERLEAVED && rot) load_weights(s.w, a.w_f32, first ? f0 + half : f0 - half, wp);
  }
  // Half layout: y = z * c[i] + partner * sn[i], the sign of the sine folded
  // in; interleaved: four angles.
  float c[8], sn[8];
  if (rot) {
    int64_t p = a.positions[t];
    p = p < 0 ? 0 : (p >= a.max_pos ? a.max_pos - 1 : p);
    const float* cs = a.table + p * a.R;
    const int i0 = INTERLEAVED ? f0 >> 1 : (first ? f0 : f0 - half);
#pragma unroll
    for (int b = 0; b < (INTERLEAVED ? 4 : 8); b += 4) {
      const float4 cv = *reinterpret_cast<const float4*>(cs + i0 + b);
      const float4 sv = *reinterpret_cast<const float4*>(cs + half + i0 + b);
      c[b] = cv.x; c[b + 1] = cv.y; c[b + 2] = cv.z; c[b + 3] = cv.w;
      sn[b] = sv.x; sn[b + 1] = sv.y; sn[b + 2] = sv.z; sn[b + 3] = sv.w;
    }
    if (!INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = (first ? -sn[i] : sn[i]) * wp[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] *= w[i];
    }
  }
  const float inv_d = 1.0f / (float)a.D;
  for (int it = 0; it < a.iters; ++it) {
    const int h = h0 + it * step;
    if (it * step + (h0 - (lane >> a.gshift)) >= s.heads) break;   // wave-uniform
    const uint4 cur = q;
    if (it + 1 < a.iters) {
      q = make_uint4(0, 0, 0, 0);
      if (holds && h + step < s.heads) q = x[(int64_t)(h + step) * d8 + j];
    }
    float v[8];
    unpack8(cur, v);
    float r = 1.0f;
    if (s.w) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
      for (int o = 1; o < G; o <<= 1) ss += __shfl_xor(ss, o);
      r = __builtin_amdgcn_rsqf(fmaf(ss, inv_d, a.eps));
    }
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
      if (rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a1 = v[2 * i], a2 = v[2 * i + 1];
          v[2 * i] = a1 * c[i] - a2 * sn[i];
          v[2 * i + 1] = a2 * c[i] + a1 * sn[i];
        }
      }
    } else {
      uint4 pq;
      pq.x = (uint32_t)__shfl((int)cur.x, srcl);
      pq.y = (uint32_t)__shfl((int)cur.y, srcl);
      pq.z = (uint32_t)__shfl((int)cur.z, srcl);
      pq.w = (uint32_t)__shfl((int)cur.w, srcl);
      if (rot) {
        float o[8];
        unpack8(pq, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r * (v[i] * c[i] + o[i] * sn[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
      }
    }
    if (holds && h < s.heads) {
      uint4 o;
      o.x = pack_bf16(v[0], v[1]);
      o.y = pack_bf16(v[2], v[3]);
      o.z = pack_bf16(v[4], v[5]);
      o.w = pack_bf16(v[6], v[7]);
      store_stream(y + ((int64_t)h * d8 + j), o);
    }
  }
}

}  // namespace

hipError_t prepare_qk_norm_rope_kernels() {
  hipError_t e = prepare_kernel(reinterpret_cast<const void*>(&qk_norm_rope_kernel<false>), 0);
  if (e == hipSuccess)
    e = prepare_kernel(reinterpret_cast<const void*>(&qk_norm_rope_kernel<true>), 0);
  return e;
}

int64_t qk_norm_rope_waves(int64_t T, int NHq, int NHk, int D) {
  const int64_t heads = (int64_t)kMostSteps * heads_of_step(D);
  return T * ((NHq + heads - 1) / heads + (NHk + heads - 1) / heads);
}

hipError_t launch_qk_norm_rope(const HeadRows& q, const HeadRows& k, const int64_t* positions,
                               const float* table, int64_t max_pos, int64_t T, int D, int R,
                               bool interleaved, bool weights_f32, float eps, int num_cus,
                               hipStream_t stream) {
  NormRopeArgs a{};
  const int step = heads_of_step(D), g = 6 - __builtin_ctz(step);
  // Steps per wave: as many as leave every SIMD four waves, at most kMostSteps.
  const int64_t steps = T * ((q.heads + step - 1) / step + (k.heads + step - 1) / step);
  int64_t iters = steps / ((int64_t)num_cus * 16);
  iters = iters < 1 ? 1 : (iters > kMostSteps ? kMostSteps : iters);
  const HeadRows* src[2] = {&q, &k};
  for (int i = 0; i < 2; ++i) {
    HeadsArgs& s = a.side[i];
    s.x = static_cast<const uint4*>(src[i]->x);
    s.y = static_cast<uint4*>(src[i]->y);
    s.x_stride8 = src[i]->x_stride / 8;
    s.y_stride8 = src[i]->y_stride / 8;
    s.w = src[i]->weight;
    s.heads = src[i]->heads;
    s.units = (int)((src[i]->heads + step * iters - 1) / (step * iters));
  }
  a.positions = positions;
  a.table = table;
  a.max_pos = max_pos;
  a.units = T * (a.side[0].units + a.side[1].units);
  a.D = D;
  a.R = R;
  a.gshift = g;
  a.iters = (int)iters;
  a.w_f32 = weights_f32;
  a.eps = eps;
  const int64_t blocks = (a.units + kWavesPerBlock - 1) / kWavesPerBlock;
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (interleaved) qk_norm_rope_kernel<true><<<grid, block, 0, stream>>>(a);
  else qk_norm_rope_kernel<false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
