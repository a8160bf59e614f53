// Attention of one query token per sequence over the paged 4-bit cache
// (layout: cache4_device.hpp).
//
// Per sequence b, query head h over kv head h / (NHq / NKV), tokens t < lens[b]:
//   s_t = scale * q . k_t,  o = sum_t softmax(s)_t v_t,  lse = log sum_t e^{s_t}
// in one pass with a running maximum m and sum l of each head in float32.
//
// HBM-bound by its bytes: 17 * D / 16 of cache per token and kv head against
// 4 * D operations per query head, so up to 16 query heads share a column
// tile.  The stream leaves a compute unit 13 cycles a token (D = 128, 5.2
// TB/s): per 32 tokens a wave reads four 16-byte pieces per lane and issues
// about 300 instructions, which several waves per SIMD have to overlap.
//
// A wave takes steps of 32 tokens (two tiles of 16).  Both products run on
// 16x16x32 bfloat16 matrix instructions; E2M1 times a power of two is exact
// in bfloat16, so the cache enters them as it stands, by one conversion per
// two values.
//  - S = K Q^T: rows are tokens.  Lane (n, g) (n = lane & 15, g = lane >> 4)
//    holds features 32g .. 32g + 31 of token n (each 128 features; 16g ..
//    16g + 15 of a last 64): one 16-byte load and one scale.  Q^T is held in
//    registers in the same order of features.
//  - O^T = V^T P^T: rows are features.  S leaves lane (n, g) with tokens
//    4g .. 4g + 3 of both tiles for head n, which is taken as the order of
//    the 32 tokens of the second product: P needs no movement between lanes.
//    The matching V operand is 8n .. 8n + 7 of the same tokens: one 16-byte
//    load per tile; a conversion gives two features of one token, a byte
//    permute pairs them by feature.
// Probabilities enter the second product as two bfloat16, the second what the
// first leaves (2^-16 relative): one alone would add as much error as the
// output's own rounding, and the matrix unit has room beside the stream.
//
// The running maximum moves only when a score passes it by more than 8 (in
// powers of two), so most steps skip the exchange between lanes and the
// rescaling; sums stay below 2^8 times the number of tokens.
//
// Tokens behind lens[b], and tokens of a page id that names no page of the
// cache, have no score; the bytes of their scales are replaced, since
// whatever lies there may read as NaN, and no address is formed from a bad
// page id.
//
// Work split: (kv head and column tile) x sequence x splits of the sequence.
// A split takes an equal share of the sequence's own steps, worked out on the
// device, so the host reads no lengths; the four waves of a workgroup
// interleave the steps of its split and join in LDS.  A sequence that one
// split holds is written at once; the partial sums of the others go to
// scratch in float32 and a second launch joins them.  Page ids come 64 at a
// time into a register, so that a step's loads wait for no other load.
//
// Measured (both launches, caches in turn so that they come from HBM): one
// sequence of 131072 tokens, 64 heads over 8 of 128: 34 us = 4.2 TB/s of cache;
// 64 sequences of up to 8192, 32 heads over 4: 47 us = 3.3 TB/s (the second
// bfloat16 of the probabilities is 4 us of it); 4 of up to 300, 16 over 2: 5.4
// us.  Page ids loaded when a step needed them: 60 us for the first.  Equal
// shares of all sequences' steps behind each other in place of equal parts of
// each: 44 us for the second, but 12.3 against 9.7 us for 4 sequences of up to
// 4000 and 17.6 against 11.3 us for 64 of up to 2048 with one kv head, since the
// prefix sum over lens and the change of sequence stand in the way of the loads.
#include "cache4_device.hpp"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kStep = 32;                  // tokens of a wave's step
constexpr int kJoinWaves = 16;
constexpr int kMaxSplits = 128;
constexpr int kOneSplit = 1024;            // tokens
constexpr int kCols = 16;                  // query heads of a column tile
constexpr int kLeast = 2 * kWaves;         // steps of a split, at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;             // the maximum moves beyond this
constexpr float kNegInf = -__builtin_inff();

struct AttendArgs {
  Cache4 c;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  uint32_t page_magic;      // ceil(2^32 / page_tiles); 0 for one tile a page
  const int32_t* lens;
  int B, NHq, G, col_tiles; // G = NHq / NKV
  float scale2;             // scale * log2(e)
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  int splits;
  float* part_o;            // [B][NHq][splits][D]
  float2* part_ml;          // [B][NHq][splits] (maximum in powers of two, sum)
};

// What a part with maximum ml.x and sum ml.y counts in a join whose maximum
// is top.  A part without a score has the sum 0; one whose scores are all NaN
// keeps the maximum -inf and the sum NaN, which has to reach the output.
__device__ __forceinline__ float join_factor(const float2& ml, float top) {
  return ml.x == kNegInf ? ml.y : __builtin_amdgcn_exp2f(ml.x - top);
}
// 1 / sum; 0 (or NaN, as above) where no score is left.
__device__ __forceinline__ float final_factor(float top, float z) {
  return top == kNegInf ? z : 1.0f / z;
}

// Steps of a split: an equal share of n steps, at least kLeast of them, so
// that the splits with work come first; all of them where one split can.
__device__ __forceinline__ int split_steps(int n, int splits) {
  const int each = (n + splits - 1) / splits;
  return each < kLeast ? kLeast : each;
}
__device__ __forceinline__ int sequence_steps(const AttendArgs& a, int b, int* len) {
  const int64_t capacity = (int64_t)a.max_pages * a.c.page_tiles * kTileTokens;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : (n > capacity ? capacity : n);
  *len = (int)n;
  return (int)((n + kStep - 1) / kStep);
}

__device__ __forceinline__ v8bf as_bf8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(v8bf, make_uint4(a, b, c, d));
}

// One step's cache bytes in registers.
template <int D>
struct StepRegs {
  static constexpr int kWide = D / 128;       // 128-feature chunks
  static constexpr bool kTail = D % 128 != 0; // a last 64
  uint4 k[2][kWide ? kWide : 1], v[2][kWide ? kWide : 1];
  uint2 k64[2], v64[2];
  uint32_t ks[2][kWide ? kWide : 1], vs[2][kWide ? kWide : 1];
  uint32_t ks64[2], vs64[2];
  bool there[2];                              // the tile is in the cache

  __device__ __forceinline__ void fetch(const uint8_t* const (&tile)[2], int n, int g) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* t = tile[i];
#pragma unroll
      for (int c = 0; c < kWide; ++c) {
        k[i][c] = *reinterpret_cast<const uint4*>(t + n * (D / 2) + c * 64 + g * 16);
        ks[i][c] = t[cache4_k_scales(D) + n * (D / 32) + c * 4 + g];
        v[i][c] = *reinterpret_cast<const uint4*>(t + cache4_v_codes(D) + c * 1024 + g * 256 + n * 16);
        vs[i][c] = *reinterpret_cast<const uint32_t*>(t + cache4_v_scales(D) +
                                                      (g * (D / 32) + c * 4 + (n >> 2)) * 4);
      }
      if constexpr (kTail) {
        k64[i] = *reinterpret_cast<const uint2*>(t + n * (D / 2) + kWide * 64 + g * 8);
        ks64[i] = t[cache4_k_scales(D) + n * (D / 32) + kWide * 4 + (g >> 1)];
        v64[i] = *reinterpret_cast<const uint2*>(t + cache4_v_codes(D) + kWide * 1024 + g * 128 + n * 8);
        vs64[i] = *reinterpret_cast<const uint32_t*>(t + cache4_v_scales(D) +
                                                     (g * (D / 32) + kWide * 4 + (n >> 3)) * 4);
      }
    }
  }
};

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v8bf fp4_row8(uint32_t codes, float s) {
  const uint4 w = fp4_unpack8(codes, s);
  return __builtin_bit_cast(v8bf, w);
}

// Byte i of a word as a scale of fp4_pair, which looks at the exponent bits
// alone: the bits of the other bytes stay where they fall.
__device__ __forceinline__ float byte_scale(uint32_t w, int i) {
  return __uint_as_float(i == 3 ? w >> 1 : w << (23 - 8 * i));
}

// Tiles 2 * BYTE and 2 * BYTE + 1 of a chunk of V^T P^T: the operand rows are
// the codes of byte BYTE of eight tokens' words.
template <int BYTE>
__device__ __forceinline__ void v_tiles(const uint32_t (&w)[8], const float (&s)[8], v8bf p, v8bf rest,
                                        v4f& even, v4f& odd) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fp4_pair<BYTE>(w[i], s[i]);
  uint32_t e[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
    o[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
  }
  const v8bf ev = as_bf8(e[0], e[1], e[2], e[3]), od = as_bf8(o[0], o[1], o[2], o[3]);
  even = mfma(ev, p, even);
  odd = mfma(od, p, odd);
  even = mfma(ev, rest, even);
  odd = mfma(od, rest, odd);
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void cache4_attend_kernel(AttendArgs a) {
  constexpr int kWide = D / 128;
  constexpr bool kTail = D % 128 != 0;
  constexpr int kSteps = D / 32;             // matrix instructions of a score tile
  constexpr int kTiles = D / 16;             // row tiles of O^T
  constexpr int kDeep = 2;                   // steps in registers
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n = lane & 15, g = lane >> 4;
  const int split = blockIdx.x;
  const int kvh = blockIdx.y / a.col_tiles;
  const int col0 = (blockIdx.y - kvh * a.col_tiles) * kCols;   // first head of the tile in its group
  const int b = blockIdx.z;
  int len;
  const int nsteps = sequence_steps(a, b, &len);
  const int each = split_steps(nsteps, a.splits);
  const int first = split * each;
  const int last = min(nsteps, first + each);
  if (first >= last && split > 0) return;
  const bool alone = nsteps <= each;           // the whole sequence is here: no join

  const int head = col0 + n;                   // in the group
  const bool mine = head < a.G;
  const int qh = kvh * a.G + head;

  // Q^T in the order of K's features
  v8bf qr[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) qr[s] = as_bf8(0, 0, 0, 0);
  if (mine) {
    const uint16_t* q = a.q + b * a.q_stride + (int64_t)qh * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = s < 4 * kWide ? (s / 4) * 128 + g * 32 + (s % 4) * 8
                                  : kWide * 128 + g * 16 + (s - 4 * kWide) * 8;
      qr[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(q + d));
    }
  }

  // Page ids, 64 columns of the table in a register from column page0 on: the
  // loads of a step wait for no other load.
  const int32_t* table = a.table + b * a.table_stride;
  const int tiles = (len + kTileTokens - 1) / kTileTokens;
  auto column_of = [&](int tl) {
    return (int)(a.page_magic ? __umulhi((uint32_t)tl, a.page_magic) : (uint32_t)tl);
  };
  int page0 = 0, pages = -1;
  auto take_pages = [&](int col) {
    page0 = col;
    pages = col + lane < a.max_pages ? table[col + lane] : -1;
  };
  auto load = [&](int step, StepRegs<D>& r) {
    if (step >= last) return;
    if (column_of(min(2 * step + 1, tiles - 1)) >= page0 + kWave) take_pages(column_of(2 * step));
    const uint8_t* tile[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tl = 2 * step + i;
      const int col = column_of(tl);
      const int page = tl < tiles ? __builtin_amdgcn_readlane(pages, col - page0) : -1;
      r.there[i] = (uint32_t)page < (uint32_t)a.c.num_pages;
      // a page that is not there is read as the cache's first tile
      const uint32_t at = ((uint32_t)page * a.c.NKV + kvh) * a.c.page_tiles + (tl - col * a.c.page_tiles);
      tile[i] = a.c.pages + (uint64_t)(r.there[i] ? at : 0u) * (uint32_t)cache4_tile_bytes(D);
    }
    r.fetch(tile, n, g);
  };

  float m = kNegInf, l = 0.0f;                 // l: this lane's tokens only
  v4f o[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) o[i] = v4f{0, 0, 0, 0};

  auto compute = [&](const StepRegs<D>& r, int step) {
    // scores
    v4f sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v4f acc = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kWide; ++c) {
        const float ks = cache4_scale(r.ks[i][c]);
        acc = mfma(fp4_row8(r.k[i][c].x, ks), qr[4 * c], acc);
        acc = mfma(fp4_row8(r.k[i][c].y, ks), qr[4 * c + 1], acc);
        acc = mfma(fp4_row8(r.k[i][c].z, ks), qr[4 * c + 2], acc);
        acc = mfma(fp4_row8(r.k[i][c].w, ks), qr[4 * c + 3], acc);
      }
      if constexpr (kTail) {
        const float ks = cache4_scale(r.ks64[i]);
        acc = mfma(fp4_row8(r.k64[i].x, ks), qr[4 * kWide], acc);
        acc = mfma(fp4_row8(r.k64[i].y, ks), qr[4 * kWide + 1], acc);
      }
      sc[i] = acc;
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3];
    const bool whole = r.there[0] && r.there[1] && (step + 1) * kStep <= len;   // uniform
    const int left = len - step * kStep - 4 * g;       // of this lane's tokens, from the first on
    auto dead = [&](int i) { return !r.there[i >> 2] || (i >> 2) * kTileTokens + (i & 3) >= left; };
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = dead(i) ? kNegInf : x[i];
    }
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                      fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * a.scale2;
    if (__any(top > m + kSlack)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float next = fmaxf(m, top);
      const float f = next == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[i] *= f;
    }
    const float base = m == kNegInf ? 0.0f : -m;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(x[i], a.scale2, base));
    l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
      lo[i] = pack_bf16(p[2 * i] - bf16_lo(hi[i]), p[2 * i + 1] - bf16_hi(hi[i]));
    }
    const v8bf pb = as_bf8(hi[0], hi[1], hi[2], hi[3]), pl = as_bf8(lo[0], lo[1], lo[2], lo[3]);
    // values
    auto scales = [&](uint32_t a0, uint32_t a1, float (&s)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = byte_scale(i < 4 ? a0 : a1, i & 3);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = dead(i) ? 1.0f : s[i];
      }
    };
#pragma unroll
    for (int c = 0; c < kWide; ++c) {
      const uint4 &v0 = r.v[0][c], &v1 = r.v[1][c];
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      float s[8];
      scales(r.vs[0][c], r.vs[1][c], s);
      v_tiles<0>(w, s, pb, pl, o[8 * c], o[8 * c + 1]);
      v_tiles<1>(w, s, pb, pl, o[8 * c + 2], o[8 * c + 3]);
      v_tiles<2>(w, s, pb, pl, o[8 * c + 4], o[8 * c + 5]);
      v_tiles<3>(w, s, pb, pl, o[8 * c + 6], o[8 * c + 7]);
    }
    if constexpr (kTail) {
      const uint2 &v0 = r.v64[0], &v1 = r.v64[1];
      const uint32_t w[8] = {v0.x & 0xFFFFu, v0.x >> 16, v0.y & 0xFFFFu, v0.y >> 16,
                             v1.x & 0xFFFFu, v1.x >> 16, v1.y & 0xFFFFu, v1.y >> 16};
      float s[8];
      scales(r.vs64[0], r.vs64[1], s);
      v_tiles<0>(w, s, pb, pl, o[8 * kWide], o[8 * kWide + 1]);
      v_tiles<1>(w, s, pb, pl, o[8 * kWide + 2], o[8 * kWide + 3]);
    }
  };

  // kDeep steps in registers: the loads of the next ones are under way while
  // one is worked on
  StepRegs<D> r[kDeep];
  int step = first + wave;
  if (step < last) {
    take_pages(column_of(2 * step));
#pragma unroll
    for (int i = 0; i < kDeep; ++i) load(step + i * kWaves, r[i]);
#pragma clang loop unroll(disable)
    while (true) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        if (step + i * kWaves < last) {
          compute(r[i], step + i * kWaves);
          load(step + (i + kDeep) * kWaves, r[i]);
        }
      }
      step += kDeep * kWaves;
      if (step >= last) break;
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // join the waves: each leaves its columns' maximum, sum and O^T in LDS
  __shared__ float2 ml[kWaves][kCols];
  extern __shared__ float lo[];                // [kWaves][cols][D + 4]
  const int cols = min(kCols, a.G);            // rows kept (the last tile's may be fewer)
  constexpr int kRow = D + 4;                  // floats; off the banks' period
  if (g == 0) ml[wave][n] = make_float2(m, l);
  if (mine) {
    float* dst = lo + (wave * cols + n) * kRow;
    // row 4g + r of tile j of a chunk is feature w * (4g + r) + j
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int i = 0; i < kTiles; i += 4) {
        const int c = i / 8;
        const int d = c < kWide ? c * 128 + 8 * (4 * g + r) + i % 8
                                : kWide * 128 + 4 * (4 * g + r);
        *reinterpret_cast<float4*>(dst + d) = make_float4(o[i][r], o[i + 1][r], o[i + 2][r], o[i + 3][r]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < min(cols, a.G - col0) * (D / 4); i += kThreads) {
    const int col = i / (D / 4), d = (i - col * (D / 4)) * 4;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[w][col].x);
    float4 sum = make_float4(0, 0, 0, 0);
    float z = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float2 s = ml[w][col];
      const float f = join_factor(s, top);
      const float4 v = *reinterpret_cast<const float4*>(lo + (w * cols + col) * kRow + d);
      z += f * s.y;
      sum.x += f * v.x; sum.y += f * v.y; sum.z += f * v.z; sum.w += f * v.w;
    }
    const int h = kvh * a.G + col0 + col;
    if (!alone) {
      const int64_t at = ((int64_t)b * a.NHq + h) * a.splits + split;
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = sum;
      if (d == 0) a.part_ml[at] = make_float2(top, z);
    } else {
      const float f = final_factor(top, z);
      uint2 w;
      w.x = pack_bf16(sum.x * f, sum.y * f);
      w.y = pack_bf16(sum.z * f, sum.w * f);
      *reinterpret_cast<uint2*>(a.out + b * a.out_stride + (int64_t)h * D + d) = w;
      if (d == 0 && a.lse)
        a.lse[(int64_t)b * a.NHq + h] = (top + __log2f(z)) * kLn2;
    }
  }
}

// Joins the splits of one head: a workgroup per (sequence, head), a lane for
// every D / 64 features, the waves (4, or 16 where there are many splits)
// taking turns at the splits.  Sequences that one split held are there already.
template <int D>
__global__ __launch_bounds__(kJoinWaves * kWave) void cache4_join_kernel(AttendArgs a) {
  constexpr int kPer = D / kWave;              // features of a lane
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int waves = blockDim.x / kWave;
  const int64_t row = blockIdx.x;              // b * NHq + h
  const int b = (int)(row / a.NHq), h = (int)(row - (int64_t)b * a.NHq);
  int len;
  const int nsteps = sequence_steps(a, b, &len);
  const int each = split_steps(nsteps, a.splits);
  if (nsteps <= each) return;
  const int parts = (nsteps + each - 1) / each;   // at most kMaxSplits
  const float2* ml = a.part_ml + row * a.splits;
  // factors of the parts: lane s of register i has that of part 64 i + s
  float2 v[kMaxSplits / kWave];
  float f[kMaxSplits / kWave], top = kNegInf, z = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kWave; ++i) {
    v[i] = i * kWave + lane < parts ? ml[i * kWave + lane] : make_float2(kNegInf, 0.0f);
    top = fmaxf(top, v[i].x);
  }
  top = wave_max(top);
#pragma unroll
  for (int i = 0; i < kMaxSplits / kWave; ++i) {
    f[i] = join_factor(v[i], top);
    z += f[i] * v[i].y;
  }
  z = wave_sum(z);
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
  const float* po = a.part_o + row * a.splits * D + lane * kPer;
  for (int s0 = wave; s0 < parts; s0 += 4 * waves) {   // four loads under way
    float x[4][kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = po[(int64_t)min(s0 + i * waves, parts - 1) * D + k];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i * waves;
      const float fs = __shfl(s < kWave ? f[0] : f[1], s & (kWave - 1));
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] += s < parts ? fs * x[i][k] : 0.0f;
    }
  }
  __shared__ float sum[kJoinWaves][D];
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum[wave][lane * kPer + k] = acc[k];
  __syncthreads();
  const float scale = final_factor(top, z);
  const int d = threadIdx.x;
  if (d < D) {
    float o = 0.0f;
    for (int w = 0; w < waves; ++w) o += sum[w][d];
    (a.out + b * a.out_stride + (int64_t)h * D)[d] = (uint16_t)pack_bf16(o * scale, 0.0f);
  }
  if (d == 0 && a.lse) a.lse[row] = (top + __log2f(z)) * kLn2;
}

int attend_lds(int D, int cols) { return kWaves * cols * (D + 4) * (int)sizeof(float); }

template <int D>
hipError_t prepare_one() {
  hipError_t e = prepare_kernel(reinterpret_cast<const void*>(&cache4_attend_kernel<D>), attend_lds(D, kCols));
  if (e == hipSuccess) e = prepare_kernel(reinterpret_cast<const void*>(&cache4_join_kernel<D>), 0);
  return e;
}

template <int D>
void launch_one(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.splits, (unsigned)(a.c.NKV * a.col_tiles), (unsigned)a.B);
  cache4_attend_kernel<D><<<grid, dim3(kThreads), attend_lds(D, a.G < kCols ? a.G : kCols),
                            stream>>>(a);
  if (a.splits > 1) {
    cache4_join_kernel<D><<<dim3((unsigned)(a.B * a.NHq)),
                            dim3(a.splits > 16 ? kJoinWaves * kWave : kThreads), 0, stream>>>(a);
  }
}

}  // namespace

hipError_t prepare_cache4_attend_kernels() {
  hipError_t e = prepare_one<64>();
  if (e == hipSuccess) e = prepare_one<128>();
  if (e == hipSuccess) e = prepare_one<192>();
  if (e == hipSuccess) e = prepare_one<256>();
  return e;
}

// Splits that a sequence may have.  Few sequences: as many as make one round
// of resident workgroups (256 compute units, 4, 3 or 2 workgroups each by the
// registers of the head size; one sequence of 131072 tokens, 8 kv heads of
// 128: 64 splits 36.1 us, 96 splits 35.2 us, 128 splits, a round and a third,
// 38.0 us).  Sixteen and more: their lengths differ, and shorter splits even
// them out (64 sequences of up to 8192, 4 kv heads: 3 splits 51.6 us, 4 splits
// 48.6 us, 6 splits 47.6 us, 8 splits 49.0 us).  At most as many as have kLeast
// steps each when the sequences are as long as the table allows; one, and one
// launch, for tables of up to kOneSplit tokens (4 sequences of up to 300 tokens:
// 5.5 us against 7.9 us with a second launch).
int cache4_attend_splits(int64_t B, int NHq, int NKV, int D, int64_t capacity) {
  const int64_t units = B * NKV * ((NHq / NKV + kCols - 1) / kCols);
  const int64_t round = 256 * (D == 64 ? 4 : (D == 128 ? 3 : 2));
  int64_t s = B < 16 ? round / units : (2 * round + units - 1) / units;
  const int64_t most = capacity / (kLeast * kStep);
  if (s > most) s = most;
  if (capacity <= kOneSplit) s = 1;
  return (int)(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}

size_t cache4_attend_workspace(int64_t B, int NHq, int D, int splits) {
  return splits > 1 ? (size_t)B * NHq * splits * (D * sizeof(float) + sizeof(float2)) : 0;
}

hipError_t launch_cache4_attend(const Cache4& c, const void* q, int64_t q_stride,
                                const int32_t* table, int64_t table_stride, int max_pages,
                                const int32_t* lens, int B, int NHq, float scale, void* out,
                                int64_t out_stride, float* lse, int splits, void* workspace,
                                hipStream_t stream) {
  AttendArgs a{};
  a.c = c;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.table = table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.page_magic = c.page_tiles == 1 ? 0u
                                   : (uint32_t)((((uint64_t)1 << 32) + c.page_tiles - 1) / c.page_tiles);
  a.lens = lens;
  a.B = B;
  a.NHq = NHq;
  a.G = NHq / c.NKV;
  a.col_tiles = (a.G + kCols - 1) / kCols;
  a.scale2 = scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.splits = splits;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)B * NHq * splits * c.D);
  switch (c.D) {
    case 64: launch_one<64>(a, stream); break;
    case 128: launch_one<128>(a, stream); break;
    case 192: launch_one<192>(a, stream); break;
    default: launch_one<256>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace moe
