// Attention of packed prompts: bfloat16 queries, keys and values, grouped
// heads, sequences of different lengths behind each other, causal (the last
// query sees the last key) or full.
//
// Per sequence of nq queries and nk keys, query row i of head h sees the keys
// j < lim(i) of kv head h / (NHq / NKV), lim(i) = nk, or, causal,
// clamp(i + 1 + nk - nq, 0, nk):
//   s_j = scale * q_i . k_j,  o_i = sum_j softmax(s)_j v_j,  lse_i = log sum_j e^{s_j}
// in one pass over the keys with a running maximum and sum of each row in
// float32; a row that sees nothing gives o = 0, lse = -inf.
//
// MFMA-bound: 4 * D operations per visible pair on 32x32x16 bfloat16 matrix
// instructions, both products transposed so that a lane owns one query row
// (column lane & 31 of every result):
//  - S^T = K Q^T: rows are keys; lane half g = lane >> 5 gets keys
//    8 (r / 4) + 4 g + r % 4 of 32 in register r.
//  - O^T = V^T P^T: registers 8u .. 8u + 7 of S^T are taken as the 16 keys of
//    its k-step u, so the probabilities stay in the lane that made them: row
//    maximum, sum and rescaling need one exchange between the two halves and
//    no LDS.  The V operand of the same keys, four keys of one feature per
//    lane, comes from row-major V by the transposing LDS read.
// Probabilities are rounded to bfloat16 for the second product (relative
// 2^-9 each, random over the keys: the output's error stays at the size of its
// own rounding); their sum is taken in float32 before that.  The running
// maximum moves only when a score passes it by more than 8 (in powers of
// two), so most tiles skip the rescaling of O^T.
//
// Work split: a workgroup of four waves takes 128 query rows of one head, 32
// rows a wave; K and V tiles are shared through LDS, two deep: the next tile's
// loads are in flight in registers while the current one is worked on.  LDS
// rows keep their 16-byte pieces XOR-ed with the row so that both the row
// reads of K and the transposing reads of V are free of bank conflicts.
// Each XCD takes a contiguous range of (head, tile) so that a kv head's keys
// stay in one L2; inside a sequence the tiles with the most keys go first.
//
// A key or value that a row does not see never reaches it: scores of masked
// pairs are replaced, and as 0 * NaN is NaN, a workgroup that ends with a
// value that is not finite starts over with the masked tiles' values taken
// apart (kCareful below); finite inputs never do.
#include "device_common.hpp"
#include "internal.hpp"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kRows = 32;                       // query rows of a wave
constexpr int kBlockRows = kWaves * kRows;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
constexpr float kNegInf = -__builtin_inff();

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Keys of a tile: 64, or 32 where two tiles of 64 would not leave room for a
// second workgroup on the compute unit (D = 192, 256).
template <int D>
constexpr int tile_keys() { return D <= 128 ? 64 : 32; }
template <int D>
constexpr int lds_bytes() { return 2 * 2 * tile_keys<D>() * D * 2; }

// Position of 16-byte piece p of a row.  The 64 banks hold 256 bytes: rows of
// 256 or 512 bytes all start at the same bank, and 16 rows that read the same
// piece need 16 different positions, while 4 rows that read 4 pieces each
// (the transposing read) need them in 4 different quarters.  Rows of 128 or
// 384 bytes alternate between the two halves of the banks.
template <int D>
__device__ __forceinline__ int swizzle(int p, int row) {
  if constexpr (D % 128 == 0) return p ^ (((row & 3) << 2) | ((row >> 2) & 3));
  const int x = row >> 1;
  return p ^ (((x & 1) << 2) | ((x >> 1) & 3));
}

__device__ __forceinline__ int seq_tiles(const PromptArgs& p, int b, int* q0, int* q1) {
  int64_t lo = p.cu_q[b], hi = p.cu_q[b + 1];
  lo = lo < 0 ? 0 : (lo > p.Tq ? p.Tq : lo);
  hi = hi < lo ? lo : (hi > p.Tq ? p.Tq : hi);
  *q0 = (int)lo;
  *q1 = (int)hi;
  return (int)((hi - lo + kBlockRows - 1) / kBlockRows);
}

// Zeroes what is not finite in a word of two bfloat16.
__device__ __forceinline__ uint32_t only_finite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

template <int D>
__global__ __launch_bounds__(kThreads, D <= 192 ? 2 : 1) void prompt_attention_kernel(
    PromptArgs a, int slots, int per_xcd) {
  constexpr int KB = tile_keys<D>();
  constexpr int kPieces = D / 8;                      // 16-byte pieces of a row
  constexpr int kLoads = KB * kPieces / kThreads;     // pieces of a thread, per K or V tile
  constexpr int kTileHalf = KB * D * 2;               // bytes of K (or V) in a buffer
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int g = lane >> 5, c = lane & 31;

  const int w = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (w >= slots * a.NHq) return;
  const int h = w / slots;
  const int x = w - h * slots;
  const int kvh = h / (a.NHq / a.NKV);

  // the sequence and tile of slot x: a running sum of the sequences' tiles
  int seq = -1, tile = 0, q0 = 0, q1 = 0, total = 0;
  for (int b0 = 0; b0 < a.B; b0 += kWave) {
    int lo = 0, hi = 0;
    const int nt = b0 + lane < a.B ? seq_tiles(a, b0 + lane, &lo, &hi) : 0;
    const int incl = wave_inclusive_sum_dpp(nt);
    const unsigned long long hit = __ballot(x >= total + incl - nt && x < total + incl);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      seq = b0 + src;
      tile = __shfl(total + incl, src) - 1 - x;       // the last tile first
      q0 = __shfl(lo, src);
      q1 = __shfl(hi, src);
      break;
    }
    total += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  seq = __builtin_amdgcn_readfirstlane(seq);
  if (seq < 0) {
    // no tile: such slots share the rows behind the last sequence
    if (!a.zero_tail) return;
    int64_t behind = a.cu_q[a.B];
    behind = behind < 0 ? 0 : behind;
    for (int64_t t = behind + (x - total); t < a.Tq; t += slots - total) {
      if ((a.zero_tail & 1) && tid < kPieces)
        reinterpret_cast<uint4*>(a.out + t * a.out_stride + (int64_t)h * D)[tid] = make_uint4(0, 0, 0, 0);
      if ((a.zero_tail & 2) && tid == 0 && a.lse) a.lse[t * a.NHq + h] = kNegInf;
    }
    return;
  }
  tile = __builtin_amdgcn_readfirstlane(tile);
  q0 = __builtin_amdgcn_readfirstlane(q0);
  q1 = __builtin_amdgcn_readfirstlane(q1);
  int64_t k0 = a.cu_k[seq], k1 = a.cu_k[seq + 1];
  k0 = k0 < 0 ? 0 : (k0 > a.Tk ? a.Tk : k0);
  k1 = k1 < k0 ? k0 : (k1 > a.Tk ? a.Tk : k1);
  const int nq = q1 - q0, nk = (int)(k1 - k0);
  // keys that in-sequence row i sees
  auto limit = [&](int i) {
    if (!a.causal) return nk;
    const int64_t l = (int64_t)i + 1 + nk - nq;
    return l < 0 ? 0 : (l > nk ? nk : (int)l);
  };
  const int block0 = tile * kBlockRows;
  const int row0 = block0 + wave * kRows;
  const int row = row0 + c;                           // in the sequence; may be past its end
  const int lim = limit(row);
  const int wave_min = limit(row0);
  const int wave_max = row0 < nq ? limit(min(row0 + kRows, nq) - 1) : 0;
  const int tiles = (limit(min(block0 + kBlockRows, nq) - 1) + KB - 1) / KB;

  v8bf q[D / 16];
  {
    const uint16_t* src = a.q + (int64_t)(q0 + min(row, nq - 1)) * a.q_stride + (int64_t)h * D + g * 8;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 16 * s));
  }
  const float scale2 = a.scale * kLog2e;
  const uint16_t* kbase = a.k + k0 * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vbase = a.v + k0 * a.v_stride + (int64_t)kvh * D;

  uint4 kr[kLoads], vr[kLoads];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = tid + i * kThreads;
      const int r = idx / kPieces, pc = idx - r * kPieces;
      const int64_t j = min(t * KB + r, nk - 1);      // rows behind the end repeat the last one
      kr[i] = *reinterpret_cast<const uint4*>(kbase + j * a.k_stride + pc * 8);
      vr[i] = *reinterpret_cast<const uint4*>(vbase + j * a.v_stride + pc * 8);
    }
  };
  auto stash = [&](int buf) {
    uint8_t* dst = smem + buf * 2 * kTileHalf;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = tid + i * kThreads;
      const int r = idx / kPieces, pc = idx - r * kPieces;
      const int at = (r * kPieces + swizzle<D>(pc, r)) * 16;
      *reinterpret_cast<uint4*>(dst + at) = kr[i];
      *reinterpret_cast<uint4*>(dst + kTileHalf + at) = vr[i];
    }
  };

  float m, l;
  v16f o[D / 32];
  // kCareful: values that are not finite are left out of the masked tiles'
  // product and added afterwards to the rows that see them.
  auto attend = [&](bool careful) {
    m = kNegInf;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    if (tiles > 0) {
      fetch(0);
      stash(0);
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      if (t + 1 < tiles) fetch(t + 1);
      const uint8_t* kt = smem + (t & 1) * 2 * kTileHalf;
      const uint8_t* vt = kt + kTileHalf;
      if (t * KB < wave_max) {                         // wave-uniform
        v16f s[KB / 32];
#pragma unroll
        for (int i = 0; i < KB / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[i][r] = 0.0f;
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {
#pragma unroll
          for (int i = 0; i < KB / 32; ++i) {
            const int r = i * 32 + c;
            const uint4 kf = *reinterpret_cast<const uint4*>(
                kt + (r * kPieces + swizzle<D>(2 * st + g, r)) * 16);
            s[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, kf), q[st], s[i], 0, 0, 0);
          }
        }
        const bool masked = (t + 1) * KB > wave_min;
        if (masked) {
#pragma unroll
          for (int i = 0; i < KB / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int key = t * KB + i * 32 + 8 * (r >> 2) + 4 * g + (r & 3);
              if (key >= lim) s[i][r] = kNegInf;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 0; i < KB / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, s[i][r]);
        top *= scale2;
        if (__any(top > m + kSlack)) {
          top = fmaxf(top, __shfl_xor(top, 32));
          const float next = fmaxf(m, top);
          const float f = next == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - next);
          m = next;
          l *= f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] *= f;
        }
        const float base = m == kNegInf ? 0.0f : -m;
        float sum = 0.0f;
        v8bf pb[KB / 16];
#pragma unroll
        for (int u = 0; u < KB / 16; ++u) {
          uint32_t pw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = (u & 1) * 8 + 2 * i;
            const float p0 = __builtin_amdgcn_exp2f(fmaf(s[u >> 1][r], scale2, base));
            const float p1 = __builtin_amdgcn_exp2f(fmaf(s[u >> 1][r + 1], scale2, base));
            sum += p0 + p1;
            pw[i] = pack_bf16(p0, p1);
          }
          pb[u] = __builtin_bit_cast(v8bf, make_uint4(pw[0], pw[1], pw[2], pw[3]));
        }
        l += sum;
#pragma unroll
        for (int u = 0; u < KB / 16; ++u) {
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            // lane: key row r0 (+ 8), features 8 * (piece) + 4 * (lane & 1) ..
            const int r0 = 16 * u + 4 * g + ((lane & 15) >> 2);
            const int pc = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            const uint8_t* a0 = vt + (r0 * kPieces + swizzle<D>(pc, r0)) * 16 + (lane & 1) * 8;
            const uint8_t* a1 = vt + ((r0 + 8) * kPieces + swizzle<D>(pc, r0 + 8)) * 16 + (lane & 1) * 8;
            const uint2 v0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)a0));
            const uint2 v1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)a1));
            uint4 vf = make_uint4(v0.x, v0.y, v1.x, v1.y);
            if (careful && masked)
              vf = make_uint4(only_finite(vf.x), only_finite(vf.y), only_finite(vf.z), only_finite(vf.w));
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, vf), pb[u], o[d], 0, 0, 0);
          }
        }
        if (careful && masked) {
          for (int key = 0; key < KB && t * KB + key < nk; ++key) {
            const bool seen = t * KB + key < lim;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const int f = 32 * d + 8 * (r >> 2) + 4 * g + (r & 3);
                const uint16_t bits = *reinterpret_cast<const uint16_t*>(
                    vt + (key * kPieces + swizzle<D>(f >> 3, key)) * 16 + (f & 7) * 2);
                if (seen && (bits & 0x7F80u) == 0x7F80u) o[d][r] += bf16_lo(bits);
              }
          }
        }
      }
      if (t + 1 < tiles) stash((t + 1) & 1);
      __syncthreads();
    }
  };

  attend(false);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd |= !(fabsf(o[i][r]) < __builtin_inff());
  if (__syncthreads_or(odd)) attend(true);

  l += __shfl_xor(l, 32);
  // a row without a score has the sum 0, one whose scores are all NaN the sum
  // NaN and the maximum -inf
  const float f = m == kNegInf ? l : 1.0f / l;
  if (row < nq) {
    uint16_t* dst = a.out + (int64_t)(q0 + row) * a.out_stride + (int64_t)h * D + 4 * g;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        uint2 v;
        v.x = pack_bf16(o[i][r] * f, o[i][r + 1] * f);
        v.y = pack_bf16(o[i][r + 2] * f, o[i][r + 3] * f);
        *reinterpret_cast<uint2*>(dst + 32 * i + 2 * r) = v;
      }
    if (a.lse && g == 0) a.lse[(int64_t)(q0 + row) * a.NHq + h] = (m + __log2f(l)) * kLn2;
  }
}

template <int D>
hipError_t prepare_one() {
  return prepare_kernel(reinterpret_cast<const void*>(&prompt_attention_kernel<D>), lds_bytes<D>());
}

template <int D>
void launch_one(const PromptArgs& p, int slots, int per_xcd, hipStream_t stream) {
  prompt_attention_kernel<D><<<dim3((unsigned)(8 * per_xcd)), dim3(kThreads), lds_bytes<D>(), stream>>>(
      p, slots, per_xcd);
}

}  // namespace

hipError_t prepare_prompt_kernels() {
  hipError_t e = prepare_one<64>();
  if (e == hipSuccess) e = prepare_one<128>();
  if (e == hipSuccess) e = prepare_one<192>();
  if (e == hipSuccess) e = prepare_one<256>();
  return e;
}

hipError_t launch_prompt_attention(const PromptArgs& p, hipStream_t stream) {
  // Each sequence ends with at most one part tile; one slot more, so that some
  // slot is left for the rows behind the last sequence.
  const int64_t slots = p.Tq / kBlockRows + p.B + (p.zero_tail ? 1 : 0);
  const int64_t per_xcd = (slots * p.NHq + 7) / 8;
  switch (p.D) {
    case 64: launch_one<64>(p, (int)slots, (int)per_xcd, stream); break;
    case 128: launch_one<128>(p, (int)slots, (int)per_xcd, stream); break;
    case 192: launch_one<192>(p, (int)slots, (int)per_xcd, stream); break;
    default: launch_one<256>(p, (int)slots, (int)per_xcd, stream); break;
  }
  return hipGetLastError();
}

}  // namespace moe
