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
// Probabilities are rounded to bfloat16 for the second product (at most 2^-8
// relative each, random over the keys: the output's error stays at the size of
// its own rounding; a second bfloat16 for the rest, as the cache's attention
// has it, would add half as many matrix instructions); their sum is taken in
// float32 before that.  The running maximum moves only when a score passes it by
// more than 8 (in powers of two), so most tiles skip the rescaling of O^T.
//
// Work split: a workgroup of eight waves takes 256 rows, 32 a wave, of one kv
// head; a row is (query, head of the group), so that the heads of a group share
// their keys and short prompts fill the rows.  K and V tiles of 64 keys (32 for
// D = 192, 256) come to LDS by direct loads into a ring of four, two tiles
// ahead; rows behind the last key repeat it.  The two waves of a SIMD work in
// opposite phases (below): a tile's two products are 32 matrix instructions
// (D = 128), its softmax about 110 vector instructions of which 32 are
// exponentials, so neither may wait for the other.  Few rows take workgroups of
// 128 or 64 rows, in which two waves share 32 rows and take half of each tile's
// keys each; their sums meet in the LDS at the end (launch_head has the
// measurements).  Few query tiles over many keys split the keys over
// workgroups; the parts go to scratch in float32 and a second launch joins them
// (prompt_splits).  Many rows of short sequences take tiles of 32 keys, with
// more workgroups on a compute unit.
//
// Measured: 8192 tokens, 32 heads over 4 of D = 128, causal, 510 us = 1.08
// PFLOP/s (D = 64, 192, 256: 0.92, 1.10, 1.11; not causal, D = 128: 1.15); a
// library product of 8192^3 reaches 1.38 on the same card.  In parts (not
// causal, D = 128, before the values were read ahead: 975 us): without the
// loads to LDS 905, without the softmax as well 858, without the LDS reads as
// well 706, which is the matrix instructions and the barriers.  What bounds it
// is the phase of the products: one wave of a SIMD at a time reads 1 KB of LDS
// per matrix instruction, 128 bytes a cycle and compute unit.  A
// tile takes 3300 cycles (2048 of matrix instructions), at a clock that falls to
// 1.5 .. 1.9 GHz under this load.
//
// A key or value that a row does not see never reaches it: scores of masked
// pairs are replaced, and a wave that ends with a value that is not finite
// looks for values among its masked pairs that 0 * NaN carried over
// (mend_rows).
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "internal.hpp"

namespace moe {
namespace {

constexpr int kRows = 32;                       // rows of a wave
constexpr int kMaxSplits = 64;
constexpr int kLeast = 4;                       // tiles of keys of a split, at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
constexpr float kNegInf = -__builtin_inff();

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
#define MOE_LDS __attribute__((address_space(3)))

// Shape of a kernel: head size, waves of a workgroup, buffers of the ring.
template <int D_, int WAVES_, int BUFS_, int PARTS_ = 1, int KB_ = D_ <= 128 ? 64 : 32>
struct Shape {
  static constexpr int D = D_, kWaves = WAVES_, kBufs = BUFS_;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kParts = PARTS_;                   // waves that share 32 rows, and a tile's keys
  static constexpr int kGroups = kWaves / kParts;         // of 32 rows
  static constexpr int kBlockRows = kGroups * kRows;
  static constexpr bool kPaired = kWaves == 8;            // two waves on a SIMD, in opposite phases
  // keys of a tile
  static constexpr int KB = KB_;
  static constexpr int KW = KB / kParts;                  // of them a wave's
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kHalf = KB * kRowBytes;            // K (or V) of a tile
  static constexpr int kLoads = 2 * kHalf / 1024 / kWaves;  // 1 KB loads of a wave per tile
  static constexpr int kAhead = kBufs - 2;                // tiles in flight
  static constexpr int kLds = kBufs * 2 * kHalf;
  static_assert(2 * kHalf % (1024 * kWaves) == 0, "whole loads per wave");
  // operands read ahead, and whether the two products take turns: as far as
  // the registers go (D = 256 would spill)
  static constexpr int kReadAhead = D == 128 || D == 192 ? 4 : 2;
  static constexpr bool kTurns = D <= 192;
  // value operands read during the softmax
  static constexpr int kPre = D == 128 ? KW / 8 : (D == 192 ? 2 : 0);
  // D = 64: two workgroups to a compute unit
  static constexpr int kWavesPerSimd = D == 64 && kPaired ? 4 : 2;
  // The 16-byte pieces of a row are XOR-ed with a function of the row inside
  // groups of kGroup.  The 64 banks hold 256 bytes: rows of 256 or 512 bytes
  // all start at the same bank; 16 rows that read the same piece need 16
  // different positions, and 4 rows that read 4 pieces each (the transposing
  // read) need them in 4 different quarters.  Rows of 128 or 384 bytes
  // alternate between the two halves of the banks.
  static constexpr int kGroup = D % 128 == 0 ? 16 : 8;
  __device__ __forceinline__ static int mix(int row) {
    if constexpr (kGroup == 16) return ((row & 3) << 2) | ((row >> 2) & 3);
    return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  }
  // byte of piece p of a row
  __device__ __forceinline__ static int at(int row, int p) {
    return row * kRowBytes + (p & ~(kGroup - 1)) * 16 + ((p & (kGroup - 1)) ^ mix(row)) * 16;
  }
};

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const MOE_LDS uint8_t*)p;
}

// 1 KB from 64 lanes' addresses (uniform base + 32-bit byte offset) to LDS at
// `lds` (uniform), lane after lane.  Written in assembly because the compiler
// would otherwise wait for every such load before its next LDS read; the
// kernel waits for them itself (wait_loads) and no register is an output.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n"
               "s_nop 0\n"
               "global_load_lds_dwordx4 %1, %0"
               :
               : "s"(base), "v"(offset), "s"(lds)
               : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// Every wave's LDS accesses so far are done, and those after stay after.
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\ns_barrier" : : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Where sequence b's queries start, and how many it has.
__device__ __forceinline__ int query_span(const PromptArgs& p, int b, int* q0) {
  int64_t lo = p.cu_q[b], hi = p.cu_q[b + 1];
  lo = lo < 0 ? 0 : (lo > p.Tq ? p.Tq : lo);
  hi = hi < lo ? lo : (hi > p.Tq ? p.Tq : hi);
  *q0 = (int)lo;
  return (int)(hi - lo);
}
__device__ __forceinline__ int key_span(const PromptArgs& p, int b, int* k0) {
  int64_t lo = p.cu_k[b], hi = p.cu_k[b + 1];
  lo = lo < 0 ? 0 : (lo > p.Tk ? p.Tk : lo);
  hi = hi < lo ? lo : (hi > p.Tk ? p.Tk : hi);
  *k0 = (int)lo;
  return (int)(hi - lo);
}
// Keys that query i of nq sees.
__device__ __forceinline__ int keys_seen(const PromptArgs& p, int i, int nq, int nk) {
  if (!p.causal) return nk;
  const int64_t l = (int64_t)i + 1 + nk - nq;
  return l < 0 ? 0 : (l > nk ? nk : (int)l);
}
// Tiles of keys of a split, of n: an equal share, kLeast at least, so that the
// splits with work come first.
__device__ __forceinline__ int split_tiles(int n, int splits) {
  const int each = (n + splits - 1) / splits;
  return each < kLeast ? kLeast : each;
}

// A finished row, or its part in a split, from a wave: lane's features d ..
template <int N>
__device__ __forceinline__ void store_row(const PromptArgs& a, bool alone, int64_t token, int h, int split,
                                          int d, const float (&o)[N], float m, float l, bool first) {
  if (alone) {
    const float f = m == kNegInf ? l : 1.0f / l;       // as at the kernel's end
    uint16_t* dst = a.out + token * a.out_stride + (int64_t)h * a.D + d;
#pragma unroll
    for (int k = 0; k < N; ++k) dst[k] = (uint16_t)pack_bf16(o[k] * f, 0.0f);
    if (first && a.lse) a.lse[token * a.NHq + h] = (m + __log2f(l)) * kLn2;
  } else {
    const int64_t at = (token * a.NHq + h) * a.splits + split;
#pragma unroll
    for (int k = 0; k < N; ++k) a.part_o[at * a.D + d + k] = o[k];
    if (first) a.part_ml[at] = make_float2(m, l);
  }
}

// Mends a wave's rows row0 .. + rows (row r is query r / G of the sequence and
// head r % G of the group) after their last tile, when one of them holds a
// value that is not finite.  A row's products ran over the keys key0 .. key1,
// with probability 0 for those it does not see: where such a key's value is
// not finite, 0 * NaN has reached it.  Those rows are computed again, a lane
// holding D / 64 features, over exactly the keys they see.  Reached by no
// finite values; kept out of line so that it costs the others no register.
template <int D>
__attribute__((noinline)) __device__ void mend_rows(PromptArgs a, int q0, int nq, int row0, int rows, int kvh,
                                                    int64_t k0, int nk, int key0, int key1, bool alone, int split) {
  constexpr int kPer = D / kWave;
  const int lane = threadIdx.x & (kWave - 1), f0 = lane * kPer;
  const int G = a.G;
  const float scale2 = a.scale * kLog2e;
  int bad = -1;                                        // the last key whose value is not finite
  for (int j = max(key0, keys_seen(a, row0 / G, nq, nk)); j < key1; ++j) {
    bool odd = false;
    for (int d = 0; d < kPer; ++d)
      odd |= (a.v[(k0 + j) * a.v_stride + (int64_t)kvh * D + f0 + d] & 0x7F80u) == 0x7F80u;
    if (__any(odd)) bad = j;
  }
  for (int r = row0; r < row0 + rows && keys_seen(a, r / G, nq, nk) <= bad; ++r) {
    const int64_t token = q0 + r / G;
    const int h = kvh * G + r % G;
    const int lim = min(key1, keys_seen(a, r / G, nq, nk));
    float q[kPer], o[kPer], m = kNegInf, l = 0.0f;
    for (int d = 0; d < kPer; ++d) {
      q[d] = bf16_lo(a.q[token * a.q_stride + (int64_t)h * D + f0 + d]);
      o[d] = 0.0f;
    }
    for (int j = key0; j < lim; ++j) {
      const uint16_t* k = a.k + (k0 + j) * a.k_stride + (int64_t)kvh * D + f0;
      const uint16_t* v = a.v + (k0 + j) * a.v_stride + (int64_t)kvh * D + f0;
      float s = 0.0f;
      for (int d = 0; d < kPer; ++d) s = fmaf(q[d], bf16_lo(k[d]), s);
      s = wave_sum(s) * scale2;
      const float next = fmaxf(m, s);
      const float f = next == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - next);
      const float p = __builtin_amdgcn_exp2f(s - (next == kNegInf ? 0.0f : next));
      m = next;
      l = l * f + p;
      for (int d = 0; d < kPer; ++d) o[d] = o[d] * f + p * bf16_lo(v[d]);
    }
    store_row(a, alone, token, h, split, f0, o, m, l, lane == 0);
  }
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void prompt_attention_kernel(
    PromptArgs a, int slots) {
  constexpr int D = S::D, KB = S::KB, KW = S::KW;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int g = lane >> 5, c = lane & 31;
  const int G = a.G;

  // Workgroup b runs on XCD b & 7.  With 1, 2, 4 or 8 kv heads (or a multiple
  // of 8) each XCD keeps to one kv head at a time, so that its keys stay in
  // that L2, and the XCDs of a head take its slots in turn: the slots with the
  // most keys go first, on all XCDs alike.
  int kvh, rest;
  if (a.xcd_shift >= 0) {                              // 8 >> xcd_shift kv heads
    const int turn = blockIdx.x & 7;
    kvh = turn & (a.NKV - 1);
    rest = ((blockIdx.x >> 3) << a.xcd_shift) + (turn >> (3 - a.xcd_shift));
  } else if (a.NKV % 8 == 0) {
    const int j = blockIdx.x >> 3, heads = a.NKV >> 3;
    rest = j / heads;
    kvh = (j - rest * heads) * 8 + (blockIdx.x & 7);
  } else {
    rest = blockIdx.x / a.NKV;
    kvh = blockIdx.x - rest * a.NKV;
  }
  const int x = a.splits == 1 ? rest : rest / a.splits, split = rest - x * a.splits;
  if (x >= slots) return;

  // the sequence and tile of slot x: a running sum of the sequences' tiles
  int seq = -1, tile = 0, q0 = 0, nq = 0, k0 = 0, nk_all = 0, total = 0;
  for (int b0 = 0; b0 < a.B; b0 += kWave) {
    int lo = 0, klo = 0, n = 0, kn = 0;
    if (b0 + lane < a.B) {
      n = query_span(a, b0 + lane, &lo);
      kn = key_span(a, b0 + lane, &klo);
    }
    const int nt = (n * G + S::kBlockRows - 1) / S::kBlockRows;
    const int incl = wave_inclusive_sum_dpp(nt);
    const unsigned long long hit = __ballot(x >= total + incl - nt && x < total + incl);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      seq = b0 + src;
      tile = __shfl(total + incl, src) - 1 - x;       // the last tile first
      q0 = __shfl(lo, src);
      nq = __shfl(n, src);
      k0 = __shfl(klo, src);
      nk_all = __shfl(kn, src);
      break;
    }
    total += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  seq = __builtin_amdgcn_readfirstlane(seq);
  if (seq < 0) {
    // no tile: such slots share the rows behind the last sequence and before
    // the first
    if (split > 0) return;
    int64_t before = a.cu_q[0], behind = a.cu_q[a.B];
    before = before < 0 ? 0 : (before > a.Tq ? a.Tq : before);
    behind = behind < before ? before : (behind > a.Tq ? a.Tq : behind);
    for (int64_t i = x - total; i < before + (a.Tq - behind); i += slots - total) {
      const int64_t t = i < before ? i : behind + (i - before);
      if (a.zero_tail & 1)
        for (int j = tid; j < G * (D / 8); j += S::kThreads)
          reinterpret_cast<uint4*>(a.out + t * a.out_stride + (int64_t)kvh * G * D)[j] = make_uint4(0, 0, 0, 0);
      if ((a.zero_tail & 2) && a.lse)
        for (int j = tid; j < G; j += S::kThreads) a.lse[t * a.NHq + kvh * G + j] = kNegInf;
    }
    return;
  }
  tile = __builtin_amdgcn_readfirstlane(tile);
  q0 = __builtin_amdgcn_readfirstlane(q0);
  nq = __builtin_amdgcn_readfirstlane(nq);
  k0 = __builtin_amdgcn_readfirstlane(k0);
  nk_all = __builtin_amdgcn_readfirstlane(nk_all);
  const int nr = nq * G;                              // rows: (query, head of the group)
  const int block0 = tile * S::kBlockRows;
  const int part = wave / S::kGroups;                 // of a tile's keys
  const int row0 = block0 + wave % S::kGroups * kRows;
  const int last_row = min(block0 + S::kBlockRows, nr) - 1;
  // this split's tiles of keys; from here on keys and limits count from its
  // first key on
  const int all_tiles = (keys_seen(a, last_row / G, nq, nk_all) + KB - 1) / KB;
  const int each = split_tiles(all_tiles, a.splits);
  const bool alone = all_tiles <= each;
  const int tiles = min(all_tiles - split * each, each);
  if (tiles <= 0 && split > 0) return;
  const int key0 = split * each * KB;
  const int nk = nk_all - key0;
  auto limit = [&](int r) {                           // keys that row r sees here
    const int l = keys_seen(a, r / G, nq, nk_all) - key0;
    return l < 0 ? 0 : min(l, tiles * KB);
  };
  const int lim = limit(min(row0 + c, nr - 1));       // lanes past the end repeat the last row
  const int wave_max = row0 < nr ? limit(min(row0 + kRows, nr) - 1) : 0;

  const float scale2 = a.scale * kLog2e;
  const uint16_t* kbase = a.k + (int64_t)(k0 + key0) * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vbase = a.v + (int64_t)(k0 + key0) * a.v_stride + (int64_t)kvh * D;

  // This wave's loads of a tile: 1 KB pieces wave, wave + kWaves, .. of K's
  // and then V's LDS image; the lane brings the 16 bytes that belong there.
  const uint32_t lds0 = lds_addr(smem);
  constexpr int kRowsOfLoad = 1024 / S::kRowBytes;    // (D = 192: not whole, kEven false)
  // Where a wave's loads of K fall on whole rounds of the waves, they differ by
  // whole rows that leave the XOR as it is: one offset does for all of them,
  // and one for those of V.
  constexpr bool kEven = S::kHalf / 1024 % S::kWaves == 0 && 1024 % S::kRowBytes == 0;
  constexpr int kHalfLoads = S::kLoads / 2;
  static_assert(!kEven || S::kWaves * kRowsOfLoad % 16 == 0, "rows of a round");
  auto load_is_v = [&](int i) { return kEven ? i >= kHalfLoads : wave + i * S::kWaves >= S::kHalf / 1024; };
  auto image_byte = [&](int i) {                      // of K or V
    return (wave + i * S::kWaves) * 1024 + lane * 16 - (load_is_v(i) ? S::kHalf : 0);
  };
  uint32_t loff[kEven ? 2 : S::kLoads];               // byte offset of the row's piece
#pragma unroll
  for (int i = 0; i < (kEven ? 2 : S::kLoads); ++i) {
    const int l = kEven ? i * kHalfLoads : i;
    const int r = image_byte(l) / S::kRowBytes, p = (image_byte(l) - r * S::kRowBytes) / 16;
    const int piece = (p & ~(S::kGroup - 1)) | ((p & (S::kGroup - 1)) ^ S::mix(r));
    loff[i] = (uint32_t)r * (uint32_t)(2 * (load_is_v(l) ? a.v_stride : a.k_stride)) + piece * 16;
  }
  auto fetch = [&](int t) {
    const uint32_t buf = lds0 + (uint32_t)(t % S::kBufs) * (2 * S::kHalf) + wave * 1024;
    const int last = nk - 1 - t * KB;                 // rows behind the last key repeat it
    const bool whole_tile = last >= KB - 1;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const bool is_v = load_is_v(i);
      const int64_t stride = is_v ? a.v_stride : a.k_stride;
      const uint16_t* base = (is_v ? vbase : kbase) + (int64_t)t * KB * stride;
      uint32_t off = loff[kEven ? i / kHalfLoads : i];
      const int rows = kEven ? i % kHalfLoads * (S::kWaves * kRowsOfLoad) : 0;   // after loff's
      if (whole_tile) {
        base += rows * stride;
      } else {
        const int r = image_byte(i) / S::kRowBytes;
        off += (uint32_t)(rows - max(r - last, 0)) * (uint32_t)(2 * stride);
      }
      load_to_lds(base, off, buf + i * (S::kWaves * 1024));
    }
  };

#pragma unroll
  for (int t = 0; t < S::kAhead; ++t)
    if (t < tiles) fetch(t);
  // The queries, behind the first tiles; they are in registers before the loop:
  // waiting for them in it would wait for the loads to LDS as well.
  v8bf q[D / 16];
  {
    const int row = min(row0 + c, nr - 1);
    const uint16_t* src = a.q + (int64_t)(q0 + row / G) * a.q_stride + (int64_t)(kvh * G + row % G) * D + g * 8;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 16 * s));
#pragma unroll
    for (int s = 0; s < D / 16; ++s) asm volatile("" : "+v"(q[s]));
  }

  // LDS bytes of the operands: K row c (+ 32 i), piece 2 st + g; V row 16 u +
  // 4 g + (lane & 15) / 4 (+ 8), piece 4 d + x.  The pieces' XOR with the row
  // leaves constants in st and d, since rows differ by multiples of 32 or 16,
  // and 8 rows further on the XOR-ed function differs in bit 1.
  const int vr = 4 * g + ((lane & 15) >> 2);
  const uint32_t kat = lds0 + part * (KW * S::kRowBytes) + S::at(c, g);
  const uint32_t vat = lds0 + S::kHalf + part * (KW * S::kRowBytes) +
                       S::at(vr, 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + (lane & 1) * 8;

  // Tiles that every row of the workgroup sees whole, and this wave's tiles.
  const int whole = limit(block0) / KB;
  const int mine = (wave_max + KB - 1) / KB;
  float m, l;
  v16f o[D / 32], s[KW / 32];
  v8bf pb[KW / 16];

  // Operands of the matrix instructions.  Scores of tile t: instruction n
  // takes K rows 32 i .. of step st; values: V^T rows 32 d .. of 16 keys u.
  // Neighbours add to different accumulators where there are several.
  constexpr int kOps = (D / 16) * (KW / 32);           // of either product
  auto key_operand = [&](uint32_t kt, int n) {
    const int st = n / (KW / 32), i = n % (KW / 32);
    const uint32_t at = (kt ^ (32 * (st % (S::kGroup / 2)))) + (2 * st / S::kGroup) * (S::kGroup * 16);
    return *(const MOE_LDS v8bf*)(uintptr_t)(at + i * 32 * S::kRowBytes);
  };
  auto value_operand = [&](uint32_t vt, int n) {
    const int d = n % (D / 32), u = n / (D / 32);
    const uint32_t far = (4 * d / S::kGroup) * (S::kGroup * 16) + u * 16 * S::kRowBytes;
    const uint32_t at0 = (vt ^ (64 * (d % (S::kGroup / 4)))) + far;
    const uint32_t at1 = ((vt + 8 * S::kRowBytes) ^ (64 * (d % (S::kGroup / 4))) ^ 32) + far;
    const uint2 v0 = __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)(uintptr_t)at0));
    const uint2 v1 = __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)(uintptr_t)at1));
    return __builtin_bit_cast(v8bf, make_uint4(v0.x, v0.y, v1.x, v1.y));
  };
  // S^T of tile t, and O^T += V^T P^T of tile t - 1 with P as the last softmax
  // left it, each on request.  Together: where two score accumulators take
  // turns (KW = 64), a quarter of the values, then two scores and a value at a
  // time, then the last values; with one, values and scores in turn (kTurns).
  // So no instruction waits for the one before it, the first ones find their
  // operands in registers (ahead, read during the softmax, when the LDS has
  // less to do) and the scores are ready when the phase ends.  Operands are
  // read kReadAhead at a time, one such group ahead of its use.  The wave goes
  // before the other one of its SIMD meanwhile, whose softmax fills the gaps.
  v8bf ahead[S::kPre ? S::kPre : 1];                   // of the first values
  auto read_ahead = [&](int t) {
    const uint32_t vt = vat + (uint32_t)(t % S::kBufs) * (2 * S::kHalf);
#pragma unroll
    for (int i = 0; i < S::kPre; ++i) ahead[i] = value_operand(vt, i);
  };
  auto multiply = [&](int t, auto scores, auto values) {
    constexpr bool kS = decltype(scores)::value, kV = decltype(values)::value;
    constexpr int kAll = (kS ? kOps : 0) + (kV ? kOps : 0), kAt = S::kReadAhead;
    // instruction n: 2 * op for scores, 2 * op + 1 for values
    auto at = [&](int n) {
      if (!kV) return 2 * n;
      if (!kS) return 2 * n + 1;
      if (!S::kTurns) return n < kOps ? 2 * n : 2 * (n - kOps) + 1;
      if (KW == 32) return n % 2 ? n - 1 : n + 1;
      constexpr int kQ = kOps / 4;
      if (n < kQ) return 2 * n + 1;
      if (n >= kAll - kQ) return 2 * (n - kOps) + 1;
      const int m = n - kQ;
      return m % 3 == 2 ? 2 * (kQ + m / 3) + 1 : 2 * (m / 3 * 2 + m % 3);
    };
    uint32_t kt = kat + (uint32_t)(t % S::kBufs) * (2 * S::kHalf);
    uint32_t vt = vat + (uint32_t)((t + S::kBufs - 1) % S::kBufs) * (2 * S::kHalf);
    __builtin_amdgcn_s_setprio(1);
    v8bf f[2][kAt];
    auto read = [&](int n) {
      // the addresses are formed again for every read: kept, they would spill
      if constexpr (D == 256) asm volatile("" : "+v"(kt), "+v"(vt));
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int op = at(n + i);
        if (op % 2 == 0) f[(n / kAt) & 1][i] = key_operand(kt, op / 2);
        else if (op / 2 >= S::kPre) f[(n / kAt) & 1][i] = value_operand(vt, op / 2);
      }
      __builtin_amdgcn_sched_barrier(0);               // reads stay ahead of the products before them
    };
    if constexpr (kS) {
#pragma unroll
      for (int i = 0; i < KW / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[i][r] = 0.0f;
    }
    read(0);
#pragma unroll
    for (int n = 0; n < kAll; n += kAt) {
      if (n + kAt < kAll) read(n + kAt);
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int op = at(n + i) / 2;
        if (at(n + i) % 2 == 0) {
          const int j = op % (KW / 32);
          s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[(n / kAt) & 1][i], q[op / (KW / 32)], s[j], 0, 0, 0);
        } else {
          const int d = op % (D / 32);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op < S::kPre ? ahead[op < S::kPre ? op : 0] : f[(n / kAt) & 1][i],
                                                         pb[op / (D / 32)], o[d], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // P of S^T, with the running maximum and sum.
  auto softmax = [&](int t) {
    if (t >= whole) {                                  // uniform
      const int left = lim - t * KB - part * KW - 4 * g;           // of this lane's keys, from register 0's on
#pragma unroll
      for (int i = 0; i < KW / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[i][r] = i * 32 + 8 * (r >> 2) + (r & 3) < left ? s[i][r] : kNegInf;
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 0; i < KW / 32; ++i)
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
#pragma unroll
    for (int u = 0; u < KW / 16; ++u) {
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
    // P is made here and not, as the compiler would have it, where the next
    // phase's products first need it
#pragma unroll
    for (int u = 0; u < KW / 16; ++u) asm volatile("" : "+v"(pb[u]));
    asm volatile("" : "+v"(l));
  };

  // Phases (kPaired).  A wave alternates between matrix products (the scores of tile t
  // and the values of tile t - 1) and the softmax of tile t; the second half
  // of the waves is one phase behind the first, so that on every SIMD one wave
  // multiplies while the other takes exponentials.  A barrier ends each phase.
  // Before barrier 2 t (first half: before the products of tile t; second
  // half: before the softmax of tile t - 1) every wave's loads of tile t have
  // arrived; after it the last reader of tile t - 2 (the second half's
  // products of tile t - 1) is done, and its buffer takes tile t + kBufs - 2.
  // Four waves have a SIMD each and no opposite phase: the odd barriers fall
  // away, and the same holds of the even ones.
  const bool late = S::kPaired && wave >= S::kWaves / 2;
  auto even = [&](int t) {
    if (t + S::kAhead <= tiles) wait_loads<(S::kAhead - 1) * S::kLoads>();
    else wait_loads<0>();
    barrier();
    if (t + S::kAhead < tiles) fetch(t + S::kAhead);
  };
  m = kNegInf;
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  auto before_softmax = [&](int t) {
    if (late) even(t + 1);
    else if (S::kPaired) barrier();
  };
  auto after_softmax = [&](int t) {
    if (late) barrier();
    else even(t + 1);
  };
  even(0);
  if (late) barrier();
  if (mine > 0) {
    multiply(0, std::true_type{}, std::false_type{});
#pragma clang loop unroll(disable)
    for (int t = 0; t < mine - 1; ++t) {
      before_softmax(t);
      read_ahead(t);
      softmax(t);
      after_softmax(t);
      multiply(t + 1, std::true_type{}, std::true_type{});
    }
    before_softmax(mine - 1);
    read_ahead(mine - 1);
    softmax(mine - 1);
    after_softmax(mine - 1);
    multiply(mine, std::false_type{}, std::true_type{});
  }
#pragma clang loop unroll(disable)
  for (int t = mine; t < tiles; ++t) {
    before_softmax(t);
    after_softmax(t);
  }
  if (S::kPaired && !late) barrier();                  // the second half's last products

  l += __shfl_xor(l, 32);
  if constexpr (S::kParts == 2) {
    // The second parts' sums go to the first through the LDS, register by
    // register, when its last reader is done.
    barrier();
    float* box = reinterpret_cast<float*>(smem) + wave % S::kGroups * (kRows * D + 2 * kWave) + lane;
    if (part) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) box[(i * 16 + r) * kWave] = o[i][r];
      box[kRows * D] = m;
      box[kRows * D + kWave] = l;
    }
    barrier();
    if (part) return;
    const float m2 = box[kRows * D], l2 = box[kRows * D + kWave], top = fmaxf(m, m2);
    // as the join of splits has it
    const float f = m == kNegInf ? l : __builtin_amdgcn_exp2f(m - top);
    const float f2 = m2 == kNegInf ? l2 : __builtin_amdgcn_exp2f(m2 - top);
    m = top;
    l = f * l + f2 * l2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = f * o[i][r] + f2 * box[(i * 16 + r) * kWave];
  }
  float odd = 0.0f;                                    // NaN as soon as one value is not finite
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd = fmaf(o[i][r], 0.0f, odd);
  int end_c = c;
  asm volatile("" : "+v"(end_c));                      // worked out again: registers of the loop
  const int row = row0 + end_c;
  const int64_t token = q0 + min(row, nr - 1) / G;
  const int h = kvh * G + min(row, nr - 1) % G;
  if (alone) {
    // a row without a score has the sum 0, one whose scores are all NaN the
    // sum NaN and the maximum -inf
    const float f = m == kNegInf ? l : 1.0f / l;
    uint16_t* dst = a.out + token * a.out_stride + (int64_t)h * D + 8 * g;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 8) {
        // registers r .. r + 3 of both halves are 8 features, r + 4 .. the next
        // 8: the halves exchange, so that each stores 16 bytes
        uint32_t x[2], y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[j] = pack_bf16(o[i][r + 2 * j] * f, o[i][r + 2 * j + 1] * f);
          y[j] = pack_bf16(o[i][r + 4 + 2 * j] * f, o[i][r + 5 + 2 * j] * f);
          const auto swapped = __builtin_amdgcn_permlane32_swap(x[j], y[j], false, false);
          x[j] = swapped[0];
          y[j] = swapped[1];
        }
        if (row < nr) *reinterpret_cast<uint4*>(dst + 32 * i + 2 * r) = make_uint4(x[0], x[1], y[0], y[1]);
      }
    if (row < nr && a.lse && g == 0) a.lse[token * a.NHq + h] = (m + __log2f(l)) * kLn2;
  } else if (row < nr) {
    const int64_t at = (token * a.NHq + h) * a.splits + split;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(a.part_o + at * D + 32 * i + 2 * r + 4 * g) =
            make_float4(o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]);
    if (g == 0) a.part_ml[at] = make_float2(m, l);
  }
  if (__any(odd != 0.0f) && mine > 0) {
    wait_loads<0>();                                   // the rows' stores above come first
    mend_rows<D>(a, q0, nq, row0, min(kRows, nr - row0), kvh, k0, nk_all, key0, min(nk_all, key0 + mine * KB),
                 alone, split);
  }
}

// Joins the splits of a row, a wave each: the block that computed it is found
// again to know how many splits had work.
template <typename S>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs a) {
  constexpr int D = S::D, KB = S::KB, kPer = D / kWave;
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (at >= a.Tq * a.NHq) return;
  const int64_t token = at / a.NHq;
  const int h = (int)(at - token * a.NHq);
  int seq = -1, q0 = 0, nq = 0;
  for (int b0 = 0; b0 < a.B && seq < 0; b0 += kWave) {
    int lo = 0;
    const int n = b0 + lane < a.B ? query_span(a, b0 + lane, &lo) : 0;
    const unsigned long long hit = __ballot(token >= lo && token < lo + n);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      seq = b0 + src;
      q0 = __shfl(lo, src);
      nq = __shfl(n, src);
    }
  }
  if (seq < 0) return;
  const int G = a.G;
  int k0;
  const int nk = key_span(a, seq, &k0);
  const int row = (int)(token - q0) * G + h % G;
  const int last_row = min((row / S::kBlockRows + 1) * S::kBlockRows, nq * G) - 1;
  const int all_tiles = (keys_seen(a, last_row / G, nq, nk) + KB - 1) / KB;
  const int each = split_tiles(all_tiles, a.splits);
  if (all_tiles <= each) return;
  const int parts = (all_tiles + each - 1) / each;   // at most kMaxSplits = 64
  const float2 v = lane < parts ? a.part_ml[at * a.splits + lane] : make_float2(kNegInf, 0.0f);
  const float m = wave_max(v.x);
  const float f = v.x == kNegInf ? v.y : __builtin_amdgcn_exp2f(v.x - m);
  const float l = wave_sum(f * v.y);
  float o[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = 0.0f;
  const float* po = a.part_o + at * a.splits * D + lane * kPer;
  for (int s0 = 0; s0 < parts; s0 += 4) {              // four loads under way
    float x[4][kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = po[(int64_t)min(s0 + i, parts - 1) * D + k];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float fs = __shfl(f, (s0 + i) & (kWave - 1));
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[k] += s0 + i < parts ? fs * x[i][k] : 0.0f;
    }
  }
  store_row(a, true, token, h, 0, lane * kPer, o, m, l, lane == 0);
}

// Each sequence ends with at most one part tile.
int64_t prompt_slots(int64_t Tq, int64_t B, int G, int rows) { return Tq * G / rows + B; }

template <typename S>
void launch_one(const PromptArgs& p, hipStream_t stream) {
  // one slot more, so that some slot is left for the rows behind the last sequence
  const int64_t slots = prompt_slots(p.Tq, p.B, p.NHq / p.NKV, S::kBlockRows) + (p.zero_tail ? 1 : 0);
  const int64_t groups = slots * p.NKV * p.splits;
  prompt_attention_kernel<S><<<dim3((unsigned)((groups + 7) / 8 * 8)), dim3(S::kThreads), S::kLds, stream>>>(
      p, (int)slots);
}

// Workgroups of 256, 128 and 64 rows.
template <int D>
using Rows256 = Shape<D, 8, 4>;
template <int D>
using Rows128 = Shape<D, D == 192 ? 4 : 8, 4, D == 192 ? 1 : 2>;
template <int D>
using Rows64 = Shape<D, 4, 4, 2>;
// 128 rows, with tiles of 32 keys: two workgroups on a compute unit (four at D
// = 64), so that the beginning and end of one run beside the others' products.
template <int D>
using Short128 = Shape<D, 4, 4, 1, 32>;

template <typename S>
hipError_t prepare_one() {
  return prepare_kernel(reinterpret_cast<const void*>(&prompt_attention_kernel<S>), S::kLds);
}
template <int D>
hipError_t prepare_head() {
  hipError_t e = prepare_one<Rows256<D>>();
  if (e == hipSuccess) e = prepare_kernel(reinterpret_cast<const void*>(&prompt_join_kernel<Rows256<D>>), 0);
  if constexpr (D < 256) {
    if (e == hipSuccess) e = prepare_one<Rows128<D>>();
  }
  if constexpr (D <= 128) {
    if (e == hipSuccess) e = prepare_one<Rows64<D>>();
    if (e == hipSuccess) e = prepare_one<Short128<D>>();
  }
  return e;
}

// Where the keys are not split, the fewest rows a workgroup that leave the rows
// in one round of the 256 compute units (two workgroups each at D = 64): the
// waves that the rows do not need share a tile's keys, so that the chain of
// tiles, which is the time then, has shorter links.  256, 128 and 64 rows, one
// sequence, 16 heads over 4 of 128: 512 tokens 20.0, 16.2, 13.6 us; 1024 tokens
// 31.8, 24.5, 21.7 us; 2048 tokens, where 64 rows take two rounds, 55.7, 41.2,
// 45.1 us; 8 x 1024 tokens (two rounds of 128) 65.9, 75.6, 106 us; D = 64, 2048
// tokens 38.6, 28.6, 24.6 us.  D = 192 has tiles of 32 keys, which do not divide
// (256 tokens, 256 and 128 rows: 18.2, 13.6 us), and 128 rows of D = 256 spill
// (1024 tokens: 37 and 41 us).
//
// More rows whose sequences have few keys (8 D on average; at D = 64 also where
// they take less than a second round) do not lose to the smaller tiles what they
// win at their beginnings and ends.  Short128 against 256 rows, 32 heads over 8
// of 128: 64 x 128 tokens 42 and 59 us, 32 x 256 51 and 66 us; 16 over 4: 16 x
// 1024 tokens 108 and 114 us, 3 x 1500 48 and 45 us, 8192 tokens 555 and 510 us;
// D = 64: 6 x 1024 tokens 33 and 37 us, 32 x 256 28 and 31 us, 8 x 1024 45 and
// 42 us.
template <int D>
void launch_head(const PromptArgs& p, hipStream_t stream) {
  const int64_t round = D == 64 ? 512 : 256, rows = p.Tq * p.NHq;
  if constexpr (D <= 128) {
    if (p.splits == 1 && rows <= round * Rows64<D>::kBlockRows) return launch_one<Rows64<D>>(p, stream);
  }
  if constexpr (D < 256) {
    if (p.splits == 1 && rows <= round * Rows128<D>::kBlockRows) return launch_one<Rows128<D>>(p, stream);
  }
  if constexpr (D <= 128) {
    const bool few_keys = p.Tk <= (int64_t)p.B * 8 * D || (D == 64 && rows < 2 * round * Short128<D>::kBlockRows);
    if (p.splits == 1 && few_keys) return launch_one<Short128<D>>(p, stream);
  }
  launch_one<Rows256<D>>(p, stream);
  if (p.splits > 1)
    prompt_join_kernel<Rows256<D>><<<dim3((unsigned)((p.Tq * p.NHq + 3) / 4)), dim3(256), 0, stream>>>(p);
}

}  // namespace

hipError_t prepare_prompt_kernels() {
  hipError_t e = prepare_head<64>();
  if (e == hipSuccess) e = prepare_head<128>();
  if (e == hipSuccess) e = prepare_head<192>();
  if (e == hipSuccess) e = prepare_head<256>();
  return e;
}

// Splits of the keys, where 256 rows a workgroup leave compute units without
// work: as many as fill them, each with kLeast tiles if a sequence had all the
// keys, and as the estimate of the time takes least, in us: a tile of a
// workgroup of 256 rows, a second launch, and the parts' way to memory and back
// at 4.5 TB/s.  None where the tiles of the workgroup of fewest rows, one after
// the other, take less than that.  Measured, whole and split, us: 1 query over
// 4096 keys, 16 heads over 2 of 128, 60.2 and 13.5; 256 queries over 4096 keys,
// 16 over 4, 62.3 and 30.1; 1024 over 8192, 8 over 1, 120 and 57; 2048 over 2048,
// 8 over 1, 35.2 and 41.2; 700 over 1500, 16 over 2, 27.9 and 32.4.
int prompt_splits(int64_t Tq, int64_t Tk, int64_t B, int NHq, int NKV, int D) {
  if (B == 0 || Tq == 0) return 1;
  const int64_t units = prompt_slots(Tq, B, NHq / NKV, Rows256<64>::kBlockRows) * NKV;
  const int64_t tiles = Tk / (D <= 128 ? 64 : 32);
  const int64_t most = std::min<int64_t>(std::min(256 / units, tiles / kLeast), kMaxSplits);
  const double whole = D == 64 ? 0.54 : (D == 128 ? 0.88 : (D == 192 ? 0.86 : 1.58));   // us a tile
  const double tile = D == 64 ? 1.0 : (D == 128 ? 1.5 : (D == 192 ? 1.16 : 1.58));
  const double part = (double)Tq * NHq * D * 8 / 4.5e6, launch = 6.0;
  double best = (double)tiles * whole;
  int splits = 1;
  for (int s = 2; s <= most; ++s) {
    const double us = tiles * tile / s + launch + s * part;
    if (us < best) {
      best = us;
      splits = s;
    }
  }
  return splits;
}

size_t prompt_workspace(int64_t Tq, int NHq, int D, int splits) {
  return splits > 1 ? (size_t)Tq * NHq * splits * (D * sizeof(float) + sizeof(float2)) : 0;
}

hipError_t launch_prompt_attention(PromptArgs p, void* workspace, hipStream_t stream) {
  p.G = p.NHq / p.NKV;
  p.xcd_shift = p.NKV == 1 ? 3 : (p.NKV == 2 ? 2 : (p.NKV == 4 ? 1 : (p.NKV == 8 ? 0 : -1)));
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.Tq * p.NHq * p.splits * p.D);
  switch (p.D) {
    case 64: launch_head<64>(p, stream); break;
    case 128: launch_head<128>(p, stream); break;
    case 192: launch_head<192>(p, stream); break;
    default: launch_head<256>(p, stream); break;
  }
  return hipGetLastError();
}

}  // namespace moe
