// Keys and values quantised as they enter the paged 4-bit cache, and read
// back (layout and codes: cache4_device.hpp).
//
// A workgroup takes 16 consecutive packed tokens of one kv head: 16 * D / 8
// threads, each 8 features of one token's key and value (one 16-byte load or
// store each, one word of codes each); four neighbouring lanes share a group
// of 32 and find its largest magnitude by two lane swaps.  Each thread finds
// its token's sequence by a binary search of cu_seqlens and its page in the
// block table, so ragged batches need no plan made on the host.  A place is
// used only if its position is not negative, lies in the table's columns and
// its page id names a page of the cache: other tokens are skipped by a write
// and read as zeros, and no address is formed from them.  HBM-bound.
#include "cache4_device.hpp"

namespace moe {
namespace {

// Sequence of packed token t: the last b with cu[b] <= t (empty sequences
// share their start with the next one and are passed over); -1 behind the
// last sequence or before the first.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
  if (t < cu[0] || t >= cu[B]) return -1;
  int lo = 0, hi = B;                       // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Place {
  uint8_t* tile;   // null: no place in the cache
  int token;       // 0..15 in the tile
  bool behind;     // behind the last sequence
};

__device__ __forceinline__ Place place_of(const Cache4& c, const CachePlaces& at, int64_t t,
                                          int h) {
  Place p{nullptr, 0, true};
  int b = (int)t;
  int64_t pos = 0;
  if (at.cu) {
    b = sequence_of(at.cu, at.B, t);
    if (b < 0) return p;
    pos = t - at.cu[b];
  }
  p.behind = false;
  pos += at.start[b];
  if (pos < 0) return p;
  const int64_t tile = pos / kTileTokens;
  const int64_t column = tile / c.page_tiles;
  if (column >= at.max_pages) return p;
  const int page = at.table[b * at.table_stride + column];
  if (page < 0 || page >= c.num_pages) return p;
  p.tile = cache4_tile(c, page, h, (int)(tile - column * c.page_tiles));
  p.token = (int)(pos % kTileTokens);
  return p;
}

// Byte offset of the V codes of features 8j .. 8j + 7 of a token: one word,
// or, in a last chunk of 64 features, two half words kV64Step apart.
constexpr int kV64Step = 8;
__device__ __forceinline__ int v_code_offset(int D, int j, int token, bool* wide) {
  const int f0 = 8 * j, chunk = f0 / 128;
  *wide = (chunk + 1) * 128 <= D;
  const int quad = token >> 2, i = token & 3;
  return cache4_v_codes(D) + chunk * 1024 +
         (*wide ? ((quad * 16 + (f0 % 128) / 8) * 4 + i) * 4
                : ((quad * 16 + (f0 % 128) / 4) * 4 + i) * 2);
}

__device__ __forceinline__ int v_scale_offset(int D, int group, int token) {
  return cache4_v_scales(D) + ((token >> 2) * (D / 32) + group) * 4 + (token & 3);
}

// Quantises eight values; every lane of the group of four takes part.
__device__ __forceinline__ uint32_t quantise(const uint4& q, uint32_t* byte) {
  float v[8] = {bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y),
                bf16_lo(q.z), bf16_hi(q.z), bf16_lo(q.w), bf16_hi(q.w)};
  // magnitudes as integers: NaN and infinity order above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, dpp::move<dpp::kSwap1, 0xF>(m));
  m = max(m, dpp::move<dpp::kSwap2, 0xF>(m));
  *byte = cache4_scale_byte(m);
  return fp4_pack8(v, cache4_scale(*byte == 255u ? 127u : *byte));
}

__global__ void cache4_write_kernel(Cache4 c, CachePlaces at, const uint4* k, int64_t k_stride8,
                                    const uint4* v, int64_t v_stride8) {
  const int d8 = c.D >> 3;
  const int j = threadIdx.x % d8;
  const int64_t t = (int64_t)blockIdx.x * kTileTokens + threadIdx.x / d8;
  const int h = blockIdx.y;
  uint4 kq = make_uint4(0, 0, 0, 0), vq = kq;
  Place p{nullptr, 0, true};
  if (t < at.T) {
    kq = k[t * k_stride8 + (int64_t)h * d8 + j];
    vq = v[t * v_stride8 + (int64_t)h * d8 + j];
    p = place_of(c, at, t, h);
  }
  uint32_t kb, vb;
  const uint32_t kc = quantise(kq, &kb), vc = quantise(vq, &vb);
  if (!p.tile) return;
  const int D = c.D;
  *reinterpret_cast<uint32_t*>(p.tile + p.token * (D / 2) + 4 * j) = kc;
  bool wide;
  uint8_t* vp = p.tile + v_code_offset(D, j, p.token, &wide);
  if (wide) {
    *reinterpret_cast<uint32_t*>(vp) = vc;
  } else {
    *reinterpret_cast<uint16_t*>(vp) = (uint16_t)vc;
    *reinterpret_cast<uint16_t*>(vp + kV64Step) = (uint16_t)(vc >> 16);
  }
  if ((j & 3) == 0) {
    p.tile[cache4_k_scales(D) + p.token * (D / 32) + (j >> 2)] = (uint8_t)kb;
    p.tile[v_scale_offset(D, j >> 2, p.token)] = (uint8_t)vb;
  }
}

__global__ void cache4_read_kernel(Cache4 c, CachePlaces at, uint4* k, int64_t k_stride8,
                                   uint4* v, int64_t v_stride8, int zero_tail) {
  const int d8 = c.D >> 3;
  const int j = threadIdx.x % d8;
  const int64_t t = (int64_t)blockIdx.x * kTileTokens + threadIdx.x / d8;
  const int h = blockIdx.y;
  if (t >= at.T) return;
  const Place p = place_of(c, at, t, h);
  if (p.behind && !zero_tail) return;
  uint4 kq = make_uint4(0, 0, 0, 0), vq = kq;
  if (p.tile) {
    const int D = c.D;
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(p.tile + p.token * (D / 2) + 4 * j);
    bool wide;
    const uint8_t* vp = p.tile + v_code_offset(D, j, p.token, &wide);
    uint32_t vc;
    if (wide) vc = *reinterpret_cast<const uint32_t*>(vp);
    else vc = *reinterpret_cast<const uint16_t*>(vp) |
              (uint32_t)*reinterpret_cast<const uint16_t*>(vp + kV64Step) << 16;
    kq = fp4_unpack8(kc, cache4_scale(p.tile[cache4_k_scales(D) + p.token * (D / 32) + (j >> 2)]));
    vq = fp4_unpack8(vc, cache4_scale(p.tile[v_scale_offset(D, j >> 2, p.token)]));
  }
  k[t * k_stride8 + (int64_t)h * d8 + j] = kq;
  v[t * v_stride8 + (int64_t)h * d8 + j] = vq;
}

dim3 cache_grid(const Cache4& c, const CachePlaces& at) {
  return dim3((unsigned)((at.T + kTileTokens - 1) / kTileTokens), (unsigned)c.NKV);
}

}  // namespace

hipError_t prepare_cache4_kernels() {
  hipError_t e = prepare_kernel(reinterpret_cast<const void*>(&cache4_write_kernel), 0);
  if (e == hipSuccess) e = prepare_kernel(reinterpret_cast<const void*>(&cache4_read_kernel), 0);
  return e;
}

hipError_t launch_cache4_write(const Cache4& c, const CachePlaces& at, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride,
                               hipStream_t stream) {
  cache4_write_kernel<<<cache_grid(c, at), dim3(2 * c.D), 0, stream>>>(
      c, at, static_cast<const uint4*>(k), k_stride / 8, static_cast<const uint4*>(v),
      v_stride / 8);
  return hipGetLastError();
}

hipError_t launch_cache4_read(const Cache4& c, const CachePlaces& at, void* k, int64_t k_stride,
                              void* v, int64_t v_stride, bool zero_tail, hipStream_t stream) {
  cache4_read_kernel<<<cache_grid(c, at), dim3(2 * c.D), 0, stream>>>(
      c, at, static_cast<uint4*>(k), k_stride / 8, static_cast<uint4*>(v), v_stride / 8,
      zero_tail);
  return hipGetLastError();
}

}  // namespace moe
