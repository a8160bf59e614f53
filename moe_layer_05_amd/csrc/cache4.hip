// Keys and values quantised as they enter the paged 4-bit cache, and read
// back (layout and codes: cache4_device.hpp).
//
// A workgroup takes 16 consecutive packed tokens of one or four kv heads:
// 16 * D / 8 threads, each 8 features of one token's key and value (one
// 16-byte load or store each, one word of codes each); four neighbouring lanes
// share a group of 32 and find its largest magnitude by two lane swaps.  Each
// thread finds its token's sequence by a binary search of cu_seqlens and its
// page in the block table, so ragged batches need no plan made on the host.  A
// place is
// used only if its position is not negative, lies in the table's columns and
// its page id names a page of the cache: other tokens are skipped by a write
// and read as zeros, and no address is formed from them.
//
// HBM-bound: 2 * 2 * D bytes of bfloat16 and 17 * D / 16 of cache a token and
// head.  The bfloat16 side is many times the L2 and goes past it, which leaves
// the L2 to the cache's lines, whose parts come from several waves.  Measured,
// 8 ragged sequences of up to 4096 tokens, 8 heads of 128 (116 MB each way):
// write 27 us = 4.2 TB/s, read 19 us = 6.0 TB/s (through the L2 31 and 28 us;
// one head a workgroup and neighbours on different XCDs 35 and 38 us).
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

// The place of packed token t for kv head 0; head h's tile is h * page_tiles
// tiles further on.
__device__ __forceinline__ Place place_of(const Cache4& c, const CachePlaces& at, int64_t t) {
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
  p.tile = cache4_tile(c, page, 0, (int)(tile - column * c.page_tiles));
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

// Workgroup of the grid (chunks of 16 tokens) x (groups of HEADS kv heads):
// each XCD takes a contiguous range of chunks, so that neighbours, which share
// a tile where a sequence does not start on one, meet in one L2.
struct Work {
  int64_t t;       // this thread's token
  int j;           // its features 8j .. 8j + 7
  int h0;          // first kv head
};
template <int HEADS>
__device__ __forceinline__ Work work_of(int D, int chunks, int per_xcd) {
  const int64_t i = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const int group = (int)(i / chunks), chunk = (int)(i - (int64_t)group * chunks);
  const int d8 = D >> 3;
  return Work{(int64_t)chunk * kTileTokens + threadIdx.x / d8, (int)(threadIdx.x % d8), group * HEADS};
}

template <int HEADS>
__global__ void cache4_write_kernel(Cache4 c, CachePlaces at, const uint4* k, int64_t k_stride8,
                                    const uint4* v, int64_t v_stride8, int chunks, int per_xcd) {
  const Work w = work_of<HEADS>(c.D, chunks, per_xcd);
  if (w.h0 >= c.NKV) return;                           // uniform
  const int D = c.D, d8 = D >> 3, j = w.j;
  uint4 kq[HEADS], vq[HEADS];
  Place p{nullptr, 0, true};
#pragma unroll
  for (int i = 0; i < HEADS; ++i) kq[i] = vq[i] = make_uint4(0, 0, 0, 0);
  if (w.t < at.T) {
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      kq[i] = load_stream(k + (w.t * k_stride8 + (int64_t)(w.h0 + i) * d8 + j));
      vq[i] = load_stream(v + (w.t * v_stride8 + (int64_t)(w.h0 + i) * d8 + j));
    }
    p = place_of(c, at, w.t);
  }
  bool wide;
  const int v_at = v_code_offset(D, j, p.token, &wide);
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    uint32_t kb, vb;
    const uint32_t kc = quantise(kq[i], &kb), vc = quantise(vq[i], &vb);
    if (!p.tile) continue;
    uint8_t* tile = p.tile + (int64_t)(w.h0 + i) * c.page_tiles * cache4_tile_bytes(D);
    *reinterpret_cast<uint32_t*>(tile + p.token * (D / 2) + 4 * j) = kc;
    if (wide) {
      *reinterpret_cast<uint32_t*>(tile + v_at) = vc;
    } else {
      *reinterpret_cast<uint16_t*>(tile + v_at) = (uint16_t)vc;
      *reinterpret_cast<uint16_t*>(tile + v_at + kV64Step) = (uint16_t)(vc >> 16);
    }
    if ((j & 3) == 0) {
      tile[cache4_k_scales(D) + p.token * (D / 32) + (j >> 2)] = (uint8_t)kb;
      tile[v_scale_offset(D, j >> 2, p.token)] = (uint8_t)vb;
    }
  }
}

template <int HEADS>
__global__ void cache4_read_kernel(Cache4 c, CachePlaces at, uint4* k, int64_t k_stride8,
                                   uint4* v, int64_t v_stride8, int zero_tail, int chunks, int per_xcd) {
  const Work w = work_of<HEADS>(c.D, chunks, per_xcd);
  if (w.h0 >= c.NKV || w.t >= at.T) return;
  const int D = c.D, d8 = D >> 3, j = w.j;
  const Place p = place_of(c, at, w.t);
  if (p.behind && !zero_tail) return;
  bool wide;
  const int v_at = v_code_offset(D, j, p.token, &wide);
  uint32_t kc[HEADS], vc[HEADS];
  uint8_t kb[HEADS], vb[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    kc[i] = vc[i] = 0;
    kb[i] = vb[i] = 0;
    if (p.tile) {
      const uint8_t* tile = p.tile + (int64_t)(w.h0 + i) * c.page_tiles * cache4_tile_bytes(D);
      kc[i] = *reinterpret_cast<const uint32_t*>(tile + p.token * (D / 2) + 4 * j);
      if (wide) vc[i] = *reinterpret_cast<const uint32_t*>(tile + v_at);
      else vc[i] = *reinterpret_cast<const uint16_t*>(tile + v_at) |
                   (uint32_t)*reinterpret_cast<const uint16_t*>(tile + v_at + kV64Step) << 16;
      kb[i] = tile[cache4_k_scales(D) + p.token * (D / 32) + (j >> 2)];
      vb[i] = tile[v_scale_offset(D, j >> 2, p.token)];
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    store_stream(k + (w.t * k_stride8 + (int64_t)(w.h0 + i) * d8 + j), fp4_unpack8(kc[i], cache4_scale(kb[i])));
    store_stream(v + (w.t * v_stride8 + (int64_t)(w.h0 + i) * d8 + j), fp4_unpack8(vc[i], cache4_scale(vb[i])));
  }
}

// kv heads of a workgroup: four share a token's search and page where that
// leaves 8 workgroups for every compute unit (4 x 1000 tokens, 4 heads of 192:
// one head 8.9 and 8.0 us, four 9.7 and 9.2 us; above, the figures at the top).
int heads_of(const Cache4& c, const CachePlaces& at) {
  const int64_t chunks = (at.T + kTileTokens - 1) / kTileTokens;
  return c.NKV % 4 == 0 && chunks * (c.NKV / 4) >= 2048 ? 4 : 1;
}
struct Grid {
  int chunks, per_xcd;
  dim3 grid() const { return dim3((unsigned)(8 * (int64_t)per_xcd)); }
};
Grid cache_grid(const Cache4& c, const CachePlaces& at, int heads) {
  const int64_t chunks = (at.T + kTileTokens - 1) / kTileTokens;
  return Grid{(int)chunks, (int)((chunks * (c.NKV / heads) + 7) / 8)};
}

}  // namespace

hipError_t prepare_cache4_kernels() {
  const void* fns[] = {reinterpret_cast<const void*>(&cache4_write_kernel<1>),
                       reinterpret_cast<const void*>(&cache4_write_kernel<4>),
                       reinterpret_cast<const void*>(&cache4_read_kernel<1>),
                       reinterpret_cast<const void*>(&cache4_read_kernel<4>)};
  for (const void* f : fns) {
    const hipError_t e = prepare_kernel(f, 0);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_cache4_write(const Cache4& c, const CachePlaces& at, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride,
                               hipStream_t stream) {
  const int heads = heads_of(c, at);
  const Grid g = cache_grid(c, at, heads);
  const auto kernel = heads == 4 ? cache4_write_kernel<4> : cache4_write_kernel<1>;
  kernel<<<g.grid(), dim3(2 * c.D), 0, stream>>>(c, at, static_cast<const uint4*>(k), k_stride / 8,
                                                 static_cast<const uint4*>(v), v_stride / 8, g.chunks, g.per_xcd);
  return hipGetLastError();
}

hipError_t launch_cache4_read(const Cache4& c, const CachePlaces& at, void* k, int64_t k_stride,
                              void* v, int64_t v_stride, bool zero_tail, hipStream_t stream) {
  const int heads = heads_of(c, at);
  const Grid g = cache_grid(c, at, heads);
  const auto kernel = heads == 4 ? cache4_read_kernel<4> : cache4_read_kernel<1>;
  kernel<<<g.grid(), dim3(2 * c.D), 0, stream>>>(c, at, static_cast<uint4*>(k), k_stride / 8,
                                                 static_cast<uint4*>(v), v_stride / 8, zero_tail, g.chunks, g.per_xcd);
  return hipGetLastError();
}

}  // namespace moe
