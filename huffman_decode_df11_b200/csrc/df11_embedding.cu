// df11_embedding.cu -- the token embedding on a compressed table: lookup of
// rows, and the table's gradient.
//
// Lookup (df11_decode_embedding): out[t] = scale * W[ids[t]].  The table is an
// ordinary compressed tensor, row-major; only the chunks that hold a row are
// decoded.  A warp takes a segment of a token's row: it finds the format block
// that holds the segment's first element (the positions are close to even, so
// 32 probes around the proportional guess nearly always hold it), the chunk in
// it from the chunk counts, and walks 32 chunks at a time, one per lane, as the
// decode kernel does.  Many short rows take a part of a warp each (launch_lookup).
//
// It reads a fraction of the table and writes the rows.  What bounds it is the walk, as
// in the decode kernels: 8192 rows of 4096 in 42 us, 0.8 weights per ns, where decoding
// all of a tensor gives 1.35, since a row begins and ends inside a chunk and a warp has to
// find its place first.  Four rows: 6 us, one pass over the chain of dependent loads.
//
// Gradient (df11_embedding_gradient): dW[v] = scale * sum of grad[t] over the
// tokens t with ids[t] = v.  The tokens are sorted by id (a stable radix sort by one
// cluster of thread blocks), so a row's tokens are a run of the sorted list.  The
// list is cut into equal pieces; a thread block sums the runs of its piece, and
// a run that crosses pieces is put together by a second kernel from the pieces'
// partial sums, in order: nothing depends on scheduling, and a token that
// half of the batch shares costs no more than any other.
//   It reads the gradients once and writes the whole table: bound by memory for a large table
// (151936 x 4096 in BF16 and 32768 tokens: 254 us, 92% of the copy bandwidth), so the
// zeros are written beside the steps that wait for latency, the sort and the join.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "df11.h"
#include "df11_device.cuh"
#include "df11_device_check.h"
#include "df11_launch.h"

using namespace df11_internal;

namespace {

constexpr int kT = 256;
constexpr int kWarps = 8;

// fp32 to BF16, to nearest, ties to even; NaN stays NaN
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// two BF16 products, rounded once: what the fp32 product is rounded to, which is exact from 2^-134
// on (16 bits above 2^-149), and below gives zero like this
__device__ __forceinline__ uint32_t bf16_product(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// ---- lookup -------------------------------------------------------------------

struct EmbedArgs {
  KTensor k;
  const void *ids;
  void *out;
  int32_t *err;
  uint64_t out_stride;
  uint32_t tokens, rows, dim;
  uint32_t segs, seg_len;   // a row's segments, and elements per segment
  uint32_t ids64, out_f32, scaled;
  float scale;
  uint32_t scale2;          // the scale twice in BF16 where it is a BF16 value, or 0
  uint32_t vec;             // rows of 16-element groups on 16-byte boundaries
  uint32_t region_bytes;
  uint32_t spin_limit;
};

__device__ __forceinline__ float scaled_value(const EmbedArgs &a, uint32_t bits) {
  const float v = __uint_as_float(bits << 16);
  return a.scaled ? v * a.scale : v;
}

__device__ __forceinline__ void embed_store(const EmbedArgs &a, size_t i, uint32_t bits) {
  if (a.out_f32) static_cast<float *>(a.out)[i] = scaled_value(a, bits);
  else static_cast<uint16_t *>(a.out)[i] =
      (uint16_t)(a.scaled ? bf16_bits(scaled_value(a, bits)) : bits);
}

// the last format block whose first element is at or before element e, and that element
__device__ __forceinline__ uint32_t find_block(const KTensor &k, uint32_t e, int lane, uint32_t &at) {
  const uint32_t guess = (uint32_t)((uint64_t)e * k.num_blocks / k.n);
  const uint32_t lo = guess > 15u ? guess - 15u : 0u;
  const uint32_t i = lo + (uint32_t)lane;
  const uint32_t v = i < k.num_blocks ? __ldg(k.block_out_pos + i) : 0xFFFFFFFFu;
  const uint32_t m = __ballot_sync(0xFFFFFFFFu, i < k.num_blocks && v <= e);
  const bool below = m == 0, above = m == 0xFFFFFFFFu && lo + 32u < k.num_blocks;
  if (!below && !above) {
    const int last = 31 - __clz(m);
    at = __shfl_sync(0xFFFFFFFFu, v, last);
    return lo + (uint32_t)last;
  }
  uint32_t first = below ? 0u : lo + 31u, last = below ? lo + 1u : k.num_blocks;
  while (last - first > 1u) {
    const uint32_t mid = first + ((last - first) >> 1);
    if (__ldg(k.block_out_pos + mid) <= e) first = mid;
    else last = mid;
  }
  at = __ldg(k.block_out_pos + first);
  return first;
}

// The same by one lane: a bracket of 32 blocks around the proportional guess where it holds
// the element, halved.
__device__ __forceinline__ uint32_t find_block_alone(const KTensor &k, uint32_t e, uint32_t &at) {
  const uint32_t guess = (uint32_t)((uint64_t)e * k.num_blocks / k.n);
  uint32_t first = guess > 15u ? guess - 15u : 0u, last = min(first + 32u, k.num_blocks);
  if (first && __ldg(k.block_out_pos + first) > e) first = 0;
  if (last < k.num_blocks && __ldg(k.block_out_pos + last) <= e) last = k.num_blocks;
  while (last - first > 1u) {
    const uint32_t mid = first + ((last - first) >> 1);
    if (__ldg(k.block_out_pos + mid) <= e) first = mid;
    else last = mid;
  }
  at = __ldg(k.block_out_pos + first);
  return first;
}

// What a lane needs of its chunk: the codewords that start in it, its words and the next one
// (as they are in memory), and the gap fields of it and the next one from bit 31 down.
template <int C>
struct Chunk {
  uint32_t cnt, gaps, w[C / 4 + 1];
  __device__ __forceinline__ void load(const KTensor &k, uint64_t chunk) {
    constexpr int NW = C / 4 + 1;
    cnt = gaps = 0;
    if (chunk >= (uint64_t)k.num_blocks * kT) return;
    cnt = __ldg(k.chunk_counts + chunk);
    const uint2 *q = reinterpret_cast<const uint2 *>(k.bitstream + chunk * C);
#pragma unroll
    for (int j = 0; j < NW / 2; ++j) {
      const uint2 v = __ldg(q + j);
      w[2 * j] = v.x;
      w[2 * j + 1] = v.y;
    }
    w[NW - 1] = __ldg(reinterpret_cast<const uint32_t *>(q + NW / 2));
    const uint64_t bit = 5ull * chunk;
    const uint32_t *g = reinterpret_cast<const uint32_t *>(k.gaps) + (bit >> 5);
    gaps = __funnelshift_l(__byte_perm(__ldg(g + 1), 0, 0x0123), __byte_perm(__ldg(g), 0, 0x0123),
                           (uint32_t)bit);
  }
};

// G lanes per segment: a warp, or for many short rows a part of it, whose rows go side by side.
template <int C, int G>
__global__ void __launch_bounds__(kWarps * 32)
    df11_embedding_kernel(const __grid_constant__ EmbedArgs a) {
  constexpr int NW = C / 4 + 1;
  extern __shared__ __align__(128) uint8_t smem[];
  const KTensor &tk = a.k;
  constexpr int kGroups = 32 / G;  // per warp
  const int tid = threadIdx.x, lane = tid & (G - 1), group = tid / G;
  const uint32_t gm = G == 32 ? 0xFFFFFFFFu : ((1u << (G & 31)) - 1u) << (tid & 31 & ~(G - 1));
  uint8_t *lens_s = smem + kOffLens;
  uint32_t *lut0_s = reinterpret_cast<uint32_t *>(smem + kOffLut0);
  const uint32_t wide = smem_addr(smem + kOffWide);
  uint8_t *region_p = smem + kOffStages + group * a.region_bytes;
  const uint32_t region = smem_addr(region_p);
  const uint32_t tbar = smem_addr(smem);
  if (tid == 0) {
    mbar_init(tbar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_arrive_expect_tx(tbar, DF11_DECODE_TABLE_BYTES);
    bulk_g2s(smem_addr(lens_s), tk.decode_table, DF11_DECODE_TABLE_BYTES, tbar);
  }
  for (uint32_t i = lane; i < a.region_bytes / 16; i += G)
    reinterpret_cast<uint4 *>(region_p)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();  // the barrier is initialised
  pdl_wait();       // the ids may come from the previous kernel, which may read the output
  pdl_launch_dependents();
  bool table = false;
  const uint64_t items = (uint64_t)a.tokens * a.segs;
  for (uint64_t item = blockIdx.x + (uint64_t)gridDim.x * group; item < items;
       item += (uint64_t)gridDim.x * kWarps * kGroups) {
    const uint32_t token = (uint32_t)(item / a.segs), seg = (uint32_t)(item - (uint64_t)token * a.segs);
    // offsets within the segment, since a row's end may be next to 2^32
    const uint32_t c_first = seg * a.seg_len, c_count = min(a.seg_len, a.dim - c_first);
    const int64_t id = a.ids64 ? static_cast<const int64_t *>(a.ids)[token]
                               : static_cast<const int32_t *>(a.ids)[token];
    const size_t out0 = (size_t)token * a.out_stride;
    if (id < 0 || id >= (int64_t)a.rows) {
      if (lane == 0) report(a.err, DF11_DEV_ERR_INDEX);
      for (uint32_t c = lane; c < c_count; c += G) {
        if (a.out_f32) static_cast<float *>(a.out)[out0 + c_first + c] = 0.f;
        else static_cast<uint16_t *>(a.out)[out0 + c_first + c] = 0;
      }
      continue;
    }
    const uint32_t row0 = (uint32_t)id * a.dim;  // elements of a tensor: below 2^32
    const uint32_t e0 = row0 + c_first, e1 = e0 + c_count;
    uint32_t P, chunk0;
    const uint32_t b = G == 32 ? find_block(tk, e0, lane, P) : find_block_alone(tk, e0, P);
    if (P > e0) {  // inconsistent positions
      if (lane == 0) report(a.err, DF11_DEV_ERR_COUNT);
      continue;
    }
    if constexpr (G == 32) {
      // the chunk of block b that holds e0: the last whose first element is at
      // or before it
      const uint2 cv = __ldg(reinterpret_cast<const uint2 *>(tk.chunk_counts + (size_t)b * kT) + lane);
      const uint32_t sum = __dp4a(cv.x, 0x01010101u, __dp4a(cv.y, 0x01010101u, 0u));
      uint32_t incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      const uint32_t off = e0 - P;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, incl - sum <= off);
      const int src = 31 - __clz(m);  // lane 0's count before is 0: m is not 0
      uint32_t before = incl - sum, j = 0;
#pragma unroll
      for (uint32_t i = 0; i < 7; ++i) {
        const uint32_t c = ((i < 4 ? cv.x : cv.y) >> (8 * (i & 3))) & 0xFFu;
        if (j == i && before + c <= off) {
          before += c;
          ++j;
        }
      }
      P += __shfl_sync(0xFFFFFFFFu, before, src);
      chunk0 = b * kT + 8u * src + __shfl_sync(0xFFFFFFFFu, j, src);
    } else {
      // the same, by 16 counts, then 4, then one
      const uint4 *q = reinterpret_cast<const uint4 *>(tk.chunk_counts + (size_t)b * kT);
      const uint32_t off = e0 - P;
      uint32_t before = 0, j = 0;
      uint4 v = __ldg(q);
      auto sum4 = [](uint32_t c) { return __dp4a(c, 0x01010101u, 0u); };
      for (uint32_t i = 0; i < kT / 16 - 1; ++i) {
        const uint32_t sum = sum4(v.x) + sum4(v.y) + sum4(v.z) + sum4(v.w);
        if (before + sum > off) break;
        before += sum;
        j += 16;
        v = __ldg(q + i + 1);
      }
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
      uint32_t c = v.x;
#pragma unroll
      for (uint32_t i = 0; i < 3; ++i) {
        const uint32_t sum = sum4(w4[i]);
        if ((j & 15u) == 4 * i && before + sum <= off) {
          before += sum;
          j += 4;
          c = w4[i + 1];
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < 3; ++i) {
        const uint32_t n = (c >> (8 * i)) & 0xFFu;
        if ((j & 3u) == i && before + n <= off) {
          before += n;
          ++j;
        }
      }
      P += before;
      chunk0 = b * kT + j;
    }
    Chunk<C> next;
    next.load(tk, (uint64_t)chunk0 + lane);
    for (uint64_t c0 = chunk0; P < e1; c0 += G) {
      const uint64_t chunk = c0 + lane;
      Chunk<C> ck = next;
      const uint32_t cnt = ck.cnt;
      uint32_t incl = cnt;
#pragma unroll
      for (int d = 1; d < G; d <<= 1) {
        const uint32_t v = __shfl_up_sync(gm, incl, d, G);
        if (lane >= d) incl += v;
      }
      const uint32_t total = __shfl_sync(gm, incl, G - 1, G);
      if (total == 0 || total > tk.n - P || __any_sync(gm, cnt > tk.max_chunk_elems)) {
        if (lane == 0) report(a.err, DF11_DEV_ERR_COUNT);
        break;
      }
      // the next 32 chunks, and the first sign/mantissa bytes, arrive during the walk
      if (P + total < e1) next.load(tk, chunk + G);
      const uint32_t E = P + incl - cnt, base = P & ~15u;
      const bool need = cnt && E < e1 && E + cnt > e0;
      // elements [lo, hi) past `base` are the row's, element i at byte i of the region
      const uint32_t lo = max(e0, P) - base, hi = min(e1 - base, P - base + total);
      const uint8_t *sm = tk.sign_mantissa + base;
      uint4 sv = make_uint4(0, 0, 0, 0);
      if (a.vec && (lo & ~15u) + 16u * lane < hi)
        sv = __ldg(reinterpret_cast<const uint4 *>(sm + (lo & ~15u)) + lane);
      int start = 0, end = 0, bad = 0;
      uint32_t w[NW];
      if (need) {
#pragma unroll
        for (int j = 0; j < NW; ++j) w[j] = __byte_perm(ck.w[j], 0, 0x0123);
        start = (int)(ck.gaps >> 27);
        end = C * 8 + (int)((ck.gaps >> 22) & 31u);
        const uint64_t bit0 = chunk * (C * 8);
        if (bit0 >= tk.total_bits) start = end = 0;
        else if ((uint64_t)end > tk.total_bits - bit0) end = (int)(tk.total_bits - bit0);
        if (tk.masked) {
#pragma unroll
          for (int j = 0; j < NW; ++j)
            w[j] |= __funnelshift_rc(0xFFFFFFFFu, 0u, (uint32_t)max(end - 32 * j, 0));
        }
      }
      if (!table) {
        table = __all_sync(gm, mbar_wait(tbar, 0, a.spin_limit));
        if (!table) {
          if (lane == 0) report(a.err, DF11_DEV_ERR_TIMEOUT);
          break;
        }
      }
      if (need) {
        const uint32_t d = E - base;
        uint32_t got;
        if (tk.masked) {
          got = decode_counted<C>(w, start, end, wide, lut0_s, lens_s, tk.luts + 256, tk.num_luts,
                                  region, d, cnt, bad);
        } else {
          got = decode_direct<kT, C, false>(w, start, end, wide, lut0_s, lens_s, tk.luts + 256,
                                            tk.num_luts, region, d, region + ((d + cnt - 1u) & ~3u),
                                            bad);
        }
        if (!bad && got != cnt) bad = DF11_DEV_ERR_COUNT;
        if (bad) report(a.err, bad);
      }
      __syncwarp(gm);
      const size_t out_base = out0 + base - row0;  // may wrap below the row: base is before it
      if (a.vec) {
        for (uint32_t i = (lo & ~15u) + 16u * lane; i < hi; i += 16u * G) {
          const uint4 rv = lds128(region + i);
          const uint4 cur = sv;  // the next group's bytes ahead
          if (i + 16u * G < hi) sv = __ldg(reinterpret_cast<const uint4 *>(sm + i + 16u * G));
          const uint2 p0 = fuse4(cur.x, rv.x), p1 = fuse4(cur.y, rv.y);
          const uint2 p2 = fuse4(cur.z, rv.z), p3 = fuse4(cur.w, rv.w);
          const uint32_t u[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
          const size_t o = out_base + i;
          if (i >= lo && i + 16u <= hi) {
            if (a.out_f32) {
              float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                q[j] = make_float4(scaled_value(a, u[2 * j] & 0xFFFFu), scaled_value(a, u[2 * j] >> 16),
                                   scaled_value(a, u[2 * j + 1] & 0xFFFFu),
                                   scaled_value(a, u[2 * j + 1] >> 16));
            } else {
              uint32_t r[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                r[j] = !a.scaled ? u[j]
                       : a.scale2
                           ? bf16_product(u[j], a.scale2)
                           : bf16_pair(scaled_value(a, u[j] & 0xFFFFu), scaled_value(a, u[j] >> 16));
              uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + o);
              q[0] = make_uint4(r[0], r[1], r[2], r[3]);
              q[1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
          } else {  // a group that two passes share
#pragma unroll
            for (uint32_t j = 0; j < 16; ++j)
              if (i + j >= lo && i + j < hi)
                embed_store(a, o + j, (u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
          }
        }
      } else {
        constexpr uint32_t kAhead = 8;  // loads before the first store
        for (uint32_t i = lo + lane; i < hi; i += G * kAhead) {
          uint32_t v[kAhead];
#pragma unroll
          for (uint32_t j = 0; j < kAhead; ++j) v[j] = i + G * j < hi ? __ldg(sm + i + G * j) : 0u;
#pragma unroll
          for (uint32_t j = 0; j < kAhead; ++j)
            if (i + G * j < hi)
              embed_store(a, out_base + i + G * j, fuse1(v[j], lds8(region + i + G * j)));
        }
      }
      __syncwarp(gm);
      // the region zero again (a walk over corrupt data may write 7 bytes more)
      for (uint32_t i = lane; i < (P - base + total + 8u + 15u) >> 4; i += G)
        sts128_zero(region + 16u * i);
      __syncwarp(gm);
      P += total;
    }
  }
  // the table's copy has landed before the thread block ends
  if (!table && tid == 0 && !mbar_wait(tbar, 0, a.spin_limit)) report(a.err, DF11_DEV_ERR_TIMEOUT);
}

// ---- gradient: sort by token ----------------------------------------------------

constexpr int kSortThreads = 1024, kSortWarps = 32, kMaxDigitBits = 9, kMaxDigits = 512;
constexpr uint32_t kBatch = 4;  // tokens of a lane loaded together

struct SortArgs {
  const void *ids;
  uint32_t *key[2], *tok[2];  // the sorted list ends in [passes & 1]
  uint32_t *crossing;         // [0]: runs that cross pieces, counted by the next kernel
  uint32_t *touched;          // a bit per row that has tokens; NULL: not wanted
  // the clusters after the first set rows zero_from .. rows - 1 of the gradient to zero
  // meanwhile, tokens or not: the last ones of the table, which the fewest tokens have
  void *out;
  uint64_t out_stride;        // in bytes
  uint32_t row_bytes, zero_from, touched_words;
  int32_t *err;
  uint32_t tokens, rows, passes, digit_bits, ids64;
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n"
               " ld.shared::cluster.u32 %0, [a];\n}\n"
               : "=r"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

// the lanes of `active` whose digit is this lane's (a vote per bit: a match instruction takes
// several times as long for 32 different digits)
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, uint32_t bits, uint32_t active) {
  uint32_t peers = active;
  for (uint32_t b = 0; b < bits; ++b) {
    const bool one = (digit >> b) & 1u;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, one);
    peers &= one ? m : ~m;
  }
  return peers;
}

struct SortShared {
  uint32_t whist[kSortWarps][kMaxDigits + 1];  // a column in 32 banks
  uint32_t own[kMaxDigits], base[kMaxDigits], warp_total[kMaxDigits / 32];
};

// Bytes that a thread block of the sort's kernel sets to zero: few enough that clusters
// which find no place at first do not end late, and more than their start costs.
constexpr uint64_t kZeroBytes = 256 * 1024;

// Rows zero_from .. rows - 1 set to zero by thread block `block` of `blocks`, 16 bytes at a
// time where the rows follow one another or start on 16-byte boundaries.
__device__ void zero_rows(const SortArgs &a, uint32_t block, uint32_t blocks) {
  uint8_t *out = static_cast<uint8_t *>(a.out) + (uint64_t)a.zero_from * a.out_stride;
  const uint4 z = make_uint4(0, 0, 0, 0);
  const bool whole = a.out_stride == a.row_bytes;
  const uint64_t n = a.rows - a.zero_from, rows = whole ? 1 : n;
  const uint64_t bytes = whole ? n * a.row_bytes : a.row_bytes;
  const bool vec = (uintptr_t)out % 16 == 0 && (whole || a.out_stride % 16 == 0);
  // a row per thread block, or all of them over one
  const uint64_t first = whole ? (uint64_t)block * kSortThreads + threadIdx.x : threadIdx.x;
  const uint64_t step = whole ? (uint64_t)blocks * kSortThreads : kSortThreads;
  for (uint64_t r = whole ? 0 : block; r < rows; r += whole ? 1 : blocks) {
    uint8_t *p = out + r * a.out_stride;
    const uint64_t quads = vec ? bytes / 16 : 0;
    for (uint64_t i = first; i < quads; i += step) reinterpret_cast<uint4 *>(p)[i] = z;
    for (uint64_t i = quads * 8 + first; i < bytes / 2; i += step)
      reinterpret_cast<uint16_t *>(p)[i] = 0;
  }
}

// The first cluster sorts (id, token) by id, least significant digit first; every
// warp keeps a contiguous part of the list, so equal ids stay in token order.
// An id outside the table sorts behind every row.
__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ SortShared sort_shared[];
  auto &whist = sort_shared->whist;
  auto &own = sort_shared->own;
  auto &base = sort_shared->base;
  auto &warp_total = sort_shared->warp_total;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const uint32_t parts = ctas * kSortWarps;
  const uint64_t per = (((uint64_t)a.tokens + parts - 1) / parts + 31) & ~31ull;
  const uint64_t begin = per * (rank * kSortWarps + warp);
  const uint64_t end = begin + per < a.tokens ? begin + per : a.tokens;
  const uint32_t digits = 1u << a.digit_bits;
  pdl_wait();  // the ids may come from the previous kernel; the workspace may still be read
  if (blockIdx.x >= ctas) {
    zero_rows(a, blockIdx.x - ctas, gridDim.x - ctas);
    pdl_launch_dependents();
    return;  // a whole cluster
  }
  if (rank == 0 && tid == 0) a.crossing[0] = 0;
  if (a.touched)
    for (uint32_t i = rank * kSortThreads + tid; i < a.touched_words; i += ctas * kSortThreads)
      a.touched[i] = 0;
  for (uint32_t p = 0; p < a.passes; ++p) {
    const uint32_t shift = p * a.digit_bits;
    const uint32_t *sk = a.key[p & 1], *st = a.tok[p & 1];
    uint32_t *dk = a.key[(p + 1) & 1], *dt = a.tok[(p + 1) & 1];
    auto load = [&](uint64_t i) -> uint32_t {
      if (p) return __ldcg(sk + i);
      const int64_t id = a.ids64 ? static_cast<const int64_t *>(a.ids)[i]
                                 : static_cast<const int32_t *>(a.ids)[i];
      return id < 0 || id >= (int64_t)a.rows ? a.rows : (uint32_t)id;
    };
    for (uint32_t d = lane; d < digits; d += 32) whist[warp][d] = 0;
    __syncwarp();
    uint32_t held[kBatch];  // the keys of the batch at hand; of the whole part if it has but one
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kBatch) {
#pragma unroll
      for (uint32_t j = 0; j < kBatch; ++j)
        if (i0 + 32 * j + lane < end) held[j] = load(i0 + 32 * j + lane);
#pragma unroll
      for (uint32_t j = 0; j < kBatch; ++j) {
        if (i0 + 32 * j >= end) break;
        const bool act = i0 + 32 * j + lane < end;
        const uint32_t digit = act ? (held[j] >> shift) & (digits - 1u) : 0u;
        const uint32_t peers = same_digit(digit, a.digit_bits, __ballot_sync(0xFFFFFFFFu, act));
        if (act && (peers >> lane) == 1u)  // the last of the peers
          whist[warp][digit] += __popc(peers);
        __syncwarp();
      }
    }
    __syncthreads();
    // per digit, the counts of the warps before and this thread block's: a warp per digit, a
    // lane per warp
    for (uint32_t d = warp; d < digits; d += kSortWarps) {
      const uint32_t v = whist[lane][d];
      uint32_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= (uint32_t)o) incl += u;
      }
      whist[lane][d] = incl - v;
      if (lane == 31) own[d] = incl;
    }
    cluster_sync();
    if (tid < kMaxDigits) {  // where each digit's tokens of this thread block begin
      uint32_t total = 0, before = 0;
      if (tid < digits)
        for (uint32_t r = 0; r < ctas; ++r) {
          const uint32_t v = ld_cluster(smem_addr(&own[tid]), r);
          if (r < rank) before += v;
          total += v;
        }
      uint32_t incl = total;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= (uint32_t)d) incl += v;
      }
      base[tid] = incl - total + before;
      if (lane == 31) warp_total[warp] = incl;
    }
    __syncthreads();
    if (tid < kMaxDigits)
      for (uint32_t w = 0; w < warp; ++w) base[tid] += warp_total[w];
    __syncthreads();
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kBatch) {
      uint32_t tok[kBatch];
#pragma unroll
      for (uint32_t j = 0; j < kBatch; ++j) {
        const uint64_t i = i0 + 32 * j + lane;
        if (i >= end) continue;
        if (per > 32 * kBatch) held[j] = load(i);
        tok[j] = p ? __ldcg(st + i) : (uint32_t)i;
      }
#pragma unroll
      for (uint32_t j = 0; j < kBatch; ++j) {
        if (i0 + 32 * j >= end) break;
        const bool act = i0 + 32 * j + lane < end;
        const uint32_t key = held[j];
        const uint32_t digit = act ? (key >> shift) & (digits - 1u) : 0u;
        const uint32_t peers = same_digit(digit, a.digit_bits, __ballot_sync(0xFFFFFFFFu, act));
        uint32_t at = 0;
        if (act) at = base[digit] + whist[warp][digit] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (act && (peers >> lane) == 1u) whist[warp][digit] += __popc(peers);
        __syncwarp();
        if (act) {
          dk[at] = key;
          dt[at] = tok[j];
        }
      }
    }
    cluster_sync();  // the list is whole, and own[] read by everyone
  }
  // the rows that have tokens, by the first token of each (all tokens' marks would meet at
  // the few words of the commonest rows)
  const uint32_t *sk = a.key[a.passes & 1];
  for (uint64_t i = rank * kSortThreads + tid; i < a.tokens; i += ctas * kSortThreads) {
    const uint32_t key = __ldcg(sk + i);
    if (i && __ldcg(sk + i - 1) == key) continue;
    if (key == a.rows) report(a.err, DF11_DEV_ERR_INDEX);
    else if (a.touched) atomicOr(a.touched + (key >> 5), 1u << (key & 31u));
  }
  pdl_launch_dependents();
}

// ---- gradient: sums of runs -------------------------------------------------------

constexpr int kRunThreads = 128;
constexpr uint32_t kMaxPiece = 32;  // tokens of the sorted list per thread block

struct RunArgs {
  const void *grad;
  void *out;
  const uint32_t *key, *tok;  // sorted
  const uint32_t *touched;    // a bit per row that has tokens
  uint32_t zero_rows, zero_step;  // rows below this without one are set to zero, some per thread block
  uint32_t *crossing;         // their number, then the pieces where runs begin that cross pieces
  float *head, *tail;         // per piece: sums of the run that began before it / that goes on
  uint64_t grad_stride, out_stride;
  uint32_t tokens, rows, dim, piece, pieces, col_tiles, part_stride;
  uint32_t join_blocks;       // thread blocks of the second kernel that put runs together
  uint32_t accumulate;
  float scale;
  int32_t *err;
  uint32_t spin_limit;
};

// V columns of a gradient's row, 16 bytes, or one
template <typename G, int V>
__device__ __forceinline__ void add_row(const uint4 &a, float (&acc)[V]) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(G) == 4) {
      acc[j] += __uint_as_float(u[j]);
    } else {
      acc[2 * j] += bf16_lo(u[j]);
      acc[2 * j + 1] += bf16_hi(u[j]);
    }
  }
}
__device__ __forceinline__ float load_one(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_one(const uint16_t *p) { return bf16_lo(__ldg(p)); }

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_lo(v); }
__device__ __forceinline__ void narrow(float *p, float v) { *p = v; }
__device__ __forceinline__ void narrow(uint16_t *p, float v) { *p = (uint16_t)bf16_bits(v); }

// dW[row], columns col .. col + V - 1: scale * sum, added to what is there or not
template <typename O, int V>
__device__ __forceinline__ void write_row(const RunArgs &a, uint32_t row, uint32_t col,
                                          const float (&s)[V]) {
  O *p = static_cast<O *>(a.out) + (size_t)row * a.out_stride + col;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = s[j] * a.scale;
  if (a.accumulate) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += widen(p[j]);
  }
  if constexpr (V == 1) {
    narrow(p, v[0]);
  } else if constexpr (sizeof(O) == 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4 *>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const uint2 u = make_uint2(bf16_pair(v[j], v[j + 1]), bf16_pair(v[j + 2], v[j + 3]));
      if (V % 8 == 0) {
        if (j % 8) continue;
        *reinterpret_cast<uint4 *>(p + j) = make_uint4(
            u.x, u.y, bf16_pair(v[j + 4], v[j + 5]), bf16_pair(v[j + 6], v[j + 7]));
      } else {
        *reinterpret_cast<uint2 *>(p + j) = u;
      }
    }
  }
}

template <int V>
__device__ __forceinline__ void write_part(float *p, const float (&s)[V]) {
  if constexpr (V == 1) {
    p[0] = s[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4 *>(p + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
  }
}

// A thread block: the runs of one piece of the sorted list, kRunThreads * V columns.  The
// piece's rows are all asked for at once, by bulk copies into shared memory (V > 1), since
// what bounds this is how much is on its way (32768 tokens of 4096 columns in BF16: 67 us,
// with four rows ahead in registers 100); kGroup rows have a barrier.
constexpr uint32_t kGroup = 8;
constexpr uint32_t kRowBytes = 16 * kRunThreads;
template <typename G, typename O, int V>
__global__ void __launch_bounds__(kRunThreads) embedding_runs_kernel(const __grid_constant__ RunArgs a) {
  __shared__ uint32_t key_s[kMaxPiece + 2], tok_s[kMaxPiece];
  __shared__ uint64_t bar_s[kMaxPiece / kGroup];
  extern __shared__ __align__(128) uint8_t rows_s[];
  const uint32_t tid = threadIdx.x, lane = tid & 31;
  const uint32_t piece = blockIdx.x / a.col_tiles, ct = blockIdx.x - piece * a.col_tiles;
  const uint32_t i0 = piece * a.piece, i1 = min(i0 + a.piece, a.tokens), n = i1 - i0;
  const uint32_t bars = smem_addr(bar_s), rows = smem_addr(rows_s);
  if (V > 1 && tid == 0) {
    for (uint32_t i = 0; i < kMaxPiece / kGroup; ++i) mbar_init(bars + 8u * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  // key_s[0]: the key before the piece, then the piece, then the key after it
  // (no row: beyond every key)
  if (tid < n) {
    key_s[tid + 1] = __ldcg(a.key + i0 + tid);
    tok_s[tid] = __ldcg(a.tok + i0 + tid);
  }
  if (tid == 32) key_s[0] = i0 ? __ldcg(a.key + i0 - 1) : 0xFFFFFFFFu;
  if (tid == 33) key_s[n + 1] = i1 < a.tokens ? __ldcg(a.key + i1) : 0xFFFFFFFFu;
  __syncthreads();
  const uint32_t col0 = ct * kRunThreads * V;
  // without the ids outside the table, at the list's end; bit i of `ends`: a run's last token
  const uint32_t valid = __popc(__ballot_sync(0xFFFFFFFFu, lane < n && key_s[lane + 1] < a.rows));
  const uint32_t ends =
      __ballot_sync(0xFFFFFFFFu, lane < n && (lane + 1 == n || key_s[lane + 2] != key_s[lane + 1]));
  if (V > 1 && tid < valid) {
    const uint32_t bytes = min((uint32_t)(kRunThreads * V), a.dim - col0) * (uint32_t)sizeof(G);
    const uint32_t bar = bars + 8u * (tid / kGroup);
    if (tid % kGroup == 0) mbar_arrive_expect_tx(bar, min(kGroup, valid - tid) * bytes);
    __syncwarp(valid == 32 ? 0xFFFFFFFFu : (1u << valid) - 1u);
    bulk_g2s(rows + tid * kRowBytes,
             static_cast<const G *>(a.grad) + (size_t)tok_s[tid] * a.grad_stride + col0, bytes, bar);
  }
  // the piece's last run goes on and began here: the next kernel puts it together (in any
  // order, since every run is by itself)
  if (ct == 0 && tid == 0 && key_s[n] < a.rows && key_s[n + 1] == key_s[n] && key_s[0] != key_s[n])
    a.crossing[1 + atomicAdd(a.crossing, 1u)] = piece;
  const uint32_t col = col0 + tid * V;
  const bool here = col < a.dim;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  bool first = true;  // the current run is the piece's first
  auto end_run = [&](uint32_t i) {
    const uint32_t key = key_s[i + 1];
    const bool before = first && key_s[0] == key, after = key_s[i + 2] == key;
    if (here) {
      if (!before && !after) write_row<O, V>(a, key, col, acc);
      else write_part<V>((before ? a.head : a.tail) + (size_t)piece * a.part_stride + col, acc);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    first = false;
  };
  if constexpr (V > 1) {
    for (uint32_t i = 0; i < valid; i += kGroup) {
      if (!mbar_wait(bars + 8u * (i / kGroup), 0, a.spin_limit)) {
        if (tid == 0) {  // the copies may still come: leave once they have, or not
          report(a.err, DF11_DEV_ERR_TIMEOUT);
          for (uint32_t g = i; g < valid; g += kGroup) mbar_wait(bars + 8u * (g / kGroup), 0, a.spin_limit);
        }
        break;
      }
      const uint32_t at = rows + i * kRowBytes + 16u * tid;
      uint4 v[kGroup];
#pragma unroll
      for (uint32_t u = 0; u < kGroup; ++u)
        if (i + u < valid) v[u] = lds128(at + u * kRowBytes);
#pragma unroll
      for (uint32_t u = 0; u < kGroup; ++u) {
        if (i + u >= valid) break;
        add_row<G, V>(v[u], acc);
        if ((ends >> (i + u)) & 1u) end_run(i + u);
      }
    }
  } else {
    const G *g = static_cast<const G *>(a.grad) + col;
    constexpr uint32_t kAhead = 4;
    for (uint32_t i = 0; i < valid; i += kAhead) {
      float v[kAhead];
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u)
        v[u] = here && i + u < valid ? load_one(g + (size_t)tok_s[i + u] * a.grad_stride) : 0.f;
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) {
        if (i + u >= valid) break;
        acc[0] += v[u];
        if ((ends >> (i + u)) & 1u) end_run(i + u);
      }
    }
  }
}

// Thread blocks below join_blocks: runs that cross pieces.  The tail in the piece where
// a run begins and the heads of the pieces after it, 32 V columns at a time; each of the four
// warps adds every fourth head, and their sums follow the tail in order.
// The others, which write while those wait for their sums: zero_step rows each, those
// without a token set to zero.
constexpr uint32_t kJoinWarps = kRunThreads / 32;
constexpr uint32_t kJoinBlocks = 148 * 12;
constexpr uint64_t kZeroStep = 16 * 1024;
template <typename O, int V>
__global__ void __launch_bounds__(kRunThreads, 12) embedding_join_kernel(const __grid_constant__ RunArgs a) {
  __shared__ uint32_t stop_s[kJoinWarps];
  __shared__ float sums[kJoinWarps][32 * V];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= a.join_blocks) {
    const uint32_t row0 = (blockIdx.x - a.join_blocks) * a.zero_step;
    const uint32_t bits = __ldg(a.touched + (row0 >> 5)) >> (row0 & 31u);
    for (uint32_t r = 0; r < a.zero_step; ++r) {
      const uint32_t row = row0 + r;
      if (row >= a.zero_rows) break;
      if ((bits >> r) & 1u) continue;
      O *p = static_cast<O *>(a.out) + (size_t)row * a.out_stride;
      if constexpr (V == 1) {
        for (uint32_t c = tid; c < a.dim; c += kRunThreads) p[c] = O(0);
      } else {
        constexpr uint32_t per = 16 / sizeof(O);  // dim is a multiple of 8
        for (uint32_t c = tid * per; c < a.dim; c += kRunThreads * per)
          *reinterpret_cast<uint4 *>(p + c) = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const uint32_t tiles = (a.dim + 32 * V - 1) / (32 * V);
  const uint64_t work = (uint64_t)__ldcg(a.crossing) * tiles;
  for (uint64_t u = blockIdx.x; u < work; u += a.join_blocks) {
    const uint32_t piece = __ldcg(a.crossing + 1 + u / tiles), tile = (uint32_t)(u % tiles);
    const uint32_t key = __ldcg(a.key + (piece + 1) * a.piece);
    // the run's last piece: the first one after this whose next token has another key; a
    // piece per thread, until some thread has it
    uint32_t last = piece + 1;
    for (;; last += kRunThreads) {
      const uint64_t e = ((uint64_t)last + tid + 1) * a.piece;  // the token after the piece
      const bool goes_on = e < a.tokens && __ldcg(a.key + e) == key;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, !goes_on);
      if (lane == 0) stop_s[warp] = m ? (tid & ~31u) + __ffs(m) - 1 : kRunThreads;
      __syncthreads();
      uint32_t first = kRunThreads;
#pragma unroll
      for (uint32_t w = 0; w < kJoinWarps; ++w) first = min(first, stop_s[w]);
      __syncthreads();
      if (first < kRunThreads) {
        last += first;
        break;
      }
    }
    const uint32_t col = (tile * 32 + lane) * V;
    float s[V];
    auto load = [&](const float *p, float (&v)[V]) {
      if constexpr (V == 1) {
        v[0] = __ldcg(p);
      } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const float4 q = __ldcg(reinterpret_cast<const float4 *>(p + j));
          v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
        }
      }
    };
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.f;
    if (col < a.dim) {
      constexpr uint32_t kAhead = 4;
      for (uint32_t p = piece + 1 + warp; p <= last; p += kAhead * kJoinWarps) {
        float v[kAhead][V];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k)
          if (p + k * kJoinWarps <= last)
            load(a.head + (size_t)(p + k * kJoinWarps) * a.part_stride + col, v[k]);
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k)
          if (p + k * kJoinWarps <= last) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += v[k][j];
          }
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sums[warp][lane * V + j] = s[j];
    __syncthreads();
    if (warp == 0 && col < a.dim) {
      load(a.tail + (size_t)piece * a.part_stride + col, s);
#pragma unroll
      for (uint32_t w = 0; w < kJoinWarps; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] += sums[w][lane * V + j];
      write_row<O, V>(a, key, col, s);
    }
    __syncthreads();
  }
}

// ---- host side --------------------------------------------------------------------

uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }
bool known_type(int32_t t) { return t == DF11_BF16 || t == DF11_F32; }
uintptr_t type_bytes(int32_t t) { return t == DF11_F32 ? 4 : 2; }

constexpr uint64_t kMaxSegment = 1u << 31;  // elements: loops over a segment's stay below 2^32

// `per_pass`: elements of a row that G chunks hold on average
template <int C, int G>
df11_status launch_embedding(EmbedArgs &a, uint64_t per_pass, int instance, cudaStream_t s) {
  auto kern = df11_embedding_kernel<C, G>;
  // G chunks from any chunk on: first element's offset, elements, the walk's slack
  a.region_bytes = (uint32_t)round_up(15 + (uint64_t)G * a.k.max_chunk_elems + 8, 16);
  const size_t smem = kOffStages + (size_t)kWarps * (32 / G) * a.region_bytes;
  uint64_t budget = 0;
  const df11_status st = prepare(kern, kWarps * 32, smem, instance, budget);
  if (st != DF11_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DF11_ERR_CUDA;
  const uint64_t sms = device_info(dev).sms, groups = kWarps * (32 / G);
  // A row in segments that one pass holds, while there are fewer rows than warps; more of a row
  // per warp otherwise, which then finds its place in the stream once.
  const uint64_t most = (a.dim + per_pass - 1) / per_pass;
  uint64_t segs = budget * groups / a.tokens;
  segs = segs < 1 || G < 32 ? 1 : (segs > most ? most : segs);
  const uint64_t len = round_up((a.dim + segs - 1) / segs, 16);
  a.seg_len = (uint32_t)(len < kMaxSegment ? len : kMaxSegment);
  a.segs = (uint32_t)(((uint64_t)a.dim + a.seg_len - 1) / a.seg_len);
  // every SM, then every warp of a thread block, then more thread blocks per SM
  const uint64_t items = (uint64_t)a.tokens * a.segs;
  uint64_t grid = (items + groups - 1) / groups;
  if (grid < sms) grid = items < sms ? items : sms;
  if (grid > budget) grid = budget;
  return launch_pdl(kern, dim3((uint32_t)grid), kWarps * 32, smem, s, a);
}

// Lanes per row: a warp's 32, unless there are more rows than the device holds warps and a row
// takes a few chunks only (3591 x 64 and 144534 tokens: 28 us with two lanes per row, 226 with a
// warp; 50000 x 256 and 20000 tokens: 18 with eight, 36).
template <int C>
df11_status launch_lookup(EmbedArgs &a, int instance, cudaStream_t s) {
  const uint64_t chunks = (uint64_t)a.k.num_blocks * kT;
  const bool many = a.tokens > 148u * 4 * kWarps;
  // chunks that a row begins in or reaches, 64 times
  const uint64_t row = 64ull * a.dim * chunks / a.k.n + 64;
  if (many && row <= 2 * 64) return launch_embedding<C, 2>(a, 1, instance + 1, s);
  if (many && row <= 4 * 64) return launch_embedding<C, 4>(a, 1, instance + 2, s);
  if (many && row <= 8 * 64) return launch_embedding<C, 8>(a, 1, instance + 3, s);
  if (many && row <= 16 * 64) return launch_embedding<C, 16>(a, 1, instance + 4, s);
  // 32 chunks hold 30 chunks' elements of a row, since it begins and ends inside a chunk
  return launch_embedding<C, 32>(a, 30ull * a.k.n / chunks + 1, instance, s);
}

struct GradPlan {
  uint32_t piece, pieces, col_tiles, part_stride, passes, digit_bits;
  uint64_t key[2], tok[2], touched, crossing, head, tail, bytes;
  int v;  // columns per thread
};

// 16-byte accesses of gradients and table rows, when every row starts on such a
// boundary and holds whole ones
int columns_per_thread(const df11_embedding_grad &op) {
  const uintptr_t gb = type_bytes(op.grad_type), ob = type_bytes(op.out_type);
  const uint32_t v = (uint32_t)(16 / gb);
  const bool ok = op.dim % 8 == 0 && aligned(op.grad, 16) && aligned(op.out, 16) &&
                  op.grad_stride * gb % 16 == 0 && op.out_stride * ob % 16 == 0;
  return ok ? (int)v : 1;
}

GradPlan grad_plan(const df11_embedding_grad &op) {
  GradPlan p{};
  p.v = columns_per_thread(op);
  p.col_tiles = (uint32_t)((op.dim + kRunThreads * p.v - 1) / (kRunThreads * p.v));
  // pieces of 32 tokens, shorter ones while that leaves SMs without work
  p.piece = kMaxPiece;
  while (p.piece > 4 && (uint64_t)op.tokens * p.col_tiles / p.piece < 592) p.piece /= 2;
  p.pieces = (op.tokens + p.piece - 1) / p.piece;
  p.part_stride = (uint32_t)round_up(op.dim, 8);
  uint32_t bits = 1;
  while ((op.rows >> bits) != 0) ++bits;  // keys 0 .. rows
  p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    p.key[i] = take(4ull * op.tokens);
    p.tok[i] = take(4ull * op.tokens);
  }
  p.touched = take((op.rows + 31ull) / 32 * 4);
  p.crossing = take(4ull * (p.pieces + 1));
  p.head = take(4ull * p.pieces * p.part_stride);
  p.tail = take(4ull * p.pieces * p.part_stride);
  p.bytes = off;
  return p;
}

df11_status check_grad(const df11_embedding_grad *op) {
  if (!op) return DF11_ERR_NULL;
  if (!known_type(op->grad_type) || !known_type(op->out_type) ||
      (op->ids_type != DF11_IDS_I32 && op->ids_type != DF11_IDS_I64))
    return DF11_ERR_INVALID;
  if (op->rows == 0 || op->dim == 0) return DF11_ERR_INVALID;
  if (op->rows >= (1u << 31) || op->tokens >= (1u << 31) || op->dim >= (1u << 30))
    return DF11_ERR_TOO_LARGE;
  if (op->out_stride < op->dim || (op->tokens && op->grad_stride < op->dim)) return DF11_ERR_INVALID;
  if (!op->out || (op->tokens && (!op->ids || !op->grad))) return DF11_ERR_NULL;
  if (!aligned(op->ids, op->ids_type == DF11_IDS_I64 ? 8 : 4) ||
      !aligned(op->grad, type_bytes(op->grad_type)) || !aligned(op->out, type_bytes(op->out_type)))
    return DF11_ERR_ALIGN;
  return DF11_OK;
}

template <typename G, typename O, int V>
df11_status launch_runs(RunArgs a, cudaStream_t s) {
  if (a.pieces) {
    const size_t smem = V > 1 ? a.piece * kRowBytes : 0;
    df11_status st = DF11_OK;
    if (V > 1) {
      uint64_t budget = 0;
      st = prepare(embedding_runs_kernel<G, O, V>, kRunThreads, kMaxPiece * kRowBytes,
                   82 + 2 * (sizeof(G) / 4) + sizeof(O) / 4, budget);
      if (st != DF11_OK) return st;
    }
    st = launch_pdl(embedding_runs_kernel<G, O, V>, dim3(a.pieces * a.col_tiles), kRunThreads, smem, s, a);
    if (st != DF11_OK) return st;
  }
  // four columns per thread at most: more threads on the few rows that many tokens share
  constexpr int J = V == 1 ? 1 : 4;
  const uint64_t most = a.pieces < 2 ? 0 : (uint64_t)a.pieces * ((a.dim + 32 * J - 1) / (32 * J));
  a.join_blocks = (uint32_t)(most < kJoinBlocks ? most : kJoinBlocks);
  // rows per thread block: up to 16 KB, so that all of them write close to one another
  // (151936 x 4096 in BF16: 254 us, with 64 KB 259, with 256 KB 271)
  a.zero_step = 32;
  while (a.zero_step > 1 && (uint64_t)a.zero_step * a.dim * sizeof(O) > kZeroStep) a.zero_step /= 2;
  const uint32_t blocks = a.join_blocks + (a.zero_rows + a.zero_step - 1) / a.zero_step;
  if (blocks == 0) return DF11_OK;
  return launch_pdl(embedding_join_kernel<O, J>, dim3(blocks), kRunThreads, 0, s, a);
}

template <typename O>
df11_status launch_runs_for(const RunArgs &a, bool grad_f32, bool vec, cudaStream_t s) {
  if (grad_f32) return vec ? launch_runs<float, O, 4>(a, s) : launch_runs<float, O, 1>(a, s);
  return vec ? launch_runs<uint16_t, O, 8>(a, s) : launch_runs<uint16_t, O, 1>(a, s);
}

}  // namespace

extern "C" {

df11_status df11_decode_embedding(const df11_tensor *table, const df11_embedding *op,
                                  int32_t *d_err, df11_stream_t stream) {
  if (!table || !op) return DF11_ERR_NULL;
  const df11_params &p = table->params;
  if (!known_type(op->out_type) || (op->ids_type != DF11_IDS_I32 && op->ids_type != DF11_IDS_I64))
    return DF11_ERR_INVALID;
  if (p.n >= (1ull << 32)) return DF11_ERR_TOO_LARGE;
  if (op->rows == 0 || op->dim == 0 || (uint64_t)op->rows * op->dim != p.n) return DF11_ERR_INVALID;
  if (op->tokens >= (1u << 31)) return DF11_ERR_TOO_LARGE;
  if (d_err && !aligned(d_err, 4)) return DF11_ERR_ALIGN;
  if (op->tokens == 0) return DF11_OK;
  if (!op->ids || !op->out) return DF11_ERR_NULL;
  if (op->out_stride < op->dim) return DF11_ERR_INVALID;
  if (!aligned(op->ids, op->ids_type == DF11_IDS_I64 ? 8 : 4) ||
      !aligned(op->out, type_bytes(op->out_type)))
    return DF11_ERR_ALIGN;
  df11_tensor v = *table;
  v.out_bf16 = reinterpret_cast<uint16_t *>(16);  // not written; passes the output checks
  df11_status st = validate(v);
  if (st != DF11_OK) return st;
  if (!table->chunk_counts || !table->decode_table || p.threads_per_block != kT ||
      (p.chunk_bytes != 8 && p.chunk_bytes != 16 && p.chunk_bytes != 24))
    return DF11_ERR_UNSUPPORTED;
  const uint64_t ob = type_bytes(op->out_type), ib = op->ids_type == DF11_IDS_I64 ? 8 : 4;
  if (share_memory(Rows{op->out, op->tokens, op->dim * ob, op->out_stride * ob},
                   Rows{op->ids, 1, op->tokens * ib, 0}))
    return DF11_ERR_INVALID;
  const void *ptrs[] = {table->bitstream, table->sign_mantissa, table->decode_table, op->ids, op->out};
  st = check_device_pointers(ptrs, 5);
  if (st != DF11_OK) return st;
  EmbedArgs a{};
  fill_tensor(a.k, *table);
  a.ids = op->ids;
  a.out = op->out;
  a.err = d_err;
  a.out_stride = op->out_stride;
  a.tokens = op->tokens;
  a.rows = op->rows;
  a.dim = op->dim;
  a.ids64 = op->ids_type == DF11_IDS_I64;
  a.out_f32 = op->out_type == DF11_F32;
  a.scaled = op->scale != 1.0f;
  a.scale = op->scale;
  uint32_t bits;
  memcpy(&bits, &op->scale, sizeof(bits));
  a.scale2 = bits & 0xFFFFu ? 0u : bits | bits >> 16;
  a.vec = op->dim % 16 == 0 && aligned(op->out, 16) &&
          op->out_stride * type_bytes(op->out_type) % 16 == 0;
  a.spin_limit = kSpinLimit;
  cudaStream_t s = (cudaStream_t)stream;
  if (p.chunk_bytes == 24) return launch_lookup<24>(a, 86, s);
  if (p.chunk_bytes == 16) return launch_lookup<16>(a, 91, s);
  return launch_lookup<8>(a, 96, s);
}

df11_status df11_embedding_gradient_workspace(const df11_embedding_grad *op, size_t *bytes) {
  if (!bytes) return DF11_ERR_NULL;
  *bytes = 0;
  const df11_status st = check_grad(op);
  if (st == DF11_OK) *bytes = grad_plan(*op).bytes;
  return st;
}

df11_status df11_embedding_gradient(const df11_embedding_grad *op, void *workspace,
                                    size_t workspace_bytes, int32_t *d_err, df11_stream_t stream) {
  df11_status st = check_grad(op);
  if (st != DF11_OK) return st;
  if (d_err && !aligned(d_err, 4)) return DF11_ERR_ALIGN;
  const GradPlan p = grad_plan(*op);
  if (!workspace) return DF11_ERR_NULL;
  if (!aligned(workspace, 256)) return DF11_ERR_ALIGN;
  if (workspace_bytes < p.bytes) return DF11_ERR_INVALID;
  // rows of the gradient are written before the last of grad and of the ids are read
  const uint64_t ob = type_bytes(op->out_type), gb = type_bytes(op->grad_type);
  const Rows out{op->out, op->rows, op->dim * ob, op->out_stride * ob};
  if (share_memory(out, Rows{op->grad, op->tokens, op->dim * gb, op->grad_stride * gb}) ||
      share_memory(out, Rows{op->ids, 1, op->tokens * (op->ids_type == DF11_IDS_I64 ? 8ull : 4ull), 0}))
    return DF11_ERR_INVALID;
  const void *ptrs[] = {op->ids, op->grad, op->out, workspace};
  st = check_device_pointers(ptrs, 4);
  if (st != DF11_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  SortArgs so{};
  so.ids = op->ids;
  for (int i = 0; i < 2; ++i) {
    so.key[i] = reinterpret_cast<uint32_t *>(ws + p.key[i]);
    so.tok[i] = reinterpret_cast<uint32_t *>(ws + p.tok[i]);
  }
  so.crossing = reinterpret_cast<uint32_t *>(ws + p.crossing);
  so.err = d_err;
  so.tokens = op->tokens;
  so.rows = op->rows;
  so.passes = p.passes;
  so.digit_bits = p.digit_bits;
  so.ids64 = op->ids_type == DF11_IDS_I64;
  // one thread block per 1024 tokens (32 per warp), up to a cluster of eight
  uint32_t ctas = 1;
  while (ctas < 8 && (uint64_t)ctas * kSortThreads < op->tokens) ctas *= 2;
  uint64_t budget = 0;
  st = prepare(embedding_sort_kernel, kSortThreads, sizeof(SortShared), 81, budget);
  if (st != DF11_OK) return st;
  // Rows set to zero beside the sort, as many as it leaves time for: it takes about 10 us, and
  // 1 us per 1300 tokens, and the other SMs write 5 MB per us (measured).  The rest is set
  // to zero beside the join, where rows with tokens are left out.
  uint32_t grid = ctas;
  if (!op->accumulate) {
    so.touched = reinterpret_cast<uint32_t *>(ws + p.touched);
    so.touched_words = (op->rows + 31) / 32;
    so.out = op->out;
    so.out_stride = op->out_stride * type_bytes(op->out_type);
    so.row_bytes = (uint32_t)(op->dim * type_bytes(op->out_type));
    uint64_t beside = (10 + op->tokens / 1300) * 5000000ull / so.row_bytes;
    if (beside > op->rows) beside = op->rows;
    so.zero_from = (uint32_t)(op->rows - beside);
    const uint64_t blocks = (beside * so.row_bytes + kZeroBytes - 1) / kZeroBytes;
    grid += (uint32_t)round_up(blocks, ctas);
  }
  st = launch_cluster(embedding_sort_kernel, grid, ctas, kSortThreads, sizeof(SortShared), s, so);
  if (st != DF11_OK) return st;
  RunArgs r{};
  r.grad = op->grad;
  r.out = op->out;
  r.key = so.key[p.passes & 1];
  r.tok = so.tok[p.passes & 1];
  r.head = reinterpret_cast<float *>(ws + p.head);
  r.tail = reinterpret_cast<float *>(ws + p.tail);
  r.grad_stride = op->grad_stride;
  r.out_stride = op->out_stride;
  r.tokens = op->tokens;
  r.rows = op->rows;
  r.dim = op->dim;
  r.piece = p.piece;
  r.pieces = p.pieces;
  r.col_tiles = p.col_tiles;
  r.crossing = so.crossing;
  r.touched = so.touched;
  r.zero_rows = so.zero_from;
  r.part_stride = p.part_stride;
  r.accumulate = op->accumulate ? 1 : 0;
  r.scale = op->scale;
  r.err = d_err;
  r.spin_limit = kSpinLimit;
  const bool gf = op->grad_type == DF11_F32, vec = p.v > 1;
  return op->out_type == DF11_F32 ? launch_runs_for<float>(r, gf, vec, s)
                                  : launch_runs_for<uint16_t>(r, gf, vec, s);
}

}  // extern "C"
