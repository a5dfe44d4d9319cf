// df11_device.cuh -- device code that the library's kernels share: the tensor
// descriptor, the decode table's place in shared memory, shared-memory and
// mbarrier primitives, bounded waits, programmatic dependent launch, the
// bitstream walks (one lane decodes one chunk) and the staging of a format
// block.  Internal to the library; every kernel file includes it.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "df11.h"

namespace {

constexpr uint32_t kSpinLimit = 1u << 20;  // x ~1 us suspend hint: ~1 s
constexpr uint32_t kSuspendHintNs = 1000;
constexpr int kWideBits = 11;              // index bits of the derived table

struct KTensor {
  const uint8_t *bitstream;
  const uint8_t *gaps;
  const uint8_t *chunk_counts;  // NULL: count by decoding
  const uint32_t *block_out_pos;
  const uint32_t *luts;
  const uint8_t *code_lengths;
  const uint8_t *sign_mantissa;
  uint16_t *out;
  const void *decode_table;  // NULL: derived by every thread block
  uint64_t total_bits;
  uint32_t n;
  uint32_t num_blocks;
  uint32_t num_luts;
  uint32_t max_block_elems;
  uint32_t max_chunk_elems;
  uint32_t max_warp_elems;   // sizes the per-warp regions of the warp-specialised kernel
  uint32_t masked;     // longest codeword > kWideBits: bits past a region may be set
  uint32_t cta_begin;  // first thread block of this tensor
  uint32_t pad;
  // fused matrix-vector product (df11_decode_gemv): y[b][r] += sum_c W[r][c] x[b][c]
  // with W the decoded tensor as rows x cols, row-major
  const uint16_t *x;  // BF16 activations, batch rows of x_stride elements
  float *y;           // batch rows of y_stride floats
  uint32_t cols, batch, x_stride, y_stride;
  uint32_t interleave_log2;  // rows interleaved per 16-column group: 2^this (0: row-major)
  uint32_t pad2;
};

// a descriptor's decode fields
inline void fill_tensor(KTensor &k, const df11_tensor &t) {
  const df11_params &p = t.params;
  k.bitstream = t.bitstream;
  k.gaps = t.gaps;
  k.chunk_counts = t.chunk_counts;
  k.block_out_pos = t.block_out_pos;
  k.luts = t.luts;
  k.code_lengths = t.code_lengths;
  k.sign_mantissa = t.sign_mantissa;
  k.decode_table = t.decode_table;
  k.total_bits = p.total_bits;
  k.n = (uint32_t)p.n;
  k.num_blocks = p.num_blocks;
  k.num_luts = p.num_luts;
  k.max_block_elems = p.max_block_elems;
  k.max_chunk_elems = p.max_chunk_elems;
  k.max_warp_elems = p.max_warp_elems;
  k.masked = p.max_len > (uint32_t)kWideBits ? 1u : 0u;
}

// ---- shared memory layout --------------------------------------------------
// [0,304)      mbarriers (full and empty per stage slot, per-warp copies, the
//              decode table's copy, the page layout's counted barriers)
// [304,560)    code lengths by rotated exponent
// [560,1584)   table 0 (rotated)
// [1584, ...)  wide table (2^WB x 8 bytes)
// then         the stage slots, the warps' exponent regions, their
//              sign/mantissa buffers and column areas (see the kernel)
constexpr uint32_t kOffLens = 304;
constexpr uint32_t kOffLut0 = 560;
constexpr uint32_t kOffWide = 1584;
constexpr uint32_t kWideBytes = 8u << kWideBits;
constexpr uint32_t kOffStages = kOffWide + kWideBytes;
// a decode table (df11_build_decode_table) is the image of [kOffLens, kOffStages)
static_assert(kOffStages - kOffLens == DF11_DECODE_TABLE_BYTES, "decode table layout");
static_assert(kOffLut0 - kOffLens == 256 && kOffWide - kOffLut0 == 1024, "decode table layout");

__device__ __forceinline__ uint32_t rot8x3(uint32_t v) {
  // rotate each of the low three bytes right by one bit
  return ((v >> 1) & 0x007F7F7Fu) | ((v << 7) & 0x00808080u);
}

__device__ __forceinline__ void report(int32_t *err, int32_t code) {
  if (err) atomicCAS(err, 0, code);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// Shared-memory accesses through 32-bit shared-window addresses.
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128_zero(uint32_t a) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts8_zero(uint32_t a) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "h"((unsigned short)0) : "memory");
}
__device__ __forceinline__ void red_or32(uint32_t a, uint32_t v) {
  asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Programmatic dependent launch: a launch of this library may start while
// the previous kernel in the stream is still running.  Each thread block
// lets the next launch start once it has queued its last block
// (launch_dependents; the next grid starts when every block has, so its
// thread blocks take the places of this grid's as they finish, and set up
// their tables and first blocks meanwhile), and waits for the previous grid
// to finish, and its writes to be visible, only before its first store to
// the output (wait): the output buffer may be one that the previous kernel
// wrote or still reads, while the compressed inputs are read-only.  Letting
// the next grid start at once measured slower on sequences of different
// launches.  Without the launch attribute both are no-ops.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The thread block's cluster: its place there, the cluster's size, and a barrier of all its
// threads after which what they wrote to shared memory is seen.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Bounded wait for phase `parity` of an mbarrier: at most `limit` polls,
// each suspending for up to about a microsecond; false on timeout.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          uint32_t limit = kSpinLimit) {
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    if (done) return true;
  }
  return false;
}

// One codeword at the start of a 32-bit window through the format's tables:
// the (rotated) exponent and the codeword length; false for an invalid one.
__device__ __forceinline__ bool decode_one(uint32_t win, const uint32_t *__restrict__ lut0,
                                           const uint8_t *__restrict__ lens,
                                           const uint32_t *sub, uint32_t num_luts,
                                           uint32_t &sym, uint32_t &len) {
  const uint32_t e = lut0[win >> 24];
  if ((e >> 24) & 15u) {
    sym = e & 0xFFu;
  } else {
    uint32_t t = e & 0xFFFFFFu, f = 0;
#pragma unroll 1
    for (int level = 1; level <= 3; ++level) {
      if (t == 0 || t >= num_luts) break;
      const uint32_t e2 = sub[(t - 1) * 256 + ((win >> (24 - 8 * level)) & 0xFFu)];
      if (e2 >> 28) {
        f = e2;
        break;
      }
      t = e2 & 0xFFFFFFu;
    }
    if (f == 0) return false;
    sym = rot8x3(f & 0xFFu);
  }
  len = lens[sym];
  return len != 0;
}

// Table 0 of the format and the code lengths into shared memory, every
// exponent byte rotated right by one bit (code lengths indexed by the
// rotated exponent).
__device__ __forceinline__ void load_tables(int tid, int nthreads, const uint32_t *luts,
                                            const uint8_t *code_lengths, uint32_t *lut0_s,
                                            uint8_t *lens_s) {
  for (int i = tid; i < 256; i += nthreads) {
    uint32_t e = luts[i] & 0x3FFFFFFFu;
    if ((e >> 24) & 15u) e = (e & 0xFF000000u) | rot8x3(e);
    lut0_s[i] = e;
    lens_s[((uint32_t)i >> 1) | (((uint32_t)i & 1u) << 7)] = code_lengths[i];
  }
}

// Derived table: entry i holds the codewords that lie wholly inside the WB
// bits i, at most MS of them: x = the first four exponents (first in bits
// 0-7), y = bits used | 8 * count << 16 | fifth exponent << 24, so that one
// add of y's low 24 bits moves both the bit position and the output bit
// offset of a packed (bit, output bit) register, and the five exponent
// bytes shift into two words with two funnel shifts.
// y == 0: the first codeword is longer than WB bits (or invalid) and takes
// the slow path.
template <int T, int MS>
__device__ void build_wide(uint2 *wide, const uint32_t *lut0, const uint8_t *lens,
                           const uint32_t *sub, uint32_t num_luts) {
  static_assert(MS >= 1 && MS <= 5, "at most five exponent bytes per entry");
  for (uint32_t i = threadIdx.x; i < (1u << kWideBits); i += T) {
    const uint32_t bits = i << (32 - kWideBits);
    uint32_t used = 0, n = 0;
    uint64_t syms = 0;
    while (n < MS) {
      const uint32_t win = bits << used;
      const uint32_t e = lut0[win >> 24];
      const uint32_t ns = e >> 28;
      if (((e >> 24) & 15u) == 0) {
        uint32_t s, l;
        if (!decode_one(win, lut0, lens, sub, num_luts, s, l) || used + l > kWideBits) break;
        syms |= (uint64_t)s << (8 * n);
        ++n;
        used += l;
        continue;
      }
      bool stop = ns == 0;
      for (uint32_t j = 0; j < ns && n < MS; ++j) {
        const uint32_t s = (e >> (8 * j)) & 0xFFu, l = lens[s];
        if (l == 0 || used + l > kWideBits) {
          stop = true;
          break;
        }
        syms |= (uint64_t)s << (8 * n);
        ++n;
        used += l;
      }
      if (stop || used >= kWideBits) break;
    }
    wide[i] = n ? make_uint2((uint32_t)syms, used | (n << 19) | ((uint32_t)(syms >> 32) << 24))
                : make_uint2(0, 0);
  }
}

// 32 stream bits starting at bit `pos` of a chunk held as big-endian words
// (the chunk and the 4 bytes after it).  Codeword starts lie below 8*C (the
// next chunk's gap covers the rest), so for C = 8 the window comes from words
// (0,1) or (1,2).
template <int C>
__device__ __forceinline__ uint32_t window(const uint32_t (&w)[C / 4 + 1], uint32_t pos) {
  if (C == 4) return __funnelshift_l(w[1], w[0], pos);
  if (C == 8) {
    const bool up = pos & 32u;
    return __funnelshift_l(up ? w[2] : w[1], up ? w[1] : w[0], pos);
  }
  const uint32_t k = pos >> 5;
  uint32_t hi = w[0], lo = w[1];
#pragma unroll
  for (int j = 1; j < C / 4; ++j)
    if (k == (uint32_t)j) {
      hi = w[j];
      lo = w[j + 1];
    }
  return __funnelshift_l(lo, hi, pos);
}

// The same walk when the thread's output place is known before it decodes
// (the format's chunk count): exponents go straight into the block's
// (zeroed) exponent array from byte d on.  Every lookup ORs its up to five
// bytes into the word that holds the next byte and the word after it (the
// part that spills over; zero when nothing does), which also merges the
// words a thread shares with its neighbours.  `pk` packs the bit position
// (bits 0-15) with the bit offset of the next byte (bits 16-31, so d stays
// below 8192); `limit` is the last word the thread may touch.  Returns the
// number of codewords decoded.
template <int T, int C, bool MASKED>
__device__ __forceinline__ uint32_t decode_direct(const uint32_t (&w)[C / 4 + 1], int start,
                                                  const int end, uint32_t wide,
                                                  const uint32_t *__restrict__ lut0,
                                                  const uint8_t *__restrict__ lens,
                                                  const uint32_t *sub, uint32_t num_luts,
                                                  uint32_t ex, uint32_t d, uint32_t limit,
                                                  int &bad) {
  uint32_t pk = (uint32_t)start | (d << 19);
  while ((int)(pk & 0xFFFFu) < end) {
    const uint32_t win = window<C>(w, pk & 0xFFFFu);
    uint2 e = lds64(wide + ((win >> (32 - kWideBits)) << 3));
    if (e.y == 0 || (!MASKED && (int)(e.y & 0xFFFFu) > end - (int)(pk & 0xFFFFu))) {
      uint32_t sym, len;
      if (!decode_one(win, lut0, lens, sub, num_luts, sym, len)) {
        bad = DF11_DEV_ERR_TABLE;
        return 0;
      }
      e = make_uint2(sym, len | (8u << 16));
    }
    const uint32_t sh = (pk >> 16) & 24u;
    const uint32_t a = min(ex + ((pk >> 21) << 2), limit);
    red_or32(a, e.x << sh);
    red_or32(a + 4u, __funnelshift_l(e.x, e.y >> 24, sh));  // with the fifth exponent
    pk += e.y & 0x00FFFFFFu;
  }
  if ((int)(pk & 0xFFFFu) != end) bad = DF11_DEV_ERR_OVERRUN;
  return (pk >> 19) - d;
}

// The direct walk for masked streams when the chunk's count is known, with
// fewer operations per lookup:
//   - the chunk's bits sit in a shifting window of NW words (next bit at the
//     top of s[0]), moved on by funnel shifts whose amount is the entry's
//     second word itself: funnel shifts use only its low five bits, which
//     hold the bits used (at most kWideBits here), and ones come in from the
//     right, so the stream stays masked past its last word;
//   - the loop ends on the element count, not the bit position: it runs
//     while the output bit offset (bits 16-31 of `pk`, bit position in bits
//     0-15) is below 8*(d+cnt).  Every iteration emits at least one element,
//     so a corrupt stream stops within cnt lookups and writes at most four
//     bytes past the thread's range (the last lookup's five bytes stay in two
//     words), which the region's slack absorbs: no clamp on the address.  Bits past `end` are ones, so
//     on valid data the last lookup stops exactly at `end` (checked after).
// Returns the number of elements written.
template <int C>
__device__ __forceinline__ uint32_t decode_counted(const uint32_t (&w)[C / 4 + 1], int start,
                                                   const int end, uint32_t wide,
                                                   const uint32_t *__restrict__ lut0,
                                                   const uint8_t *__restrict__ lens,
                                                   const uint32_t *sub, uint32_t num_luts,
                                                   uint32_t ex, uint32_t d, uint32_t cnt,
                                                   int &bad) {
  constexpr int NW = C / 4 + 1;
  uint32_t s[NW];
#pragma unroll
  for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(w[j + 1], w[j], (uint32_t)start);
  s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, w[NW - 1], (uint32_t)start);
  uint32_t pk = (uint32_t)start | ((8u * d) << 16);
  const uint32_t lim = (8u * (d + cnt)) << 16;
  while (pk < lim) {
    uint2 e = lds64(wide + ((s[0] >> (32 - kWideBits)) << 3));
    if (e.y == 0) {
      // rare: a codeword longer than the derived table's index.  Shift by
      // half its length here and the rest below (both at most 16 bits, in
      // the funnel shifts' range).
      uint32_t sym, len;
      if (!decode_one(s[0], lut0, lens, sub, num_luts, sym, len)) {
        bad = DF11_DEV_ERR_TABLE;
        return 0;
      }
      const uint32_t half = len >> 1;
#pragma unroll
      for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(s[j + 1], s[j], half);
      s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, s[NW - 1], half);
      pk += half;
      e = make_uint2(sym, (len - half) | (8u << 16));
    }
    const uint32_t sh = pk >> 16;  // funnel shifts use sh & 31: the bit offset in the word
    const uint32_t a = ex + ((pk >> 21) << 2);
    red_or32(a, __funnelshift_l(0u, e.x, sh));
    red_or32(a + 4u, __funnelshift_l(e.x, e.y >> 24, sh));  // with the fifth exponent
#pragma unroll
    for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(s[j + 1], s[j], e.y);
    s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, s[NW - 1], e.y);
    pk += e.y & 0x00FFFFFFu;
  }
  // a count that disagrees with the stream ends the walk short of `end`
  // (too small) or past it (too large, or a corrupt stream)
  const int pos = (int)(pk & 0xFFFFu);
  if (pos != end) bad = pos < end ? DF11_DEV_ERR_COUNT : DF11_DEV_ERR_OVERRUN;
  return (pk >> 19) - d;
}

// The walk of the format as the pages state it (no chunk counts): a thread
// learns where its output goes only once every warp of the block has
// counted, so it decodes into its own column of the warp's column area
// (its byte j at word (j/4)*32 + lane: the lanes' reductions never share a
// bank) and counts.  The window moves as in decode_counted; the walk stops
// at the chunk's end bit, or when `cap` bytes (the format's
// max_chunk_elems) are written, beyond which the data are inconsistent.
// Unmasked streams (every codeword within the derived table's index) check
// each entry against the end.  Returns the number of codewords.
template <int C, bool MASKED>
__device__ __forceinline__ uint32_t decode_column(const uint32_t (&w)[C / 4 + 1], int start,
                                                  const int end, uint32_t wide,
                                                  const uint32_t *__restrict__ lut0,
                                                  const uint8_t *__restrict__ lens,
                                                  const uint32_t *sub, uint32_t num_luts,
                                                  uint32_t col, uint32_t cap, int &bad) {
  constexpr int NW = C / 4 + 1;
  uint32_t s[NW];
#pragma unroll
  for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(w[j + 1], w[j], (uint32_t)start);
  s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, w[NW - 1], (uint32_t)start);
  uint32_t pk = (uint32_t)start;          // bit position | 8 * bytes written << 16
  const uint32_t lim = (8u * cap) << 16;  // pk < lim: fewer than cap bytes written
  while ((int)(pk & 0xFFFFu) < end && pk < lim) {
    uint2 e = lds64(wide + ((s[0] >> (32 - kWideBits)) << 3));
    if (e.y == 0 || (!MASKED && (int)(e.y & 0xFFFFu) > end - (int)(pk & 0xFFFFu))) {
      // a codeword longer than the derived table's index, or (unmasked
      // streams) an entry that runs past the end: one codeword through the
      // format's own tables, the window moved by half its length here
      uint32_t sym, len;
      if (!decode_one(s[0], lut0, lens, sub, num_luts, sym, len)) {
        bad = DF11_DEV_ERR_TABLE;
        return 0;
      }
      const uint32_t half = len >> 1;
#pragma unroll
      for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(s[j + 1], s[j], half);
      s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, s[NW - 1], half);
      pk += half;
      e = make_uint2(sym, (len - half) | (8u << 16));
    }
    const uint32_t sh = pk >> 16;
    const uint32_t a = col + ((pk >> 21) << 7);
    red_or32(a, __funnelshift_l(0u, e.x, sh));
    red_or32(a + 128u, __funnelshift_l(e.x, e.y >> 24, sh));
#pragma unroll
    for (int j = 0; j < NW - 1; ++j) s[j] = __funnelshift_l(s[j + 1], s[j], e.y);
    s[NW - 1] = __funnelshift_l(0xFFFFFFFFu, s[NW - 1], e.y);
    pk += e.y & 0x00FFFFFFu;
  }
  const int pos = (int)(pk & 0xFFFFu);
  if (pos != end) bad = pos < end ? DF11_DEV_ERR_COUNT : DF11_DEV_ERR_OVERRUN;
  return pk >> 19;
}

// A lane's `cnt` exponent bytes, from its column (word k at col + 128k),
// into the warp's element-order region from byte d on: whole words are
// stored, the first and last (shared with the neighbouring lanes' ranges)
// ORed into the zeroed region.  Column bytes past cnt are zero.  Each column
// word is zeroed once read, for the next block.
__device__ __forceinline__ void column_to_region(uint32_t col, uint32_t cnt, uint32_t region,
                                                 uint32_t d) {
  if (!cnt) return;
  const uint32_t r8 = (d & 3u) * 8u;
  const uint32_t words = ((d & 3u) + cnt + 3u) >> 2;  // destination words
  const uint32_t held = (cnt + 3u) >> 2;              // column words with bytes
  uint32_t prev = 0, dst = region + (d & ~3u);
  for (uint32_t j = 0; j < words; ++j, dst += 4u) {
    uint32_t cur = 0;
    if (j < held) {
      cur = lds32(col + 128u * j);
      sts32(col + 128u * j, 0u);
    }
    const uint32_t v = __funnelshift_l(prev, cur, r8);  // bytes 4j - (d & 3) ..
    if (j == 0 || j + 1 == words) red_or32(dst, v);
    else sts32(dst, v);
    prev = cur;
  }
}

// four sign/mantissa bytes and four rotated exponents -> four BF16 words:
// the four low bytes (E0 | mantissa) and the four high bytes (sign | E7..E1)
// are two bitwise selects, then two byte permutes interleave them
__device__ __forceinline__ uint2 fuse4(uint32_t sm4, uint32_t er4) {
  const uint32_t lo = (sm4 & 0x7F7F7F7Fu) | (er4 & 0x80808080u);
  const uint32_t hi = (er4 & 0x7F7F7F7Fu) | (sm4 & 0x80808080u);
  return make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
}

__device__ __forceinline__ uint16_t fuse1(uint32_t sm, uint32_t er) {
  const uint32_t lo = (sm & 0x7Fu) | (er & 0x80u), hi = (er & 0x7Fu) | (sm & 0x80u);
  return (uint16_t)__byte_perm(lo, hi, 0x3340);
}

__device__ __forceinline__ void bulk_prefetch_l2(const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------------------
// Warp-specialised decode for tensors that carry chunk counts.
//
// With the counts in shared memory every warp can work out where its output
// goes on its own, so the thread block needs no block-wide barrier per format
// block.  One producer warp (one lane) keeps kWsStages stage slots filled
// (bitstream slice, gap fields, chunk counts, positions and the block's
// sign/mantissa bytes), each guarded by a "full" mbarrier (completed by the
// bulk copies) and an "empty" mbarrier (one arrival per consumer warp when it
// is done with the block).  Each of the T/32 consumer warps, per format block:
//   - sums the block's chunk counts before its own chunks and over the whole
//     block (two warp reductions over T bytes) and scans its lanes' counts;
//   - decodes straight into its private exponent region (zeroed; words shared
//     by two lanes merged with OR) and checks every count;
//   - writes its own output range from shared memory: whole 16-element
//     groups with 16-byte stores, the two ragged edge groups one element per
//     lane; then releases the slot.
constexpr int kWsStages = 2;

// Where the output of the warp-specialised kernel finds a block's sign/
// mantissa bytes: in the stage slot (one bulk copy per block by the
// producer), in global memory (L2-prefetched by the producer), or in a
// buffer of the warp's own, filled by one bulk copy of the warp's output
// range that the warp issues before it decodes.  The host takes the first
// that keeps the most thread blocks resident.
enum SmMode { kSmSlot = 0, kSmGlobal = 1, kSmWarp = 2 };

template <int T, int C>
struct WsLayout {
  static constexpr uint32_t bits_bytes = T * C + 16;
  static constexpr uint32_t gaps_bytes = T * 5 / 8 + 16;
  static constexpr uint32_t counts_bytes = T;
  static constexpr uint32_t meta_bytes = 16;
  // the block's sign/mantissa bytes follow (KBatch::sm_bytes of them)
  static constexpr uint32_t head_bytes = bits_bytes + gaps_bytes + counts_bytes + meta_bytes;
  static_assert(head_bytes % 16 == 0, "alignment");
};

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int T, int C, int SM, bool COUNTS>
__device__ __forceinline__ void ws_issue(const KTensor &tk, uint32_t b, uint8_t *slot,
                                         uint32_t full, uint32_t sm_capacity) {
  using L = WsLayout<T, C>;
  const uint32_t P0 = tk.block_out_pos[b], P1 = tk.block_out_pos[b + 1];
  const uint32_t expected = P1 - P0;
  // a warp's exponents fit its region whatever the block: every chunk count
  // is checked against max_chunk_elems before decoding
  const bool ok = P1 >= P0 && P1 <= tk.n && expected <= tk.max_block_elems &&
                  (SM != kSmSlot || expected + 32 <= sm_capacity);
  // bits of the stream inside this block: all of them but in the last block
  const uint64_t bit0 = (uint64_t)b * (T * C * 8);
  const uint32_t valid_bits = tk.total_bits - bit0 < (uint64_t)(T * C * 8)
                                  ? (uint32_t)(tk.total_bits - bit0)
                                  : 0xFFFFFFFFu;
  *reinterpret_cast<uint4 *>(slot + L::bits_bytes + L::gaps_bytes + L::counts_bytes) =
      make_uint4(P0, P1, ok ? 1u : 0u, valid_bits);
  if (!ok) {
    mbar_arrive_expect_tx(full, 0);
    return;
  }
  const uint32_t sm_begin = P0 & ~15u;
  const uint32_t sm_bytes = ((P1 + 15u) & ~15u) - sm_begin;
  mbar_arrive_expect_tx(full, L::bits_bytes + L::gaps_bytes + (COUNTS ? L::counts_bytes : 0u) +
                                  (SM == kSmSlot ? sm_bytes : 0u));
  bulk_g2s(smem_addr(slot), tk.bitstream + (size_t)b * (T * C), L::bits_bytes, full);
  bulk_g2s(smem_addr(slot + L::bits_bytes), tk.gaps + (size_t)b * (T * 5 / 8), L::gaps_bytes,
           full);
  if (COUNTS)
    bulk_g2s(smem_addr(slot + L::bits_bytes + L::gaps_bytes), tk.chunk_counts + (size_t)b * T,
             L::counts_bytes, full);
  if (SM == kSmGlobal) {
    if (sm_bytes) bulk_prefetch_l2(tk.sign_mantissa + sm_begin, sm_bytes);
  } else if (SM == kSmSlot && sm_bytes) {
    bulk_g2s(smem_addr(slot + L::head_bytes), tk.sign_mantissa + sm_begin, sm_bytes, full);
  }
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

}  // namespace
