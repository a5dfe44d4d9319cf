// df11_linear.cu -- the linear product of a model's layer on compressed weights:
// y = act(W x + bias) * multiplier + residual, for any number of tokens.
//
// The weight is encoded in the tile order of this product: for each block of
// 16 rows and each group of 64 columns, the 16 rows' 64 elements one after
// another (rows and columns padded with zeros to whole tiles).  A tile is 64
// groups of 16 elements, and lane l of a warp that takes groups l and l + 32 of
// a tile holds, for rows l/4 and l/4 + 8, the 16 columns 16 (l mod 4) .. + 15:
// the A fragments of four m16n8k16 products, with no exchange between lanes
// and without a bank conflict on the way.
//
// Two paths, chosen by the number of tokens (see kFusedMax):
//   few tokens    one kernel decodes the weight and multiplies it from
//                 registers; the warps' sums over their parts of a row block go
//                 to a workspace, and a second kernel adds them in a fixed order
//                 and applies the epilogue.
//   more tokens   the weight is decoded into the workspace by the decode kernel
//                 and multiplied by a tcgen05 kernel with the epilogue on its
//                 accumulators.
// Every sum runs in fp32 in an order that the sizes and the device fix, so a
// call repeats bit for bit.  The result is rounded once, to the output's type.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "df11.h"
#include "df11_device.cuh"
#include "df11_device_check.h"
#include "df11_launch.h"

using namespace df11_internal;

namespace {

constexpr int kT = 256;            // chunks per format block
constexpr int kWarps = kT / 32;    // consumer warps of the fused kernel
constexpr uint32_t kTileRows = 16, kTileCols = 64, kTileElems = kTileRows * kTileCols;

// ---- epilogue ---------------------------------------------------------------

struct Epilogue {
  const void *bias, *mul, *res;  // NULL: absent
  void *y;
  uint32_t mul_stride, res_stride, y_stride;
  uint32_t act;                  // DF11_ACT_*
  uint32_t flags;                // kBiasF32 ...
};
constexpr uint32_t kBiasF32 = 1, kMulF32 = 2, kResF32 = 4, kOutF32 = 8;

__device__ __forceinline__ float load_any(const void *p, size_t i, bool f32) {
  return f32 ? __ldg(static_cast<const float *>(p) + i)
             : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
}

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

// The activations in fp32.  gelu through the complementary error function and
// the tanh form as a logistic function: neither loses digits in the negative
// tail, where 1 + erf and 1 + tanh cancel.
__device__ __forceinline__ float activate(float v, uint32_t act) {
  switch (act) {
    case DF11_ACT_RELU: return v < 0.f ? 0.f : v;  // NaN stays
    case DF11_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case DF11_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
      return v / (1.f + expf(-2.f * u));
    }
    case DF11_ACT_SILU: return v / (1.f + expf(-v));
    default: return v;
  }
}

__device__ __forceinline__ float finish(const Epilogue &e, float v, uint32_t token, uint32_t row) {
  if (e.bias) v += load_any(e.bias, row, e.flags & kBiasF32);
  v = activate(v, e.act);
  if (e.mul) v *= load_any(e.mul, (size_t)token * e.mul_stride + row, e.flags & kMulF32);
  if (e.res) {
    // the residual may be the output itself: a plain load
    const size_t i = (size_t)token * e.res_stride + row;
    v += e.flags & kResF32
             ? static_cast<const float *>(e.res)[i]
             : __uint_as_float((uint32_t)static_cast<const uint16_t *>(e.res)[i] << 16);
  }
  return v;
}

__device__ __forceinline__ void store_any(const Epilogue &e, float v, uint32_t token,
                                          uint32_t row) {
  const size_t i = (size_t)token * e.y_stride + row;
  if (e.flags & kOutF32) static_cast<float *>(e.y)[i] = v;
  else static_cast<uint16_t *>(e.y)[i] = (uint16_t)bf16_bits(v);
}

// ---- activations whose rows the kernels cannot load 16 bytes at a time -----

struct PackArgs {
  const uint16_t *x;
  uint16_t *out;
  uint32_t cols, out_cols, batch;
  uint64_t x_stride;
};

// rows of x into rows of out_cols columns, zeros past the last column
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ PackArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const uint64_t all = (uint64_t)a.batch * a.out_cols;
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < all; i += gridDim.x * 256ull) {
    const uint32_t b = (uint32_t)(i / a.out_cols), c = (uint32_t)(i - (uint64_t)b * a.out_cols);
    a.out[i] = c < a.cols ? a.x[b * a.x_stride + c] : (uint16_t)0;
  }
}

// ---- few tokens: decode and multiply in one kernel ----------------------------

struct LTensor {
  KTensor k;      // decode fields; x, x_stride, batch; cols: the columns that x holds
  float *part;    // partial sums: [thread block][slot][warp][token][16 rows]
  uint32_t ncg;   // 64-column groups per row block
  uint32_t slots; // row blocks that one thread block's range can touch
};

struct LBatch {
  LTensor t[DF11_MAX_BATCH];
  int32_t *err;
  int count;
  uint32_t cta_end;
  uint32_t region_bytes;  // each warp's exponent region, and its sign/mantissa buffer
  uint32_t spin_limit;
};

__device__ __forceinline__ uint32_t first_block(uint32_t cta, uint32_t blocks, uint32_t ctas) {
  return (uint32_t)((uint64_t)cta * blocks / ctas);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the bytes [lo, hi) of a 16-byte group kept, the others zero
__device__ __forceinline__ uint4 keep_bytes(uint4 v, uint32_t lo, uint32_t hi) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m = 0xFFFFFFFFu;
    if (lo > 4u * j) m = lo >= 4u * j + 4u ? 0u : m << (8u * (lo - 4u * j));
    if (hi < 4u * j + 4u) m = hi <= 4u * j ? 0u : m & (0xFFFFFFFFu >> (8u * (4u * j + 4u - hi)));
    w[j] &= m;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread block decodes a contiguous range of one tensor's format blocks
// with the decode kernel's warps (a producer warp that stages blocks, eight
// consumer warps that each walk 32 chunks into their own exponent region), and
// each consumer warp multiplies the groups of its part straight from
// registers: 4 m16n8k16 products per tile and 8 tokens.  A warp's sums are for
// one block of 16 rows at a time; when its range leaves a row block it writes
// them to the block's slot of the workspace.
template <int C, int NB>
__global__ void __launch_bounds__(kT + 32, NB > 2 ? 2 : 3)
    df11_linear_kernel(const __grid_constant__ LBatch lb) {
  using L = WsLayout<kT, C>;
  constexpr int NW = C / 4 + 1;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem);  // full[2], empty[2], warp[8], table
  uint8_t *lens_s = smem + kOffLens;
  uint32_t *lut0_s = reinterpret_cast<uint32_t *>(smem + kOffLut0);
  uint8_t *stages = smem + kOffStages;
  uint8_t *regions = stages + kWsStages * L::head_bytes;
  uint8_t *warp_sm = regions + kWarps * lb.region_bytes;

  int ti = 0;
  for (int i = 1; i < lb.count; ++i)
    if (blockIdx.x >= lb.t[i].k.cta_begin) ti = i;
  const LTensor &lt = lb.t[ti];
  const KTensor &tk = lt.k;
  const uint32_t ctas = (ti + 1 < lb.count ? lb.t[ti + 1].k.cta_begin : lb.cta_end) - tk.cta_begin;
  const uint32_t cta = blockIdx.x - tk.cta_begin;
  const uint32_t b0 = first_block(cta, tk.num_blocks, ctas);
  const uint32_t b1 = first_block(cta + 1, tk.num_blocks, ctas);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const uint32_t tbar = smem_addr(&bars[2 * kWsStages + kWarps]);
  if (tid == 0) {
    for (int i = 0; i < kWsStages; ++i) {
      mbar_init(smem_addr(&bars[i]), 1);
      mbar_init(smem_addr(&bars[kWsStages + i]), kWarps);
    }
    for (int i = 0; i < kWarps; ++i) mbar_init(smem_addr(&bars[2 * kWsStages + i]), 1);
    mbar_init(tbar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t issued = 0;
  if (warp == kWarps && lane == 0) {
    mbar_arrive_expect_tx(tbar, DF11_DECODE_TABLE_BYTES);
    bulk_g2s(smem_addr(lens_s), tk.decode_table, DF11_DECODE_TABLE_BYTES, tbar);
    for (uint32_t b = b0; b < b1 && issued < kWsStages; ++b, ++issued)
      ws_issue<kT, C, kSmWarp, true>(tk, b, stages + issued * L::head_bytes,
                                     smem_addr(&bars[issued]), 0);
  }
  for (uint32_t i = tid; i < kWarps * lb.region_bytes / 16; i += kT + 32)
    reinterpret_cast<uint4 *>(regions)[i] = make_uint4(0, 0, 0, 0);
  const bool tables_ok = mbar_wait(tbar, 0, lb.spin_limit);
  if (!__syncthreads_and(tables_ok)) {
    if (tid == 0) report(lb.err, DF11_DEV_ERR_TIMEOUT);
    return;
  }

  if (warp == kWarps) {  // producer
    if (lane == 0) {
      uint32_t k = issued;
      for (uint32_t b = b0 + issued; b < b1; ++b, ++k) {
        const uint32_t s = k % kWsStages, par = (k / kWsStages) & 1u;
        if (!mbar_wait(smem_addr(&bars[kWsStages + s]), par ^ 1u, lb.spin_limit)) {
          report(lb.err, DF11_DEV_ERR_TIMEOUT);
          break;
        }
        ws_issue<kT, C, kSmWarp, true>(tk, b, stages + s * L::head_bytes, smem_addr(&bars[s]), 0);
      }
      pdl_launch_dependents();
      // no copy in flight into this thread block's shared memory when it ends
      for (uint32_t j = k > kWsStages ? k - kWsStages : 0; j < k; ++j)
        if (!mbar_wait(smem_addr(&bars[j % kWsStages]), (j / kWsStages) & 1u, lb.spin_limit))
          report(lb.err, DF11_DEV_ERR_TIMEOUT);
    }
    return;
  }

  const uint32_t region = smem_addr(regions + warp * lb.region_bytes);
  uint8_t *region_p = regions + warp * lb.region_bytes;
  const uint32_t wide = smem_addr(smem + kOffWide);
  const uint32_t wsm = smem_addr(warp_sm + warp * lb.region_bytes);
  const uint32_t wbar = smem_addr(&bars[2 * kWsStages + warp]);
  const uint32_t *sub = tk.luts + 256;
  // this thread block's row blocks: slots 0 .. last of the workspace
  const uint32_t rb_elems = lt.ncg * kTileElems;
  const uint32_t rb0 = __ldg(tk.block_out_pos + b0) / rb_elems;
  const uint32_t e_end = __ldg(tk.block_out_pos + b1);
  const uint32_t last = min(e_end > rb0 * rb_elems ? (e_end - 1) / rb_elems - rb0 : 0u,
                            lt.slots - 1);
  float *part = lt.part + ((size_t)cta * lt.slots * kWarps + warp) * (16 * 8 * NB);
  const int g = lane >> 2, t4 = lane & 3;
  float acc[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  uint32_t slot = 0;
  // this warp's sums of the current slot to the workspace, [token][row]
  auto flush = [&]() {
    float *p = part + (size_t)slot * (kWarps * 16 * 8 * NB);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float *q = p + (8 * j + 2 * t4) * 16 + g;
      q[0] = acc[j][0];
      q[16] = acc[j][1];
      q[8] = acc[j][2];
      q[24] = acc[j][3];
      acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    }
    ++slot;
  };

  uint32_t wph = 0, k = 0;
  bool waited = false;
  for (uint32_t b = b0; b < b1; ++b, ++k) {
    const uint32_t s = k % kWsStages, par = (k / kWsStages) & 1u;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&bars[s]), par, lb.spin_limit))) {
      if (lane == 0) report(lb.err, DF11_DEV_ERR_TIMEOUT);
      return;  // whole warp
    }
    const uint32_t slot_sa = smem_addr(stages + s * L::head_bytes);
    const uint32_t counts_sa = slot_sa + L::bits_bytes + L::gaps_bytes;
    const uint4 m = lds128(counts_sa + L::counts_bytes);
    const uint32_t P0 = m.x, expected = m.y - m.x;
    const uint32_t release = smem_addr(&bars[kWsStages + s]);
    int start, end;
    {
      const uint32_t bit = 5u * (uint32_t)tid;
      const uint32_t ga = slot_sa + L::bits_bytes + 4u * (bit >> 5);
      const uint32_t v = __funnelshift_l(__byte_perm(lds32(ga + 4u), 0, 0x0123),
                                         __byte_perm(lds32(ga), 0, 0x0123), bit);
      start = (int)(v >> 27);
      end = C * 8 + (int)((v >> 22) & 31u);
    }
    uint32_t w[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j)
      w[j] = __byte_perm(lds32(slot_sa + (uint32_t)tid * C + 4u * j), 0, 0x0123);
    const uint2 cv = lds64(counts_sa + 8u * lane);
    const uint32_t lsum = __dp4a(cv.x, 0x01010101u, __dp4a(cv.y, 0x01010101u, 0u));
    const uint32_t cnt = lds8(counts_sa + tid);
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp * 32 / kWarps ? lsum : 0u);
    const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, lsum);
    uint32_t incl = cnt;
#pragma unroll
    for (int dd = 1; dd < 32; dd <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, dd);
      if (lane >= dd) incl += v;
    }
    const uint32_t warp_total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (!m.z || total != expected || warp_total > tk.max_warp_elems ||
        __any_sync(0xFFFFFFFFu, cnt > tk.max_chunk_elems)) {
      if (lane == 0)
        report(lb.err, m.z && total != expected ? DF11_DEV_ERR_COUNT : DF11_DEV_ERR_CAPACITY);
      __syncwarp();
      if (lane == 0) mbar_arrive(release);
      continue;
    }
    if (m.w != 0xFFFFFFFFu) {  // the block that holds the end of the stream
      const uint32_t bit0 = (uint32_t)tid * (C * 8);
      if (bit0 >= m.w) start = end = 0;
      else if ((uint32_t)end > m.w - bit0) end = (int)(m.w - bit0);
    }
    if (tk.masked) {  // ones from bit `end` on
      if (end >= C * 8) {
        w[NW - 1] |= __funnelshift_rc(0xFFFFFFFFu, 0u, (uint32_t)(end - C * 8));
      } else {
#pragma unroll
        for (int j = 0; j < NW; ++j)
          w[j] |= __funnelshift_rc(0xFFFFFFFFu, 0u, (uint32_t)max(end - 32 * j, 0));
      }
    }
    // the slot's bytes are in registers: it can be refilled
    __syncwarp();
    if (lane == 0) mbar_arrive(release);
    const uint32_t G0 = P0 + before;
    const uint32_t head = G0 & 15u, span = head + warp_total;
    const uint32_t d = head + incl - cnt;
    const uint32_t wsm_bytes = (span + 15u) & ~15u;
    if (wsm_bytes && lane == 0) {
      mbar_arrive_expect_tx(wbar, wsm_bytes);
      bulk_g2s(wsm, tk.sign_mantissa + (G0 & ~15u), wsm_bytes, wbar);
    }
    int bad = 0;
    uint32_t got;
    if (tk.masked) {
      got = decode_counted<C>(w, start, end, wide, lut0_s, lens_s, sub, tk.num_luts, region, d, cnt,
                              bad);
    } else {
      const uint32_t limit = region + ((d + (cnt ? cnt : 1u) - 1u) & ~3u);
      got = decode_direct<kT, C, false>(w, start, end, wide, lut0_s, lens_s, sub, tk.num_luts,
                                        region, d, limit, bad);
    }
    if (!bad && got != cnt) bad = DF11_DEV_ERR_COUNT;
    if (wsm_bytes) {
      const bool landed = __all_sync(0xFFFFFFFFu, mbar_wait(wbar, wph & 1u, lb.spin_limit));
      ++wph;
      if (!landed) {
        if (lane == 0) report(lb.err, DF11_DEV_ERR_TIMEOUT);
        return;  // whole warp; the buffer may still be written
      }
    }
    if (__any_sync(0xFFFFFFFFu, bad != 0)) {
      if (bad) report(lb.err, bad);
      __syncwarp();
      for (uint32_t i = lane; i < (span + 8u + 15u) >> 4; i += 32)
        reinterpret_cast<uint4 *>(region_p)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      continue;
    }
    __syncwarp();
    if (!waited) {  // the previous kernel may have written x, or still read the workspace
      pdl_wait();
      waited = true;
    }

    // multiply: groups 0 .. ng-1 of the region are the stream's groups q0 ..
    const uint32_t ng = (span + 15u) >> 4, q0 = G0 >> 4;
    if (ng) {
      uint32_t tile = q0 >> 6;
      const uint32_t tile_end = (q0 + ng - 1u) >> 6;
      uint32_t rb = tile / lt.ncg, cg = tile - rb * lt.ncg;
      for (; tile <= tile_end; ++tile) {
        // sums of the row blocks before this tile's; beyond the range only
        // when the positions are inconsistent
        if (rb - rb0 > last) {
          if (lane == 0) report(lb.err, DF11_DEV_ERR_COUNT);
          break;
        }
        while (slot < rb - rb0) flush();
        const uint32_t col = cg * kTileCols + 16u * t4;
        uint4 xv[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if ((uint32_t)g < tk.batch && col < tk.cols) {
          const uint4 *xp = reinterpret_cast<const uint4 *>(tk.x + (size_t)g * tk.x_stride + col);
          xv[0] = __ldg(xp);
          xv[1] = __ldg(xp + 1);
        }
        uint32_t wv[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t gi = (tile << 6) + 32u * h + lane - q0;  // wraps below the range
          uint4 sv = make_uint4(0, 0, 0, 0), rv = make_uint4(0, 0, 0, 0);
          if (gi < ng) {
            sv = lds128(wsm + 16u * gi);
            rv = lds128(region + 16u * gi);
            sts128_zero(region + 16u * gi);
            // the first and last groups may hold neighbours' elements
            if ((gi == 0 && head) || (gi == ng - 1 && (span & 15u)))
              sv = keep_bytes(sv, gi == 0 ? head : 0u, gi == ng - 1 ? span - 16u * gi : 16u);
          }
          const uint2 a = fuse4(sv.x, rv.x), c = fuse4(sv.y, rv.y);
          const uint2 e = fuse4(sv.z, rv.z), f = fuse4(sv.w, rv.w);
          wv[h][0] = a.x; wv[h][1] = a.y; wv[h][2] = c.x; wv[h][3] = c.y;
          wv[h][4] = e.x; wv[h][5] = e.y; wv[h][6] = f.x; wv[h][7] = f.y;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          mma_bf16(acc[j], wv[0][0], wv[1][0], wv[0][1], wv[1][1], xv[0].x, xv[0].y);
          mma_bf16(acc[j], wv[0][2], wv[1][2], wv[0][3], wv[1][3], xv[0].z, xv[0].w);
          mma_bf16(acc[j], wv[0][4], wv[1][4], wv[0][5], wv[1][5], xv[1].x, xv[1].y);
          mma_bf16(acc[j], wv[0][6], wv[1][6], wv[0][7], wv[1][7], xv[1].z, xv[1].w);
          if (j + 1 < NB) {
            xv[0] = xv[1] = make_uint4(0, 0, 0, 0);
            const uint32_t n = 8u * (j + 1) + g;
            if (n < tk.batch && col < tk.cols) {
              const uint4 *xp = reinterpret_cast<const uint4 *>(tk.x + (size_t)n * tk.x_stride + col);
              xv[0] = __ldg(xp);
              xv[1] = __ldg(xp + 1);
            }
          }
        }
        if (++cg == lt.ncg) {
          cg = 0;
          ++rb;
        }
      }
      __syncwarp();  // the region is zero again before the next walk
    }
  }
  if (!waited) pdl_wait();
  while (slot <= last) flush();
}

// The warps' sums of every row block added in a fixed order, and the epilogue.
struct FTensor {
  Epilogue e;
  const float *part;
  const uint32_t *block_out_pos;
  uint32_t num_blocks, ctas, slots, rb_elems;
  uint32_t rows, batch;
  uint32_t rb_begin;  // first row block of this tensor in the grid
};
struct FBatch {
  FTensor t[DF11_MAX_BATCH];
  int count;
  uint32_t nb;  // groups of 8 tokens in the workspace's layout
};

// 128 threads per row block and group of 8 tokens: thread (n, r) is token n, row r
__global__ void __launch_bounds__(128) df11_linear_finish_kernel(const __grid_constant__ FBatch fb) {
  __shared__ uint32_t range[2];
  int ti = 0;
  for (int i = 1; i < fb.count; ++i)
    if (blockIdx.x >= fb.t[i].rb_begin) ti = i;
  const FTensor &ft = fb.t[ti];
  const uint32_t rb = blockIdx.x - ft.rb_begin;
  const uint32_t token = 8u * blockIdx.y + (threadIdx.x >> 4), r = threadIdx.x & 15u;
  // the thread blocks whose ranges touch this row block, from the positions at
  // the ranges' ends (inputs of the call, so before the wait)
  if (threadIdx.x < 2) {
    const uint32_t e = threadIdx.x == 0 ? rb * ft.rb_elems : (rb + 1) * ft.rb_elems - 1u;
    // the last thread block whose range starts at or before element e
    uint32_t lo = 0, hi = ft.ctas;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (__ldg(ft.block_out_pos + first_block(mid, ft.num_blocks, ft.ctas)) <= e) lo = mid;
      else hi = mid;
    }
    range[threadIdx.x] = lo;
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t row = 16u * rb + r;
  if (token >= ft.batch || row >= ft.rows) return;
  const uint32_t per_warp = 16u * 8u * fb.nb;
  float sum = 0.f;
  for (uint32_t c = range[0]; c <= range[1]; ++c) {
    const uint32_t rb0 =
        __ldg(ft.block_out_pos + first_block(c, ft.num_blocks, ft.ctas)) / ft.rb_elems;
    const uint32_t slot = rb - rb0;
    if (slot >= ft.slots) continue;  // inconsistent positions, reported by the product kernel
    const float *p = ft.part + ((size_t)c * ft.slots + slot) * kWarps * per_warp + token * 16u + r;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += __ldcg(p + w * per_warp);
  }
  store_any(ft.e, finish(ft.e, sum, token, row), token, row);
}

// ---- more tokens: tcgen05 product of the decoded tiles ------------------------
//
// D[token][row] = sum_c x[token][c] W[row][c]: A is x (128 tokens, TMA from the
// caller's rows), B the decoded tiles (BN rows; a 16 x 64 tile is 16 rows of 128
// bytes, so a TMA box of BN/16 row blocks is BN rows of 64 columns), both in the
// 128-byte swizzle, K in steps of 64.  One warp issues the copies, one the
// products, four move finished accumulators (two, in turn) out through the
// epilogue: a lane is a token, its columns consecutive rows of W.
constexpr int kGemmTokens = 128;
constexpr int kGemmThreads = 6 * 32;  // warps 0-3: epilogue, 4: copies, 5: products

struct GemmArgs {
  Epilogue e;
  uint32_t tokens, rows, ncg;         // ncg: 64-column steps
  uint32_t tiles_m, tiles;            // token tiles, all tiles
  uint32_t vec;                       // rows of y, multiplier and residual take 16-byte accesses
  int32_t *err;
  uint32_t spin_limit;
};

template <int BN>
struct GemmLayout {
  static constexpr uint32_t a_bytes = kGemmTokens * 128, b_bytes = BN * 128;
  static constexpr uint32_t stage_bytes = a_bytes + b_bytes;
  static constexpr int stages = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr uint32_t smem = 1024 + stages * stage_bytes + 256;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// K-major operand in the 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// 16 consecutive rows of one token: loads of 16 bytes where aligned
__device__ __forceinline__ void load16(const void *p, size_t i, bool f32, float (&v)[16]) {
  if (f32) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 a = q[j];
      v[4 * j] = a.x; v[4 * j + 1] = a.y; v[4 * j + 2] = a.z; v[4 * j + 3] = a.w;
    }
  } else {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 a = q[j];
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        v[8 * j + 2 * l] = __uint_as_float(u[l] << 16);
        v[8 * j + 2 * l + 1] = __uint_as_float(u[l] & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ void finish16(const Epilogue &e, float (&v)[16], uint32_t token,
                                         uint32_t row) {
  float t[16];
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += load_any(e.bias, row + j, e.flags & kBiasF32);
  }
  if (e.act != DF11_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = activate(v[j], e.act);
  }
  if (e.mul) {
    load16(e.mul, (size_t)token * e.mul_stride + row, e.flags & kMulF32, t);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= t[j];
  }
  if (e.res) {
    load16(e.res, (size_t)token * e.res_stride + row, e.flags & kResF32, t);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += t[j];
  }
  const size_t i = (size_t)token * e.y_stride + row;
  if (e.flags & kOutF32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(e.y) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(e.y) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      q[j] = make_uint4(bf16_pair(v[8 * j], v[8 * j + 1]), bf16_pair(v[8 * j + 2], v[8 * j + 3]),
                        bf16_pair(v[8 * j + 4], v[8 * j + 5]), bf16_pair(v[8 * j + 6], v[8 * j + 7]));
  }
}

template <int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    df11_linear_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                            const __grid_constant__ CUtensorMap map_w,
                            const __grid_constant__ GemmArgs ga) {
  using L = GemmLayout<BN>;
  constexpr int S = L::stages;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S * L::stage_bytes;
  // full[S], empty[S], acc_full[2], acc_empty[2], the tensor-memory address
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (S + i); };
  auto acc_full = [&](int i) { return bars + 8u * (2 * S + i); };
  auto acc_empty = [&](int i) { return bars + 8u * (2 * S + 2 + i); };
  const uint32_t taddr_s = bars + 8u * (2 * S + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(taddr_s),
                 "r"(2u * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(taddr_s);
  pdl_wait();  // the decoded weight, and x, come from the kernels before
  bool failed = false;

  if (warp == 4) {
    if (lane == 0) {
      uint32_t k = 0;
      for (uint32_t tile = blockIdx.x; tile < ga.tiles && !failed; tile += gridDim.x) {
        const uint32_t tn = tile / ga.tiles_m, tm = tile - tn * ga.tiles_m;
        for (uint32_t c = 0; c < ga.ncg; ++c, ++k) {
          const uint32_t s = k % S, par = (k / S) & 1u;
          if (!mbar_wait(empty(s), par ^ 1u, ga.spin_limit)) {
            failed = true;
            break;
          }
          mbar_arrive_expect_tx(full(s), L::stage_bytes);
          tma_load_2d(base + s * L::stage_bytes, &map_x, (int)(64u * c), (int)(tm * kGemmTokens),
                      full(s));
          tma_load_4d(base + s * L::stage_bytes + L::a_bytes, &map_w, 0, 0, (int)c,
                      (int)(tn * (BN / 16)), full(s));
        }
      }
      pdl_launch_dependents();
      // no copy in flight into this thread block's shared memory when it ends
      for (uint32_t j = k > S ? k - S : 0; j < k; ++j)
        if (!mbar_wait(full(j % S), (j / S) & 1u, ga.spin_limit)) failed = true;
      if (failed) report(ga.err, DF11_DEV_ERR_TIMEOUT);
    }
  } else if (warp == 5) {
    // fp32 accumulators, BF16 operands, both K-major
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((BN / 8) << 17) |
                               ((kGemmTokens / 16) << 24);
    uint32_t k = 0, n = 0;
    for (uint32_t tile = blockIdx.x; tile < ga.tiles && !failed; tile += gridDim.x, ++n) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_empty(n & 1), ((n >> 1) & 1u) ^ 1u,
                                              ga.spin_limit))) {
        failed = true;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (n & 1u) * BN;
      for (uint32_t c = 0; c < ga.ncg; ++c, ++k) {
        const uint32_t s = k % S;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(full(s), (k / S) & 1u, ga.spin_limit))) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t ad = sw128_desc(base + s * L::stage_bytes);
          const uint64_t bd = sw128_desc(base + s * L::stage_bytes + L::a_bytes);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // K = 16: 32 bytes on
            const uint32_t add = c || j ? 1u : 0u;
            asm volatile(
                "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                "l"(ad + 2u * j), "l"(bd + 2u * j), "r"(idesc), "r"(add)
                : "memory");
          }
          asm volatile(
              "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                  empty(s))
              : "memory");
          if (c + 1 == ga.ncg)
            asm volatile(
                "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                    acc_full(n & 1))
                : "memory");
        }
        __syncwarp();
      }
    }
    // no product in flight when the tensor memory goes
    for (uint32_t j = k > S ? k - S : 0; j < k; ++j)
      if (!mbar_wait(empty(j % S), (j / S) & 1u, ga.spin_limit)) failed = true;
    if (failed && lane == 0) report(ga.err, DF11_DEV_ERR_TIMEOUT);
  } else {
    uint32_t n = 0;
    for (uint32_t tile = blockIdx.x; tile < ga.tiles; tile += gridDim.x, ++n) {
      const uint32_t tn = tile / ga.tiles_m, tm = tile - tn * ga.tiles_m;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full(n & 1), (n >> 1) & 1u, ga.spin_limit))) {
        failed = true;
        break;
      }
      tc_fence_after();
      const uint32_t token = tm * kGemmTokens + 32u * warp + lane;
      const uint32_t src = tmem + ((32u * warp) << 16) + (n & 1u) * BN;
      for (uint32_t c = 0; c < BN; c += 16) {
        const uint32_t row = tn * BN + c;
        if (row >= ga.rows) break;
        uint32_t u[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
            "%11, %12, %13, %14, %15}, [%16];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
              "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]),
              "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
            : "r"(src + c)
            : "memory");
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(u[j]);
        if (token >= ga.tokens) {
          // a row of the tile past the last token
        } else if (ga.vec && row + 16 <= ga.rows) {
          finish16(ga.e, v, token, row);
        } else {
#pragma unroll 1
          for (int j = 0; j < 16; ++j)
            if (row + j < ga.rows) {
              float o = v[0];
#pragma unroll
              for (int l = 1; l < 16; ++l) o = l == j ? v[l] : o;
              store_any(ga.e, finish(ga.e, o, token, row + j), token, row + j);
            }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(n & 1));
    }
    if (failed && lane == 0) report(ga.err, DF11_DEV_ERR_TIMEOUT);
  }
  // every warp is here before the tensor memory goes
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2u * BN)
                 : "memory");
  }
}

// ---- host side ------------------------------------------------------------------

// Tokens up to which a call decodes and multiplies in one kernel.
constexpr uint32_t kFusedMax = 32;

uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

uint32_t region_bytes_for(uint32_t max_warp_elems) {
  return (15u + max_warp_elems + 8u + 15u) & ~15u;
}

// x as the kernels read it: 16-byte loads of whole 16-column groups
bool needs_pack(const df11_linear &op) {
  return op.cols % 16 || op.x_stride % 8 || !aligned(op.x, 16);
}

struct Plan {
  bool fused = false;
  uint32_t nb = 1;                       // groups of 8 tokens (fused)
  uint64_t ctas[DF11_MAX_BATCH] = {};    // thread blocks per tensor (fused)
  uint32_t slots[DF11_MAX_BATCH] = {};
  uint64_t part[DF11_MAX_BATCH] = {};    // workspace offsets: partial sums or decoded weight
  uint64_t packed[DF11_MAX_BATCH] = {};  // packed activations
  uint64_t bytes = 0;
  uint32_t region = 0;
  size_t smem = 0;
};

template <int C, int NB>
void (*linear_kernel())(LBatch) { return df11_linear_kernel<C, NB>; }

using LinearKernel = void (*)(LBatch);
LinearKernel pick_kernel(uint32_t C, uint32_t nb, int &instance) {
  const int ci = C == 8 ? 0 : (C == 16 ? 1 : 2), ni = nb == 1 ? 0 : (nb == 2 ? 1 : 2);
  static const LinearKernel k[3][3] = {
      {linear_kernel<8, 1>(), linear_kernel<8, 2>(), linear_kernel<8, 4>()},
      {linear_kernel<16, 1>(), linear_kernel<16, 2>(), linear_kernel<16, 4>()},
      {linear_kernel<24, 1>(), linear_kernel<24, 2>(), linear_kernel<24, 4>()}};
  instance = 66 + 3 * ci + ni;
  return k[ci][ni];
}

// Everything a group of at most DF11_MAX_BATCH tensors needs from the
// workspace.  `want_launch`: also query the kernel (needs a device).
df11_status make_plan(const df11_tensor *ts, const df11_linear *ops, int count, Plan &pl) {
  uint32_t max_batch = 0, max_warp = 0, C = 0;
  uint64_t off = 0;
  for (int i = 0; i < count; ++i) {
    max_batch = max_batch > ops[i].batch ? max_batch : ops[i].batch;
    const df11_params &p = ts[i].params;
    max_warp = max_warp > p.max_warp_elems ? max_warp : p.max_warp_elems;
    C = p.chunk_bytes;
    pl.packed[i] = off;
    if (needs_pack(ops[i]))
      off += round_up(2ull * ops[i].batch * round_up(ops[i].cols, kTileCols), 256);
  }
  pl.fused = max_batch <= kFusedMax;
  if (!pl.fused) {
    for (int i = 0; i < count; ++i) {
      pl.part[i] = off;
      off += round_up(2ull * ts[i].params.n, 256);
    }
    pl.bytes = off;
    return DF11_OK;
  }
  pl.nb = max_batch <= 8 ? 1 : (max_batch <= 16 ? 2 : 4);
  pl.region = region_bytes_for(max_warp);
  const size_t head = C == 8 ? WsLayout<kT, 8>::head_bytes
                             : (C == 16 ? WsLayout<kT, 16>::head_bytes : WsLayout<kT, 24>::head_bytes);
  pl.smem = kOffStages + kWsStages * head + 2ull * kWarps * pl.region;
  if (pl.smem > 227 * 1024) return DF11_ERR_TOO_LARGE;
  int instance = 0;
  uint64_t budget = 0;
  const LinearKernel kern = pick_kernel(C, pl.nb, instance);
  const df11_status st = prepare(kern, kT + 32, pl.smem, instance, budget);
  if (st != DF11_OK) return st;
  // one wave, split so that the busiest thread block has as few format blocks
  // as possible
  uint32_t blocks[DF11_MAX_BATCH];
  for (int i = 0; i < count; ++i) blocks[i] = ts[i].params.num_blocks;
  split_blocks(blocks, count, budget, pl.ctas);
  for (int i = 0; i < count; ++i) {
    const df11_params &p = ts[i].params;
    const uint64_t per = (p.num_blocks + pl.ctas[i] - 1) / pl.ctas[i];
    const uint64_t rb_elems = round_up(ops[i].cols, kTileCols) * kTileRows;
    uint64_t elems = per * p.max_block_elems;
    if (elems > p.n) elems = p.n;
    uint64_t slots = (elems + rb_elems - 1) / rb_elems + 1;
    const uint64_t all = p.n / rb_elems;
    if (slots > all) slots = all;
    pl.slots[i] = (uint32_t)slots;
    pl.part[i] = off;
    off += round_up(pl.ctas[i] * slots * kWarps * 16 * 8 * pl.nb * sizeof(float), 256);
  }
  pl.bytes = off;
  return DF11_OK;
}

Epilogue make_epilogue(const df11_linear &op) {
  Epilogue e{};
  e.bias = op.bias;
  e.mul = op.multiplier;
  e.res = op.residual;
  e.y = op.y;
  e.mul_stride = op.multiplier_stride;
  e.res_stride = op.residual_stride;
  e.y_stride = op.y_stride;
  e.act = (uint32_t)op.activation;
  e.flags = (op.bias_type == DF11_F32 ? kBiasF32 : 0u) |
            (op.multiplier_type == DF11_F32 ? kMulF32 : 0u) |
            (op.residual_type == DF11_F32 ? kResF32 : 0u) | (op.y_type == DF11_F32 ? kOutF32 : 0u);
  return e;
}

bool known_type(int32_t t) { return t == DF11_BF16 || t == DF11_F32; }
uintptr_t type_bytes(int32_t t) { return t == DF11_F32 ? 4 : 2; }

// One tensor and its operation; DF11_OK for one that does nothing, too.
df11_status check_op(const df11_tensor &t, const df11_linear &op) {
  const df11_params &p = t.params;
  if (op.activation < DF11_ACT_NONE || op.activation > DF11_ACT_SILU) return DF11_ERR_INVALID;
  if (!known_type(op.y_type) || (op.bias && !known_type(op.bias_type)) ||
      (op.multiplier && !known_type(op.multiplier_type)) ||
      (op.residual && !known_type(op.residual_type)))
    return DF11_ERR_INVALID;
  if (p.n >= (1ull << 32)) return DF11_ERR_TOO_LARGE;
  if (op.rows == 0 || op.cols == 0 ||
      round_up(op.rows, kTileRows) * round_up(op.cols, kTileCols) != p.n)
    return DF11_ERR_INVALID;
  if (op.batch == 0) return DF11_OK;
  if (op.batch > DF11_LINEAR_MAX_BATCH) return DF11_ERR_TOO_LARGE;
  if (!op.x || !op.y) return DF11_ERR_NULL;
  if (op.x_stride < op.cols || op.y_stride < op.rows ||
      (op.multiplier && op.multiplier_stride < op.rows) ||
      (op.residual && op.residual_stride < op.rows))
    return DF11_ERR_INVALID;
  if (!aligned(op.x, 2) || !aligned(op.y, type_bytes(op.y_type)) ||
      !aligned(op.bias, type_bytes(op.bias_type)) ||
      !aligned(op.multiplier, type_bytes(op.multiplier_type)) ||
      !aligned(op.residual, type_bytes(op.residual_type)))
    return DF11_ERR_ALIGN;
  df11_tensor v = t;
  v.out_bf16 = reinterpret_cast<uint16_t *>(16);  // not written; passes the output checks
  const df11_status st = validate(v);
  if (st != DF11_OK) return st;
  if (!t.chunk_counts || !t.decode_table || p.threads_per_block != kT ||
      (p.chunk_bytes != 8 && p.chunk_bytes != 16 && p.chunk_bytes != 24))
    return DF11_ERR_UNSUPPORTED;
  return DF11_OK;
}

// The tensors of a call that have work, checked; groups of them are launched
// together.
df11_status check_call(const df11_tensor *tensors, const df11_linear *ops, int count) {
  if (count < 0) return DF11_ERR_INVALID;
  if (count && (!tensors || !ops)) return DF11_ERR_NULL;
  uint32_t C = 0;
  for (int i = 0; i < count; ++i) {
    const df11_status st = check_op(tensors[i], ops[i]);
    if (st != DF11_OK) return st;
    if (ops[i].batch == 0) continue;
    if (C && C != tensors[i].params.chunk_bytes) return DF11_ERR_INVALID;
    C = tensors[i].params.chunk_bytes;
  }
  return DF11_OK;
}

// calls f(tensors, ops, count) for the next group of at most DF11_MAX_BATCH
// tensors with work, until one fails
template <typename F>
df11_status for_groups(const df11_tensor *tensors, const df11_linear *ops, int count, F f) {
  df11_tensor ts[DF11_MAX_BATCH];
  df11_linear os[DF11_MAX_BATCH];
  int m = 0;
  for (int i = 0; i < count; ++i) {
    if (ops[i].batch) {
      ts[m] = tensors[i];
      os[m] = ops[i];
      ++m;
    }
    if (m && (m == DF11_MAX_BATCH || i + 1 == count)) {
      const df11_status st = f(ts, os, m);
      if (st != DF11_OK) return st;
      m = 0;
    }
  }
  return DF11_OK;
}

df11_status launch_fused(const df11_tensor *ts, const df11_linear *ops, int count, const Plan &pl,
                         uint8_t *ws, const uint16_t *const *x, const uint32_t *x_stride,
                         const uint32_t *x_cols, int32_t *d_err, cudaStream_t s) {
  LBatch lb{};
  FBatch fb{};
  lb.err = d_err;
  lb.count = fb.count = count;
  lb.region_bytes = pl.region;
  lb.spin_limit = kSpinLimit;
  fb.nb = pl.nb;
  uint32_t cta = 0, rbs = 0;
  for (int i = 0; i < count; ++i) {
    LTensor &l = lb.t[i];
    fill_tensor(l.k, ts[i]);
    l.k.cta_begin = cta;
    cta += (uint32_t)pl.ctas[i];
    l.k.x = x[i];
    l.k.x_stride = x_stride[i];
    l.k.cols = x_cols[i];
    l.k.batch = ops[i].batch;
    l.ncg = (uint32_t)(round_up(ops[i].cols, kTileCols) / kTileCols);
    l.slots = pl.slots[i];
    l.part = reinterpret_cast<float *>(ws + pl.part[i]);
    FTensor &f = fb.t[i];
    f.e = make_epilogue(ops[i]);
    f.part = l.part;
    f.block_out_pos = l.k.block_out_pos;
    f.num_blocks = l.k.num_blocks;
    f.ctas = (uint32_t)pl.ctas[i];
    f.slots = l.slots;
    f.rb_elems = l.ncg * kTileElems;
    f.rows = ops[i].rows;
    f.batch = ops[i].batch;
    f.rb_begin = rbs;
    rbs += (ops[i].rows + 15u) / 16u;
  }
  lb.cta_end = cta;
  int instance = 0;
  const LinearKernel kern = pick_kernel(ts[0].params.chunk_bytes, pl.nb, instance);
  df11_status st = launch_pdl(kern, dim3(cta), kT + 32, pl.smem, s, lb);
  if (st != DF11_OK) return st;
  return launch_pdl(df11_linear_finish_kernel, dim3(rbs, pl.nb), 128, 0, s, fb);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiled) nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

template <int BN>
df11_status launch_gemm_bn(const CUtensorMap &mx, CUtensorMap mw, GemmArgs ga, int sms,
                           int instance, cudaStream_t s) {
  auto kern = df11_linear_gemm_kernel<BN>;
  uint64_t budget = 0;
  const df11_status st = prepare(kern, kGemmThreads, GemmLayout<BN>::smem, instance, budget);
  if (st != DF11_OK) return st;
  ga.tiles = ga.tiles_m * ((ga.rows + BN - 1) / BN);
  const uint32_t grid = ga.tiles < (uint32_t)sms ? ga.tiles : (uint32_t)sms;
  return launch_pdl(kern, dim3(grid), kGemmThreads, GemmLayout<BN>::smem, s, mx, mw, ga);
}

df11_status launch_gemm(const df11_linear &op, const uint16_t *w, const uint16_t *x,
                        uint32_t x_stride, uint32_t x_cols, int32_t *d_err, cudaStream_t s) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return DF11_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DF11_ERR_CUDA;
  const int sms = device_info(dev).sms;
  GemmArgs ga{};
  ga.e = make_epilogue(op);
  ga.tokens = op.batch;
  ga.rows = op.rows;
  ga.ncg = (uint32_t)(round_up(op.cols, kTileCols) / kTileCols);
  ga.tiles_m = (op.batch + kGemmTokens - 1) / kGemmTokens;
  ga.err = d_err;
  ga.spin_limit = kSpinLimit;
  auto vec_ok = [](const void *p, uint32_t stride, int32_t type) {
    return !p || (aligned(p, 16) && stride * type_bytes(type) % 16 == 0);
  };
  ga.vec = vec_ok(op.y, op.y_stride, op.y_type) &&
           vec_ok(op.multiplier, op.multiplier_stride, op.multiplier_type) &&
           vec_ok(op.residual, op.residual_stride, op.residual_type);
  // the widest tile whose rounds over the SMs cost least (a round costs about
  // its tile's rows; narrow tiles read x more often)
  uint32_t best = 64;
  uint64_t cost = ~0ull;
  for (uint32_t bn : {256u, 128u, 64u}) {
    const uint64_t tiles = (uint64_t)ga.tiles_m * ((op.rows + bn - 1) / bn);
    const uint64_t c = (tiles + sms - 1) / sms * (bn + 32);
    if (c < cost) {
      cost = c;
      best = bn;
    }
  }
  CUtensorMap mx, mw;
  {
    const cuuint64_t dims[2] = {x_cols, op.batch}, strides[1] = {2ull * x_stride};
    const cuuint32_t box[2] = {64, kGemmTokens}, one[2] = {1, 1};
    if (encode(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(x), dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return DF11_ERR_CUDA;
  }
  {
    const cuuint64_t dims[4] = {64, 16, ga.ncg, (op.rows + 15u) / 16u};
    const cuuint64_t strides[3] = {128, 2048, 2048ull * ga.ncg};
    const cuuint32_t box[4] = {64, 16, 1, best / 16}, one[4] = {1, 1, 1, 1};
    if (encode(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(w), dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return DF11_ERR_CUDA;
  }
  if (best == 256) return launch_gemm_bn<256>(mx, mw, ga, sms, 75, s);
  if (best == 128) return launch_gemm_bn<128>(mx, mw, ga, sms, 76, s);
  return launch_gemm_bn<64>(mx, mw, ga, sms, 77, s);
}

df11_status check_linear_devices(const df11_tensor *ts, const df11_linear *ops, int count,
                                 const void *ws) {
  for (int i = 0; i < count; ++i) {
    const void *ptrs[] = {ts[i].bitstream, ts[i].sign_mantissa, ts[i].decode_table,
                          ops[i].x,        ops[i].y,            ops[i].bias,
                          ops[i].multiplier, ops[i].residual,   i ? nullptr : ws};
    const df11_status st = check_device_pointers(ptrs, (int)(sizeof(ptrs) / sizeof(*ptrs)));
    if (st != DF11_OK) return st;
  }
  return DF11_OK;
}

}  // namespace

extern "C" {

df11_status df11_linear_workspace(const df11_tensor *tensors, const df11_linear *ops, int count,
                                  size_t *bytes) {
  if (!bytes) return DF11_ERR_NULL;
  *bytes = 0;
  df11_status st = check_call(tensors, ops, count);
  if (st != DF11_OK) return st;
  size_t most = 0;
  st = for_groups(tensors, ops, count, [&](const df11_tensor *ts, const df11_linear *os, int m) {
    Plan pl;
    const df11_status r = make_plan(ts, os, m, pl);
    if (r == DF11_OK && pl.bytes > most) most = pl.bytes;
    return r;
  });
  if (st == DF11_OK) *bytes = most;
  return st;
}

df11_status df11_decode_linear(const df11_tensor *tensors, const df11_linear *ops, int count,
                               void *workspace, size_t workspace_bytes, int32_t *d_err,
                               df11_stream_t stream) {
  df11_status st = check_call(tensors, ops, count);
  if (st != DF11_OK) return st;
  if (d_err && !aligned(d_err, 4)) return DF11_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  // checked for every group before anything is queued
  st = for_groups(tensors, ops, count, [&](const df11_tensor *ts, const df11_linear *os, int m) {
    Plan pl;
    df11_status r = make_plan(ts, os, m, pl);
    if (r != DF11_OK) return r;
    if (!workspace) return DF11_ERR_NULL;
    if (!aligned(workspace, 256)) return DF11_ERR_ALIGN;
    if (pl.bytes > workspace_bytes) return DF11_ERR_INVALID;
    return check_linear_devices(ts, os, m, workspace);
  });
  if (st != DF11_OK) return st;
  return for_groups(tensors, ops, count, [&](const df11_tensor *ts, const df11_linear *os, int m) {
    Plan pl;
    df11_status r = make_plan(ts, os, m, pl);
    if (r != DF11_OK) return r;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const uint16_t *x[DF11_MAX_BATCH];
    uint32_t x_stride[DF11_MAX_BATCH], x_cols[DF11_MAX_BATCH];
    for (int i = 0; i < m; ++i) {
      x[i] = os[i].x;
      x_stride[i] = os[i].x_stride;
      x_cols[i] = os[i].cols;
      if (!needs_pack(os[i])) continue;
      PackArgs pa{};
      pa.x = os[i].x;
      pa.out = reinterpret_cast<uint16_t *>(ws + pl.packed[i]);
      pa.cols = os[i].cols;
      pa.out_cols = x_stride[i] = x_cols[i] = (uint32_t)round_up(os[i].cols, kTileCols);
      pa.batch = os[i].batch;
      pa.x_stride = os[i].x_stride;
      x[i] = pa.out;
      const uint64_t blocks = ((uint64_t)pa.batch * pa.out_cols + 255) / 256;
      r = launch_pdl(linear_pack_kernel, dim3((uint32_t)(blocks < 592 ? blocks : 592)), 256, 0, s, pa);
      if (r != DF11_OK) return r;
    }
    if (pl.fused) return launch_fused(ts, os, m, pl, ws, x, x_stride, x_cols, d_err, s);
    df11_tensor out[DF11_MAX_BATCH];
    for (int i = 0; i < m; ++i) {
      out[i] = ts[i];
      out[i].out_bf16 = reinterpret_cast<uint16_t *>(ws + pl.part[i]);
    }
    r = df11_decode_batched(out, m, d_err, stream);
    for (int i = 0; i < m && r == DF11_OK; ++i)
      r = launch_gemm(os[i], out[i].out_bf16, x[i], x_stride[i], x_cols[i], d_err, s);
    return r;
  });
}

}  // extern "C"
