// df11_linear.cu -- the linear product of a model's layer on compressed weights:
// y = act(W x + bias) * multiplier + residual, for any number of tokens.
//
// The weight has a compressed form of its own (df11_linear_weight_begin): like the decode
// kernels' format a Huffman code of the exponents, with sign and mantissa kept as a byte,
// but limited to 8-bit codewords and cut by elements instead of bits.  The matrix, padded
// with zeros to whole tiles of 16 rows and 64 columns, is taken in units of four tiles
// along a block of 16 rows (the last one may be shorter).  One warp decodes a unit: lane l
// has a bitstream of its own with the 32 elements of every tile that belong to it, rows
// l/4 and l/4 + 8 and the 16 columns from 16 (l mod 4) on.  Those are the A fragments of
// four m16n8k16 products, so a decoded weight goes from the table to the tensor core in
// registers: no chunk counts, scans, shared-memory exponents or exchange between lanes.
// The lanes' streams of a unit are stored word by word across the lanes, each padded to
// the longest of the 32 (about 0.3 bits per weight; chunk counts and gaps cost 0.2).
//
// Two paths, chosen by the number of tokens (see kFusedMax):
//   few tokens    one kernel decodes the weight and multiplies it from registers; the
//                 warps' sums over their parts of a row block go to a workspace, and a
//                 second kernel adds them in a fixed order and applies the epilogue.
//   more tokens   the weight is decoded into the workspace and multiplied by a
//                 tcgen05 kernel with the epilogue on its accumulators.
// Every sum runs in fp32 in an order that the sizes and the device fix, so a call
// repeats bit for bit.  The result is rounded once, to the output's type.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <vector>

#include "df11.h"
#include "df11_codebook.h"
#include "df11_device.cuh"
#include "df11_device_check.h"
#include "df11_launch.h"

using namespace df11_internal;

namespace {

constexpr uint32_t kTileRows = 16, kTileCols = 64, kTileElems = kTileRows * kTileCols;
constexpr uint32_t kUnitTiles = 4;
// Warps of a thread block (W below), of which an SM holds one: one per row block of a group.
// Decoding is a chain of dependent lookups, so its rate follows the warps: 260 us with 32
// warps, 284 with 24, 335 with 16 for 151936 x 4096 and 8 tokens.  16 where the streams are
// too long for more, and above 8 tokens, where the activations of a tile need the registers
// (12288 x 4096, 16 tokens: 43.1 us with 16 warps, 46.5 with 32).
constexpr int kManyWarps = 32, kFewWarps = 16;

// ---- the code and its decode table ------------------------------------------------
//
// Codewords of at most 8 bits (0.08 bits longer on average than the unlimited code of
// Gaussian weights), so that a table of 256 entries has every one of them, and small enough
// that each lane of a warp has a copy in its own bank of shared memory: entry i of lane l at
// byte 256 i + 4 l.  A lookup then costs one wavefront (a table shared by the lanes: 3.4
// for 32 lanes at independent places), and four codewords need at most the 32 bits
// of one window.  The streams are filled from bit 0 of a word up, a codeword's first
// bit lowest.
// An entry: bits 0-3 the codeword's length, bits 7-14 the exponent, where a BF16 word has
// it; the others zero, so that a sum of four entries has the lengths' sum in its low six
// bits.  The sign and mantissa bits of four weights are one word: those of the first two
// where a pair of BF16 words has them, those of the other two where the pair has exponents,
// so that a rotation by a byte puts them in place.
//   The steps are bound by the ALU pipe (half rate), so what can be a multiply-add is one.
constexpr int kMaxLength = 8;
constexpr uint32_t kEntries = 1u << kMaxLength;
constexpr uint32_t kTableBytes = 256u * kEntries;  // in shared memory; 128 of each 256 used
constexpr uint32_t kExponents = 0x7F807F80u;
// Words of a lane's stream in a unit, at most.
constexpr uint32_t kMaxWords = kUnitTiles * 32u * kMaxLength / 32u;
struct LinearTable {
  uint32_t entry[kEntries];
  uint8_t code[256];    // by exponent: the codeword, first bit lowest, and its length
  uint8_t length[256];  // (for the builder)
};
static_assert(sizeof(LinearTable) == DF11_LINEAR_TABLE_BYTES, "table layout");

// ---- epilogue ---------------------------------------------------------------

struct Epilogue {
  const void *bias, *mul, *res;  // NULL: absent
  void *y;
  uint32_t mul_stride, res_stride, y_stride;
  uint32_t act;                  // DF11_ACT_*
  uint32_t flags;                // kBiasF32 ...
};
constexpr uint32_t kBiasF32 = 1, kMulF32 = 2, kResF32 = 4, kOutF32 = 8;
constexpr uint32_t kBiasVec = 16;  // the bias starts on a 16-byte boundary

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
// tail, where 1 + erf and 1 + tanh cancel.  v / (1 + exp(-t)) is written with exp(-|t|), so that the
// divisor is between 1 and 2, where the approximate division is within two units in the last
// place (the exact one is half of an epilogue's instructions; beyond 2^126 the approximate one
// gives zero, where silu(-88) is still a normal number).
__device__ __forceinline__ float relu(float v) { return v < 0.f ? 0.f : v; }  // NaN stays
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }
__device__ __forceinline__ float logistic(float v, float t) {
  const float e = expf(-0.5f * fabsf(t));  // squared where it is used: exp(-|t|) loses digits below 2^-126
  return __fdividef(t < 0.f ? v * e * e : v, 1.f + e * e);
}
__device__ __forceinline__ float gelu_tanh(float v) {
  const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
  return logistic(v, 2.f * u);
}
__device__ __forceinline__ float silu(float v) { return logistic(v, v); }
// one branch for all values, so that their chains of instructions run side by side
template <int N>
__device__ __forceinline__ void activate(float *v, uint32_t act) {
#define DF11_EACH(f)            \
  _Pragma("unroll") for (int j = 0; j < N; ++j) v[j] = f(v[j]); \
  break
  switch (act) {
    case DF11_ACT_RELU: DF11_EACH(relu);
    case DF11_ACT_GELU: DF11_EACH(gelu);
    case DF11_ACT_GELU_TANH: DF11_EACH(gelu_tanh);
    case DF11_ACT_SILU: DF11_EACH(silu);
    default: break;
  }
#undef DF11_EACH
}

// An output's operands, and the epilogue on a sum.  The loads stand before what they wait
// beside.
struct Operands {
  float bias = 0.f, mul = 0.f, res = 0.f;
};
__device__ __forceinline__ Operands load_operands(const Epilogue &e, uint32_t token, uint32_t row) {
  Operands o;
  if (e.bias) o.bias = load_any(e.bias, row, e.flags & kBiasF32);
  if (e.mul) o.mul = load_any(e.mul, (size_t)token * e.mul_stride + row, e.flags & kMulF32);
  if (e.res) {
    // the residual may be the output itself: a plain load
    const size_t i = (size_t)token * e.res_stride + row;
    o.res = e.flags & kResF32
                ? static_cast<const float *>(e.res)[i]
                : __uint_as_float((uint32_t)static_cast<const uint16_t *>(e.res)[i] << 16);
  }
  return o;
}
template <int N>
__device__ __forceinline__ void finish(const Epilogue &e, float (&v)[N], const Operands (&o)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (e.bias) v[j] += o[j].bias;
  activate<N>(v, e.act);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (e.mul) v[j] *= o[j].mul;
    if (e.res) v[j] += o[j].res;
  }
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

// rows of x into rows of out_cols columns, zeros past the last column: 256 columns of a row
// per step of a warp, all loads before the first store
__device__ __forceinline__ void pack_rows(const PackArgs &a, uint64_t warp, uint64_t warps) {
  const uint32_t lane = threadIdx.x & 31, segs = (a.out_cols + 255u) / 256u;
  for (uint64_t i = warp; i < (uint64_t)a.batch * segs; i += warps) {
    const uint32_t b = (uint32_t)(i / segs), c0 = 256u * (uint32_t)(i - (uint64_t)b * segs) + lane;
    const uint16_t *x = a.x + b * a.x_stride;
    uint16_t *out = a.out + (uint64_t)b * a.out_cols;
    uint16_t v[8];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) v[j] = c0 + 32u * j < a.cols ? x[c0 + 32u * j] : (uint16_t)0;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (c0 + 32u * j < a.out_cols) out[c0 + 32u * j] = v[j];
  }
}
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ PackArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  pack_rows(a, (blockIdx.x * 256ull + threadIdx.x) / 32, gridDim.x * 8ull);
}

// ---- one lane's stream -------------------------------------------------------------

struct LWeight {
  const uint32_t *streams;        // rows of 32 words
  const uint32_t *unit_rows;      // first row of each unit
  const uint8_t *sign_mantissa;   // per tile: rows 0-7 (16 bytes per lane), rows 8-15
  const LinearTable *table;
  uint32_t rbs, ncg, upr;         // row blocks, tiles and units per row block
  uint32_t max_words, stream_rows;
  uint32_t one, k64;              // 1 and 65536 (see next4)
};

// Two words of the lane's stream, b after a, with the next bit at bit (p & 31) of a, and
// where the word after them is.  Bits 6 and up of p are not kept clean (the table's entries
// are added whole).
struct LaneBits {
  uint32_t a, b, p, addr;
  // to position `t`, at most 32 bits on, which is past a word when bit 5 changes: without a
  // branch, since in most steps some lane has reached its word's end
  __device__ __forceinline__ void move(uint32_t t, uint32_t one) {
    asm volatile(
        "{\n .reg .pred q;\n .reg .b32 x;\n"
        " xor.b32 x, %2, %4;\n and.b32 x, x, 32;\n setp.ne.b32 q, x, 0;\n"
        " @q mul.lo.u32 %0, %1, %5;\n @q ld.shared.b32 %1, [%3];\n"
        " @q mad.lo.u32 %3, %5, 128, %3;\n mov.b32 %2, %4;\n}\n"
        : "+r"(a), "+r"(b), "+r"(p), "+r"(addr)
        : "r"(t), "r"(one));
  }
};

// A value that the compiler keeps in a register instead of computing it again: it would
// take the shared-memory window's base anew for every lookup.
__device__ __forceinline__ uint32_t keep(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// The entry of the codeword at the start of a window: `table` is the lane's copy, which
// starts at a multiple of 64 KB plus 4 times the lane, so one byte permute has the address.
__device__ __forceinline__ uint32_t look_up(uint32_t table, uint32_t window) {
  return lds32(__byte_perm(window, table, 0x7604));
}

// The next four weights, two BF16 per word, from their sign and mantissa bits.  The shifts
// use an entry's low five bits: the length.  `one` and `k64` are 1 and 65536, arguments of
// the launch because the compiler would not multiply by constants like these.
__device__ __forceinline__ void next4(LaneBits &s, uint32_t table, uint32_t one, uint32_t k64,
                                      uint32_t sm, uint32_t &w0, uint32_t &w1) {
  uint32_t w = __funnelshift_r(s.a, s.b, s.p);
  const uint32_t e0 = look_up(table, w);
  w = __funnelshift_r(w, 0u, e0);
  const uint32_t e1 = look_up(table, w);
  w = __funnelshift_r(w, 0u, e1);
  const uint32_t e2 = look_up(table, w);
  w = __funnelshift_r(w, 0u, e2);
  const uint32_t e3 = look_up(table, w);
  s.move(e3 * one + (e2 * one + (e1 * one + (e0 * one + s.p))), one);
  w0 = ((e1 * k64 + e0) & kExponents) | (sm & ~kExponents);
  w1 = ((e3 * k64 + e2) & kExponents) | (__byte_perm(sm, 0, 0x0321) & ~kExponents);
}

// 16 weights of a lane
__device__ __forceinline__ void next16(LaneBits &s, uint32_t table, uint32_t one, uint32_t k64,
                                       const uint4 &sm, uint32_t (&w)[8]) {
  const uint32_t v[4] = {sm.x, sm.y, sm.z, sm.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) next4(s, table, one, k64, v[j], w[2 * j], w[2 * j + 1]);
}

// 16 bytes that are read once
__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A warp's walk over its units: thread block `cta` of `ctas` has an equal, contiguous
// share of the units in the order (group of W row blocks, unit along the rows, row block of
// the group), and warp w of it those of the group's row block w.  So the warps of a
// thread block are at the same columns of x at about the same time.
__device__ __host__ __forceinline__ uint64_t first_unit(uint64_t cta, uint64_t units, uint64_t ctas) {
  return cta * units / ctas;
}
// units in that order, row blocks past the last included
__device__ __host__ __forceinline__ uint64_t ordered_units(uint32_t rbs, uint32_t upr, uint32_t w) {
  return (uint64_t)((rbs + w - 1) / w) * upr * w;
}

// Shared memory: barriers (two per warp), the warps' buffers (two units each) on both sides
// of the table, which starts at a multiple of its size, and room for what a lane of an
// inconsistent stream can read past its buffer before a tile's check stops it (at most 8
// refills, two words ahead).
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kOverrun = 128u * (8u + 2u);
static_assert(kBarBytes >= 16 * kManyWarps && kBarBytes % 128 == 0, "barriers");

__device__ __host__ constexpr uint32_t decode_smem(uint32_t max_words, uint32_t warps) {
  // the space before the table is below the table's size, and holds all buffers or leaves
  // less than one warp's free
  const uint32_t buffers = (warps + 1) * 2u * max_words * 128u;
  return kBarBytes + (buffers > kTableBytes ? buffers : kTableBytes) + kTableBytes + kOverrun;
}

// The decoding side of both kernels: `use.load(cg)` and `use(rb, cg, w0, w1)` get every
// tile of the warp's units in order, before and after it is decoded (w0: rows 0-7, w1: rows
// 8-15), `moved(j)` is called for every group j of row blocks of the thread block's range once
// the warp's units there are done, and `start()` once before anything is used.
// A unit's streams are copied into one of the warp's two buffers while it decodes the
// other; the rows of the unit after that and the next tile's sign/mantissa bytes are
// loaded ahead along a row block.
template <int W, typename Start, typename Use, typename Moved>
__device__ __forceinline__ void decode_units(const LWeight &lw, uint32_t cta, uint32_t ctas,
                                             int32_t *err, uint32_t spin_limit, uint8_t *smem,
                                             Start start, Use use, Moved moved) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bars = keep(smem_addr(smem)), wbar = bars + 16u * warp;
  const uint32_t bytes = lw.max_words * 128u;
  const uint32_t at = (bars + kBarBytes + kTableBytes - 1u) & ~(kTableBytes - 1u);
  const uint32_t before = min((at - bars - kBarBytes) / (2u * bytes), (uint32_t)W);
  const uint32_t buf = keep(warp < before ? bars + kBarBytes + warp * 2u * bytes
                                          : at + kTableBytes + (warp - before) * 2u * bytes);
  const uint32_t table = keep(at + 4u * lane), one = lw.one, k64 = lw.k64;
  if (lane < 2) {  // the warp's own barriers
    mbar_init(wbar + 8u * lane, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  const uint64_t units = ordered_units(lw.rbs, lw.upr, W);
  const uint64_t o0 = first_unit(cta, units, ctas), o1 = first_unit(cta + 1, units, ctas);
  const uint32_t per_group = lw.upr * W;
  const uint32_t g0 = (uint32_t)(o0 / per_group), g1 = (uint32_t)((o1 + per_group - 1) / per_group);
  // this warp's units: q = group * upr + (unit along the rows), [q0, q1), without those of
  // row blocks past the last
  const uint32_t q0 = (uint32_t)((o0 + W - 1 - warp) / W);
  const uint32_t mine = warp < lw.rbs ? ((lw.rbs - 1 - warp) / W + 1) * lw.upr : 0u;
  const uint32_t q1 = min((uint32_t)((o1 + W - 1 - warp) / W), mine);
  // rows [r0, r1) of a unit into buffer i, and its sign/mantissa bytes (from byte `sm` on)
  // into L2; returns the words, 0 when the table of rows is inconsistent
  auto fetch = [&](uint32_t r0, uint32_t r1, uint32_t i, uint32_t sm, uint32_t tiles) -> uint32_t {
    const uint32_t n = r1 - r0;
    if (r1 < r0 || n > lw.max_words || n == 0 || r1 > lw.stream_rows) {
      if (lane == 0) report(err, DF11_DEV_ERR_CAPACITY);
      return 0u;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(wbar + 8u * i, n * 128u);
      bulk_g2s(buf + i * bytes, lw.streams + (size_t)r0 * 32u, n * 128u, wbar + 8u * i);
      bulk_prefetch_l2(lw.sign_mantissa + sm, tiles * kTileElems);
    }
    return n;
  };
  // the bytes of the warp's unit q, and the words of a unit's streams once they are asked for
  auto bytes_of = [&](uint32_t rb, uint32_t cg) {  // below 2^32: the weight's elements
    return (rb * lw.ncg + cg) * kTileElems;
  };
  uint32_t words = 0;
  if (q0 < q1) {
    const uint32_t rb = q0 / lw.upr * W + warp, ku = q0 % lw.upr;
    const uint32_t *rows = lw.unit_rows + (rb * lw.upr + ku);
    words = fetch(__ldg(rows), __ldg(rows + 1), 0, bytes_of(rb, ku * kUnitTiles),
                  min(kUnitTiles, lw.ncg - ku * kUnitTiles));
  }
#pragma unroll
  for (uint32_t e = 0; e < kEntries; e += W)  // every lane's copy of the table
    sts32(table + 256u * (e + warp), __ldg(lw.table->entry + e + warp));
  __syncthreads();
  bool running = true;
  start();
  uint32_t done = g0, bad = 0;
  uint32_t i = 0, phase = 0;  // buffer of the current unit; bit j: parity of buffer j's next wait
  for (uint32_t q = q0; q < q1 && running;) {
    // the units of one row block
    const uint32_t group = q / lw.upr, ku = q - group * lw.upr, count = min(lw.upr - ku, q1 - q);
    const uint32_t rb = group * W + warp;
    q += count;
    for (; done < group; ++done) moved(done - g0);
    const uint32_t rows = rb * lw.upr + ku;
    uint32_t cg = ku * kUnitTiles;
    uint32_t smo = bytes_of(rb, cg) + 16u * lane;
    uint32_t r1 = __ldg(lw.unit_rows + rows + 1), r2 = count > 1 ? __ldg(lw.unit_rows + rows + 2) : 0u;
    uint4 sm0 = ldg_stream(lw.sign_mantissa + smo), sm1 = ldg_stream(lw.sign_mantissa + smo + 512u);
    if (q > q0 + count)  // the first one is on its way
      words = fetch(__ldg(lw.unit_rows + rows), r1, i, bytes_of(rb, cg), min(kUnitTiles, lw.ncg - cg));
    for (uint32_t u = 1; u <= count; ++u, i ^= 1u) {
      uint32_t next_words = 0;
      __syncwarp();  // every lane is done with the other buffer
      if (u < count) {
        next_words = fetch(r1, r2, i ^ 1u, bytes_of(rb, cg + kUnitTiles),
                           min(kUnitTiles, lw.ncg - cg - kUnitTiles));
        r1 = r2;
        if (u + 1 < count) r2 = __ldg(lw.unit_rows + rows + u + 2);
      }
      if (words) {
        running = __all_sync(0xFFFFFFFFu, mbar_wait(wbar + 8u * i, (phase >> i) & 1u, spin_limit));
        phase ^= 1u << i;
        if (!running) {
          // the copy may still come: leave, once the other one has landed or not
          if (lane == 0) {
            report(err, DF11_DEV_ERR_TIMEOUT);
            if (next_words) mbar_wait(wbar + 8u * (i ^ 1u), (phase >> (i ^ 1u)) & 1u, spin_limit);
          }
          break;
        }
      }
      const uint32_t row0 = buf + i * bytes + 4u * lane;
      LaneBits s{lds32(row0), lds32(row0 + 128u), 0u, row0 + 256u};
      const uint32_t cg1 = min(cg + kUnitTiles, lw.ncg);
      for (; cg < cg1; ++cg) {
        if (s.addr - row0 > bytes + 256u) {  // read past the unit's words
          bad = 1u;
          s.addr = row0;
        }
        // the next tile's bytes, or a tile's that is there for the last one of the row block
        if (cg + 1 < lw.ncg) smo += kTileElems;
        uint32_t w0[8], w1[8];
        use.load(cg);
        next16(s, table, one, k64, sm0, w0);
        sm0 = ldg_stream(lw.sign_mantissa + smo);
        next16(s, table, one, k64, sm1, w1);
        sm1 = ldg_stream(lw.sign_mantissa + smo + 512u);
        if (words) use(rb, cg, w0, w1);
      }
      // the longest stream ends in the unit's last word
      const uint32_t used = ((s.addr - row0 - 256u) >> 7) + (s.p & 31u ? 1u : 0u);
      if (words && __reduce_max_sync(0xFFFFFFFFu, used) != words) bad = 1u;
      words = next_words;
    }
  }
  for (; done < g1; ++done) moved(done - g0);
  if (bad) report(err, DF11_DEV_ERR_COUNT);
}

// ---- few tokens: decode and multiply in one kernel ----------------------------------
//
// 2 cols operations per weight and token on 1.35 bytes per weight: up to 32 tokens the
// least time is that of reading the compressed weight.  What bounds the kernel is not the
// memory but the decoding's chain of four lookups, each waiting for the one before, over
// the 32 warps that an SM's registers hold: 151936 x 4096 and 8 tokens in 262 us, half of
// the copy bandwidth (16 warps: 335 us; a table of pairs shared by the lanes, which has
// half as many lookups but 3.4 wavefronts each: 285 us).  12288 x 4096 and 24 tokens take
// 49 us, 6144 x 4096 and one token 21 us, of which 4 us are the second kernel and its launch.
//   With 32 warps a thread has 64 registers, and the compiler keeps 28 bytes of it in local memory.

struct LTensor {
  LWeight w;
  const uint16_t *x;
  float *part;        // partial sums: [thread block][slot][warp][token][16 rows]
  uint32_t x_stride, x_cols, batch;  // x_cols: the columns that x holds, a multiple of 16
  uint32_t slots;     // groups of row blocks that one thread block's range can touch
  uint32_t cta_begin;
};

struct LBatch {
  LTensor t[DF11_MAX_BATCH];
  int32_t *err;
  int count;
  uint32_t cta_end;
  uint32_t spin_limit;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The products of a tile: x as B fragments, token 8 j + lane / 4 and the lane's 16 columns
template <int NB>
struct Multiply {
  float (&acc)[NB][4];
  const uint8_t *x;
  uint32_t offset;  // of the lane's token and columns; 32 rows of x end below 2^32 bytes
  uint32_t step;    // from token n to token n + 8
  uint32_t tiles;   // tiles in which x has the lane's columns
  uint32_t tokens;  // of the lane: n = lane / 4 + 8 j, j below this
  uint4 xv[NB][2];
  __device__ __forceinline__ Multiply(const LTensor &lt, uint32_t lane, float (&a)[NB][4]) : acc(a) {
    const uint32_t n = lane >> 2, c = 16u * (lane & 3u);
    x = reinterpret_cast<const uint8_t *>(lt.x);
    offset = 2u * (n * lt.x_stride + c);
    step = 16u * lt.x_stride;
    tokens = lt.batch > n ? (lt.batch - n + 7u) / 8u : 0u;
    tiles = lt.x_cols > c && tokens ? (lt.x_cols - c + kTileCols - 1) / kTileCols : 0u;
  }
  // issued where it stands, before the tile is decoded: the compiler would move plain loads
  // down to the products
  __device__ __forceinline__ void load(uint32_t cg) {
#pragma unroll
    for (uint32_t j = 0; j < NB; ++j) {
      const uint8_t *p = x + (offset + j * step + cg * (2u * kTileCols));
      const uint32_t there = (j == 0 || j < tokens) && cg < tiles;
      asm volatile(
          "{\n .reg .pred q;\n setp.ne.u32 q, %9, 0;\n"
          " mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
          " mov.b32 %4, 0;\n mov.b32 %5, 0;\n mov.b32 %6, 0;\n mov.b32 %7, 0;\n"
          " @q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%8];\n"
          " @q ld.global.nc.v4.b32 {%4, %5, %6, %7}, [%8 + 16];\n}\n"
          : "=&r"(xv[j][0].x), "=&r"(xv[j][0].y), "=&r"(xv[j][0].z), "=&r"(xv[j][0].w),
            "=&r"(xv[j][1].x), "=&r"(xv[j][1].y), "=&r"(xv[j][1].z), "=&r"(xv[j][1].w)
          : "l"(p), "r"(there));
    }
  }
  // A tile's products are summed from zero and then added in fp32: the tensor cores cut off
  // what an addition leaves below their accumulator, so a long chain of products drifts
  // towards zero (relative error 3.8e-6 at 4096 columns; 2e-7 like this).
  __device__ __forceinline__ void operator()(uint32_t, uint32_t, const uint32_t (&w0)[8],
                                             const uint32_t (&w1)[8]) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      mma_bf16(t, w0[0], w1[0], w0[1], w1[1], xv[j][0].x, xv[j][0].y);
      mma_bf16(t, w0[2], w1[2], w0[3], w1[3], xv[j][0].z, xv[j][0].w);
      mma_bf16(t, w0[4], w1[4], w0[5], w1[5], xv[j][1].x, xv[j][1].y);
      mma_bf16(t, w0[6], w1[6], w0[7], w1[7], xv[j][1].z, xv[j][1].w);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][k] += t[k];
    }
  }
};

template <int NB, int W>
__global__ void __launch_bounds__(32 * W, 1)
    df11_linear_kernel(const __grid_constant__ LBatch lb) {
  extern __shared__ __align__(128) uint8_t smem[];
  int ti = 0;
  for (int i = 1; i < lb.count; ++i)
    if (blockIdx.x >= lb.t[i].cta_begin) ti = i;
  const LTensor &lt = lb.t[ti];
  const uint32_t ctas = (ti + 1 < lb.count ? lb.t[ti + 1].cta_begin : lb.cta_end) - lt.cta_begin;
  const uint32_t cta = blockIdx.x - lt.cta_begin;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  // the warp's sums of a group's row block to the workspace, [token][row]
  auto moved = [&](uint32_t slot) {
    float *q = lt.part + (((size_t)cta * lt.slots + slot) * W + warp) * (16 * 8 * NB) +
               2u * (lane & 3u) * 16u + (lane >> 2);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      q[128 * j] = acc[j][0];
      q[128 * j + 16] = acc[j][1];
      q[128 * j + 8] = acc[j][2];
      q[128 * j + 24] = acc[j][3];
      acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    }
  };
  // x may come from the previous kernel, which may still read the workspace
  auto start = [&]() {
    pdl_wait();
    pdl_launch_dependents();
  };
  decode_units<W>(lt.w, cta, ctas, lb.err, lb.spin_limit, smem, start, Multiply<NB>(lt, lane, acc), moved);
}

// The warps' sums of every row block added in a fixed order, and the epilogue.
struct FTensor {
  Epilogue e;
  const float *part;
  uint32_t ctas, slots, rbs, upr;
  uint32_t rows, batch;
  uint32_t block_begin;  // first thread block of this tensor in the grid
};
struct FBatch {
  FTensor t[DF11_MAX_BATCH];
  int count;
  uint32_t nb, warps;  // groups of 8 tokens, warps per thread block in the workspace's layout
};
constexpr int kFinishThreads = 128;

// a thread per output: 16 rows of a token next to each other, tokens of a row block next
__global__ void __launch_bounds__(kFinishThreads)
    df11_linear_finish_kernel(const __grid_constant__ FBatch fb) {
  int ti = 0;
  for (int i = 1; i < fb.count; ++i)
    if (blockIdx.x >= fb.t[i].block_begin) ti = i;
  const FTensor &ft = fb.t[ti];
  // at most 2^26 rows and kFusedMax tokens: below 2^32
  const uint32_t i = (blockIdx.x - ft.block_begin) * kFinishThreads + threadIdx.x;
  const uint32_t r = i & 15u, rb = (i >> 4) / ft.batch;
  const uint32_t token = (i >> 4) - rb * ft.batch, row = 16u * rb + r;
  const bool here = rb < ft.rbs && row < ft.rows;
  // the thread blocks that hold units of the row block's group
  const uint64_t units = ordered_units(ft.rbs, ft.upr, fb.warps), per_group = (uint64_t)ft.upr * fb.warps;
  const uint64_t group = rb / fb.warps;
  auto holder = [&](uint64_t o) { return (uint32_t)(((o + 1) * ft.ctas - 1) / units); };
  const uint32_t c0 = holder(group * per_group), c1 = holder((group + 1) * per_group - 1);
  const uint32_t per_warp = 16u * 8u * fb.nb;
  // slot of the group in a thread block's part: 0 but for those that begin before it
  const uint64_t slot = group - first_unit(c0, units, ft.ctas) / per_group;
  const float *p = ft.part + (size_t)(rb % fb.warps) * per_warp + token * 16u + r;
  const size_t stride = (size_t)ft.slots * fb.warps * per_warp;
  pdl_wait();
  pdl_launch_dependents();
  if (!here) return;
  const Operands o[1] = {load_operands(ft.e, token, row)};
  float sum = __ldcg(p + c0 * stride + slot * fb.warps * per_warp);
  constexpr uint32_t kAhead = 8;  // loads before the first addition
  for (uint32_t c = c0 + 1; c <= c1; c += kAhead) {
    float v[kAhead];
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j) v[j] = c + j <= c1 ? __ldcg(p + (c + j) * stride) : 0.f;
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j)
      if (c + j <= c1) sum += v[j];
  }
  float v[1] = {sum};
  finish(ft.e, v, o);
  store_any(ft.e, v[0], token, row);
}

// ---- decoding into tiles --------------------------------------------------------------
//
// The same walk with stores in place of products: 4096 x 12288 in 34 us, 3.35 bytes per weight.

struct UArgs {
  LWeight w[DF11_MAX_BATCH];
  uint16_t *out[DF11_MAX_BATCH];  // tiles of 16 rows x 64 columns, along the rows
  uint32_t cta_begin[DF11_MAX_BATCH + 1];
  PackArgs x[DF11_MAX_BATCH];     // activations to pack beside; batch 0: none
  int32_t *err;
  int count;
  uint32_t spin_limit;
};

struct StoreTile {
  uint16_t *out;
  uint32_t ncg, lane;
  __device__ __forceinline__ void load(uint32_t) {}
  __device__ __forceinline__ void operator()(uint32_t rb, uint32_t cg, const uint32_t (&w0)[8],
                                             const uint32_t (&w1)[8]) {
    uint4 *q = reinterpret_cast<uint4 *>(out + ((size_t)rb * ncg + cg) * kTileElems) +
               2u * lane;
    q[0] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    q[1] = make_uint4(w0[4], w0[5], w0[6], w0[7]);
    q[64] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    q[65] = make_uint4(w1[4], w1[5], w1[6], w1[7]);
  }
};

template <int W>
__global__ void __launch_bounds__(32 * W, 1)
    df11_linear_unpack_kernel(const __grid_constant__ UArgs ua) {
  extern __shared__ __align__(128) uint8_t smem[];
  int ti = 0;
  for (int i = 1; i < ua.count; ++i)
    if (blockIdx.x >= ua.cta_begin[i]) ti = i;
  auto start = [&]() {  // the previous kernel may still read the output, or write x
    pdl_wait();
    pdl_launch_dependents();
    for (int i = 0; i < ua.count; ++i)
      pack_rows(ua.x[i], (uint64_t)blockIdx.x * W + threadIdx.x / 32, (uint64_t)gridDim.x * W);
  };
  decode_units<W>(ua.w[ti], blockIdx.x - ua.cta_begin[ti], ua.cta_begin[ti + 1] - ua.cta_begin[ti],
                  ua.err, ua.spin_limit, smem, start, StoreTile{ua.out[ti], ua.w[ti].ncg, threadIdx.x & 31u},
                  [](uint32_t) {});
}

// ---- building the compressed form --------------------------------------------------------

struct PackWeight {
  const uint16_t *w;       // rows x cols
  const LinearTable *table;
  uint32_t *unit_rows;
  uint32_t *streams;
  uint8_t *sign_mantissa;
  uint32_t rows, cols, rbs, ncg, upr;
  uint32_t stream_rows;    // that `streams` has
  uint32_t vec;            // rows of the weight on 16-byte boundaries
};

// a lane's 16 elements of a half tile, zeros past the matrix
__device__ __forceinline__ void load_half(const PackWeight &a, uint32_t row, uint32_t col,
                                          uint32_t (&v)[8]) {
  const uint16_t *p = a.w + (size_t)row * a.cols + col;
  if (a.vec && row < a.rows && col + 16u <= a.cols) {
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < 8; ++j) {
    const uint32_t lo = row < a.rows && col + 2 * j < a.cols ? p[2 * j] : 0u;
    const uint32_t hi = row < a.rows && col + 2 * j + 1 < a.cols ? p[2 * j + 1] : 0u;
    v[j] = lo | hi << 16;
  }
}

// A warp per unit.  WRITE = false: the longest lane's words into unit_rows[unit];
// WRITE: the lanes' streams from row unit_rows[unit] on, and the sign/mantissa bytes.
template <bool WRITE>
__global__ void __launch_bounds__(256) linear_encode_kernel(const __grid_constant__ PackWeight a) {
  __shared__ uint32_t code_s[256], len_s[256];
  for (uint32_t i = threadIdx.x; i < 256; i += 256) {
    code_s[i] = a.table->code[i];
    len_s[i] = a.table->length[i];
  }
  __syncthreads();
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t units = (uint64_t)a.rbs * a.upr;
  for (uint64_t u = (blockIdx.x * 256ull + threadIdx.x) >> 5; u < units; u += gridDim.x * 8ull) {
    const uint32_t rb = (uint32_t)(u / a.upr), ku = (uint32_t)(u - (uint64_t)rb * a.upr);
    const uint32_t cg0 = ku * kUnitTiles, cg1 = min(cg0 + kUnitTiles, a.ncg);
    uint32_t bits = 0;
    uint32_t row = WRITE ? a.unit_rows[u] : 0u;
    const uint32_t end = WRITE ? min(a.unit_rows[u + 1], a.stream_rows) : 0u;
    uint64_t buf = 0;  // the next bits, `bits` of them
    for (uint32_t cg = cg0; cg < cg1; ++cg) {
#pragma unroll 1
      for (uint32_t h = 0; h < 2; ++h) {
        uint32_t v[8], sm[4] = {};
        load_half(a, 16u * rb + 8u * h + (lane >> 2), 64u * cg + 16u * (lane & 3u), v);
#pragma unroll
        for (uint32_t j = 0; j < 16; ++j) {
          const uint32_t e16 = (v[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
          const uint32_t exp = (e16 >> 7) & 0xFFu;
          if constexpr (!WRITE) {
            bits += len_s[exp];
          } else {
            const uint32_t sign = e16 >> 15, man = e16 & 0x7Fu;
            const uint32_t bits4 = (j & 3) == 0   ? man | sign << 15
                                   : (j & 3) == 1 ? man << 16 | sign << 31
                                   : (j & 3) == 2 ? man << 8 | sign << 23
                                                  : man << 24 | sign << 7;
            sm[j >> 2] = (j & 3) ? sm[j >> 2] | bits4 : bits4;
            buf |= (uint64_t)code_s[exp] << bits;
            bits += len_s[exp];
            if (bits >= 32) {
              // within the unit's rows, even if the words are not those that were counted
              if (row < end) a.streams[(size_t)row * 32u + lane] = (uint32_t)buf;
              ++row;
              buf >>= 32;
              bits -= 32;
            }
          }
        }
        if (WRITE)
          *reinterpret_cast<uint4 *>(a.sign_mantissa + ((size_t)rb * a.ncg + cg) * kTileElems +
                                     512u * h + 16u * lane) = make_uint4(sm[0], sm[1], sm[2], sm[3]);
      }
    }
    if constexpr (WRITE) {
      for (; row < end; ++row) {
        a.streams[(size_t)row * 32u + lane] = (uint32_t)buf;
        buf = 0;
      }
    } else {
      const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, (bits + 31u) >> 5);
      if (lane == 0) a.unit_rows[u] = most;
    }
  }
}

// unit_rows[0 .. units - 1] (words of each unit) to the units' first rows, unit_rows[units]
// the total; result: the total and the longest unit.  One thread block.
__global__ void __launch_bounds__(1024) linear_rows_kernel(uint32_t *unit_rows, uint64_t units,
                                                           uint32_t *result) {
  __shared__ uint32_t sums[32], most_s[32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t base = 0, most = 0;
  for (uint64_t u0 = 0; u0 < units; u0 += 1024) {
    const uint64_t u = u0 + tid;
    const uint32_t v = u < units ? unit_rows[u] : 0u;
    most = max(most, v);
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= (uint32_t)d) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (uint32_t w = 0; w < 32; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (u < units) unit_rows[u] = base + before + incl - v;
    base += all;
    __syncthreads();
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) most_s[warp] = most;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < 32; ++w) most = max(most, most_s[w]);
    unit_rows[units] = base;
    result[0] = base;
    result[1] = most;
  }
}

// ---- more tokens: tcgen05 product of the decoded tiles ------------------------
//
// D[token][row] = sum_c x[token][c] W[row][c]: A is x (128 tokens, TMA from the
// caller's rows), B the decoded tiles (bn rows; a 16 x 64 tile is 16 rows of 128
// bytes, so a TMA box of bn/16 row blocks is bn rows of 64 columns), both in the
// 128-byte swizzle, K in steps of 64.  One warp issues the copies, one the
// products, twelve move finished accumulators (two, in turn) out through the
// epilogue: a lane is a token, its columns consecutive rows of W, three warps
// taking groups of 16 in turn (with eight warps the epilogue takes longer than the product
// of 4096 columns where an activation is in it).
//   Of more than kPart steps the accumulators are moved out every kPart steps and added in
// registers (SUMS), because the tensor cores cut off what an addition leaves below their
// accumulator: one chain drifts by 1e-5 at 12288 columns and in proportion to the length, which a
// BF16 output shows as well, as values next to a border and where a residual cancels the sum.
// Tiles are then at most 240 rows wide: 80 sums of a thread in registers, for which the
// epilogue's threads take registers from the issuing ones.  What that costs is the epilogue, of
// which only two parts' products run ahead (4096 x 12288, 2048 tokens and a residual: 190 us for
// the call against 187 with one chain; 12288 x 4096 with silu and a multiplier: 198 and 190).
//   4096 x 12288 and 2048 tokens: 159 us for this kernel by itself, 1.30 PFLOP/s (one chain, BF16:
// 152), 190 for the call with the decoding, 224 where calls follow one another for seconds, under
// the power limit.  The copies of the next stages bound it (four of 240 rows fit).
constexpr int kGemmTokens = 128;
constexpr int kEpilogueWarps = 12;  // then a warp for the copies and one for the products
constexpr uint32_t kColStep = 4 * kEpilogueWarps;  // columns from one group of 16 of a warp to its next
constexpr int kGemmThreads = (kEpilogueWarps + 4) * 32;  // whole groups of four warps
// Registers of a thread while the roles run (SUMS): the launch's 128 shared out so that an
// epilogue thread's 80 sums and what it works with fit.  Spilled ones go past what the shared
// memory leaves of L1 and cost as much as the product.
constexpr int kLaunchRegs = 128, kSumRegs = 160, kIssueRegs = 32;
static_assert(kEpilogueWarps * kSumRegs + 4 * kIssueRegs <= (kEpilogueWarps + 4) * kLaunchRegs,
              "registers given out");
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct GemmArgs {
  Epilogue e;
  uint32_t tokens, rows, ncg;         // ncg: 64-column steps
  uint32_t bn, stages, tmem_cols;     // rows of W per tile, stages of shared memory
  uint32_t tiles_m, tiles;            // token tiles, all tiles
  uint32_t x_bytes;                   // of x per stage: the rows that a tile of tokens has at most
  int32_t *err;
  uint32_t spin_limit;
};

constexpr uint32_t kXBytes = kGemmTokens * 128;
constexpr uint32_t kPart = 8;      // steps of 64 columns between accumulators (SUMS)
constexpr uint32_t kSumRows = 240; // rows of a tile whose sums are in registers (SUMS)
constexpr uint32_t kSplitRows = 128;  // of a tile that thread blocks share
constexpr uint32_t kMaxStages = 8;
// an epilogue warp's buffer of 32 tokens and 16 rows: 16 bytes more per token, so that no
// two accesses meet in a bank
constexpr uint32_t kBufRow = 80, kBufBytes = 32 * kBufRow;
// barriers: full and empty per stage, two accumulators' full and empty; the tensor-memory
// address
constexpr uint32_t kGemmTail = 8 * (2 * kMaxStages + 4) + 16;
static_assert(kGemmTail % 16 == 0, "the epilogue's buffers stand behind");
constexpr uint32_t gemm_smem(uint32_t bn, uint32_t stages, bool buffers) {
  return 1024 + stages * (kXBytes + bn * 128) + kGemmTail + (buffers ? kEpilogueWarps * kBufBytes : 0);
}

// The warps that issue copies and products run their loops as whole warps, and one elected lane
// issues, by a predicate: operands that are known to be the same in every lane come from
// uniform registers, where a branch for one lane moves each of them there anew (4096 x 4096
// and 40 tokens: 17 us for the product, with branches 29 us).
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(e));
  return e;
}
__device__ __forceinline__ void expect_tx(uint32_t elected, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t elected, uint32_t dst, const CUtensorMap *map,
                                            int x, int y, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
      " @q cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];\n}\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t elected, uint32_t dst, const CUtensorMap *map,
                                            int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %7, 0;\n"
      " @q cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4, %5}], [%6];\n}\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void umma(uint32_t elected, uint32_t d, uint64_t a, uint64_t b,
                                     uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(elected)
      : "memory");
}

// K-major operand in the 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// The epilogue of a lane's token and 16 rows, 16 bytes at a time, its operands asked for first.
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
__device__ __forceinline__ void epilogue16(const Epilogue &e, float (&v)[16], uint32_t token,
                                           uint32_t row) {
  float m[16], r[16];
  if (e.mul) load16(e.mul, (size_t)token * e.mul_stride + row, e.flags & kMulF32, m);
  if (e.res) load16(e.res, (size_t)token * e.res_stride + row, e.flags & kResF32, r);
  if (e.bias) {
    float b[16];
    if (e.flags & kBiasVec) {
      load16(e.bias, row, e.flags & kBiasF32, b);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 16; ++j) b[j] = load_any(e.bias, row + j, e.flags & kBiasF32);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += b[j];
  }
  activate<16>(v, e.act);
  if (e.mul) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= m[j];
  }
  if (e.res) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += r[j];
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

// The epilogue where rows are not on 16-byte boundaries or end early, and where sums take the
// registers: 32 tokens and 16 rows, which lie in the warp's buffer, so that the lanes'
// accesses are next to one another.  A lane has four consecutive rows of every eighth token
// (4099 x 4096 and 1024 tokens with silu, multiplier and residual: 62 us for the call; with
// operands widened as each arrives and a branch per activation 82).
__device__ __forceinline__ void sts128(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w)
               : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 v = lds128(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}

// four values in another thread block's shared memory
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n"
      " ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// A lane's four values of each of its four tokens as they are in memory, and what they stand
// for: what widens them waits for them, so it stands behind all of the loads.  VEC: 16-byte
// boundaries and all four there; otherwise the first `n`, one by one.
template <bool VEC>
struct Quads {
  uint32_t w[4][4];
  // `there`: bit k for token k
  __device__ __forceinline__ void load(const void *p, size_t i, size_t step, bool f32, uint32_t there,
                                       uint32_t n) {
    const uint8_t *q = static_cast<const uint8_t *>(p) + (f32 ? 4 * i : 2 * i);
    step *= f32 ? 4 : 2;
    if (!VEC) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k, q += step)
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          if (j < n && there >> k & 1u)
            w[k][j] = f32 ? reinterpret_cast<const uint32_t *>(q)[j] : reinterpret_cast<const uint16_t *>(q)[j];
    } else if (f32) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k, q += step)
        if (there >> k & 1u) {
          const uint4 u = *reinterpret_cast<const uint4 *>(q);
          w[k][0] = u.x, w[k][1] = u.y, w[k][2] = u.z, w[k][3] = u.w;
        }
    } else {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k, q += step)
        if (there >> k & 1u) {
          const uint2 u = *reinterpret_cast<const uint2 *>(q);
          w[k][0] = u.x, w[k][1] = u.y;
        }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(bool f32, F f) const {
    if (VEC && !f32) {
#pragma unroll
      for (uint32_t j = 0; j < 16; ++j)
        f(j, __uint_as_float(j % 2 ? w[j / 4][j % 4 / 2] & 0xFFFF0000u : w[j / 4][j % 4 / 2] << 16));
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 16; ++j) f(j, __uint_as_float(w[j / 4][j % 4] << (f32 ? 0 : 16)));
    }
  }
};

template <bool VEC>
__device__ __forceinline__ void epilogue_block(const Epilogue &e, uint32_t buf, uint32_t token0,
                                               uint32_t row0, uint32_t tokens, uint32_t rows) {
  const uint32_t lane = threadIdx.x & 31, row = row0 + 4u * (lane & 3u), token = token0 + (lane >> 2);
  const uint32_t at = buf + (lane >> 2) * kBufRow + 16u * (lane & 3u);
  const uint32_t n = row < rows ? (VEC ? 4u : min(rows - row, 4u)) : 0u;
  const bool mul32 = e.flags & kMulF32, res32 = e.flags & kResF32;
  uint32_t there = 0;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) there |= n && token + 8u * k < tokens ? 1u << k : 0u;
  Quads<VEC> m, r;
  if (e.mul) m.load(e.mul, (size_t)token * e.mul_stride + row, 8ull * e.mul_stride, mul32, there, n);
  if (e.res) r.load(e.res, (size_t)token * e.res_stride + row, 8ull * e.res_stride, res32, there, n);
  __syncwarp();  // the buffer is written
  float v[16];
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {
    const float4 q = lds_f4(at + 8u * k * kBufRow);
    v[4 * k] = q.x, v[4 * k + 1] = q.y, v[4 * k + 2] = q.z, v[4 * k + 3] = q.w;
  }
  if (e.bias) {
    float b[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) b[j] = j < n ? load_any(e.bias, row + j, e.flags & kBiasF32) : 0.f;
#pragma unroll
    for (uint32_t j = 0; j < 16; ++j) v[j] += b[j & 3u];
  }
  activate<8>(v, e.act);
  activate<8>(v + 8, e.act);
  if (e.mul) m.each(mul32, [&](uint32_t j, float f) { v[j] *= f; });
  if (e.res) r.each(res32, [&](uint32_t j, float f) { v[j] += f; });
  uint8_t *p = static_cast<uint8_t *>(e.y);
  const size_t i = (size_t)token * e.y_stride + row;
  p += e.flags & kOutF32 ? 4 * i : 2 * i;
  const size_t step = e.flags & kOutF32 ? 32ull * e.y_stride : 16ull * e.y_stride;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k, p += step) {
    if (!(there >> k & 1u)) continue;
    const float *q = v + 4 * k;
    if (e.flags & kOutF32) {
      float *y = reinterpret_cast<float *>(p);
      if (VEC) *reinterpret_cast<float4 *>(y) = make_float4(q[0], q[1], q[2], q[3]);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (!VEC && j < n) y[j] = q[j];
    } else {
      uint16_t *y = reinterpret_cast<uint16_t *>(p);
      if (VEC) *reinterpret_cast<uint2 *>(y) = make_uint2(bf16_pair(q[0], q[1]), bf16_pair(q[2], q[3]));
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (!VEC && j < n) y[j] = (uint16_t)bf16_bits(q[j]);
    }
  }
  __syncwarp();  // the buffer may be written again
}

// SPLIT: a cluster of thread blocks shares a tile, each with a part of the columns of x; the
// parts' sums meet in shared memory, and each thread block adds a share of the tile's rows
// of W over the cluster, in order, for the epilogue.
// VEC: rows of y, multiplier and residual take 16-byte accesses, and W's end with a group of four.
template <bool SUMS, bool SPLIT, bool VEC>
__global__ void __launch_bounds__(kGemmThreads, 1)
    df11_linear_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                            const __grid_constant__ CUtensorMap map_w,
                            const __grid_constant__ GemmArgs ga) {
  const uint32_t S = ga.stages, bn = ga.bn, stage_bytes = kXBytes + bn * 128u;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S * stage_bytes;
  // full[S], empty[S], acc_full[2], acc_empty[2], the tensor-memory address
  auto full = [&](uint32_t i) { return bars + 8u * i; };
  auto empty = [&](uint32_t i) { return bars + 8u * (kMaxStages + i); };
  auto acc_full = [&](uint32_t i) { return bars + 8u * (2 * kMaxStages + i); };
  auto acc_empty = [&](uint32_t i) { return bars + 8u * (2 * kMaxStages + 2 + i); };
  const uint32_t taddr_s = bars + 8u * (2 * kMaxStages + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), kEpilogueWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kEpilogueWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(taddr_s),
                 "r"(ga.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(taddr_s);
  pdl_wait();  // the decoded weight, and x, come from the kernels before
  bool failed = false;
  // the tiles of this thread block and its steps of 64 columns: asked for where they are used,
  // so that they stay in uniform registers
  auto first_tile = [&]() { return SPLIT ? blockIdx.x / cluster_size() : blockIdx.x; };
  auto tile_step = [&]() { return SPLIT ? ga.tiles : gridDim.x; };
  auto col_begin = [&]() { return SPLIT ? ga.ncg * cluster_rank() / cluster_size() : 0u; };
  auto col_end = [&]() { return SPLIT ? ga.ncg * (cluster_rank() + 1) / cluster_size() : ga.ncg; };

  constexpr bool kShare = SUMS && !SPLIT;
  auto leave = [&]() {  // every warp is here before the tensor memory goes
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kEpilogueWarps + 1) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(ga.tmem_cols)
                   : "memory");
    }
  };
  if (warp < kEpilogueWarps) {
    if constexpr (kShare) more_registers<kSumRegs>();
    uint32_t n = 0;
    const uint32_t quarter = warp & 3, half = 16u * (warp >> 2);
    const uint32_t lanes = tmem + ((32u * quarter) << 16);
    // 16 of the lane's columns
    auto read16 = [&](uint32_t src, float (&v)[16]) {
      uint32_t u[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
          "%11, %12, %13, %14, %15}, [%16];"
          : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
            "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]),
            "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
          : "r"(src)
          : "memory");
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(u[j]);
    };
    const uint32_t buf = bars + kGemmTail + kBufBytes * warp;
    // the epilogue of the warp's 32 tokens and 16 rows, some of them there
    auto write16 = [&](float (&v)[16], uint32_t token0, uint32_t row) {
      if (!SUMS && VEC && row + 16 <= ga.rows) {
        if (token0 + lane < ga.tokens) epilogue16(ga.e, v, token0 + lane, row);
      } else {
        const uint32_t p = buf + lane * kBufRow;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          sts128(p + 16u * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        epilogue_block<VEC>(ga.e, buf, token0, row, ga.tokens, ga.rows);
      }
    };
    auto acquire = [&]() {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full(n & 1), (n >> 1) & 1u, ga.spin_limit)))
        failed = true;
      tc_fence_after();
      return !failed;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(n & 1));
      ++n;
    };
    for (uint32_t tile = first_tile(); tile < ga.tiles && !failed; tile += tile_step()) {
      const uint32_t tn = tile / ga.tiles_m, tm = tile - tn * ga.tiles_m;
      const uint32_t token0 = tm * kGemmTokens + 32u * quarter;
      const bool some = token0 < ga.tokens;
      if constexpr (SUMS) {
        // groups of 16 rows of W that a warp has
        constexpr uint32_t kGroups = ((SPLIT ? kSplitRows : kSumRows) + kColStep - 1) / kColStep;
        float sum[kGroups][16];
        const uint32_t cb = col_begin();
#pragma unroll
        for (uint32_t g = 0; g < kGroups; ++g)
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[g][j] = 0.f;
        for (uint32_t c0 = cb; c0 < col_end(); c0 += kPart) {
          if (!acquire()) break;
#pragma unroll
          for (uint32_t g = 0; g < kGroups; ++g) {
            if (kColStep * g + half >= bn) break;
            float v[16];
            read16(lanes + (n & 1u) * bn + kColStep * g + half, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[g][j] += v[j];
          }
          release();
        }
        if (failed) break;
        if constexpr (SPLIT) {
          // every product is done, so the stages' memory is free: [token][row], 4 rows more
#pragma unroll
          for (uint32_t g = 0; g < kGroups; ++g) {
            if (kColStep * g + half >= bn) break;
            const uint32_t p = base + 4u * ((32u * quarter + lane) * (bn + 4u) + kColStep * g + half);
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              sts128(p + 16u * j, sum[g][4 * j], sum[g][4 * j + 1], sum[g][4 * j + 2], sum[g][4 * j + 3]);
          }
        } else {
#pragma unroll 1  // one copy of the epilogue, the sums moved to its registers
          for (uint32_t c = half; some && c < bn && tn * bn + c < ga.rows; c += kColStep) {
            write16(sum[0], token0, tn * bn + c);
#pragma unroll
            for (uint32_t g = 0; g + 1 < kGroups; ++g)
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[g][j] = sum[g + 1][j];
          }
        }
      } else {
        if (!acquire()) break;
        for (uint32_t c = half; c < bn && tn * bn + c < ga.rows; c += kColStep) {
          float v[16];
          read16(lanes + (n & 1u) * bn + c, v);
          if (some) write16(v, token0, tn * bn + c);
        }
        release();
      }
    }
    if (failed && lane == 0) report(ga.err, DF11_DEV_ERR_TIMEOUT);
    // in the branch: code behind it would have to do with the fewer registers
    if constexpr (kShare) leave();
  } else {  // one group of four warps, two of them without work
    if constexpr (kShare) fewer_registers<kIssueRegs>();
    if (warp == kEpilogueWarps) {
      const uint32_t elected = elect();
      uint32_t k = 0, s = 0, par = 0;  // copies so far; the stage, and its uses' parity
      for (uint32_t tile = first_tile(); tile < ga.tiles && !failed; tile += tile_step()) {
        const uint32_t tn = tile / ga.tiles_m, tm = tile - tn * ga.tiles_m;
        for (uint32_t c = col_begin(); c < col_end(); ++c, ++k) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty(s), par ^ 1u, ga.spin_limit))) {
            failed = true;
            break;
          }
          const uint32_t dst = base + s * stage_bytes;
          expect_tx(elected, full(s), ga.x_bytes + bn * 128u);
          tma_load_2d(elected, dst, &map_x, (int)(64u * c), (int)(tm * kGemmTokens), full(s));
          tma_load_4d(elected, dst + kXBytes, &map_w, 0, 0, (int)c, (int)(tn * (bn / 16)), full(s));
          if (++s == S) {
            s = 0;
            par ^= 1u;
          }
        }
      }
      pdl_launch_dependents();
      // no copy in flight into this thread block's shared memory when it ends
      for (uint32_t j = k > S ? k - S : 0; j < k; ++j)
        if (!mbar_wait(full(j % S), (j / S) & 1u, ga.spin_limit)) failed = true;
      if (failed && lane == 0) report(ga.err, DF11_DEV_ERR_TIMEOUT);
    } else if (warp == kEpilogueWarps + 1) {
      // fp32 accumulators, BF16 operands, both K-major
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((bn / 8) << 17) |
                             ((kGemmTokens / 16) << 24);
      const uint32_t elected = elect();
      uint32_t k = 0, n = 0, s = 0, par = 0;
      for (uint32_t tile = first_tile(); tile < ga.tiles && !failed; tile += tile_step()) {
        uint32_t d = 0;
        for (uint32_t c = col_begin(); c < col_end(); ++c, ++k) {
          const uint32_t cb = col_begin(), ce = col_end();
          const bool first = SUMS ? (c - cb) % kPart == 0 : c == cb;  // into the other accumulator
          const bool last = c + 1 == ce || (SUMS && (c + 1 - cb) % kPart == 0);
          if (first) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_empty(n & 1), ((n >> 1) & 1u) ^ 1u,
                                                    ga.spin_limit))) {
              failed = true;
              break;
            }
            tc_fence_after();
            d = tmem + (n & 1u) * bn;
          }
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(full(s), par, ga.spin_limit))) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint64_t ad = sw128_desc(base + s * stage_bytes);
          const uint64_t bd = sw128_desc(base + s * stage_bytes + kXBytes);
  #pragma unroll
          for (int j = 0; j < 4; ++j)  // K = 16: 32 bytes on
            umma(elected, d, ad + 2u * j, bd + 2u * j, idesc, !first || j ? 1u : 0u);
          umma_commit(elected, empty(s));
          if (last) umma_commit(elected, acc_full(n & 1));
          if (last) ++n;
          if (++s == S) {
            s = 0;
            par ^= 1u;
          }
        }
      }
      // no product in flight when the tensor memory goes
      for (uint32_t j = k > S ? k - S : 0; j < k; ++j)
        if (!mbar_wait(empty(j % S), (j / S) & 1u, ga.spin_limit)) failed = true;
      if (failed && lane == 0) report(ga.err, DF11_DEV_ERR_TIMEOUT);
    }
    if constexpr (kShare) leave();
  }
  if constexpr (SPLIT) {
    cluster_sync();
    if (warp < kEpilogueWarps) {
      const uint32_t buf = bars + kGemmTail + kBufBytes * warp;
      const uint32_t ctas = cluster_size(), rank = cluster_rank(), tile = first_tile();
      const uint32_t tn = tile / ga.tiles_m, tm = tile - tn * ga.tiles_m, share = bn / ctas;
      for (uint32_t b = warp; b < 4u * (share / 16u); b += kEpilogueWarps) {
        const uint32_t t0 = 32u * (b & 3u), c0 = rank * share + 16u * (b >> 2);
        if (tm * kGemmTokens + t0 >= ga.tokens || tn * bn + c0 >= ga.rows) continue;
        const uint32_t p = base + 4u * ((t0 + (lane >> 2)) * (bn + 4u) + c0 + 4u * (lane & 3u));
        float4 sum[4];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t r = 0; r < ctas; ++r) {
          float4 v[4];
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) v[k] = ld_cluster_f4(p + 32u * k * (bn + 4u), r);
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            sum[k].x += v[k].x, sum[k].y += v[k].y, sum[k].z += v[k].z, sum[k].w += v[k].w;
        }
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          sts128(buf + (8u * k + (lane >> 2)) * kBufRow + 16u * (lane & 3u), sum[k].x, sum[k].y, sum[k].z,
                 sum[k].w);
        epilogue_block<VEC>(ga.e, buf, tm * kGemmTokens + t0, tn * bn + c0, ga.tokens, ga.rows);
      }
    }
    cluster_sync();  // nobody reads this thread block's sums any more
  }
  if constexpr (!kShare) leave();
}

// ---- host side ------------------------------------------------------------------

// Tokens up to which a call decodes and multiplies in one kernel (12288 x 4096: 48 us for
// 24 tokens; decoded first, the decoding takes 34 us and the product 18).
constexpr uint32_t kFusedMax = 32;

uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Longest row of x that the fused kernel takes: it reads 32 rows by 32-bit offsets.
constexpr uint32_t kMaxStride = 1u << 25;

// x as the kernels read it: 16-byte loads of whole 16-column groups
bool needs_pack(const df11_linear &op, uint32_t cols) {
  return cols % 16 || op.x_stride % 8 || !aligned(op.x, 16) || op.x_stride > kMaxStride;
}

LWeight device_weight(const df11_linear_weight &w) {
  const df11_linear_params &p = w.params;
  LWeight l{};
  l.streams = w.streams;
  l.unit_rows = w.unit_rows;
  l.sign_mantissa = w.sign_mantissa;
  l.table = static_cast<const LinearTable *>(w.table);
  l.rbs = (p.rows + kTileRows - 1) / kTileRows;
  l.ncg = (p.cols + kTileCols - 1) / kTileCols;
  l.upr = (l.ncg + kUnitTiles - 1) / kUnitTiles;
  l.max_words = p.max_words;
  l.stream_rows = p.stream_rows;
  l.one = 1;
  l.k64 = 65536;
  return l;
}

uint64_t padded(const df11_linear_params &p) {
  return round_up(p.rows, kTileRows) * round_up(p.cols, kTileCols);
}

// the thread blocks of a launch over its weights, by units
void split_units(const df11_linear_weight *ws, int count, uint32_t warps, uint64_t budget,
                 uint64_t *ctas) {
  uint32_t units[DF11_MAX_BATCH];
  for (int i = 0; i < count; ++i) {
    const LWeight l = device_weight(ws[i]);
    units[i] = (uint32_t)ordered_units(l.rbs, l.upr, warps);
  }
  split_blocks(units, count, budget, ctas);
}

uint32_t longest_stream(const df11_linear_weight *ws, int count) {
  uint32_t m = 1;
  for (int i = 0; i < count; ++i) m = ws[i].params.max_words > m ? ws[i].params.max_words : m;
  return m;
}

struct Plan {
  bool fused = false;
  uint32_t nb = 1, warps = 0;            // groups of 8 tokens, warps per thread block (fused)
  uint64_t ctas[DF11_MAX_BATCH] = {};    // thread blocks per weight (fused)
  uint32_t slots[DF11_MAX_BATCH] = {};
  uint64_t part[DF11_MAX_BATCH] = {};    // workspace offsets: partial sums or decoded weight
  uint64_t packed[DF11_MAX_BATCH] = {};  // packed activations
  uint64_t bytes = 0;
  size_t smem = 0;
};

// warps per thread block whose buffers fit in shared memory beside the table
uint32_t warps_for(uint32_t max_words) {
  return decode_smem(max_words, kManyWarps) <= 227 * 1024 ? kManyWarps : kFewWarps;
}

// Percentage of the SM's memory asked for as shared memory: no more than the kernels need,
// since the activations are read through the rest (5% on 151936 x 4096 and 8 tokens).
int carveout(uint32_t warps) { return warps == kManyWarps ? 80 : 60; }

using LinearKernel = void (*)(LBatch);
LinearKernel pick_kernel(uint32_t nb, uint32_t warps, int &instance) {
  instance = nb == 1 ? (warps == kManyWarps ? 66 : 67) : (nb == 2 ? 68 : 69);
  if (nb == 1) return warps == kManyWarps ? df11_linear_kernel<1, kManyWarps> : df11_linear_kernel<1, kFewWarps>;
  return nb == 2 ? df11_linear_kernel<2, kFewWarps> : df11_linear_kernel<4, kFewWarps>;
}

// What a group of at most DF11_MAX_BATCH weights needs from the workspace.
df11_status make_plan(const df11_linear_weight *ws, const df11_linear *ops, int count, Plan &pl) {
  uint32_t max_batch = 0, max_cols = 0;
  uint64_t off = 0;
  for (int i = 0; i < count; ++i) {
    max_batch = max_batch > ops[i].batch ? max_batch : ops[i].batch;
    max_cols = max_cols > ws[i].params.cols ? max_cols : ws[i].params.cols;
    pl.packed[i] = off;
    if (needs_pack(ops[i], ws[i].params.cols))
      off += round_up(2ull * ops[i].batch * round_up(ws[i].params.cols, kTileCols), 256);
  }
  pl.fused = max_batch <= kFusedMax && max_cols <= kMaxStride;
  if (!pl.fused) {
    for (int i = 0; i < count; ++i) {
      pl.part[i] = off;
      off += round_up(2ull * padded(ws[i].params), 256);
    }
    pl.bytes = off;
    return DF11_OK;
  }
  pl.nb = max_batch <= 8 ? 1 : (max_batch <= 16 ? 2 : 4);
  const uint32_t words = longest_stream(ws, count);
  pl.warps = pl.nb > 1 ? kFewWarps : warps_for(words);
  pl.smem = decode_smem(words, pl.warps);
  int instance = 0;
  uint64_t budget = 0;
  const LinearKernel kern = pick_kernel(pl.nb, pl.warps, instance);
  const df11_status st = prepare(kern, 32 * pl.warps, pl.smem, instance, budget, carveout(pl.warps));
  if (st != DF11_OK) return st;
  split_units(ws, count, pl.warps, budget, pl.ctas);
  for (int i = 0; i < count; ++i) {
    const LWeight l = device_weight(ws[i]);
    const uint64_t units = ordered_units(l.rbs, l.upr, pl.warps);
    const uint64_t per_group = (uint64_t)l.upr * pl.warps;
    const uint64_t per = (units + pl.ctas[i] - 1) / pl.ctas[i];
    uint64_t slots = (per + per_group - 2) / per_group + 1;
    if (slots > units / per_group) slots = units / per_group;
    pl.slots[i] = (uint32_t)slots;
    pl.part[i] = off;
    off += round_up(pl.ctas[i] * slots * pl.warps * 16 * 8 * pl.nb * sizeof(float), 256);
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
            (op.residual_type == DF11_F32 ? kResF32 : 0u) | (op.y_type == DF11_F32 ? kOutF32 : 0u) |
            (aligned(op.bias, 16) ? kBiasVec : 0u);
  return e;
}

bool known_type(int32_t t) { return t == DF11_BF16 || t == DF11_F32; }
uintptr_t type_bytes(int32_t t) { return t == DF11_F32 ? 4 : 2; }

df11_status check_shape(uint32_t rows, uint32_t cols) {
  if (rows == 0 || cols == 0) return DF11_ERR_INVALID;
  if (round_up(rows, kTileRows) * round_up(cols, kTileCols) >= (1ull << 32)) return DF11_ERR_TOO_LARGE;
  return DF11_OK;
}

df11_status check_weight(const df11_linear_weight &w) {
  const df11_linear_params &p = w.params;
  const df11_status st = check_shape(p.rows, p.cols);
  if (st != DF11_OK) return st;
  if (!w.streams || !w.unit_rows || !w.sign_mantissa || !w.table) return DF11_ERR_NULL;
  if (!aligned(w.streams, 16) || !aligned(w.sign_mantissa, 16) || !aligned(w.table, 16) ||
      !aligned(w.unit_rows, 4))
    return DF11_ERR_ALIGN;
  if (p.max_words < 1 || p.max_words > kMaxWords) return DF11_ERR_FORMAT;
  const LWeight l = device_weight(w);
  if (p.stream_rows > (uint64_t)l.rbs * l.upr * p.max_words) return DF11_ERR_FORMAT;
  return DF11_OK;
}

// One weight and its operation; DF11_OK for one that does nothing, too.
df11_status check_op(const df11_linear_weight &w, const df11_linear &op) {
  if (op.activation < DF11_ACT_NONE || op.activation > DF11_ACT_SILU) return DF11_ERR_INVALID;
  if (!known_type(op.y_type) || (op.bias && !known_type(op.bias_type)) ||
      (op.multiplier && !known_type(op.multiplier_type)) ||
      (op.residual && !known_type(op.residual_type)))
    return DF11_ERR_INVALID;
  const df11_status st = check_weight(w);
  if (st != DF11_OK) return st;
  if (op.batch == 0) return DF11_OK;
  if (op.batch > DF11_LINEAR_MAX_BATCH) return DF11_ERR_TOO_LARGE;
  if (!op.x || !op.y) return DF11_ERR_NULL;
  const uint32_t rows = w.params.rows;
  if (op.x_stride < w.params.cols || op.y_stride < rows ||
      (op.multiplier && op.multiplier_stride < rows) || (op.residual && op.residual_stride < rows))
    return DF11_ERR_INVALID;
  if (!aligned(op.x, 2) || !aligned(op.y, type_bytes(op.y_type)) ||
      !aligned(op.bias, type_bytes(op.bias_type)) ||
      !aligned(op.multiplier, type_bytes(op.multiplier_type)) ||
      !aligned(op.residual, type_bytes(op.residual_type)))
    return DF11_ERR_ALIGN;
  return DF11_OK;
}

// y is written while other thread blocks still read x, the bias and the rows of the other
// operands; those may be y itself, since every element is read by the thread that writes it.
bool output_is_read(const df11_linear_weight &w, const df11_linear &op) {
  const uint64_t rows = w.params.rows, yb = type_bytes(op.y_type);
  const Rows y{op.y, op.batch, rows * yb, op.y_stride * yb};
  if (share_memory(y, Rows{op.x, op.batch, 2ull * w.params.cols, 2ull * op.x_stride})) return true;
  if (share_memory(y, Rows{op.bias, 1, rows * type_bytes(op.bias_type), 0})) return true;
  auto other = [&](const void *p, uint64_t stride, int32_t type) {
    if (p == op.y && type == op.y_type && (op.batch == 1 || stride == op.y_stride)) return false;
    return share_memory(y, Rows{p, op.batch, rows * type_bytes(type), stride * type_bytes(type)});
  };
  return other(op.multiplier, op.multiplier_stride, op.multiplier_type) ||
         other(op.residual, op.residual_stride, op.residual_type);
}

df11_status check_call(const df11_linear_weight *ws, const df11_linear *ops, int count) {
  if (count < 0) return DF11_ERR_INVALID;
  if (count && (!ws || !ops)) return DF11_ERR_NULL;
  for (int i = 0; i < count; ++i) {
    const df11_status st = check_op(ws[i], ops[i]);
    if (st != DF11_OK) return st;
  }
  return DF11_OK;
}

// calls f(weights, ops, count) for the next group of at most DF11_MAX_BATCH weights
// with work, until one fails
template <typename F>
df11_status for_groups(const df11_linear_weight *ws, const df11_linear *ops, int count, F f) {
  df11_linear_weight w[DF11_MAX_BATCH];
  df11_linear o[DF11_MAX_BATCH];
  int m = 0;
  for (int i = 0; i < count; ++i) {
    if (ops[i].batch) {
      w[m] = ws[i];
      o[m] = ops[i];
      ++m;
    }
    if (m && (m == DF11_MAX_BATCH || i + 1 == count)) {
      const df11_status st = f(w, o, m);
      if (st != DF11_OK) return st;
      m = 0;
    }
  }
  return DF11_OK;
}

// activations as the kernels read them: the caller's, or packed
struct Activations {
  const uint16_t *x;
  uint32_t stride, cols;
};

df11_status launch_fused(const df11_linear_weight *ws, const df11_linear *ops, int count,
                         const Plan &pl, uint8_t *work, const Activations *x, int32_t *d_err,
                         cudaStream_t s) {
  LBatch lb{};
  FBatch fb{};
  lb.err = d_err;
  lb.count = fb.count = count;
  lb.spin_limit = kSpinLimit;
  fb.nb = pl.nb;
  fb.warps = pl.warps;
  uint32_t cta = 0, blocks = 0;
  for (int i = 0; i < count; ++i) {
    LTensor &l = lb.t[i];
    l.w = device_weight(ws[i]);
    l.x = x[i].x;
    l.x_stride = x[i].stride;
    l.x_cols = x[i].cols;
    l.batch = ops[i].batch;
    l.slots = pl.slots[i];
    l.part = reinterpret_cast<float *>(work + pl.part[i]);
    l.cta_begin = cta;
    cta += (uint32_t)pl.ctas[i];
    FTensor &f = fb.t[i];
    f.e = make_epilogue(ops[i]);
    f.part = l.part;
    f.ctas = (uint32_t)pl.ctas[i];
    f.slots = l.slots;
    f.rbs = l.w.rbs;
    f.upr = l.w.upr;
    f.rows = ws[i].params.rows;
    f.batch = ops[i].batch;
    f.block_begin = blocks;
    blocks += (l.w.rbs * 16u * ops[i].batch + kFinishThreads - 1) / kFinishThreads;
  }
  lb.cta_end = cta;
  int instance = 0;
  const LinearKernel kern = pick_kernel(pl.nb, pl.warps, instance);
  const df11_status st = launch_pdl(kern, dim3(cta), 32 * pl.warps, pl.smem, s, lb);
  if (st != DF11_OK) return st;
  return launch_pdl(df11_linear_finish_kernel, dim3(blocks), kFinishThreads, 0, s, fb);
}

// the weights decoded into tiles and activations packed, one launch
df11_status launch_unpack(const df11_linear_weight *ws, int count, uint16_t *const *out,
                          const PackArgs *x, int32_t *d_err, cudaStream_t s) {
  UArgs ua{};
  const uint32_t words = longest_stream(ws, count), warps = warps_for(words);
  const size_t smem = decode_smem(words, warps);
  uint64_t budget = 0, ctas[DF11_MAX_BATCH];
  void (*kern)(UArgs) = warps == kManyWarps ? df11_linear_unpack_kernel<kManyWarps>
                                            : df11_linear_unpack_kernel<kFewWarps>;
  const df11_status st = prepare(kern, 32 * warps, smem, warps == kManyWarps ? 71 : 72, budget,
                                 carveout(warps));
  if (st != DF11_OK) return st;
  split_units(ws, count, warps, budget, ctas);
  ua.err = d_err;
  ua.count = count;
  ua.spin_limit = kSpinLimit;
  for (int i = 0; i < count; ++i) {
    ua.w[i] = device_weight(ws[i]);
    ua.out[i] = out[i];
    if (x) ua.x[i] = x[i];
    ua.cta_begin[i + 1] = ua.cta_begin[i] + (uint32_t)ctas[i];
  }
  return launch_pdl(kern, dim3(ua.cta_begin[count]), 32 * warps, smem, s, ua);
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

using GemmKernel = void (*)(CUtensorMap, CUtensorMap, GemmArgs);
// variant: one chain per tile, sums in parts, tiles shared by a cluster
GemmKernel pick_gemm(int variant, bool vec) {
  if (variant == 2) return vec ? df11_linear_gemm_kernel<true, true, true> : df11_linear_gemm_kernel<true, true, false>;
  if (variant == 1) return vec ? df11_linear_gemm_kernel<true, false, true> : df11_linear_gemm_kernel<true, false, false>;
  return vec ? df11_linear_gemm_kernel<false, false, true> : df11_linear_gemm_kernel<false, false, false>;
}

df11_status launch_gemm(const df11_linear &op, uint32_t rows, uint32_t cols, const uint16_t *w,
                        const Activations &x, int32_t *d_err, cudaStream_t s) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return DF11_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DF11_ERR_CUDA;
  const int sms = device_info(dev).sms;
  GemmArgs ga{};
  ga.e = make_epilogue(op);
  ga.tokens = op.batch;
  ga.rows = rows;
  ga.ncg = (uint32_t)(round_up(cols, kTileCols) / kTileCols);
  ga.tiles_m = (op.batch + kGemmTokens - 1) / kGemmTokens;
  ga.err = d_err;
  ga.spin_limit = kSpinLimit;
  auto vec_ok = [](const void *p, uint32_t stride, int32_t type) {
    return !p || (aligned(p, 16) && stride * type_bytes(type) % 16 == 0);
  };
  const bool vec = rows % 4 == 0 && vec_ok(op.y, op.y_stride, op.y_type) &&
           vec_ok(op.multiplier, op.multiplier_stride, op.multiplier_type) &&
           vec_ok(op.residual, op.residual_stride, op.residual_type);
  // The tile width and the number of thread blocks that share a tile for which the rounds over
  // the SMs cost least, in cycles: a step of 64 columns takes about 250 and two per row
  // (measured from 32 to 240 rows), a tile 1000 and 20 per row for its epilogue, and a
  // shared one 10000 more.  The wider and less shared one of two.  (500 x 8192 and 40 tokens:
  // 12 us with shared tiles, 27 without; 4096 x 4096 and 256 tokens: 25 and 19.)
  uint64_t cost = ~0ull;
  const bool sums = ga.ncg > kPart;
  uint32_t split = 1;
  for (uint32_t ctas = 1; ctas <= 8; ctas *= 2) {
    for (uint32_t bn = ctas > 1 ? kSplitRows : (sums ? kSumRows : 256); bn >= 16 * ctas; bn -= 16 * ctas) {
      const uint64_t tiles = (uint64_t)ga.tiles_m * ((rows + bn - 1) / bn);
      // whole clusters do not reach every SM
      if (ctas > 1 && (tiles * ctas > (uint64_t)sms * 7 / 8 || ga.ncg < 4 * ctas)) break;
      const uint64_t steps = (ga.ncg + ctas - 1) / ctas, rounds = (tiles * ctas + sms - 1) / sms;
      const uint64_t c = rounds * (steps * (250 + 2 * bn) + 1000 + 20 * bn) + (ctas > 1 ? 10000 : 0);
      if (c < cost) {
        cost = c;
        split = ctas;
        ga.bn = bn;
        ga.tiles = (uint32_t)tiles;
      }
    }
  }
  ga.stages = kMaxStages;
  const bool buffers = sums || split > 1 || !vec || rows % 16;
  while (gemm_smem(ga.bn, ga.stages, buffers) > 226 * 1024) --ga.stages;
  ga.tmem_cols = 32;
  while (ga.tmem_cols < 2 * ga.bn) ga.tmem_cols *= 2;
  CUtensorMap mx, mw;
  {
    const cuuint64_t dims[2] = {x.cols, op.batch}, strides[1] = {2ull * x.stride};
    // up to 128 tokens: only the rows that there are.  The others of the tile are whatever the
    // shared memory holds, and so are the accumulators' lanes of theirs, which nothing reads
    const uint32_t box_rows = op.batch < kGemmTokens ? (op.batch + 7u) / 8u * 8u : kGemmTokens;
    const cuuint32_t box[2] = {64, box_rows}, one[2] = {1, 1};
    ga.x_bytes = box_rows * 128u;
    if (encode(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(x.x), dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return DF11_ERR_CUDA;
  }
  {
    const cuuint64_t dims[4] = {64, 16, ga.ncg, (rows + 15u) / 16u};
    const cuuint64_t strides[3] = {128, 2048, 2048ull * ga.ncg};
    const cuuint32_t box[4] = {64, 16, 1, ga.bn / 16}, one[4] = {1, 1, 1, 1};
    if (encode(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(w), dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return DF11_ERR_CUDA;
  }
  const size_t smem = gemm_smem(ga.bn, ga.stages, buffers);
  uint64_t budget = 0;
  const int variant = split > 1 ? 2 : (sums ? 1 : 0);
  const GemmKernel kern = pick_gemm(variant, vec);
  const df11_status st = prepare(kern, kGemmThreads, smem, 73 + 2 * variant + vec, budget);
  if (st != DF11_OK) return st;
  if (split > 1)
    return launch_cluster(kern, ga.tiles * split, split, kGemmThreads, smem, s, mx, mw, ga);
  const uint32_t grid = ga.tiles < (uint32_t)sms ? ga.tiles : (uint32_t)sms;
  return launch_pdl(kern, dim3(grid), kGemmThreads, smem, s, mx, mw, ga);
}

df11_status check_linear_devices(const df11_linear_weight *ws, const df11_linear *ops, int count,
                                 const void *work) {
  for (int i = 0; i < count; ++i) {
    const void *ptrs[] = {ws[i].streams, ws[i].unit_rows, ws[i].sign_mantissa, ws[i].table,
                          ops[i].x,      ops[i].y,        ops[i].bias,         ops[i].multiplier,
                          ops[i].residual, i ? nullptr : work};
    const df11_status st = check_device_pointers(ptrs, (int)(sizeof(ptrs) / sizeof(*ptrs)));
    if (st != DF11_OK) return st;
  }
  return DF11_OK;
}

// The decode table of a code: its lengths (at most kMaxLength) and right-aligned codewords.
void make_table(const uint8_t len[256], const uint32_t code[256], LinearTable &t) {
  // bits that no codeword begins with (a code of one symbol has such): a length of one
  for (uint32_t &e : t.entry) e = 1;
  for (uint32_t e = 0; e < 256; ++e) {
    uint32_t c = 0;
    for (uint32_t i = 0; i < len[e]; ++i) c |= (code[e] >> i & 1u) << (len[e] - 1 - i);
    t.code[e] = (uint8_t)c;
    t.length[e] = len[e];
    if (len[e])
      for (uint32_t i = c; i < kEntries; i += 1u << len[e]) t.entry[i] = e << 7 | len[e];
  }
}

PackWeight pack_weight(const uint16_t *d_w, const df11_linear_params &p, uint32_t *unit_rows,
                       const void *table) {
  PackWeight a{};
  a.w = d_w;
  a.table = static_cast<const LinearTable *>(table);
  a.unit_rows = unit_rows;
  a.rows = p.rows;
  a.cols = p.cols;
  a.rbs = (p.rows + kTileRows - 1) / kTileRows;
  a.ncg = (p.cols + kTileCols - 1) / kTileCols;
  a.upr = (a.ncg + kUnitTiles - 1) / kUnitTiles;
  a.vec = p.cols % 8 == 0 && aligned(d_w, 16);
  return a;
}

uint32_t encode_grid(const PackWeight &a) {
  const uint64_t blocks = ((uint64_t)a.rbs * a.upr + 7) / 8;
  return (uint32_t)(blocks < 148 * 8 ? blocks : 148 * 8);
}

}  // namespace

extern "C" {

df11_status df11_linear_sizes(uint32_t rows, uint32_t cols, uint64_t *unit_rows_count,
                              uint64_t *sign_mantissa_bytes) {
  if (!unit_rows_count || !sign_mantissa_bytes) return DF11_ERR_NULL;
  const df11_status st = check_shape(rows, cols);
  if (st != DF11_OK) return st;
  *unit_rows_count = round_up(rows, kTileRows) / kTileRows *
                         (round_up(cols, kUnitTiles * kTileCols) / (kUnitTiles * kTileCols)) +
                     3;  // the units', the total, two results of the builder
  *sign_mantissa_bytes = round_up(rows, kTileRows) * round_up(cols, kTileCols);
  return DF11_OK;
}

df11_status df11_linear_weight_begin(const uint16_t *d_w, uint32_t rows, uint32_t cols,
                                     uint32_t *unit_rows, void *table, df11_linear_params *params,
                                     df11_stream_t stream) {
  if (!d_w || !unit_rows || !table || !params) return DF11_ERR_NULL;
  df11_status st = check_shape(rows, cols);
  if (st != DF11_OK) return st;
  if (!aligned(d_w, 2) || !aligned(unit_rows, 4) || !aligned(table, 16)) return DF11_ERR_ALIGN;
  const void *ptrs[] = {d_w, unit_rows, table};
  st = check_device_pointers(ptrs, 3);
  if (st != DF11_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  df11_linear_params p{};
  p.rows = rows;
  p.cols = cols;
  const uint64_t n = (uint64_t)rows * cols;
  uint64_t hist[256];
  st = df11_exponent_histogram(d_w, n, hist, stream);
  if (st != DF11_OK) return st;
  hist[0] += padded(p) - n;
  try {
    uint8_t len[256];
    uint32_t code[256];
    limited_code(hist, kMaxLength, len, code);
    std::vector<LinearTable> t(1);
    make_table(len, code, t[0]);
    if (cudaMemcpyAsync(table, t.data(), sizeof(LinearTable), cudaMemcpyHostToDevice, s) !=
            cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return DF11_ERR_CUDA;
  } catch (...) {
    return DF11_ERR_NOMEM;
  }
  const PackWeight a = pack_weight(d_w, p, unit_rows, table);
  const uint64_t units = (uint64_t)a.rbs * a.upr;
  uint32_t *result = unit_rows + units + 1;
  linear_encode_kernel<false><<<encode_grid(a), 256, 0, s>>>(a);
  linear_rows_kernel<<<1, 1024, 0, s>>>(unit_rows, units, result);
  uint32_t got[2] = {0, 0};
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyAsync(got, result, sizeof(got), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return DF11_ERR_CUDA;
  p.stream_rows = got[0];
  p.max_words = got[1];
  *params = p;
  return DF11_OK;
}

df11_status df11_linear_weight_finish(const uint16_t *d_w, const df11_linear_weight *weight,
                                      df11_stream_t stream) {
  if (!d_w || !weight) return DF11_ERR_NULL;
  df11_status st = check_weight(*weight);
  if (st != DF11_OK) return st;
  if (!aligned(d_w, 2)) return DF11_ERR_ALIGN;
  const void *ptrs[] = {d_w, weight->streams, weight->unit_rows, weight->sign_mantissa, weight->table};
  st = check_device_pointers(ptrs, 5);
  if (st != DF11_OK) return st;
  PackWeight a = pack_weight(d_w, weight->params, const_cast<uint32_t *>(weight->unit_rows),
                             weight->table);
  a.streams = const_cast<uint32_t *>(weight->streams);
  a.stream_rows = weight->params.stream_rows;
  a.sign_mantissa = const_cast<uint8_t *>(weight->sign_mantissa);
  linear_encode_kernel<true><<<encode_grid(a), 256, 0, (cudaStream_t)stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return DF11_ERR_CUDA;
  return queue_after_writes((cudaStream_t)stream);  // a product may be the next launch
}

df11_status df11_linear_unpack(const df11_linear_weight *weight, uint16_t *tiles, int32_t *d_err,
                               df11_stream_t stream) {
  if (!weight || !tiles) return DF11_ERR_NULL;
  df11_status st = check_weight(*weight);
  if (st != DF11_OK) return st;
  if (!aligned(tiles, 16) || (d_err && !aligned(d_err, 4))) return DF11_ERR_ALIGN;
  const void *ptrs[] = {tiles, weight->streams, weight->unit_rows, weight->sign_mantissa, weight->table};
  st = check_device_pointers(ptrs, 5);
  if (st != DF11_OK) return st;
  return launch_unpack(weight, 1, &tiles, nullptr, d_err, (cudaStream_t)stream);
}

df11_status df11_linear_workspace(const df11_linear_weight *weights, const df11_linear *ops,
                                  int count, size_t *bytes) {
  if (!bytes) return DF11_ERR_NULL;
  *bytes = 0;
  df11_status st = check_call(weights, ops, count);
  if (st != DF11_OK) return st;
  size_t most = 0;
  st = for_groups(weights, ops, count, [&](const df11_linear_weight *w, const df11_linear *o, int m) {
    Plan pl;
    for (int i = 0; i < m; ++i)
      if (output_is_read(w[i], o[i])) return DF11_ERR_INVALID;
    const df11_status r = make_plan(w, o, m, pl);
    if (r == DF11_OK && pl.bytes > most) most = pl.bytes;
    return r;
  });
  if (st == DF11_OK) *bytes = most;
  return st;
}

uint64_t df11_capture_id(df11_stream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo((cudaStream_t)stream, &status, &id) != cudaSuccess) {
    (void)cudaGetLastError();  // the legacy stream beside a capture: not in one
    return 0;
  }
  return status == cudaStreamCaptureStatusNone ? 0 : id;
}

int df11_event_done(void *event) {
  if (!event) return -1;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return -1;
  const cudaError_t e = cudaEventQuery(static_cast<cudaEvent_t>(event));
  (void)cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) (void)cudaGetLastError();  // clear this call's (non-sticky) error
  return e == cudaSuccess ? 1 : (e == cudaErrorNotReady ? 0 : -1);
}

df11_status df11_decode_linear(const df11_linear_weight *weights, const df11_linear *ops, int count,
                               void *workspace, size_t workspace_bytes, int32_t *d_err,
                               df11_stream_t stream) {
  df11_status st = check_call(weights, ops, count);
  if (st != DF11_OK) return st;
  if (d_err && !aligned(d_err, 4)) return DF11_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  // checked for every group before anything is queued
  st = for_groups(weights, ops, count, [&](const df11_linear_weight *w, const df11_linear *o, int m) {
    Plan pl;
    for (int i = 0; i < m; ++i)
      if (output_is_read(w[i], o[i])) return DF11_ERR_INVALID;
    df11_status r = make_plan(w, o, m, pl);
    if (r != DF11_OK) return r;
    if (!workspace) return DF11_ERR_NULL;
    if (!aligned(workspace, 256)) return DF11_ERR_ALIGN;
    if (pl.bytes > workspace_bytes) return DF11_ERR_INVALID;
    return check_linear_devices(w, o, m, workspace);
  });
  if (st != DF11_OK) return st;
  return for_groups(weights, ops, count, [&](const df11_linear_weight *w, const df11_linear *o, int m) {
    Plan pl;
    df11_status r = make_plan(w, o, m, pl);
    if (r != DF11_OK) return r;
    uint8_t *work = static_cast<uint8_t *>(workspace);
    Activations x[DF11_MAX_BATCH];
    PackArgs packs[DF11_MAX_BATCH] = {};
    for (int i = 0; i < m; ++i) {
      const uint32_t cols = w[i].params.cols;
      x[i] = Activations{o[i].x, o[i].x_stride, cols};
      if (!needs_pack(o[i], cols)) continue;
      PackArgs &pa = packs[i];
      pa.x = o[i].x;
      pa.out = reinterpret_cast<uint16_t *>(work + pl.packed[i]);
      pa.cols = cols;
      pa.out_cols = (uint32_t)round_up(cols, kTileCols);
      pa.batch = o[i].batch;
      pa.x_stride = o[i].x_stride;
      x[i] = Activations{pa.out, pa.out_cols, pa.out_cols};
      if (!pl.fused) continue;  // beside the decoding
      const uint64_t blocks = ((uint64_t)pa.batch * ((pa.out_cols + 255) / 256) + 7) / 8;
      r = launch_pdl(linear_pack_kernel, dim3((uint32_t)(blocks < 592 ? blocks : 592)), 256, 0, s, pa);
      if (r != DF11_OK) return r;
    }
    if (pl.fused) return launch_fused(w, o, m, pl, work, x, d_err, s);
    uint16_t *tiles[DF11_MAX_BATCH];
    for (int i = 0; i < m; ++i) tiles[i] = reinterpret_cast<uint16_t *>(work + pl.part[i]);
    r = launch_unpack(w, m, tiles, packs, d_err, s);
    for (int i = 0; i < m && r == DF11_OK; ++i)
      r = launch_gemm(o[i], w[i].params.rows, w[i].params.cols, tiles[i], x[i], d_err, s);
    return r;
  });
}

}  // extern "C"
