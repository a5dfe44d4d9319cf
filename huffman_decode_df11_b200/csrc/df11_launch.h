// df11_launch.h -- host code that the library's entry points share: checks of a
// tensor descriptor, the per-device launch state and the launch itself.
// Internal to the library.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include "df11.h"
#include "df11_device_check.h"

namespace df11_internal {

inline bool supported(uint32_t C, uint32_t T) {
  if (T == 256) return C == 4 || C == 8 || C == 16 || C == 24;
  if (T == 128 || T == 512) return C == 8;
  return false;
}

inline uint32_t stage_bytes_for(uint32_t max_block_elems) {
  return (max_block_elems + 32u + 15u) & ~15u;
}

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// `count` rows of `bytes` bytes, `stride` bytes apart, that do not overlap one another
struct Rows {
  const void *p;
  uint64_t count, bytes, stride;
};

// whether two sets of rows share a byte (columns of one buffer, say, do not)
inline bool share_memory(Rows a, Rows b) {
  if (!a.p || !b.p || !a.count || !b.count || !a.bytes || !b.bytes) return false;
  const uint64_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y + (b.count - 1) * b.stride + b.bytes || y >= x + (a.count - 1) * a.stride + a.bytes)
    return false;
  if (a.count == 1) a.stride = b.stride;
  if (b.count == 1) b.stride = a.stride;
  if (a.count == 1 && b.count == 1) return true;
  if (a.stride == b.stride) {
    // a's row i starts r behind b's row q + i, and reaches the one after it or not
    const int64_t s = (int64_t)a.stride, d = (int64_t)(x - y);
    const int64_t q = d >= 0 ? d / s : -((s - 1 - d) / s), r = d - q * s;
    const int64_t na = (int64_t)a.count, nb = (int64_t)b.count;
    auto meet = [&](int64_t first) {  // some row i of a and row first + i of b
      return (first < 0 ? -first : 0) < (na < nb - first ? na : nb - first);
    };
    return (r < (int64_t)b.bytes && meet(q)) || (r + (int64_t)a.bytes > s && meet(q + 1));
  }
  for (uint64_t i = 0; i < a.count; ++i) {  // the row of b at or before the row of a, and the next
    const uint64_t lo = x + i * a.stride, j = lo > y ? (lo - y) / b.stride : 0;
    for (uint64_t k = j; k < b.count && k <= j + 1; ++k)
      if (lo < y + k * b.stride + b.bytes && y + k * b.stride < lo + a.bytes) return true;
  }
  return false;
}

inline df11_status validate(const df11_tensor &t) {
  const df11_params &p = t.params;
  if (p.n == 0) return DF11_OK;
  if (p.n >= (1ull << 32)) return DF11_ERR_TOO_LARGE;
  if (!t.bitstream || !t.gaps || !t.block_out_pos || !t.luts || !t.code_lengths ||
      !t.sign_mantissa || !t.out_bf16)
    return DF11_ERR_NULL;
  if (!aligned(t.bitstream, 16) || !aligned(t.gaps, 16) || !aligned(t.luts, 16) ||
      !aligned(t.chunk_counts, 16) || !aligned(t.decode_table, 16) ||
      !aligned(t.sign_mantissa, 16) || !aligned(t.out_bf16, 16) || !aligned(t.block_out_pos, 4))
    return DF11_ERR_ALIGN;
  if (!supported(p.chunk_bytes, p.threads_per_block)) return DF11_ERR_UNSUPPORTED;
  const uint64_t block_bits = 8ull * p.chunk_bytes * p.threads_per_block;
  if (p.total_bits < p.n || p.total_bits > 32ull * p.n) return DF11_ERR_FORMAT;
  if ((uint64_t)p.num_blocks != (p.total_bits + block_bits - 1) / block_bits) return DF11_ERR_FORMAT;
  if (p.num_luts < 1 || p.num_luts >= (1u << 24)) return DF11_ERR_FORMAT;
  if (p.max_block_elems == 0 || p.max_block_elems > 8ull * p.chunk_bytes * p.threads_per_block)
    return DF11_ERR_FORMAT;
  if (p.max_chunk_elems == 0 || p.max_chunk_elems > 8ull * p.chunk_bytes) return DF11_ERR_FORMAT;
  if (p.max_warp_elems == 0 || p.max_warp_elems > 32ull * p.max_chunk_elems)
    return DF11_ERR_FORMAT;
  if (t.chunk_counts && 8ull * p.chunk_bytes > 255) return DF11_ERR_FORMAT;
  if (p.max_len < 1 || p.max_len > 32) return DF11_ERR_FORMAT;
  return DF11_OK;
}

// Per-device launch state, indexed by kernel instance: the warp-specialised
// kernels use 3 * i + mode with i = 3-8 (decode with counts), 12-14 (fused
// matrix-vector product) and 15-20 (decode without counts); the
// tensor-core product 64-65, the linear product 66-69 and 71-78, the embedding's
// gradient 81-85 and its lookup 86-100.
constexpr int kInstances = 104;
struct DeviceInfo {
  int sms = 0;
  std::atomic<size_t> configured[kInstances];  // shared-memory limit set, per kernel instance
  // (smem << 8 | blocks per SM) of the last two shared-memory sizes, per instance
  std::atomic<uint64_t> occupancy[kInstances][2];
};

inline DeviceInfo &device_info(int dev) {
  static DeviceInfo info[64];
  DeviceInfo &d = info[dev & 63];
  if (d.sms == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    d.sms = v > 0 ? v : 1;
  }
  return d;
}

// Thread blocks per tensor (c[0 .. n-1]): one wave (at most `budget`, the
// resident count), at least one per tensor, and as few format blocks per thread
// block as possible, since a launch lasts as long as its busiest thread block.
// Shares in proportion to the format blocks, rounded down, then thread
// blocks moved to where the most format blocks per thread block remain.
inline void split_blocks(const uint32_t *blocks, int n, uint64_t budget, uint64_t *c) {
  uint64_t total = 0, sum = 0;
  for (int i = 0; i < n; ++i) total += blocks[i];
  if (budget < (uint64_t)n) budget = n;
  for (int i = 0; i < n; ++i) {
    c[i] = budget * blocks[i] / total;
    if (c[i] < 1) c[i] = 1;
    if (c[i] > blocks[i]) c[i] = blocks[i];
    sum += c[i];
  }
  auto per = [&](int i, uint64_t ci) { return (blocks[i] + ci - 1) / ci; };
  while (sum > budget) {  // only from the at-least-one rule: take from the idlest
    int best = -1;
    for (int i = 0; i < n; ++i)
      if (c[i] > 1 && (best < 0 || per(i, c[i] - 1) < per(best, c[best] - 1))) best = i;
    if (best < 0) break;
    --c[best];
    --sum;
  }
  while (sum < budget) {  // the rest to the busiest tensor that can use one
    int best = -1;
    for (int i = 0; i < n; ++i)
      if (c[i] < blocks[i] && (best < 0 || per(i, c[i]) > per(best, c[best]))) best = i;
    if (best < 0) break;
    ++c[best];
    ++sum;
  }
}

// Launch with programmatic stream serialization: the kernel may begin while
// the previous one in the stream finishes (see pdl_wait).  DF11_PDL=0 in the
// environment launches without it.
inline bool pdl_enabled() {
  static const bool on = [] {
    const char *v = std::getenv("DF11_PDL");
    return !(v && v[0] == '0');
  }();
  return on;
}

template <typename... Args>
df11_status launch_pdl(void (*kern)(Args...), dim3 grid, uint32_t threads, size_t smem,
                       cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DF11_OK : DF11_ERR_CUDA;
}

// After a kernel that writes what the library's launches read before they wait for the previous
// kernel (streams, decode tables): a kernel that does nothing, launched plainly, starts when
// those writes are done and visible, and is the one that a launch above may overlap.
static __global__ void after_writes_kernel() {}
inline df11_status queue_after_writes(cudaStream_t s) {
  after_writes_kernel<<<1, 32, 0, s>>>();
  return cudaGetLastError() == cudaSuccess ? DF11_OK : DF11_ERR_CUDA;
}

// The same for a grid of clusters of `ctas` thread blocks (at most 8).
template <typename... Args>
df11_status launch_cluster(void (*kern)(Args...), uint32_t grid, uint32_t ctas, uint32_t threads,
                           size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DF11_OK : DF11_ERR_CUDA;
}

// The kernel's shared-memory limit raised to `smem` where needed, and the thread blocks of
// it that the device holds.  `carveout`: percentage of the SM's memory asked for as shared
// memory; the default is all of it, since most kernels here keep their working set there,
// and the occupancy query assumes this split.
template <typename K>
df11_status prepare(K kern, int threads, size_t smem, int instance, uint64_t &budget,
                    int carveout = 100) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DF11_ERR_CUDA;
  DeviceInfo &di = device_info(dev);
  if (instance < 0 || instance >= kInstances) return DF11_ERR_INVALID;
  if (smem > 48 * 1024 && di.configured[instance].load() < smem) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout) !=
            cudaSuccess)
      return DF11_ERR_CUDA;
    di.configured[instance].store(smem);
  }
  // occupancy queries cost microseconds of host time: one per instance and
  // shared-memory size (a layer-by-layer decode loop repeats the sizes)
  int per_sm = 0;
  const uint64_t c0 = di.occupancy[instance][0].load(), c1 = di.occupancy[instance][1].load();
  if (c0 && (c0 >> 8) == (uint64_t)smem) {
    per_sm = (int)(c0 & 0xFF);
  } else if (c1 && (c1 >> 8) == (uint64_t)smem) {
    per_sm = (int)(c1 & 0xFF);
  } else {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) !=
        cudaSuccess)
      return DF11_ERR_CUDA;
    // keep the most recent size in slot 0, the one before in slot 1
    di.occupancy[instance][1].store(c0);
    di.occupancy[instance][0].store(((uint64_t)smem << 8) | (uint64_t)(per_sm & 0xFF));
  }
  if (per_sm < 1) return DF11_ERR_TOO_LARGE;
  budget = (uint64_t)di.sms * per_sm;
  return DF11_OK;
}

}  // namespace df11_internal
