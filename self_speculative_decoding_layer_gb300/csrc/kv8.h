// Host-side launch interface of the 8-bit KV cache's kernels (internal; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.cuh"

namespace ssd {

// Launch with programmatic serialization: the kernel may start while its predecessor in the stream drains, and each of
// these kernels calls griddep_wait() in every thread before it touches global memory.  cluster > 1: clusters of that
// many CTAs along x.  False if the launch failed.
template <typename... KArgs, typename... Args>
inline bool launch_kv8(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                       const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

// Rows to append to a cache (k, v are read) or values to read from it (k, v are written), 16-byte aligned.
struct Kv8RowsArgs {
  void* k;
  void* v;
  size_t ld_k, ld_v;  // elements between rows
  int first, rows;    // slots first .. first + rows - 1
};

struct Kv8SelectArgs {
  const float* weight;  // [n_kv][ld_weight]
  size_t ld_weight;
  int n, keep, recent;
  int* index;           // [n_kv][keep]
  float* kept_weight;   // [n_kv][keep] or null
};

struct Kv8AttnArgs {
  Kv8View c;
  const void* q;    // [rows][ld_q], query heads of hd
  void* out;        // [rows][ld_out]
  float* lse;       // [rows][n_q] or null, ld_lse and step_lse apart; the weights kernel reads it
  size_t ld_q, ld_out, ld_lse, step_lse;
  int n_q, group, rows;
  int prefix, base;
  float scale, cap;          // cap 0: none
  unsigned long long any;    // union of the masks
  int n_split;               // key splits
  int split_tiles;           // tiles of a split (set by the launcher)
  float* part_o;             // partial results for a second kernel, [n_kv * queries][n_split][hd]; null: none
  float2* part_ml;           // [n_kv * queries][n_split]: running maximum (log2) and sum
  // weights kernel
  const float* w_in;         // [n_kv][ld_w] or null
  float* w_out;
  size_t ld_w;
  int n_take;                // query rows that count
  unsigned char take[kMaxRows];
  unsigned long long mask[kMaxRows];

  __device__ __forceinline__ size_t lse_at(int row, int head) const { return row * ld_lse + head * step_lse; }
};

// io: ssd_dtype of q / out, k / v rows.
bool launch_kv8_append(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st);
bool launch_kv8_read(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st);
bool launch_kv8_evict(const Kv8View& src, const Kv8View& dst, const Kv8SelectArgs& a, cudaStream_t st);
// Key splits of an attention launch over `slots` slots, whether they merge through device scratch (else in the
// distributed shared memory of a cluster), and whether the tensor-core kernel runs it.
struct Kv8Splits {
  int n;
  bool scratch, tc;
};
Kv8Splits kv8_attention_splits(int rows, int group, int n_kv, int slots, int io);
bool launch_kv8_attention(const Kv8AttnArgs& a, int io, bool tc, cudaStream_t st);
bool launch_kv8_attention_tc(const Kv8AttnArgs& a, int io, cudaStream_t st);
bool launch_kv8_weights(const Kv8AttnArgs& a, int io, cudaStream_t st);

}  // namespace ssd
