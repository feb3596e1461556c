// host_common.h - argument checks and launch helpers for the libdspark entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <utility>
#include <stdint.h>

#include "../../include/dspark.h"

#define DS_REQUIRE(cond)                 \
  do {                                   \
    if (!(cond)) return DSPARK_EINVAL;   \
  } while (0)

#define DS_CUDA_TRY(expr)                        \
  do {                                           \
    if ((expr) != cudaSuccess) {                 \
      (void)cudaGetLastError();                  \
      return DSPARK_ECUDA;                       \
    }                                            \
  } while (0)

static inline dspark_status ds_launch_status() {
  return (cudaGetLastError() == cudaSuccess) ? DSPARK_OK : DSPARK_ECUDA;
}

static inline int ds_dtype_size(dspark_dtype d) { return d == DSPARK_BF16 ? 2 : 4; }
static inline bool ds_dtype_ok(dspark_dtype d) { return d == DSPARK_BF16 || d == DSPARK_F32; }

static inline int64_t ds_ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static inline bool ds_aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Whether `na` bytes from a and `nb` bytes from b (null: none) share one.
static inline bool ds_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Poll limit of the first wait for a tile's tensor-core MMAs (lattice and dense walk); lowered only
// by the test hook dspark_test_set_first_wait_polls.
extern std::atomic<uint32_t> g_ds_first_wait_polls;

// Streaming multiprocessors of the current device (cached per device; thread-safe).
int ds_num_sms();

// Raises `func`'s dynamic shared-memory limit on the current device to at least `bytes` (each
// (device, kernel) pair is configured once; thread-safe). Kernel attributes are per device, so a
// process driving several GPUs, or calling from several threads, configures each one it uses.
cudaError_t ds_ensure_smem(const void* func, size_t bytes);

// cuTensorMapEncodeTiled, from the driver through the runtime (no link against the driver library);
// null when the driver has none.
using DsEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
DsEncodeFn ds_encode_fn();

// Launches `kern` on `stream` with programmatic stream serialization: it may start while the
// previous kernel on the stream is still running (see ds_pdl_trigger / ds_pdl_wait).
template <typename... KArgs, typename... Args>
static inline cudaError_t ds_launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                   cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Checks of a dspark_kvcache that every cache entry point makes (`layers`: the layer count is used).
static inline bool ds_cache_ok(const dspark_kvcache* c, bool layers) {
  if (!c || !c->k || !c->v || !c->page_table || !ds_dtype_ok(c->dtype)) return false;
  const size_t e = size_t(ds_dtype_size(c->dtype));
  return ds_aligned(c->k, e) && ds_aligned(c->v, e) && c->page_stride >= 0 && c->token_stride >= 0 &&
         c->head_stride >= 0 && c->num_pages >= 1 && c->num_pages <= INT32_MAX && c->page_size >= 1 &&
         c->page_size <= 65536 && c->heads >= 1 && c->heads <= 1024 && c->head_dim >= 8 && c->head_dim <= 256 &&
         c->head_dim % 8 == 0 && c->table_pages >= 1 && c->ld_table >= c->table_pages && (!layers || (c->n_layers >= 1 && c->layer_stride >= 0));
}

// new_len of a commit may overlap nothing that the blocks of other buffers and layers read after one block has written it. Without a path
// there is one block a request, which has read its count by then: new_len may be n_accepted itself.
static inline bool ds_commit_len_ok(const int32_t* new_len, const int32_t* ctx_len, const int32_t* n_accepted, const int32_t* path, int64_t R,
                                    int32_t T) {
  const size_t n = size_t(R) * 4;
  if (ds_overlap(new_len, n, ctx_len, n) || ds_overlap(new_len, n, path, n * size_t(T))) return false;
  return (!path && new_len == n_accepted) || !ds_overlap(new_len, n, n_accepted, n);
}

// Every row of every head of the cache starts on a 16-byte boundary.
static inline bool ds_cache_vec(const dspark_kvcache* c) {
  const int64_t e = ds_dtype_size(c->dtype);
  return ds_aligned(c->k, 16) && ds_aligned(c->v, 16) && (c->page_stride * e) % 16 == 0 &&
         (c->token_stride * e) % 16 == 0 && (c->head_stride * e) % 16 == 0 && (c->layer_stride * e) % 16 == 0;
}
