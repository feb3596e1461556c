// tree.cu - trees of drafted nodes: ancestor mask and positions (dspark_tree_mask) and greedy
// acceptance along the target's choices (dspark_tree_accept).
//
// openvino.genai PR #4847, Change > Sampled drafting and Fixes > Split validation windows: the
// target validates a request's drafted candidates in one pass, row j after candidate j. A chain of
// candidates is the tree parent[i] = i - 1; alternatives at a position are siblings.
#include "dspark_common.cuh"
#include "host_common.h"

namespace {

constexpr int TR_MAXT = 512;


DS_DEV int32_t tr_nodes(const int32_t* n_nodes, int64_t r, int32_t T, int32_t* status) {
  int32_t n = n_nodes ? n_nodes[r] : T;
  if (n < 0 || n > T) {
    if (threadIdx.x == 0) ds_set_error(status, DSPARK_EINVAL);
    n = 0;
  }
  return n;
}

// One block per request, one thread per node. Node i keeps the set A_i of the nodes from it up to,
// but without, its jump node J_i (at first {i} and the parent); a round sets A_i |= A_{J_i} and
// J_i = J_{J_i}, so ceil(log2(depth)) rounds of shared-memory reads make the whole closure instead of
// a walk of `depth` dependent steps per node. The sets are bit words, in registers while a round
// reads the others' (W is the words' number, a power of two so that the loops unroll).
template <int W>
__global__ void __launch_bounds__(TR_MAXT) tree_mask_kernel(const int32_t* parent, const int32_t* n_nodes,
                                                            const int32_t* base, int32_t T, uint32_t* mask,
                                                            int32_t* pos, int32_t* status) {
  __shared__ uint32_t s_anc[32 * W * (W + 1)];                 // rows one word apart in banks
  __shared__ int32_t s_jump[32 * W];
  const int64_t r = blockIdx.x;
  const int i = threadIdx.x;
  ds_pdl_trigger();
  ds_pdl_wait();
  const int32_t n = tr_nodes(n_nodes, r, T, status);
  int32_t jump = -1;
  if (i < n) {
    jump = parent ? parent[r * T + i] : i - 1;
    if (jump < -1 || jump >= i) {
      ds_set_error(status, DSPARK_EINVAL);
      jump = -1;
    }
  }
  uint32_t anc[W];
#pragma unroll
  for (int w = 0; w < W; ++w) anc[w] = (i < n && w == (i >> 5)) ? 1u << (i & 31) : 0u;
  uint32_t* mine = s_anc + i * (W + 1);
  for (;;) {
#pragma unroll
    for (int w = 0; w < W; ++w) mine[w] = anc[w];
    s_jump[i] = jump;
    if (!__syncthreads_or(jump >= 0)) break;
    if (jump >= 0) {
      const uint32_t* other = s_anc + jump * (W + 1);
#pragma unroll
      for (int w = 0; w < W; ++w) anc[w] |= other[w];
      jump = s_jump[jump];
    }
    __syncthreads();
  }
  if (i < T) {
    int32_t d = -1;
#pragma unroll
    for (int w = 0; w < W; ++w) d += __popc(anc[w]);
    pos[r * T + i] = i < n ? (base ? base[r] : 0) + d : 0;
  }
  const int words = (T + 31) >> 5;                   // the sets go out as one contiguous stretch
  uint32_t* out = mask + r * T * words;
  for (int u = i; u < T * words; u += blockDim.x) out[u] = s_anc[(u / words) * (W + 1) + u % words];
}

// One block per request. Every node looks up whether its token is the choice at its parent and the
// lowest such child of each node is kept (a shared-memory minimum, the same whatever the order), all
// in parallel; what is left of the walk is one thread following `next` in shared memory.
__global__ void __launch_bounds__(128) tree_accept_kernel(const int32_t* tokens, const int32_t* parent,
                                                          const int32_t* best, const int32_t* n_nodes, int32_t T,
                                                          int32_t* out_tokens, int32_t* n_accepted, int32_t* path,
                                                          int32_t* status) {
  __shared__ int32_t s_best[TR_MAXT], s_next[TR_MAXT], s_path[TR_MAXT];
  __shared__ int32_t s_n;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  ds_pdl_trigger();
  ds_pdl_wait();
  const int32_t n = tr_nodes(n_nodes, r, T, status);
  constexpr int PER = TR_MAXT / 128;
  int32_t tok[PER], par[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = tid + u * 128;
    tok[u] = par[u] = -1;
    if (i < n) {
      tok[u] = tokens[r * T + i];
      par[u] = parent ? parent[r * T + i] : i - 1;
      s_best[i] = best[r * T + i];
      s_next[i] = TR_MAXT;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = tid + u * 128;
    if (i < n && par[u] >= 0 && par[u] < i && s_best[par[u]] == tok[u]) atomicMin(&s_next[par[u]], i);
  }
  __syncthreads();
  if (tid == 0) {
    int k = 0;
    if (n > 0) {
      for (int cur = 0; cur < TR_MAXT; cur = s_next[cur]) s_path[k++] = cur;   // indices rise: at most n steps
    }
    s_n = k;
  }
  __syncthreads();
  const int k = s_n;
  if (tid == 0) n_accepted[r] = k - 1;
  for (int i = tid; i < T; i += 128) {
    path[r * T + i] = i < k ? s_path[i] : -1;
    out_tokens[r * T + i] = i < k ? s_best[s_path[i]] : -1;   // the choice at a node is the next node's token
  }
}

}  // namespace

extern "C" dspark_status dspark_tree_mask(const int32_t* parent, const int32_t* n_nodes, const int32_t* base, int64_t R,
                                          int32_t T, uint32_t* mask, int32_t* pos, int32_t* dev_status,
                                          dspark_stream_t stream) {
  DS_REQUIRE(R >= 0 && R <= INT32_MAX && T >= 1 && T <= TR_MAXT);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(mask && pos && dev_status);
  const int W = T <= 32 ? 1 : T <= 64 ? 2 : T <= 128 ? 4 : T <= 256 ? 8 : 16;
  const dim3 grid{unsigned(R)}, block{unsigned(ds_ceil_div(T, 32) * 32)};
  switch (W) {
    case 1: DS_CUDA_TRY(ds_launch(tree_mask_kernel<1>, grid, block, 0, stream, parent, n_nodes, base, T, mask, pos, dev_status)); break;
    case 2: DS_CUDA_TRY(ds_launch(tree_mask_kernel<2>, grid, block, 0, stream, parent, n_nodes, base, T, mask, pos, dev_status)); break;
    case 4: DS_CUDA_TRY(ds_launch(tree_mask_kernel<4>, grid, block, 0, stream, parent, n_nodes, base, T, mask, pos, dev_status)); break;
    case 8: DS_CUDA_TRY(ds_launch(tree_mask_kernel<8>, grid, block, 0, stream, parent, n_nodes, base, T, mask, pos, dev_status)); break;
    default: DS_CUDA_TRY(ds_launch(tree_mask_kernel<16>, grid, block, 0, stream, parent, n_nodes, base, T, mask, pos, dev_status)); break;
  }
  return DSPARK_OK;
}

extern "C" dspark_status dspark_tree_accept(const int32_t* tokens, const int32_t* parent, const int32_t* best,
                                            const int32_t* n_nodes, int64_t R, int32_t T, int32_t* out_tokens,
                                            int32_t* n_accepted, int32_t* path, int32_t* dev_status,
                                            dspark_stream_t stream) {
  DS_REQUIRE(R >= 0 && R <= INT32_MAX && T >= 1 && T <= TR_MAXT);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(tokens && best && out_tokens && n_accepted && path && dev_status);
  DS_CUDA_TRY(ds_launch(tree_accept_kernel, dim3(unsigned(R)), dim3(128), 0, stream, tokens, parent, best, n_nodes, T,
                        out_tokens, n_accepted, path, dev_status));
  return DSPARK_OK;
}
