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
  int32_t n = n_nodes ? __ldg(n_nodes + r) : T;
  if (n < 0 || n > T) {
    if (threadIdx.x == 0) ds_set_error(status, DSPARK_EINVAL);
    n = 0;
  }
  return n;
}

// One block per request, one thread per node, one warp per 32 nodes ("a word": the nodes' bits of a mask
// word). 1. Every warp closes its own word by pointer doubling over shuffles: each node gets its ancestors
// inside the word and the first one outside, `up`, which lies in an earlier word. 2. Word after word, the
// warp takes the words of `up`'s finished row from shared memory: a row is read and written once, instead of
// once per doubling step over whole rows (256 trees of 512 nodes: 12.4 us that way, 8.2 us this way, 1.4 us
// being what the outputs' bytes need). Rows lie an odd number of words apart, so a warp's rows start in 32
// banks. Bound by the latency of the T / 32 steps.
__global__ void __launch_bounds__(TR_MAXT) tree_mask_kernel(const int32_t* parent, const int32_t* n_nodes,
                                                            const int32_t* base, int32_t T, uint32_t* mask,
                                                            int32_t* pos, int32_t* status) {
  __shared__ uint32_t s_anc[TR_MAXT * (TR_MAXT / 32 + 1)];
  const int64_t r = blockIdx.x;
  const int i = threadIdx.x, lane = i & 31, word = i >> 5;
  const int words = (T + 31) >> 5, ld = words | 1;
  ds_pdl_trigger();
  ds_pdl_wait();
  const int32_t given = i < T && parent ? parent[r * T + i] : i - 1;   // the three loads together
  const int32_t first = base ? base[r] : 0;
  const int32_t n = tr_nodes(n_nodes, r, T, status);
  int32_t par = -1;
  if (i < n) {
    par = given;
    if (par < -1 || par >= i) {
      ds_set_error(status, DSPARK_EINVAL);
      par = -1;
    }
  }
  uint32_t bits = i < n ? 1u << lane : 0u;             // the path from the node up to, but without, `jump`
  int32_t jump = par >= word * 32 ? par & 31 : -1;     // a lane of this word, or -1: the path has left it
  int32_t up = jump < 0 ? par : -1;
#pragma unroll
  for (int d = 0; d < 5; ++d) {
    const int src = jump < 0 ? lane : jump;
    const uint32_t b = __shfl_sync(0xFFFFFFFFu, bits, src);
    const int32_t j = __shfl_sync(0xFFFFFFFFu, jump, src), u = __shfl_sync(0xFFFFFFFFu, up, src);
    if (jump >= 0) {
      bits |= b;
      jump = j;
      up = u;
    }
  }
  uint32_t* mine = s_anc + i * ld;
  int32_t d = __popc(bits) - 1;
  if (i < T) {
    mine[word] = bits;
    for (int w = word + 1; w < words; ++w) mine[w] = 0u;
  }
  for (int k = 1; k < words; ++k) {                    // word 0 is complete
    __syncthreads();
    if (word == k && i < T) {
      const uint32_t* other = s_anc + max(up, 0) * ld;
#pragma unroll 4
      for (int w = 0; w < k; ++w) {
        const uint32_t x = up >= 0 ? other[w] : 0u;
        mine[w] = x;
        d += __popc(x);
      }
    }
  }
  if (i < T) pos[r * T + i] = i < n ? first + d : 0;
  __syncthreads();
  uint32_t* out = mask + r * T * words;                // the rows go out as one contiguous stretch
  int row = i / words, w = i - row * words;
  const int srow = int(blockDim.x) / words, sw = int(blockDim.x) - srow * words;
  for (int u = i; u < T * words; u += blockDim.x) {
    out[u] = s_anc[row * ld + w];
    row += srow;
    w += sw;
    if (w >= words) {
      w -= words;
      ++row;
    }
  }
}

// One block per request. Every node looks up whether its token is the choice at its parent and the
// lowest such child of each node is kept (a shared-memory minimum, the same whatever the order), all
// in parallel; what is left of the walk is one thread following `next` in shared memory. Bound by latency:
// 512 trees of 512 nodes 2.7 us (their bytes: 0.8 us), 8 trees of 16 nodes 1.4 us.
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
  constexpr int PER = TR_MAXT / 128;
  int32_t tok[PER], par[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {                      // slots past the nodes are loaded and not used
    const int i = tid + u * 128;
    tok[u] = par[u] = -1;
    if (i < T) {
      tok[u] = tokens[r * T + i];
      par[u] = parent ? parent[r * T + i] : i - 1;
      s_best[i] = best[r * T + i];
      s_next[i] = TR_MAXT;
    }
  }
  const int32_t n = tr_nodes(n_nodes, r, T, status);
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
  DS_CUDA_TRY(ds_launch(tree_mask_kernel, dim3(unsigned(R)), dim3(unsigned(ds_ceil_div(T, 32) * 32)), 0, stream, parent,
                        n_nodes, base, T, mask, pos, dev_status));
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
