// tree_attn_q8_tc.cu - dspark_tree_attention_q8 on the tensor cores for many query rows a key head (tree_attn_tc.cuh).
#include "tree_attn_tc.cuh"

cudaError_t ta_launch_q8_tc(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  return a.c.head_dim <= 64 ? ta_dispatch_tc<64, true>(a, grid, k, v, st) : ta_dispatch_tc<128, true>(a, grid, k, v, st);
}
