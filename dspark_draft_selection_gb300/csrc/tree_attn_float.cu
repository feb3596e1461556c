// tree_attn_float.cu - dspark_tree_attention in float32 arithmetic (tree_attn_float.cuh).
#include "tree_attn_float.cuh"

cudaError_t ta_launch_float(const TaArgs& a, int grid, cudaStream_t st) {
  return a.c.dtype == DSPARK_BF16 ? tf_rows<__nv_bfloat16, false>(a, grid, st) : tf_rows<float, false>(a, grid, st);
}
