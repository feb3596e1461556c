// tree_attn_q8_float.cu - dspark_tree_attention_q8 in float32 arithmetic (tree_attn_float.cuh).
#include "tree_attn_float.cuh"

cudaError_t ta_launch_float_q8(const TaArgs& a, int grid, cudaStream_t st) {
  return a.c.dtype == DSPARK_BF16 ? tf_rows<__nv_bfloat16, true>(a, grid, st) : tf_rows<float, true>(a, grid, st);
}
