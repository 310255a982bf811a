// tree_attention_umma.cu -- the tensor-core kernels of tree attention.
#include "tree_attention_umma.cuh"

namespace mtp {

int attn_umma_bn(int D) { return D == 256 ? 64 : 128; }

UmmaPlan attn_umma_plan(int D, int rows) { return umma_plan<false>(D, rows, rows); }

}  // namespace mtp
