// prefix_attention_umma.cu -- the tensor-core kernels of shared prefixes.
#include "tree_attention_umma.cuh"

namespace mtp {

UmmaPlan prefix_umma_plan(int D, int rows, long long most) { return umma_plan<true>(D, rows, most); }

}  // namespace mtp
