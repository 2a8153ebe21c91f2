// Ring kernels of one norm operator and type (qk_norm_ring.cuh).
#include "qk_norm_ring.cuh"

namespace qk {
NormTable norm_shapes_bwd_bf16(bool vec) {
  static const NormShape vectors[] = {QK_NORM_BWD_VECTOR_SHAPES(kAddNormBwd, __nv_bfloat16)};
  static const NormShape elements[] = {QK_NORM_ELEMENT_SHAPES(kAddNormBwd, __nv_bfloat16)};
  return vec ? NormTable{vectors, int(sizeof(vectors) / sizeof(NormShape))}
             : NormTable{elements, int(sizeof(elements) / sizeof(NormShape))};
}
}  // namespace qk
