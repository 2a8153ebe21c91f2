// Ring kernels of one norm operator and type (qk_norm_ring.cuh).
#include "qk_norm_ring.cuh"

namespace qk {
NormTable norm_shapes_add_f32(bool vec) {
  static const NormShape vectors[] = {QK_NORM_VECTOR_SHAPES(kAddNorm, float)};
  static const NormShape elements[] = {QK_NORM_ELEMENT_SHAPES(kAddNorm, float)};
  return vec ? NormTable{vectors, int(sizeof(vectors) / sizeof(NormShape))}
             : NormTable{elements, int(sizeof(elements) / sizeof(NormShape))};
}
}  // namespace qk
