// The gradients of the norms of bf16 rows.
#include "norm_bwd.cuh"

namespace mp {
template mp_status_t norm_backward<__nv_bfloat16>(const NormCall &, int &);
}
