// The gradients of the norms of fp32 rows.
#include "norm_bwd.cuh"

namespace mp {
template mp_status_t norm_backward<float>(const NormCall &, int &);
}
