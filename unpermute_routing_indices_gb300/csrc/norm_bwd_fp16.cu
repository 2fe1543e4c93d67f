// The gradients of the norms of fp16 rows.
#include "norm_bwd.cuh"

namespace mp {
template mp_status_t norm_backward<__half>(const NormCall &, int &);
}
