// kv_attend_q8.cu -- il_kv_attend over a Q8 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_q8(const KvAttendPlan& p, int dim, bool wide, int ctas, Launch* out) {
  return attend::prepare_format<true>(p, dim, wide, ctas, out);
}

}  // namespace il
