// kv_attend_a4.cu -- il_kv_attend over an A4 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_a4(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out) {
  return attend::prepare_format<IL_A4, false>(p, dim, blocks, ctas, out);
}

}  // namespace il
