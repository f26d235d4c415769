// kv_attend_q8_scored.cu -- il_kv_attend_scored over a Q8 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_q8_scored(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out) {
  return attend::prepare_format<attend::kQ8Columns, true>(p, dim, blocks, ctas, out);
}

}  // namespace il
