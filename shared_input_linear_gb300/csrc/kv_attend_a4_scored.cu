// kv_attend_a4_scored.cu -- il_kv_attend_scored over an A4 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_a4_scored(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out) {
  return attend::prepare_format<IL_A4, true>(p, dim, blocks, ctas, out);
}

}  // namespace il
