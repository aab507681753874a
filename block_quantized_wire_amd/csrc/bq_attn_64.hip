// bq_attn_64.hip -- attention over the 4-bit cache, heads of 64 numbers.
#include "bq_attn.h"

namespace bq {
namespace attn {

hipError_t launch_width(std::integral_constant<int, 64>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream) {
    return launch_any<64>(a, p, f16, stream);
}

}  // namespace attn
}  // namespace bq
