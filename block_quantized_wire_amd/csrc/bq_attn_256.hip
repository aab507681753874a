// bq_attn_256.hip -- attention over the 4-bit cache, heads of 256 numbers.
#include "bq_attn.h"

namespace bq {
namespace attn {

hipError_t launch_width(std::integral_constant<int, 256>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream) {
    return launch_any<256>(a, p, f16, stream);
}

}  // namespace attn
}  // namespace bq
