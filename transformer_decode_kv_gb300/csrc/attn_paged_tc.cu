// The 128-row tensor-core tiles of the attention over a paged cache: no shape takes them yet, the
// 16-row tiles (attn_paged.cu) serve every call.
#include "paged.h"

namespace llm {

bool attn_paged_tc_ok(int32_t, int32_t, int32_t) { return false; }
bool launch_attn_paged_tc(const AttnPagedArgs&, cudaStream_t) { return false; }

}  // namespace llm
