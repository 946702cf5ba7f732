// attn_gather_bf16_kv16.hip - the gathering attention kernels for bf16 queries over the 16-bit cache.
#include "attn_gather.h"

namespace bs {

template int launch_attn_gather<Bf16, false>(const GatherArgs&, int, int, bool, hipStream_t);

}  // namespace bs
