// attn_gather_bf16_kv4.hip - the gathering attention kernels for bf16 queries over the 4-bit cache.
#include "attn_gather.h"

namespace bs {

template int launch_attn_gather<Bf16, kForm4>(const GatherArgs&, int, int, bool, hipStream_t);

}  // namespace bs
