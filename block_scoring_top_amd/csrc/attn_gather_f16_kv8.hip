// attn_gather_f16_kv8.hip - the gathering attention kernels for f16 queries over the 8-bit cache.
#include "attn_gather.h"

namespace bs {

template int launch_attn_gather<F16, kForm8>(const GatherArgs&, int, int, bool, hipStream_t);

}  // namespace bs
