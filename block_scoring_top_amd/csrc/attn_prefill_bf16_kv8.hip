// attn_prefill_bf16_kv8.hip - the prefill attention kernels for bf16 queries over the 8-bit cache.
#include "attn_prefill.h"

namespace bs {

template int launch_attn_prefill<Bf16, kForm8>(const PrefillArgs&, int, int, uint32_t, hipStream_t);

}  // namespace bs
