// attn_prefill_f16_kv16.hip - the prefill attention kernels for f16 queries over the 16-bit cache.
#include "attn_prefill.h"

namespace bs {

template int launch_attn_prefill<F16, false>(const PrefillArgs&, int, int, uint32_t, hipStream_t);

}  // namespace bs
