// Attention over a paged key/value cache held in OCP E4M3 with a power-of-two
// scale per block of tokens and head.  The walks are those over bf16 rows
// (attention.hip tells their mathematics): a row's codes are fetched into
// registers and enter LDS as the bf16 values they stand for, code times scale in
// one instruction per pair (exact: three fraction bits, and the scale only moves
// the exponent), so what follows is the same, to the last bit, as over a bf16
// cache of those values.
#include <hip/hip_runtime.h>

#include "attention_core.h"

namespace vla {

hipError_t launch_attn_shared_e4m3(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s) {
    prepare_attn_shared(a, p, ws);
    const bool wide = (static_cast<uint64_t>(a.num_pages) << a.page_log2) * a.Hkv * a.D > kNoOffset;
    const hipError_t e = launch_walks<PagedCodes>(a, p, wide, s);
    return e != hipSuccess || a.parts == 1 ? e : launch_attn_join(a, p, s);
}

}  // namespace vla
