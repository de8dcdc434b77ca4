// The paged KV cache's checks, shared by the append (paged.cu) and the attention (paged_attention.cu).
#pragma once
#include "verify.h"

namespace vp {

// Shapes, pointers and alignment of the host descriptor (the page table itself is device memory).
vp_status check_cache(const vp_paged_cache* c);

}  // namespace vp
