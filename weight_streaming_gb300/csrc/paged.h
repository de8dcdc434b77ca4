// The paged KV caches' checks, shared by the appends (paged.cu) and the attentions (paged_attention.cu, rows_attention.cu).
#pragma once
#include "verify.h"

namespace vp {

// Shapes, pointers and alignment of the host descriptors (the page table itself is device memory).
vp_status check_cache(const vp_paged_cache* c);
vp_status check_cache_fp8(const vp_paged_cache_fp8* c);

}  // namespace vp
