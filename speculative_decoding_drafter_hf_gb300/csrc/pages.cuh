// The paged cache (hf_pages): checks shared by its calls and its readers.
#pragma once

#include "common.cuh"

namespace hf {

constexpr int kMaxRequests = 4096;

// Why the calls refuse this descriptor, or NULL. Pointers are checked too when
// `buffers` is set.
const char* pages_bad(const hf_pages* p, bool buffers);

inline long long pages_block(const hf_pages* p) {  // elements of one page of one layer's K or V
  return (long long)p->n_kv_heads * p->page * p->head_dim;
}

}  // namespace hf
