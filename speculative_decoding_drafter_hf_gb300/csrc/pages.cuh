// The paged cache (hf_pages): checks shared by its calls and its readers.
#pragma once

#include "common.cuh"

namespace hf {

constexpr int kMaxRequests = 4096;

// Why the calls refuse this descriptor, or NULL. Pointers are checked too when
// `buffers` is set. e4m3: the cache of an hf_pages8, else HF_F32 or HF_BF16.
const char* pages_bad(const hf_pages* p, bool buffers, bool e4m3 = false);
const char* pages8_bad(const hf_pages8* p, bool buffers);

// Scales of an 8-bit cache [n_layers, n_pages, n_kv_heads], NULL of any other.
struct PageScales {
  float* k;
  float* v;
};

// hf_pages_extend, _fork, _truncate and _compact of a cache of either kind.
hf_status pages_extend(const hf_pages* p, bool e4m3, PageScales s, const int32_t* requests, const int32_t* counts,
                       int32_t n, void* stream);
hf_status pages_fork(const hf_pages* p, bool e4m3, const int32_t* from, const int32_t* into, int32_t n, void* stream);
hf_status pages_truncate(const hf_pages* p, bool e4m3, const int32_t* requests, const int32_t* keep, int32_t n,
                         void* stream);
hf_status pages_compact(const hf_pages* p, bool e4m3, PageScales s, int32_t* n_used, void* stream);
size_t pages_work_ints(const hf_pages* p, bool e4m3);
// The first `shared` tokens of request req[0] (NULL: 0) of an 8-bit cache as bf16 rows [shared, n_kv_heads * head_dim].
cudaError_t launch_prefix_values(const hf_pages& p, PageScales sc, int layer, const int32_t* req, int shared, void* k,
                                 void* v, cudaStream_t st);

// Pages that a length fills (lengths near 2^31 too).
__host__ __device__ __forceinline__ int pages_of(int len, int page) { return len / page + (len % page > 0); }

__device__ __forceinline__ void pages_flag(const hf_pages& p, int bit) {
  if (p.status) atomicOr(p.status, bit);
}

// The last index in [0, n) with first(i) <= t (rising), by one warp: 32 of them are looked at side by
// side, so that three dependent loads do for 4096.
template <typename F>
__device__ __forceinline__ int pages_find(int n, int t, F&& first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, count = n;
  while (count > 1) {
    const int step = (count + 31) / 32, i = lane * step;
    const bool before = i < count && first(lo + i) <= t;
    const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, before)));
    lo += k * step;
    count = min(step, count - k * step);
  }
  return lo;
}

__host__ __device__ inline int pages_esize(int dtype) { return dtype == HF_F32 ? 4 : dtype == HF_BF16 ? 2 : 1; }

inline long long pages_block(const hf_pages* p) {  // elements of one page of one layer's K or V
  return (long long)p->n_kv_heads * p->page * p->head_dim;
}

}  // namespace hf
