// The paged cache's book-keeping and copies (hf_pages_*).
//
// No arithmetic, only order: which page a request gets must not depend on which
// CTA comes first, so pages are ranked by prefix sums (the k-th page needed
// takes the k-th free page) and atomics are used only for reference counts,
// whose final values do not depend on order. Lists that must not repeat a
// request are checked with one bit per request in shared memory.
//
// truncate, fork: every CTA checks the whole list (at most 4096 entries), then
// works on its share of the table entries; the last CTA (ticket in work[0], left
// at zero) writes the lengths that the others still read. extend and compact:
// one CTA plans (prefix sums over the lists and over refs), then a wide launch
// moves the pages. write: one warp per row and a few layers of it.
#include <cstdio>

#include "pages.cuh"

namespace hf {

const char* pages_bad(const hf_pages* p, bool buffers) {
  if (!p) return "NULL cache";
  if (p->dtype != HF_F32 && p->dtype != HF_BF16) return "cache dtype must be HF_F32 or HF_BF16";
  if (p->n_layers < 1 || p->n_pages < 1 || p->n_kv_heads < 1 || p->table_ld < 1)
    return "cache: n_layers, n_pages, n_kv_heads and table_ld must be positive";
  if (p->page != 8 && p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
    return "cache: page must be 8, 16, 32, 64 or 128";
  if (p->head_dim < 8 || p->head_dim % 8 || p->head_dim > 256)
    return "cache: head_dim must be a multiple of 8, <= 256";
  if (p->n_kv_heads > 1024) return "cache: n_kv_heads must be <= 1024";
  if (p->n_requests < 1 || p->n_requests > kMaxRequests) return "cache: n_requests must be 1..4096";
  if ((long long)p->n_pages * p->n_kv_heads * p->page > 0x7fffffffLL ||
      (long long)p->table_ld * p->page > 0x7fffffffLL || (long long)p->n_requests * p->table_ld > 0x7fffffffLL)
    return "cache: n_pages * n_kv_heads * page, table_ld * page and n_requests * table_ld must be < 2^31";
  if (!buffers) return nullptr;
  if (!p->k || !p->v || !p->table || !p->lens || !p->refs || !p->work) return "cache: NULL buffer";
  auto off = [](const void* q, size_t n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
  if (off(p->k, 16) || off(p->v, 16)) return "cache: k and v must be 16-byte aligned";
  if (off(p->table, 4) || off(p->lens, 4) || off(p->refs, 4) || off(p->work, 4) || off(p->status, 4))
    return "cache: table, lens, refs, work and status must be 4-byte aligned";
  return nullptr;
}

namespace {

constexpr int PT = 1024;  // threads of the planning CTAs
constexpr int CT = 256;   // threads of the copying CTAs
// work: [0] ticket, [1] moves planned, [16 ..) source pages, then target pages
constexpr int kMoves = 16;

__device__ __forceinline__ int move_room(const hf_pages& p) { return max(p.n_pages, p.n_requests); }
// (lengths near 2^31 too)
__device__ __forceinline__ int pages_of(int len, int page) { return len / page + (len % page > 0); }
__device__ __forceinline__ void flag(const hf_pages& p, int bit) {
  if (p.status) atomicOr(p.status, bit);
}

// Whether the list names requests in range, none twice and none of `others` (NULL:
// no such list); each entry also has to pass ok(i, request). Same answer in every
// thread.
template <typename F>
__device__ __forceinline__ bool list_ok(const hf_pages& p, const int32_t* list, const int32_t* others, int n,
                                        F&& ok) {
  __shared__ uint32_t seen[kMaxRequests / 32];
  for (int i = threadIdx.x; i < kMaxRequests / 32; i += blockDim.x) seen[i] = 0;
  __syncthreads();
  bool good = true;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int r = list ? __ldcg(&list[i]) : i;
    if (r < 0 || r >= p.n_requests) {
      good = false;
    } else {
      const uint32_t bit = 1u << (r & 31);
      if (atomicOr(&seen[r >> 5], bit) & bit) good = false;
      if (!ok(i, r)) good = false;
    }
  }
  if (others) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int r = __ldcg(&others[i]);
      if (r < 0 || r >= p.n_requests || (seen[r >> 5] >> (r & 31) & 1)) good = false;
    }
  }
  return __syncthreads_and(good);
}

// True in every thread of the last CTA of the grid to come here; the ticket is
// left at zero.
__device__ __forceinline__ bool last_cta(const hf_pages& p) {
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(&p.work[0], 1) == (int)gridDim.x - 1;
    if (last) p.work[0] = 0;
  }
  __syncthreads();
  __threadfence();
  return last != 0;
}

// Exclusive prefix sum over the CTA's threads of v; total in every thread.
__device__ __forceinline__ int cta_scan(int v, int& total) {
  __shared__ int sums[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // sums of an earlier call have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < nw ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  total = sums[nw - 1];
  return x - v + (warp ? sums[warp - 1] : 0);
}

// ------------------------------------------------------------------ truncate
__global__ void __launch_bounds__(CT) truncate_kernel(hf_pages p, const int32_t* req, const int32_t* keep, int n) {
  pdl_trigger();
  pdl_wait();
  const bool ok = list_ok(p, req, nullptr, n, [&](int i, int r) {
    const int k = __ldcg(&keep[i]), len = __ldcg(&p.lens[r]);
    return k >= 0 && k <= len && pages_of(len, p.page) <= p.table_ld;
  });
  if (ok) {
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const int r = req ? __ldcg(&req[i]) : i;
      const int j1 = pages_of(__ldcg(&p.lens[r]), p.page);
      for (int j = pages_of(__ldcg(&keep[i]), p.page) + threadIdx.x; j < j1; j += CT) {
        int32_t* e = p.table + (size_t)r * p.table_ld + j;
        const int id = *e;
        *e = -1;
        if (id >= 0 && id < p.n_pages)
          atomicSub(&p.refs[id], 1);
        else
          flag(p, HF_S_BAD);
      }
    }
  }
  if (!last_cta(p)) return;
  if (ok) {
    for (int i = threadIdx.x; i < n; i += CT) p.lens[req ? __ldcg(&req[i]) : i] = __ldcg(&keep[i]);
  } else if (threadIdx.x == 0) {
    flag(p, HF_S_BAD);
  }
}

// ---------------------------------------------------------------------- fork
__global__ void __launch_bounds__(CT) fork_kernel(hf_pages p, const int32_t* from, const int32_t* into, int n) {
  pdl_trigger();
  pdl_wait();
  const bool ok = list_ok(p, into, from, n, [&](int i, int r) {
    const int s = __ldcg(&from[i]);
    if (s < 0 || s >= p.n_requests) return false;
    const int len = __ldcg(&p.lens[s]);
    return __ldcg(&p.lens[r]) == 0 && len >= 0 && pages_of(len, p.page) <= p.table_ld;
  });
  if (ok) {
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const int s = __ldcg(&from[i]), r = __ldcg(&into[i]);
      const int j1 = pages_of(__ldcg(&p.lens[s]), p.page);
      for (int j = threadIdx.x; j < j1; j += CT) {
        const int id = __ldcg(&p.table[(size_t)s * p.table_ld + j]);
        p.table[(size_t)r * p.table_ld + j] = id;
        if (id >= 0 && id < p.n_pages)
          atomicAdd(&p.refs[id], 1);
        else
          flag(p, HF_S_BAD);
      }
    }
  }
  if (!last_cta(p)) return;
  if (ok) {
    // no source is one of the targets, so the lengths read here are final
    for (int i = threadIdx.x; i < n; i += CT) p.lens[__ldcg(&into[i])] = __ldcg(&p.lens[__ldcg(&from[i])]);
  } else if (threadIdx.x == 0) {
    flag(p, HF_S_BAD);
  }
}

// -------------------------------------------------------------------- extend
// One CTA. Entry i needs `copy` (0 or 1: its partly filled last page is held by
// others) + new pages; ranks over the list give each its place in the order of the free
// pages, which come from scanning refs. Bound by the latency of its dependent loads: the
// list's are made once and kept, the first 8192 counts are on their way meanwhile, and the
// order of the free pages stays in shared memory as far as it fits.
__global__ void __launch_bounds__(PT) extend_plan(hf_pages p, const int32_t* req, const int32_t* counts, int n) {
  constexpr int PER = kMaxRequests / PT, NEAR = 4096;
  __shared__ int32_t s_free[NEAR];
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int32_t* src = p.work + kMoves;
  int32_t* dst = src + move_room(p);
  auto free_bits = [&](int b0) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (b0 + k < p.n_pages && __ldcg(&p.refs[b0 + k]) == 0) bits |= 1u << k;
    return bits;
  };
  uint32_t is_free = free_bits(tid * 8);
  bool full = false, ok = true;
  // entries i = tid * per + k, in list order
  const int per = (n + PT - 1) / PT;
  int req_[PER], len_[PER], cnt_[PER], last_[PER], need[PER], copy[PER], mine = 0, copies = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = tid * per + k;
    req_[k] = -1;
    need[k] = copy[k] = len_[k] = cnt_[k] = 0;
    last_[k] = -1;
    if (k >= per || i >= n) continue;
    const int r = req ? __ldcg(&req[i]) : i, c = __ldcg(&counts[i]);
    if (r < 0 || r >= p.n_requests || c < 0) {
      ok = false;
      continue;
    }
    const int len = __ldcg(&p.lens[r]);
    if (len < 0) {
      ok = false;
      continue;
    }
    req_[k] = r;
    len_[k] = len;
    cnt_[k] = c;
    if ((long long)len + c > (long long)p.table_ld * p.page) {
      full = true;
      continue;
    }
    if (c == 0) continue;
    const int have = pages_of(len, p.page);
    need[k] = pages_of(len + c, p.page) - have;
    if (len % p.page) {
      const int id = __ldcg(&p.table[(size_t)r * p.table_ld + have - 1]);
      if (id < 0 || id >= p.n_pages)
        ok = false;
      else
        copy[k] = __ldcg(&p.refs[id]) > 1;
      last_[k] = id;
    }
    need[k] += copy[k];
    mine += need[k];
    copies += copy[k];
  }
  // (checks the list for repeats)
  ok = list_ok(p, req, nullptr, n, [&](int, int) { return true; }) && __syncthreads_and(ok);
  full = __syncthreads_or(full);
  int total = 0, ncopy = 0, at = 0, cat = 0;
  if (ok && !full) {
    at = cta_scan(mine, total);
    cat = cta_scan(copies, ncopy);
    // the free pages among the first ones, until enough are found; each thread looks at 8
    // neighbouring pages a step
    int found = 0;
    for (int base = 0; base < p.n_pages && found < total; base += PT * 8) {
      const int b0 = base + tid * 8;
      if (base) is_free = free_bits(b0);
      int sum;
      int rank = found + cta_scan(__popc(is_free), sum);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (is_free >> k & 1) {
          if (rank < total) (rank < NEAR ? s_free : dst)[rank] = b0 + k;  // the order of free pages
          ++rank;
        }
      found += sum;
    }
    full = found < total;
  }
  __syncthreads();  // the order has been written by all threads of this CTA
  if (!ok || full) {
    if (tid == 0) {
      p.work[1] = 0;
      flag(p, ok ? HF_S_FULL : HF_S_BAD);
    }
    return;
  }
  auto page_at = [&](int rank) { return rank < NEAR ? s_free[rank] : dst[rank]; };
  // an entry's copy comes first, then its new pages
  int cdst[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    cdst[k] = -1;
    if (req_[k] < 0 || cnt_[k] == 0) continue;
    const int have = pages_of(len_[k], p.page);
    int32_t* row = p.table + (size_t)req_[k] * p.table_ld;
    if (copy[k]) {
      cdst[k] = page_at(at);
      row[have - 1] = cdst[k];
      p.refs[cdst[k]] = 1;
      atomicSub(&p.refs[last_[k]], 1);
    }
    for (int j = copy[k]; j < need[k]; ++j) {
      const int id = page_at(at + j);
      row[have + j - copy[k]] = id;
      p.refs[id] = 1;
    }
    at += need[k];
    p.lens[req_[k]] = len_[k] + cnt_[k];
  }
  __syncthreads();  // the order of free pages has been read: the moves take its place
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (cdst[k] >= 0) {
      src[cat] = last_[k];
      dst[cat] = cdst[k];
      ++cat;
    }
  if (tid == 0) p.work[1] = ncopy;
}

// Planned moves src[m] -> dst[m] of whole pages, in every layer, K and V; the
// tables follow when `remap` is set (compact: entries at or behind `used` move).
__device__ __forceinline__ void move_pages(const hf_pages& p, int moves) {
  const int32_t* src = p.work + kMoves;
  const int32_t* dst = src + move_room(p);
  const long long bytes = (long long)p.n_kv_heads * p.page * p.head_dim * (p.dtype == HF_F32 ? 4 : 2);
  const int vecs = (int)(bytes / 16);  // a page of 8 rows of 8 elements is already 128 bytes
  const int per = (vecs + CT * 4 - 1) / (CT * 4);  // pieces of 16 KB
  const long long units = (long long)moves * p.n_layers * 2 * per;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % per);
    long long w = u / per;
    const int kv = (int)(w & 1);
    w >>= 1;
    const int layer = (int)(w % p.n_layers), m = (int)(w / p.n_layers);
    uint8_t* base = static_cast<uint8_t*>(kv ? p.v : p.k) + (long long)layer * p.n_pages * bytes;
    const uint4* s = reinterpret_cast<const uint4*>(base + (long long)__ldcg(&src[m]) * bytes);
    uint4* d = reinterpret_cast<uint4*>(base + (long long)__ldcg(&dst[m]) * bytes);
    const int i0 = piece * CT * 4 + threadIdx.x;
    uint4 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * CT < vecs) r[k] = __ldcs(s + i0 + k * CT);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * CT < vecs) d[i0 + k * CT] = r[k];
  }
}

__global__ void __launch_bounds__(CT) extend_copy(hf_pages p) {
  pdl_trigger();
  pdl_wait();
  move_pages(p, __ldcg(&p.work[1]));
}

// ------------------------------------------------------------------- compact
// One CTA: L = pages in use; the j-th used page at or behind L goes to the j-th
// free page before it (there are as many of one as of the other). `src` and `dst`
// come in rising order.
__global__ void __launch_bounds__(PT) compact_plan(hf_pages p, int32_t* n_used) {
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int32_t* src = p.work + kMoves;
  int32_t* dst = src + move_room(p);
  int c = 0;
  for (int i = tid; i < p.n_pages; i += PT) c += __ldcg(&p.refs[i]) > 0;
  int used;
  cta_scan(c, used);
  int moves = 0, holes = 0;
  for (int base = 0; base < p.n_pages; base += PT * 8) {
    const int b0 = base + tid * 8;
    uint32_t high = 0, hole = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (b0 + k < p.n_pages) {
        const bool in_use = __ldcg(&p.refs[b0 + k]) > 0;
        if (in_use && b0 + k >= used) high |= 1u << k;
        if (!in_use && b0 + k < used) hole |= 1u << k;
      }
    // both counts in one scan: at most 8 * 1024 = 2^13 each
    int sum;
    const int at = cta_scan(__popc(high) << 16 | __popc(hole), sum);
    int rh = moves + (at >> 16), ro = holes + (at & 0xffff);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (high >> k & 1) src[rh++] = b0 + k;
      if (hole >> k & 1) dst[ro++] = b0 + k;
    }
    moves += sum >> 16;
    holes += sum & 0xffff;
  }
  __syncthreads();
  for (int m = tid; m < moves; m += PT) {
    const int s = src[m], d = dst[m];
    p.refs[d] = p.refs[s];
    p.refs[s] = 0;
  }
  if (tid == 0) {
    p.work[1] = moves;
    p.work[2] = used;
    if (n_used) *n_used = used;
  }
}

__global__ void __launch_bounds__(CT) compact_move(hf_pages p) {
  pdl_trigger();
  pdl_wait();
  const int moves = __ldcg(&p.work[1]), used = __ldcg(&p.work[2]);
  if (moves == 0) return;
  const int32_t* src = p.work + kMoves;
  const int32_t* dst = src + move_room(p);
  // tables: an entry at or behind `used` names src[m] for some m (src rises)
  for (int r = blockIdx.x; r < p.n_requests; r += gridDim.x) {
    const int j1 = min(pages_of(max(__ldcg(&p.lens[r]), 0), p.page), p.table_ld);
    for (int j = threadIdx.x; j < j1; j += CT) {
      int32_t* e = p.table + (size_t)r * p.table_ld + j;
      const int id = *e;
      if (id < used || id >= p.n_pages) continue;
      int lo = 0, hi = moves;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(&src[mid]) < id)
          lo = mid + 1;
        else
          hi = mid;
      }
      if (lo < moves && __ldcg(&src[lo]) == id)
        *e = __ldcg(&dst[lo]);
      else
        flag(p, HF_S_BAD);  // a page in a table that nobody counts
    }
  }
  move_pages(p, moves);
}

// --------------------------------------------------------------------- write
struct WriteArgs {
  const uint8_t* k;
  const uint8_t* v;
  long long ld, layer_stride;  // bytes
  const int32_t* req;
  const int32_t* off;
  int n, total, layer, layers;
};

// The last index in [0, n) whose offset is at or before t (offsets rise), by one warp: 32
// of them are looked at side by side, so that three dependent loads do for 4096.
__device__ __forceinline__ int find_entry(const int32_t* off, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, count = n;
  while (count > 1) {
    const int step = (count + 31) / 32, i = lane * step;
    const bool before = i < count && __ldcg(&off[lo + i]) <= t;
    const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, before)));
    lo += k * step;
    count = min(step, count - k * step);
  }
  return lo;
}

// One warp per row and up to kCopies of its (layer, K or V): heads * head_dim elements go
// to as many places of head_dim elements as there are heads. Small calls are bound by the
// dependent look-ups, so they are made once for several copies; large ones by the copies.
constexpr int kCopies = 8;
__global__ void __launch_bounds__(CT) write_kernel(hf_pages p, WriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int groups = (2 * a.layers + kCopies - 1) / kCopies;
  const long long units = (long long)a.total * groups;
  const int esize = p.dtype == HF_F32 ? 4 : 2;
  const int hv = p.head_dim * esize / 16, vecs = p.n_kv_heads * hv;  // 16-byte pieces of a head, of a row
  const long long block = (long long)p.n_kv_heads * p.page * hv;
  // bounds that decrease name rows twice, or name entries that the search does not find
  bool falls = false, range = true;
  for (int i = threadIdx.x; i <= a.n; i += CT) {
    const int x = __ldcg(&a.off[i]);
    falls = falls || (i > 0 && x < __ldcg(&a.off[i - 1]));
    range = range && x >= 0 && x <= a.total;
  }
  if (blockIdx.x == 0 && (falls || !range)) flag(p, HF_S_BAD);
  if (__syncthreads_or(falls)) return;
  for (long long u = (long long)blockIdx.x * (CT / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (CT / 32)) {
    const int t = (int)(u / groups), c0 = (int)(u % groups) * kCopies;
    const int e = find_entry(a.off, a.n, t);
    const int o0 = __ldcg(&a.off[e]), o1 = __ldcg(&a.off[e + 1]), r = a.req ? __ldcg(&a.req[e]) : e;
    if (t < o0 || t >= o1) continue;  // nobody's row
    bool ok = o0 >= 0 && o1 <= a.total && r >= 0 && r < p.n_requests;
    if (a.req)  // named twice: its rows would have two sources
      for (int i = lane; i < a.n; i += 32) ok = ok && (i == e || __ldcg(&a.req[i]) != r);
    ok = __all_sync(0xffffffffu, ok);
    int id = -1, at = -1;
    if (ok) {
      const int len = __ldcg(&p.lens[r]);
      at = len - o1 + t;
      ok = at >= 0 && len - o1 + o0 >= 0 && at / p.page < p.table_ld;
      if (ok) id = __ldcg(&p.table[(size_t)r * p.table_ld + at / p.page]);
      ok = ok && id >= 0 && id < p.n_pages;
    }
    if (!ok) {
      if (lane == 0) flag(p, HF_S_BAD);
      continue;
    }
    const long long row = (long long)t * a.ld;
    const long long to = (long long)id * block + (long long)(at % p.page) * hv;
    const int c1 = min(c0 + kCopies, 2 * a.layers);
    for (int i = lane; i < vecs; i += 32) {
      const long long d = to + (long long)(i / hv) * p.page * hv + i % hv;
      uint4 x[kCopies];
#pragma unroll
      for (int k = 0; k < kCopies; ++k)
        if (c0 + k < c1) {
          const int c = c0 + k;
          x[k] = __ldcs(reinterpret_cast<const uint4*>((c & 1 ? a.v : a.k) + (long long)(c >> 1) * a.layer_stride + row) + i);
        }
#pragma unroll
      for (int k = 0; k < kCopies; ++k)
        if (c0 + k < c1) {
          const int c = c0 + k;
          (reinterpret_cast<uint4*>(c & 1 ? p.v : p.k) + (long long)(a.layer + (c >> 1)) * p.n_pages * block)[d] = x[k];
        }
    }
  }
}

hf_status refuse(const char* m) {
  set_thread_error(m);
  return HF_EINVAL;
}
hf_status done(cudaError_t e) {
  if (e == cudaSuccess) return HF_OK;
  set_thread_error(cudaGetErrorString(e));
  return HF_ECUDA;
}
bool off4(const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 != 0; }

const char* list_bad(const hf_pages* p, int32_t n) {
  if (const char* m = pages_bad(p, true)) return m;
  if (n < 0 || n > p->n_requests) return "n must be 0..n_requests";
  return nullptr;
}

}  // namespace
}  // namespace hf

extern "C" size_t hf_pages_work_ints(const hf_pages* p) {
  if (hf::pages_bad(p, false)) return 0;
  return hf::kMoves + 2 * (size_t)std::max(p->n_pages, p->n_requests);
}

extern "C" hf_status hf_pages_truncate(const hf_pages* p, const int32_t* requests, const int32_t* keep,
                                       int32_t n, void* stream) {
  using namespace hf;
  if (const char* m = list_bad(p, n)) return refuse(m);
  if (n == 0) return HF_OK;
  if (!keep) return refuse("NULL buffer");
  if (off4(requests) || off4(keep)) return refuse("lists must be 4-byte aligned");
  return done(launch_pdl(truncate_kernel, dim3(std::min(n, 152)), dim3(CT), 0, (cudaStream_t)stream, *p, requests,
                         keep, (int)n));
}

extern "C" hf_status hf_pages_fork(const hf_pages* p, const int32_t* from, const int32_t* into, int32_t n,
                                   void* stream) {
  using namespace hf;
  if (const char* m = list_bad(p, n)) return refuse(m);
  if (n == 0) return HF_OK;
  if (!from || !into) return refuse("NULL buffer");
  if (off4(from) || off4(into)) return refuse("lists must be 4-byte aligned");
  return done(launch_pdl(fork_kernel, dim3(std::min(n, 152)), dim3(CT), 0, (cudaStream_t)stream, *p, from, into,
                         (int)n));
}

extern "C" hf_status hf_pages_extend(const hf_pages* p, const int32_t* requests, const int32_t* counts,
                                     int32_t n, void* stream) {
  using namespace hf;
  if (const char* m = list_bad(p, n)) return refuse(m);
  if (n == 0) return HF_OK;
  if (!counts) return refuse("NULL buffer");
  if (off4(requests) || off4(counts)) return refuse("lists must be 4-byte aligned");
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(extend_plan, dim3(1), dim3(PT), 0, st, *p, requests, counts, (int)n);
  // at most one copied page per request, in pieces of 16 KB
  const long long pieces = (pages_block(p) * (p->dtype == HF_F32 ? 4 : 2) / 16 + CT * 4 - 1) / (CT * 4);
  const long long units = (long long)n * p->n_layers * 2 * pieces;
  if (e == cudaSuccess)
    e = launch_pdl(extend_copy, dim3((unsigned)std::min<long long>(units, 152 * 8)), dim3(CT), 0, st, *p);
  return done(e);
}

extern "C" hf_status hf_pages_compact(const hf_pages* p, int32_t* n_used, void* stream) {
  using namespace hf;
  if (const char* m = pages_bad(p, true)) return refuse(m);
  if (off4(n_used)) return refuse("n_used must be 4-byte aligned");
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(compact_plan, dim3(1), dim3(PT), 0, st, *p, n_used);
  if (e == cudaSuccess) e = launch_pdl(compact_move, dim3(152 * 8), dim3(CT), 0, st, *p);
  return done(e);
}

extern "C" hf_status hf_pages_write(const hf_pages* p, int32_t layer, int32_t layers, const void* k,
                                    const void* v, int64_t ld, int64_t layer_stride, const int32_t* requests,
                                    const int32_t* offsets, int32_t n, int32_t total, void* stream) {
  using namespace hf;
  if (const char* m = list_bad(p, n)) return refuse(m);
  if (layer < 0 || layers < 0 || layer > p->n_layers || layers > p->n_layers - layer)
    return refuse("layer .. layer + layers - 1 must be layers of the cache");
  if (total < 0) return refuse("total must be >= 0");
  if (n == 0 || layers == 0 || total == 0) return HF_OK;
  const int esize = p->dtype == HF_F32 ? 4 : 2;
  if (!k || !v || !offsets) return refuse("NULL buffer");
  if (ld < (int64_t)p->n_kv_heads * p->head_dim || layer_stride < 0 || ld > (1LL << 40) ||
      layer_stride > (1LL << 48))
    return refuse("ld must be >= n_kv_heads * head_dim, layer_stride >= 0");
  if (ld * esize % 16 || layer_stride * esize % 16 || reinterpret_cast<uintptr_t>(k) % 16 ||
      reinterpret_cast<uintptr_t>(v) % 16)
    return refuse("k and v must be 16-byte aligned, their strides multiples of 16 bytes");
  if (off4(requests) || off4(offsets)) return refuse("lists must be 4-byte aligned");
  WriteArgs a{};
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.ld = ld * esize;
  a.layer_stride = layer_stride * esize;
  a.req = requests;
  a.off = offsets;
  a.n = n;
  a.total = total;
  a.layer = layer;
  a.layers = layers;
  const long long warps = (long long)total * ((2 * layers + kCopies - 1) / kCopies);
  const long long grid = std::min<long long>((warps + CT / 32 - 1) / (CT / 32), 152 * 8);
  return done(launch_pdl(write_kernel, dim3((unsigned)grid), dim3(CT), 0, (cudaStream_t)stream, *p, a));
}
