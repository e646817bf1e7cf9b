// The 8-bit cache (hf_pages8): rows quantised as they are written, and read back.
//
//   s = max(s_old if rows before the written ones stay, least 2^e with max |x| <= 448 2^e)
//   code = nearest e4m3 to x / s
// for each page and KV head that rows go to. A power of two as the scale makes x / s exact, so a code
// is rounded once, and codes of an old scale carry over to a larger one without loss down
// to the smallest codes. Bound by the reads of the rows and the writes of the codes.
#include <cstdio>

#include "e4m3.cuh"
#include "pages.cuh"

namespace hf {

const char* pages8_bad(const hf_pages8* p, bool buffers) {
  if (!p) return "NULL cache";
  if (const char* m = pages_bad(&p->pages, buffers, true)) return m;
  if (p->pages.head_dim % 16) return "cache: head_dim must be a multiple of 16";
  if (p->rows != HF_F32 && p->rows != HF_BF16) return "cache: rows must be HF_F32 or HF_BF16";
  if (p->reserved) return "cache: reserved must be 0";
  if (!buffers) return nullptr;
  if (!p->k_scale || !p->v_scale) return "cache: NULL buffer";
  if (reinterpret_cast<uintptr_t>(p->k_scale) % 4 || reinterpret_cast<uintptr_t>(p->v_scale) % 4)
    return "cache: k_scale and v_scale must be 4-byte aligned";
  return nullptr;
}

namespace {

constexpr int CT = 256;

struct RowsArgs {
  hf_pages p;
  PageScales sc;
  uint8_t* k;  // rows
  uint8_t* v;
  long long ld, layer_stride;  // bytes
  const int32_t* req;
  const int32_t* first;  // read
  const int32_t* off;
  int n, total, layer, layers;
};

// 16 bytes of a row as values.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& w, float* x) {
  if constexpr (sizeof(T) == 4) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  } else {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
}

// Bounds that decrease; by one CTA. Bounds out of range are reported by CTA 0.
__device__ __forceinline__ bool offsets_fall(const RowsArgs& a) {
  bool falls = false, range = true;
  for (int i = threadIdx.x; i <= a.n; i += CT) {
    const int x = __ldcg(&a.off[i]);
    falls = falls || (i > 0 && x < __ldcg(&a.off[i - 1]));
    range = range && x >= 0 && x <= a.total;
  }
  if (blockIdx.x == 0 && (falls || !range)) pages_flag(a.p, HF_S_BAD);
  return __syncthreads_or(falls);
}

// One warp per page that an entry's rows go to, layer, K or V, and KV head. An entry of c rows reaches
// at most c / page + 2 pages: it owns the slots [off / page + 2 e, ..) of all, no prefix sum needed.
template <typename T>
__global__ void __launch_bounds__(CT) write8_kernel(RowsArgs a) {
  constexpr int VE = 16 / sizeof(T);
  pdl_trigger();
  pdl_wait();
  const hf_pages& p = a.p;
  const int lane = threadIdx.x & 31, H = p.n_kv_heads, dh = p.head_dim, hv = dh / VE;
  if (offsets_fall(a)) return;
  auto first_slot = [&](int e) { return min(max(__ldcg(&a.off[e]), 0), a.total) / p.page + 2 * e; };
  const long long per = (long long)a.layers * 2 * H;
  const long long units = ((long long)a.total / p.page + 2 * a.n) * per;
  for (long long u = (long long)blockIdx.x * (CT / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (CT / 32)) {
    const int slot = (int)(u / per);
    int w = (int)(u % per);
    const int h = w % H;
    w /= H;
    const int kv = w & 1, l = w >> 1;
    const int e = pages_find(a.n, slot, first_slot);
    const int o0 = __ldcg(&a.off[e]), o1 = __ldcg(&a.off[e + 1]), r = a.req ? __ldcg(&a.req[e]) : e;
    if (o1 == o0) continue;
    bool ok = o0 >= 0 && o1 <= a.total && r >= 0 && r < p.n_requests;
    if (a.req)  // named twice: its rows would have two sources
      for (int i = lane; i < a.n; i += 32) ok = ok && (i == e || __ldcg(&a.req[i]) != r);
    ok = __all_sync(0xffffffffu, ok);
    int id = -1, r0 = 0, r1 = 0, src = 0;
    if (ok) {
      const int len = __ldcg(&p.lens[r]), c = o1 - o0, j = slot - first_slot(e);
      ok = len >= c && pages_of(len, p.page) <= p.table_ld;
      if (ok) {
        const int page = (len - c) / p.page + j;
        const long long base = (long long)page * p.page;
        if (base >= len) continue;
        r0 = (int)max(0LL, len - c - base);
        r1 = (int)min((long long)p.page, len - base);
        src = o0 + (int)(base + r0 - (len - c));
        id = __ldcg(&p.table[(size_t)r * p.table_ld + page]);
        ok = id >= 0 && id < p.n_pages;
      }
    }
    if (!ok) {
      if (lane == 0) pages_flag(p, HF_S_BAD);
      continue;
    }
    const uint8_t* rows = (kv ? a.v : a.k) + (long long)l * a.layer_stride + (long long)src * a.ld + (long long)h * dh * sizeof(T);
    const size_t block = ((size_t)(a.layer + l) * p.n_pages + id) * H + h;
    uint8_t* codes = static_cast<uint8_t*>(kv ? p.v : p.k) + block * p.page * dh;
    float* scale = (kv ? a.sc.v : a.sc.k) + block;
    const int vecs = (r1 - r0) * hv;
    float top = 0.f;
    for (int i = lane; i < vecs; i += 32) {
      float x[VE];
      unpack16<T>(__ldcg(reinterpret_cast<const uint4*>(rows + (long long)(i / hv) * a.ld) + i % hv), x);
#pragma unroll
      for (int k = 0; k < VE; ++k) top = fmaxf(top, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.f);
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    float s = scale_for(top);
    if (r0 > 0) {
      const float old = held_scale(__ldcg(scale));
      if (s > old) {  // the rows that stay, again
        const float f = old / s;
        for (int i = lane; i < r0 * dh / 16; i += 32) {
          uint4 c = reinterpret_cast<uint4*>(codes)[i];
          uint32_t* cw = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 lo = from_e4m3x2(cw[k] & 0xffff), hi = from_e4m3x2(cw[k] >> 16);
            cw[k] = to_e4m3x2(lo.x * f, lo.y * f) | to_e4m3x2(hi.x * f, hi.y * f) << 16;
          }
          reinterpret_cast<uint4*>(codes)[i] = c;
        }
      }
      s = fmaxf(s, old);
    }
    const float inv = 1.f / s;  // (a power of two)
    for (int i = lane; i < vecs; i += 32) {
      float x[VE];
      unpack16<T>(__ldcg(reinterpret_cast<const uint4*>(rows + (long long)(i / hv) * a.ld) + i % hv), x);
      uint32_t c[VE / 4];
#pragma unroll
      for (int k = 0; k < VE; ++k) x[k] = no_inf(x[k]) * inv;
#pragma unroll
      for (int k = 0; k < VE / 4; ++k)
        c[k] = to_e4m3x2(x[4 * k], x[4 * k + 1]) | to_e4m3x2(x[4 * k + 2], x[4 * k + 3]) << 16;
      uint8_t* to = codes + (size_t)r0 * dh + (size_t)i * VE;
      if constexpr (VE == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = c[0];
    }
    if (lane == 0) *scale = s;
  }
}

// One warp per row and (layer, K or V): 16 codes a lane and step.
template <typename T>
__global__ void __launch_bounds__(CT) read8_kernel(RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const hf_pages& p = a.p;
  const int lane = threadIdx.x & 31, H = p.n_kv_heads, dh = p.head_dim, hv = dh / 16;
  if (offsets_fall(a)) return;
  const long long units = (long long)a.total * a.layers * 2;
  for (long long u = (long long)blockIdx.x * (CT / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (CT / 32)) {
    const int t = (int)(u / (2 * a.layers)), w = (int)(u % (2 * a.layers)), kv = w & 1, l = w >> 1;
    const int e = pages_find(a.n, t, [&](int i) { return __ldcg(&a.off[i]); });
    const int o0 = __ldcg(&a.off[e]), o1 = __ldcg(&a.off[e + 1]), r = a.req ? __ldcg(&a.req[e]) : e;
    if (t < o0 || t >= o1) continue;  // nobody's row
    bool ok = o0 >= 0 && o1 <= a.total && r >= 0 && r < p.n_requests;
    int id = -1, at = 0;
    if (ok) {
      const int len = __ldcg(&p.lens[r]), f = __ldcg(&a.first[e]);
      ok = f >= 0 && len >= 0 && f <= len && o1 - o0 <= len - f && pages_of(len, p.page) <= p.table_ld;
      if (ok) {
        at = f + t - o0;
        id = __ldcg(&p.table[(size_t)r * p.table_ld + at / p.page]);
        ok = id >= 0 && id < p.n_pages;
      }
    }
    if (!ok) {
      if (lane == 0) pages_flag(p, HF_S_BAD);
      continue;
    }
    const size_t block = ((size_t)(a.layer + l) * p.n_pages + id) * H;
    const uint8_t* codes = static_cast<const uint8_t*>(kv ? p.v : p.k) + (block * p.page + at % p.page) * dh;
    const float* scale = (kv ? a.sc.v : a.sc.k) + block;
    uint8_t* row = (kv ? a.v : a.k) + (long long)l * a.layer_stride + (long long)t * a.ld;
    for (int i = lane; i < H * hv; i += 32) {
      const int h = i / hv;
      const uint4 c = __ldcg(reinterpret_cast<const uint4*>(codes + (size_t)h * p.page * dh) + i % hv);
      const float s = __ldcg(&scale[h]);
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
      uint4* to = reinterpret_cast<uint4*>(row + (size_t)i * 16 * sizeof(T));
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = from_e4m3x2(cw[k] & 0xffff), hi = from_e4m3x2(cw[k] >> 16);
          reinterpret_cast<float4*>(to)[k] = make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s);
        }
      } else {
        uint4 y[2];
        __nv_bfloat162* y2 = reinterpret_cast<__nv_bfloat162*>(y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = from_e4m3x2(cw[k] & 0xffff), hi = from_e4m3x2(cw[k] >> 16);
          y2[2 * k] = __floats2bfloat162_rn(lo.x * s, lo.y * s);
          y2[2 * k + 1] = __floats2bfloat162_rn(hi.x * s, hi.y * s);
        }
        to[0] = y[0];
        to[1] = y[1];
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

// The checks and arguments that write and read share; *run is false where there is nothing to do.
const char* rows_args(const hf_pages8* p, int32_t layer, int32_t layers, const void* k, const void* v, int64_t ld,
                      int64_t layer_stride, const int32_t* requests, const int32_t* first, bool reads,
                      const int32_t* offsets, int32_t n, int32_t total, RowsArgs& a, bool* run) {
  *run = false;
  if (const char* m = pages8_bad(p, true)) return m;
  const hf_pages& c = p->pages;
  // (a read may name a request as often as it likes)
  if (n < 0 || (reads ? n > (1 << 20) : n > c.n_requests)) return reads ? "n must be 0..1048576" : "n must be 0..n_requests";
  if (reads && !requests && n > c.n_requests) return "n must be <= n_requests without a list of requests";
  if (layer < 0 || layers < 0 || layer > c.n_layers || layers > c.n_layers - layer)
    return "layer .. layer + layers - 1 must be layers of the cache";
  if (total < 0) return "total must be >= 0";
  if (n == 0 || layers == 0 || total == 0) return nullptr;
  const int esize = pages_esize(p->rows);
  if (!k || !v || !offsets || (reads && !first)) return "NULL buffer";
  if (ld < (int64_t)c.n_kv_heads * c.head_dim || layer_stride < 0 || ld > (1LL << 40) || layer_stride > (1LL << 48))
    return "ld must be >= n_kv_heads * head_dim, layer_stride >= 0";
  if (ld * esize % 16 || layer_stride * esize % 16 || reinterpret_cast<uintptr_t>(k) % 16 ||
      reinterpret_cast<uintptr_t>(v) % 16)
    return "k and v must be 16-byte aligned, their strides multiples of 16 bytes";
  if (off4(requests) || off4(offsets) || off4(first)) return "lists must be 4-byte aligned";
  a.p = c;
  a.sc = {p->k_scale, p->v_scale};
  a.k = static_cast<uint8_t*>(const_cast<void*>(k));
  a.v = static_cast<uint8_t*>(const_cast<void*>(v));
  a.ld = ld * esize;
  a.layer_stride = layer_stride * esize;
  a.req = requests;
  a.first = first;
  a.off = offsets;
  a.n = n;
  a.total = total;
  a.layer = layer;
  a.layers = layers;
  *run = true;
  return nullptr;
}

dim3 grid_of(long long warps) { return dim3((unsigned)std::min<long long>((warps + CT / 32 - 1) / (CT / 32), 152 * 8)); }

}  // namespace
}  // namespace hf

extern "C" size_t hf_pages8_work_ints(const hf_pages8* p) {
  return hf::pages8_bad(p, false) ? 0 : hf::pages_work_ints(&p->pages, true);
}

extern "C" hf_status hf_pages8_extend(const hf_pages8* p, const int32_t* requests, const int32_t* counts, int32_t n,
                                      void* stream) {
  if (const char* m = hf::pages8_bad(p, true)) return hf::refuse(m);
  return hf::pages_extend(&p->pages, true, {p->k_scale, p->v_scale}, requests, counts, n, stream);
}

extern "C" hf_status hf_pages8_fork(const hf_pages8* p, const int32_t* from, const int32_t* into, int32_t n,
                                    void* stream) {
  if (const char* m = hf::pages8_bad(p, true)) return hf::refuse(m);
  return hf::pages_fork(&p->pages, true, from, into, n, stream);
}

extern "C" hf_status hf_pages8_truncate(const hf_pages8* p, const int32_t* requests, const int32_t* keep, int32_t n,
                                        void* stream) {
  if (const char* m = hf::pages8_bad(p, true)) return hf::refuse(m);
  return hf::pages_truncate(&p->pages, true, requests, keep, n, stream);
}

extern "C" hf_status hf_pages8_compact(const hf_pages8* p, int32_t* n_used, void* stream) {
  if (const char* m = hf::pages8_bad(p, true)) return hf::refuse(m);
  return hf::pages_compact(&p->pages, true, {p->k_scale, p->v_scale}, n_used, stream);
}

extern "C" hf_status hf_pages8_write(const hf_pages8* p, int32_t layer, int32_t layers, const void* k, const void* v,
                                     int64_t ld, int64_t layer_stride, const int32_t* requests, const int32_t* offsets,
                                     int32_t n, int32_t total, void* stream) {
  using namespace hf;
  RowsArgs a{};
  bool run;
  if (const char* m = rows_args(p, layer, layers, k, v, ld, layer_stride, requests, nullptr, false, offsets, n, total, a, &run))
    return refuse(m);
  if (!run) return HF_OK;
  const dim3 grid = grid_of((total / a.p.page + 2LL * n) * layers * 2 * a.p.n_kv_heads);
  auto* kern = p->rows == HF_F32 ? write8_kernel<float> : write8_kernel<__nv_bfloat16>;
  return done(launch_pdl(kern, grid, dim3(CT), 0, (cudaStream_t)stream, a));
}

extern "C" hf_status hf_pages8_read(const hf_pages8* p, int32_t layer, int32_t layers, void* k, void* v, int64_t ld,
                                    int64_t layer_stride, const int32_t* requests, const int32_t* first,
                                    const int32_t* offsets, int32_t n, int32_t total, void* stream) {
  using namespace hf;
  RowsArgs a{};
  bool run;
  if (const char* m = rows_args(p, layer, layers, k, v, ld, layer_stride, requests, first, true, offsets, n, total, a, &run))
    return refuse(m);
  if (!run) return HF_OK;
  auto* kern = p->rows == HF_F32 ? read8_kernel<float> : read8_kernel<__nv_bfloat16>;
  return done(launch_pdl(kern, grid_of((long long)total * layers * 2), dim3(CT), 0, (cudaStream_t)stream, a));
}
