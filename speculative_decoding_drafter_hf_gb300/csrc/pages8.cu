// The 8-bit cache (hf_pages8): rows quantised as they are written, and read back.
//
//   s = max(s_old if rows before the written ones stay, least 2^e with max |x| <= 448 2^e)
//   code = nearest e4m3 to x / s
// for each page and KV head that rows go to. A power of two as the scale makes x / s exact, so a code
// is rounded once, and codes of an old scale carry over to a larger one without loss down
// to the smallest codes.
//
// Few rows: bound by the chain of look-ups (bounds, length, page, rows), one launch each way: 64 x 8 rows into three
// layers 10.1 us, and 64 x 8 to 23 rows of them back 10.2. Many: 10732 rows of 10 heads of 128 written in 21 us
// (3.9 TB/s, instructions issued in 65% of the cycles), read back in 20 (4.1 TB/s); 54198 rows of 8 heads
// in three layers read back in 165 us (6.0 TB/s, the memory). Tried and no faster: neighbouring units to one warp,
// so that it looks a page up once (170 -> 200 then), codes to bf16 by their bits (169 -> 173).
#include <cstdio>

#include "attn.cuh"
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
  int slots;  // places for the pages of all entries
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

// 16 bytes of a row with NaN for its infinities; out of line, as few rows need it.
template <typename T>
__device__ __noinline__ uint4 no_inf16(uint4 y) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      if ((w[k] & 0x7fffffffu) == 0x7f800000u) w[k] = 0x7fffffffu;
    } else {
      if ((w[k] & 0x7fffu) == 0x7f80u) w[k] |= 0x7fffu;
      if ((w[k] & 0x7fff0000u) == 0x7f800000u) w[k] |= 0x7fff0000u;
    }
  }
  return y;
}

// i / d of 0 <= i < 2^24, 1 <= d <= 256.
struct Over {
  uint32_t by;
  __device__ __forceinline__ explicit Over(int d) : by((uint32_t)((0x100000000ULL + d - 1) / d)) {}
  __device__ __forceinline__ int operator()(int i) const { return by ? (int)__umulhi((uint32_t)i, by) : i; }
};

// Magnitudes as bits: their order is that of unsigned integers, and what is not finite comes behind.
template <typename T>
struct Bits;
template <>
struct Bits<float> {
  static constexpr uint32_t kOdd = 0x7f800000u;  // the first that is not finite
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
  static __device__ __forceinline__ uint32_t one(uint32_t m) { return m; }
};
template <>
struct Bits<__nv_bfloat16> {  // two in a word
  static constexpr uint32_t kOdd = 0x7f800000u;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
  static __device__ __forceinline__ uint32_t one(uint32_t m) { return max(m & 0xffff0000u, m << 16); }
};

// Pieces of 16 bytes that a lane has at a time. Writing keeps them in registers between the two looks at them
// (10732 rows of 10 heads of 128, pages of 64: 24.2 us, with four 32.9); reading back 20.6 us with four, 24.6
// with eight.
constexpr int KEEP = 8, READ = 4;
constexpr int kListed = kMaxRequests;  // entries whose bounds a CTA keeps in shared memory

// The list of a call as a CTA has it: bounds in shared memory (few entries) or where they lie.
struct Entries {
  const RowsArgs& a;
  int* s_off;
  int shift;  // of the page
  __device__ __forceinline__ int off(int i) const { return a.n <= kListed ? s_off[i] : __ldcg(&a.off[i]); }
  // An entry of c rows reaches at most c / page + 2 pages: it owns the slots [off / page + 2 e, ..) of all, so
  // that no prefix sum is needed.
  __device__ __forceinline__ int first_slot(int e) const { return (min(max(off(e), 0), a.total) >> shift) + 2 * e; }
};

// Loads the bounds; true where they decrease (names rows twice, or entries that no search finds). Bounds out of
// range are reported by CTA 0. By one CTA.
__device__ __forceinline__ bool load_entries(const RowsArgs& a, int* s_off) {
  bool falls = false, range = true;
  for (int i = threadIdx.x; i <= a.n; i += CT) {
    const int x = __ldcg(&a.off[i]);
    if (a.n <= kListed) s_off[i] = x;
    falls = falls || (i > 0 && x < __ldcg(&a.off[i - 1]));
    range = range && x >= 0 && x <= a.total;
  }
  if (blockIdx.x == 0 && (falls || !range)) pages_flag(a.p, HF_S_BAD);
  return __syncthreads_or(falls);
}

// Which requests the list names twice, one bit each. By one CTA.
__device__ __forceinline__ void load_twice(const RowsArgs& a, uint32_t* seen, uint32_t* twice) {
  for (int i = threadIdx.x; i < kMaxRequests / 32; i += CT) seen[i] = twice[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += CT) {
    const int r = __ldcg(&a.req[i]);
    if (r < 0 || r >= a.p.n_requests) continue;
    const uint32_t bit = 1u << (r & 31);
    if (atomicOr(&seen[r >> 5], bit) & bit) atomicOr(&twice[r >> 5], bit);
  }
  __syncthreads();
}

// One page of an entry, as the call sees it: rows r0 .. r1 - 1 of page `id` and rows src .. of the caller. False:
// nothing there; an entry that breaks a rule is reported.
struct PageOf {
  int id, r0, r1, src;
};
template <bool WRITE>
__device__ __forceinline__ bool page_of(const Entries& E, int slot, const uint32_t* twice, bool report, PageOf& g) {
  const RowsArgs& a = E.a;
  const hf_pages& p = a.p;
  const int e = pages_find(a.n, slot, [&](int i) { return E.first_slot(i); });
  const int o0 = E.off(e), o1 = E.off(e + 1), r = a.req ? __ldcg(&a.req[e]) : e;
  const int c = o1 - o0;
  if (c == 0) return false;
  bool ok = o0 >= 0 && o1 <= a.total && r >= 0 && r < p.n_requests;
  if (WRITE && a.req) ok = ok && !(twice[r >> 5] >> (r & 31) & 1);  // (its rows would have two sources)
  int first = 0;
  if (ok) {
    const int len = __ldcg(&p.lens[r]);
    first = WRITE ? len - c : __ldcg(&a.first[e]);
    ok = first >= 0 && first <= len && c <= len - first && pages_of(len, p.page) <= p.table_ld;
  }
  if (ok) {
    const int page = (first >> E.shift) + slot - E.first_slot(e);
    const long long base = (long long)page << E.shift, end = (long long)first + c;
    if (base >= end) return false;
    g.r0 = (int)max(0LL, first - base);
    g.r1 = (int)min((long long)p.page, end - base);
    g.src = o0 + (int)(base + g.r0 - first);
    g.id = __ldcg(&p.table[(size_t)r * p.table_ld + page]);
    ok = g.id >= 0 && g.id < p.n_pages;
  }
  if (!ok && report) pages_flag(p, HF_S_BAD);
  return ok;
}

// WPU warps per page that an entry's rows go to, layer, K or V, and KV head: as many as hold its rows in
// registers between the maximum and the codes (page of 64 x 128 bf16: four; what is more, 128 rows of
// 256 fp32 values, is read twice).
template <typename T, int WPU>
__global__ void __launch_bounds__(CT, 4) write8_kernel(RowsArgs a) {
  constexpr int VE = 16 / sizeof(T), UNITS = CT / 32 / WPU;
  extern __shared__ int s_off[];
  __shared__ uint32_t s_seen[kMaxRequests / 32], s_twice[kMaxRequests / 32];
  __shared__ uint32_t s_top[CT / 32];
  pdl_trigger();
  pdl_wait();
  const hf_pages& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPU, H = p.n_kv_heads, dh = p.head_dim, hv = dh / VE;
  if (load_entries(a, s_off)) return;
  if (a.req) load_twice(a, s_seen, s_twice);
  const Entries E{a, s_off, 31 - __clz(p.page)};
  const Over over_hv(hv);
  const int per = a.layers * 2 * H, units = a.slots * per;
  for (int u0 = blockIdx.x * UNITS; u0 < units; u0 += gridDim.x * UNITS) {
    const int u = u0 + warp / WPU, slot = u / per;
    int w = u - slot * per;
    const int h = w % H;
    w /= H;
    const int kv = w & 1, l = w >> 1;
    PageOf g{};
    const bool on = u < units && page_of<true>(E, slot, s_twice, lane == 0, g);
    const uint8_t* rows = nullptr;
    uint8_t* codes = nullptr;
    float* scale = nullptr;
    uint4 x[KEEP];
    float old = 0.f;
    uint32_t m[2] = {0, 0};  // the largest magnitude
    auto look = [&](const uint4& y) {
      m[0] = Bits<T>::most(Bits<T>::most(m[0], y.x), y.y);
      m[1] = Bits<T>::most(Bits<T>::most(m[1], y.z), y.w);
    };
    const int vecs = on ? (g.r1 - g.r0) * hv : 0, i0 = sub * 32 + lane;
    auto vec = [&](int i) {
      const int r = over_hv(i);
      return __ldcg(reinterpret_cast<const uint4*>(rows + (long long)r * a.ld) + i - r * hv);
    };
    if (on) {
      rows = (kv ? a.v : a.k) + (long long)l * a.layer_stride + (long long)g.src * a.ld + (long long)h * dh * sizeof(T);
      const size_t block = ((size_t)(a.layer + l) * p.n_pages + g.id) * H + h;
      codes = static_cast<uint8_t*>(kv ? p.v : p.k) + block * p.page * dh;
      scale = (kv ? a.sc.v : a.sc.k) + block;
      if (g.r0 > 0) old = held_scale(__ldcg(scale));
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        const int i = i0 + k * WPU * 32;
        x[k] = i < vecs ? vec(i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < KEEP; ++k) look(x[k]);
      for (int i = i0 + KEEP * WPU * 32; i < vecs; i += WPU * 32) look(vec(i));
    }
    __syncwarp();
    // the largest of the unit's warps
    auto join = [&](uint32_t t) {
      t = __reduce_max_sync(0xffffffffu, t);
      if constexpr (WPU > 1) {
        if (lane == 0) s_top[warp] = t;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WPU; ++k) t = max(t, s_top[warp - sub + k]);
        __syncthreads();  // (read before the next unit's)
      }
      return t;
    };
    uint32_t top = join(Bits<T>::one(Bits<T>::most(m[0], m[1])));
    const bool odd = top >= Bits<T>::kOdd;  // infinities or NaN among the values: they do not count
    bool any = odd;
    if constexpr (WPU > 1) any = __syncthreads_or(odd);
    if (any) {
      float t = 0.f;
      auto careful = [&](const uint4& y) {
        float v[VE];
        unpack16<T>(y, v);
#pragma unroll
        for (int k = 0; k < VE; ++k) t = fmaxf(t, fabsf(v[k]) < INFINITY ? fabsf(v[k]) : 0.f);
      };
      if (on) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) careful(x[k]);
        for (int i = i0 + KEEP * WPU * 32; i < vecs; i += WPU * 32) careful(vec(i));
      }
      __syncwarp();
      top = join(__float_as_uint(t));
    }
    if (!on) continue;
    const float s = fmaxf(scale_for(__uint_as_float(top)), old);
    if (s > old && old > 0.f) {  // the rows that stay, again
      const float f = old / s;
      for (int i = i0; i < g.r0 * dh / 16; i += WPU * 32) {
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
    const float inv = 1.f / s;  // (a power of two)
    auto put = [&](int i, uint4 y) {
      float v[VE];
      if (odd) y = no_inf16<T>(y);
      unpack16<T>(y, v);
      uint32_t c[VE / 4];
#pragma unroll
      for (int k = 0; k < VE; k += 2) {
        const float2 z = unpair(mul2(pair(v[k], v[k + 1]), pair(inv, inv)));
        v[k] = z.x;
        v[k + 1] = z.y;
      }
#pragma unroll
      for (int k = 0; k < VE / 4; ++k)
        c[k] = to_e4m3x2(v[4 * k], v[4 * k + 1]) | to_e4m3x2(v[4 * k + 2], v[4 * k + 3]) << 16;
      uint8_t* to = codes + (size_t)g.r0 * dh + (size_t)i * VE;
      if constexpr (VE == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = c[0];
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (i0 + k * WPU * 32 < vecs) put(i0 + k * WPU * 32, x[k]);
    for (int i = i0 + KEEP * WPU * 32; i < vecs; i += WPU * 32) put(i, vec(i));
    if (lane == 0 && sub == 0) *scale = s;
  }
}

// 2 KB of a page's codes (rows r0 .. r1 - 1 of them) to rows of values, by one warp. ZERO: rows of zeros.
template <typename T, bool ZERO = false>
__device__ __forceinline__ void read_piece(const uint4* codes, const float* scale, uint8_t* rows, long long ld, int piece,
                                           int r0, int r1, int hv, Over over_hv, int shift, int vecs) {
  const int lane = threadIdx.x & 31;
  uint4 c[READ];
  float s[READ];
  uint8_t* to[READ];  // NULL: not asked for
#pragma unroll
  for (int k = 0; k < READ; ++k) {
    const int i = piece * READ * 32 + k * 32 + lane, hr = over_hv(i), r = hr & ((1 << shift) - 1), h = hr >> shift;
    to[k] = i < vecs && r >= r0 && r < r1 ? rows + (long long)(r - r0) * ld + (size_t)(h * hv + i - hr * hv) * 16 * sizeof(T)
                                          : nullptr;
    if (ZERO) {
      c[k] = make_uint4(0, 0, 0, 0);
      s[k] = 0.f;
    } else if (to[k]) {
      c[k] = __ldcg(codes + i);
      s[k] = held_scale(__ldcg(&scale[h]));
    }
  }
#pragma unroll
  for (int k = 0; k < READ; ++k) {
    if (!to[k]) continue;
    const uint32_t cw[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 lo = from_e4m3x2(cw[q] & 0xffff), hi = from_e4m3x2(cw[q] >> 16);
        reinterpret_cast<float4*>(to[k])[q] = make_float4(lo.x * s[k], lo.y * s[k], hi.x * s[k], hi.y * s[k]);
      }
    } else {
      uint4 y[2];
      __nv_bfloat162* y2 = reinterpret_cast<__nv_bfloat162*>(y);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 lo = from_e4m3x2(cw[q] & 0xffff), hi = from_e4m3x2(cw[q] >> 16);
        y2[2 * q] = __floats2bfloat162_rn(lo.x * s[k], lo.y * s[k]);
        y2[2 * q + 1] = __floats2bfloat162_rn(hi.x * s[k], hi.y * s[k]);
      }
      reinterpret_cast<uint4*>(to[k])[0] = y[0];
      reinterpret_cast<uint4*>(to[k])[1] = y[1];
    }
  }
}

// One warp per 2 KB of codes of a page (all heads), layer, K or V.
template <typename T>
__global__ void __launch_bounds__(CT) read8_kernel(RowsArgs a) {
  extern __shared__ int s_off[];
  pdl_trigger();
  pdl_wait();
  const hf_pages& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = p.n_kv_heads, dh = p.head_dim, hv = dh / 16;
  if (load_entries(a, s_off)) return;
  const int shift = 31 - __clz(p.page), vecs = (H * hv) << shift, pieces = (vecs + READ * 32 - 1) / (READ * 32);
  const Entries E{a, s_off, shift};
  const Over over_hv(hv);
  const int per = a.layers * 2 * pieces, units = a.slots * per;
  for (int u = blockIdx.x * (CT / 32) + warp; u < units; u += gridDim.x * (CT / 32)) {
    const int slot = u / per;
    int w = u - slot * per;
    const int piece = w % pieces;
    w /= pieces;
    const int kv = w & 1, l = w >> 1;
    PageOf g{};
    const bool on = page_of<false>(E, slot, nullptr, lane == 0, g);
    __syncwarp();
    if (!on) continue;
    const size_t block = ((size_t)(a.layer + l) * p.n_pages + g.id) * H;
    const uint4* codes = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? p.v : p.k) + (block * dh << shift));
    const float* scale = (kv ? a.sc.v : a.sc.k) + block;
    uint8_t* rows = (kv ? a.v : a.k) + (long long)l * a.layer_stride + (long long)g.src * a.ld;
    read_piece<T>(codes, scale, rows, a.ld, piece, g.r0, g.r1, hv, over_hv, shift, vecs);
  }
}

// The first tokens of entry 0 as rows of values, for products that many rows share (its pages that are out of
// range are reported and read as zeros, as by the kernels that take codes).
__global__ void __launch_bounds__(CT) prefix8_kernel(RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const hf_pages& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = p.n_kv_heads, dh = p.head_dim, hv = dh / 16;
  const int shift = 31 - __clz(p.page), vecs = (H * hv) << shift, pieces = (vecs + READ * 32 - 1) / (READ * 32);
  const int r = a.req ? __ldcg(a.req) : 0;
  if (r < 0 || r >= p.n_requests) return;  // (an entry that breaks a rule is reported by the attention)
  const int len = __ldcg(&p.lens[r]);
  const int units = (a.total >> shift) * 2 * pieces;
  for (int u = blockIdx.x * (CT / 32) + warp; u < units; u += gridDim.x * (CT / 32)) {
    const int piece = u % pieces, kv = u / pieces & 1, j = u / pieces / 2;
    const int id = __ldcg(&p.table[(size_t)r * p.table_ld + j]);  // (the table reaches that far, whatever the length)
    if (len < a.total || pages_of(len, p.page) > p.table_ld) return;
    uint8_t* rows = (kv ? a.v : a.k) + (long long)j * p.page * a.ld;
    if (id < 0 || id >= p.n_pages) {
      if (lane == 0) pages_flag(p, HF_S_BAD);
      read_piece<__nv_bfloat16, true>(nullptr, nullptr, rows, a.ld, piece, 0, p.page, hv, Over(hv), shift, vecs);
      continue;
    }
    const size_t block = ((size_t)a.layer * p.n_pages + id) * H;
    const uint4* codes = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? p.v : p.k) + (block * dh << shift));
    read_piece<__nv_bfloat16>(codes, (kv ? a.sc.v : a.sc.k) + block, rows, a.ld, piece, 0, p.page, hv, Over(hv), shift, vecs);
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
  const long long slots = (long long)total / c.page + 2LL * n;
  if (slots * layers * 2 * c.n_kv_heads * ((c.page * c.head_dim + 511) / 512) > 0x3fffffffLL)
    return "total, n or layers is too large";
  a.slots = (int)slots;
  *run = true;
  return nullptr;
}

cudaError_t launch_rows(void (*kern)(RowsArgs), const RowsArgs& a, long long warps, cudaStream_t st) {
  const long long grid = std::min<long long>((warps + CT / 32 - 1) / (CT / 32), 152 * 8);
  const size_t smem = a.n <= kListed ? ((size_t)a.n + 1) * sizeof(int) : 0;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(CT), smem, st, a);
}

template <typename T>
cudaError_t launch_write(const RowsArgs& a, cudaStream_t st) {
  const long long units = (long long)a.slots * a.layers * 2 * a.p.n_kv_heads;
  const int kb = a.p.page * a.p.head_dim * (int)sizeof(T) / 1024;
  if (kb <= 4) return launch_rows(write8_kernel<T, 1>, a, units, st);
  if (kb <= 8) return launch_rows(write8_kernel<T, 2>, a, units * 2, st);
  if (kb <= 16) return launch_rows(write8_kernel<T, 4>, a, units * 4, st);
  return launch_rows(write8_kernel<T, 8>, a, units * 8, st);
}

}  // namespace

cudaError_t launch_prefix_values(const hf_pages& p, PageScales sc, int layer, const int32_t* req, int shared, void* k,
                                 void* v, cudaStream_t st) {
  RowsArgs a{};
  a.p = p;
  a.sc = sc;
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.ld = 2LL * p.n_kv_heads * p.head_dim;
  a.req = req;
  a.total = shared;
  a.layer = layer;
  const long long warps = (long long)shared / p.page * 2 * ((p.n_kv_heads * p.page * p.head_dim / 16 + READ * 32 - 1) / (READ * 32));
  return launch_pdl(prefix8_kernel, dim3((unsigned)std::min<long long>((warps + CT / 32 - 1) / (CT / 32), 152 * 8)), dim3(CT),
                    0, st, a);
}

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
  return done(p->rows == HF_F32 ? launch_write<float>(a, (cudaStream_t)stream)
                               : launch_write<__nv_bfloat16>(a, (cudaStream_t)stream));
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
  const int pieces = (a.p.n_kv_heads * a.p.page * a.p.head_dim / 16 + READ * 32 - 1) / (READ * 32);
  return done(launch_rows(p->rows == HF_F32 ? read8_kernel<float> : read8_kernel<__nv_bfloat16>, a, (long long)a.slots * a.layers * 2 * pieces,
                          (cudaStream_t)stream));
}
