// Rotary positions of the target's queries and keys (hf_rotary).
//
//   (a, b) -> f (a cos - b sin, b cos + a sin),  angle = position * w_i
// w_i / (2 pi) is held in units of 2^-64 turns: the product with the position wraps at whole turns by
// itself and loses nothing but what is below 2^-32 turns, where an angle formed in 32 bits
// would be off by 0.06 at 10^6 and one in 64-bit floating point would wait for that unit. The table's entries are 64-bit
// floating-point results, good to about 2^-55 of a turn, so a position adds that often: 2^-32 turns at 2^23, 2^-24
// at 2^31. The reduced angle is rounded to 24 bits for the functions.
//
// A thread holds the cosines and sines of its pairs and turns them in one head after the other.
// Bound by the reads and writes where the rows are many (5.96 TB/s), by the launch where they are few (one
// token 2.3 us in a graph).
#include <cmath>
#include <cstring>

#include "common.cuh"

namespace hf {
namespace {

constexpr int RT = 256;

struct RotaryArgs {
  const uint8_t* q;
  const uint8_t* k;
  uint8_t* qo;
  uint8_t* ko;
  long long q_ld, k_ld, qo_ld, ko_ld;  // elements
  const unsigned long long* turns;
  const int32_t* pos;
  float f;
  int rows, hq, hkv, dh, dim;
  int per, step;  // chunks of a head; every step-th head is the same thread's
};

// VE values of 2 to 16 bytes in all, at once.
template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <typename T, int VE>
__device__ __forceinline__ void load(const T* p, float* x) {
  using W = typename Word<VE * sizeof(T)>::type;
  const W w = *reinterpret_cast<const W*>(p);
  const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < VE; ++i) x[i] = to_f(v[i]);
}
template <typename T, int VE>
__device__ __forceinline__ void store(T* p, const float* x) {
  using W = typename Word<VE * sizeof(T)>::type;
  W w;
  T* v = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = from_f<T>(x[i]);
  *reinterpret_cast<W*>(p) = w;
}

// VE: values of a load. A thread's chunk is two loads, halves: VE values of the first half
// and their partners; interleaved: 2 VE neighbours. Chunks behind dim are copied.
template <typename T, int VE, bool INTER>
__global__ void __launch_bounds__(RT) rotary_kernel(RotaryArgs a) {
  pdl_trigger();
  pdl_wait();
  const long long all = (long long)a.rows * a.per * a.step;
  const int half = a.dim / 2, turned = half / VE, H = a.hq + a.hkv;
  for (long long u = (long long)blockIdx.x * RT + threadIdx.x; u < all; u += (long long)gridDim.x * RT) {
    const int c = (int)(u % a.per), h0 = (int)(u / a.per % a.step);
    const long long row = u / a.per / a.step;
    // columns of the two loads (x1 < 0: one only)
    int x0, x1;
    if (c < turned) {
      x0 = INTER ? 2 * c * VE : c * VE;
      x1 = INTER ? x0 + VE : x0 + half;
    } else {
      x0 = a.dim + 2 * (c - turned) * VE;
      x1 = x0 + VE < a.dh ? x0 + VE : -1;
    }
    float cs[VE], sn[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (c < turned) {
      const long long pos = a.pos[row];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const int angle = (int)(((unsigned long long)pos * a.turns[c * VE + i]) >> 32);  // 2^-32 turns, signed
        sincospif((float)angle * 4.656612873077393e-10f, &sn[i], &cs[i]);                // 2^-31
        cs[i] *= a.f;
        sn[i] *= a.f;
      }
    }
    for (int h = h0; h < H; h += a.step) {
      const bool isq = h < a.hq;
      const int g = isq ? h : h - a.hq;
      const T* src = reinterpret_cast<const T*>(isq ? a.q : a.k) + row * (isq ? a.q_ld : a.k_ld) + (long long)g * a.dh;
      T* dst = reinterpret_cast<T*>(isq ? a.qo : a.ko) + row * (isq ? a.qo_ld : a.ko_ld) + (long long)g * a.dh;
      if (c >= turned && src == dst) continue;  // in place
      float x[2 * VE];
      load<T, VE>(src + x0, x);
      if (x1 >= 0) load<T, VE>(src + x1, x + VE);
      if (c < turned) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          float& p = INTER ? x[2 * i] : x[i];
          float& r = INTER ? x[2 * i + 1] : x[VE + i];
          const float y = p * cs[i] - r * sn[i];
          r = r * cs[i] + p * sn[i];
          p = y;
        }
      }
      store<T, VE>(dst + x0, x);
      if (x1 >= 0) store<T, VE>(dst + x1, x + VE);
    }
  }
}

hf_status refuse(const char* m) {
  set_thread_error(m);
  return HF_EINVAL;
}

template <typename T, int VE>
cudaError_t launch_wide(RotaryArgs a, bool inter, cudaStream_t st) {
  const int H = a.hq + a.hkv;
  a.per = a.dim / 2 / VE + ((a.dh - a.dim) / VE + 1) / 2;
  // threads enough to fill the GPU four times, then heads one after the other (26005 tokens of 40 heads of 128 89.4
  // us, 5.96 TB/s; threads for once 93.8; four heads at a time 127: more registers, fewer threads)
  const long long cells = (long long)a.rows * a.per;
  a.step = (int)std::max<long long>(1, std::min<long long>(H, (152LL * 8192 + cells - 1) / cells));
  const long long grid = std::min<long long>((cells * a.step + RT - 1) / RT, 1 << 20);
  return launch_pdl(inter ? rotary_kernel<T, VE, true> : rotary_kernel<T, VE, false>, dim3((unsigned)grid), dim3(RT), 0, st, a);
}

// As many values a load as the pairs' halves, the heads and their places allow (`align` bytes of them).
template <typename T>
cudaError_t launch(const RotaryArgs& a, bool inter, int align, cudaStream_t st) {
  auto fits = [&](int ve) { return align % (ve * (int)sizeof(T)) == 0 && a.dim / 2 % ve == 0 && a.dh % ve == 0; };
  if constexpr (sizeof(T) == 2)
    if (fits(8)) return launch_wide<T, 8>(a, inter, st);
  if (fits(4)) return launch_wide<T, 4>(a, inter, st);
  if (fits(2)) return launch_wide<T, 2>(a, inter, st);
  return launch_wide<T, 1>(a, inter, st);
}

}  // namespace
}  // namespace hf

extern "C" hf_status hf_rotary_table(int32_t dim, double base, const hf_rotary_scaling* scaling, uint64_t* turns,
                                     float* attention) {
  using namespace hf;
  if (dim < 2 || dim % 2 || dim > 256) return refuse("dim must be even, 2..256");
  if (!(base > 1.0) || !std::isfinite(base)) return refuse("base must be above 1 and finite");
  if (!turns || !attention) return refuse("NULL buffer");
  hf_rotary_scaling s{};
  if (scaling) s = *scaling;
  if (s.kind < HF_ROTARY_NONE || s.kind > HF_ROTARY_BANDS) return refuse("scaling: unknown kind");
  if (s.kind == HF_ROTARY_NONE) s.factor = 1.0;
  if (!(s.factor >= 1.0) || !std::isfinite(s.factor)) return refuse("scaling: factor must be >= 1 and finite");
  if (!(s.attention >= 0.0) || !(s.attention <= 1e30)) return refuse("scaling: attention must be 0..1e30");
  const bool ramps = s.kind == HF_ROTARY_YARN || s.kind == HF_ROTARY_BANDS;
  if (ramps) {
    if (s.original < 1) return refuse("scaling: original must be >= 1");
    if (s.fast == 0.0) s.fast = s.kind == HF_ROTARY_YARN ? 32.0 : 4.0;
    if (s.slow == 0.0) s.slow = 1.0;
    if (!(s.slow > 0.0) || !(s.fast > s.slow) || !std::isfinite(s.fast))
      return refuse("scaling: fast > slow > 0 is needed");
  }
  const double two_pi = 6.283185307179586476925;
  if (s.kind == HF_ROTARY_NTK) {
    if (dim == 2) return refuse("scaling: NTK needs dim > 2");
    base *= std::pow(s.factor, (double)dim / (dim - 2));
    if (!std::isfinite(base)) return refuse("scaling: factor is too large");
  }
  double lo = 0, hi = 0;
  if (s.kind == HF_ROTARY_YARN) {
    auto pair_of = [&](double t) { return dim * std::log(s.original / (two_pi * t)) / (2 * std::log(base)); };
    lo = std::max(std::floor(pair_of(s.fast)), 0.0);
    hi = std::min(std::ceil(pair_of(s.slow)), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / dim);
    if (s.kind == HF_ROTARY_LINEAR) w /= s.factor;
    if (s.kind == HF_ROTARY_YARN) {
      const double r = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      w = w * (1 - r) + w / s.factor * r;
    }
    if (s.kind == HF_ROTARY_BANDS) {
      const double t = std::min(std::max((s.original * w / two_pi - s.slow) / (s.fast - s.slow), 0.0), 1.0);
      w = w * t + w / s.factor * (1 - t);
    }
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(w / two_pi, 64));  // (below 2^62: w <= 1)
  }
  *attention = (float)(s.attention > 0.0 ? s.attention : s.kind == HF_ROTARY_YARN ? 0.1 * std::log(s.factor) + 1.0 : 1.0);
  return HF_OK;
}

extern "C" hf_status hf_rotary(int32_t dtype, int32_t interleaved, int32_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                               int32_t head_dim, int32_t dim, const uint64_t* turns, float attention,
                               const int32_t* positions, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                               void* q_out, int64_t q_out_ld, void* k_out, int64_t k_out_ld, void* stream) {
  using namespace hf;
  if (dtype != HF_F32 && dtype != HF_BF16) return refuse("dtype must be HF_F32 or HF_BF16");
  if (interleaved != 0 && interleaved != 1) return refuse("interleaved must be 0 or 1");
  if (rows < 0) return refuse("rows must be >= 0");
  if (n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > (1 << 16) || n_kv_heads > (1 << 16))
    return refuse("n_q_heads and n_kv_heads must be 0..65536");
  if (head_dim < 2 || head_dim > 256) return refuse("head_dim must be 2..256");
  if (dim < 2 || dim % 2 || dim > head_dim) return refuse("dim must be even, 2..head_dim");
  if (!(std::fabs(attention) <= 1e30f)) return refuse("attention must be finite");
  if (rows == 0 || n_q_heads + n_kv_heads == 0) return HF_OK;
  if (!turns || !positions || (n_q_heads && (!q || !q_out)) || (n_kv_heads && (!k || !k_out))) return refuse("NULL buffer");
  const int esize = dtype == HF_F32 ? 4 : 2;
  auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(turns, 8) || off(positions, 4)) return refuse("turns must be 8-byte, positions 4-byte aligned");
  uintptr_t places = 16;  // bits of all that has to be divisible
  for (int i = 0; i < 4; ++i) {
    const void* p = i == 0 ? q : i == 1 ? q_out : i == 2 ? k : k_out;
    const int64_t ld = i == 0 ? q_ld : i == 1 ? q_out_ld : i == 2 ? k_ld : k_out_ld;
    const int64_t least = (int64_t)(i < 2 ? n_q_heads : n_kv_heads) * head_dim;
    if (least == 0) continue;
    if (ld < least || ld > (1LL << 36)) return refuse("a row stride is smaller than heads * head_dim, or above 2^36");
    if (off(p, esize)) return refuse("q, k and their outputs must be aligned to their type");
    places |= reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * esize);
  }
  RotaryArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.qo = static_cast<uint8_t*>(q_out);
  a.ko = static_cast<uint8_t*>(k_out);
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.qo_ld = q_out_ld;
  a.ko_ld = k_out_ld;
  a.turns = reinterpret_cast<const unsigned long long*>(turns);
  a.pos = positions;
  a.f = attention;
  a.rows = rows;
  a.hq = n_q_heads;
  a.hkv = n_kv_heads;
  a.dh = head_dim;
  a.dim = dim;
  cudaStream_t st = (cudaStream_t)stream;
  const int align = (int)(places & (~places + 1));  // the largest power of two that divides them, 16 at most
  const cudaError_t e = dtype == HF_F32 ? launch<float>(a, interleaved, align, st)
                                        : launch<__nv_bfloat16>(a, interleaved, align, st);
  if (e == cudaSuccess) return HF_OK;
  set_thread_error(cudaGetErrorString(e));
  return HF_ECUDA;
}
