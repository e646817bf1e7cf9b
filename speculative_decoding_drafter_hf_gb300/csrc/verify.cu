// Verification of drafted tokens by speculative sampling (hf_verify_tokens).
//
// Per request: p_s = softmax(x_s / T), q_s = softmax(y_s / T); draft s passes
// iff u_s q_s(d_s) < p_s(d_s); the next token is argmax_i w_i / e_i with
// w = max(p_a - q_a, 0) at the first slot a that did not pass (w = p_a when all
// did). The race w_i / e_i draws i with probability w_i / sum(w) and needs no
// prefix sum over the vocabulary: its result depends on two neighbouring
// scores only, not on the order in which a sum was formed.
//
// Two launches. verify_stats reads every logit once: (row, chunk) CTAs form
// the chunk's maximum and sum of exponentials (T = 0: maximum and its lowest
// index, or that the chunk holds a NaN or +infinity; target rows only). verify_race: each (request, chunk) CTA joins its
// request's chunks, finds the stop slot, and runs the race over its chunk of
// that slot's rows; the request's last CTA (ticket) joins the chunks. Bound by the
// reads of the logits: 64 requests x 7 drafts, 100352 tokens, bf16 and fp32 logits, 282 MB
// in 48.7 us (5.8 TB/s) for the statistics; one request by latency, 15 us in all. Drafts
// chosen greedily have no logits to read: 64 x 7 41 us, at T = 0 30 us.
#include <cstdio>

#include "common.cuh"

namespace hf {
namespace {

constexpr int VT = 256;         // threads per CTA
constexpr int VMAXS = 16;       // drafted tokens per request
constexpr float kNegInf = -INFINITY;

struct VArgs {
  const void* x;  // target logits
  const void* y;  // draft logits (or NULL)
  long long x_ld, y_ld, e_ld;
  const int32_t* tok;
  const int32_t* n_draft;
  const float* u;
  const float* e;  // noise
  const float* temp;
  int B, S, V;
  int chunk, nchunk;    // stats: vocabulary entries per CTA
  int rchunk, nrchunk;  // race
  float2* stats;        // [B * (2S + 1)][nchunk]: target rows, then draft rows, per request
  float2* race;         // [B][nrchunk]: best score, its index
  int* tickets;         // [B]
  int32_t* n_acc;
  int32_t* out;
  int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Inputs may be outputs of the launch before (drafts and logits of hf_draft_tokens among
// them): they are read after pdl_wait and never through the non-coherent path. A request's few
// numbers, which many CTAs read, go through the L1, logits and noise past it.

// (a T below the normal numbers would make 1 / T infinite)
__device__ __forceinline__ bool temp_ok(float t) { return t == 0.f || (t >= 1.17549435e-38f && t < INFINITY); }

// The entries [i0, i1) of a row: single ones up to a 16-byte boundary and behind the
// last whole 16 bytes go to one(index, value); of the rest, each thread gets UN 16-byte
// loads at a time, as some(index, values, how many): load k's values are at index +
// k * VT * VE.
template <typename T, int UN, typename F, typename G>
__device__ __forceinline__ void for_row(const T* row, int i0, int i1, F&& one, G&& some) {
  constexpr int VE = 16 / (int)sizeof(T);
  const int tid = threadIdx.x;
  const int off = (int)((reinterpret_cast<uintptr_t>(row + i0) & 15) / sizeof(T));
  const int head = min(i1 - i0, off ? VE - off : 0);
  if (tid < head) one(i0 + tid, to_f(row[i0 + tid]));
  const int b0 = i0 + head, nv = (i1 - b0) / VE;
  const uint4* p = reinterpret_cast<const uint4*>(row + b0);
  uint4 r[UN];
#pragma unroll
  for (int k = 0; k < UN; ++k)
    if (tid + k * VT < nv) r[k] = __ldcg(p + tid + k * VT);
  for (int v0 = tid; v0 < nv; v0 += VT * UN) {
    const int v1 = v0 + VT * UN;  // the next loads are on their way meanwhile
    uint4 next[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (v1 + k * VT < nv) next[k] = __ldcg(p + v1 + k * VT);
    float x[UN * VE];
    const int n = min(UN, (nv - v0 + VT - 1) / VT);
#pragma unroll
    for (int k = 0; k < UN; ++k)
#pragma unroll
      for (int j = 0; j < VE; ++j)
        x[k * VE + j] = k < n ? to_f(reinterpret_cast<const T*>(&r[k])[j]) : kNegInf;
    some(b0 + v0 * VE, x, n);
#pragma unroll
    for (int k = 0; k < UN; ++k) r[k] = next[k];
  }
  const int t0 = b0 + nv * VE;
  if (t0 + tid < i1) one(t0 + tid, to_f(row[t0 + tid]));
}

// (m, l) of two parts: maximum and sum of 2^((x - m) c). A part without
// anything above -infinity has m = -infinity, l = 0.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2, float c) {
  const float mm = fmaxf(m, m2);
  if (mm > kNegInf) {
    l = (m > kNegInf ? l * ex2((m - mm) * c) : l) + (m2 > kNegInf ? l2 * ex2((m2 - mm) * c) : l2);
  } else {
    l += l2;
  }
  m = mm;
}

// (value, lowest index) of the larger of two.
__device__ __forceinline__ void best(float& v, int& i, float v2, int i2) {
  if (i2 >= 0 && (i < 0 || v2 > v || (v2 == v && i2 < i))) {
    v = v2;
    i = i2;
  }
}
// The same for parts of a row (T = 0): kOdd, a NaN or +infinity in it, stays.
constexpr int kOdd = -2;
__device__ __forceinline__ void best_logit(float& v, int& i, float v2, int i2) {
  if (i2 == kOdd)
    i = kOdd;
  else if (i != kOdd)
    best(v, i, v2, i2);
}

template <typename T>
__device__ __forceinline__ void stats_cta(const VArgs& a, const T* row, float t, int chunk, float2* out) {
  __shared__ float sm[VT / 32], sl[VT / 32];
  __shared__ int si[VT / 32];
  const int i0 = chunk * a.chunk, i1 = min(a.V, i0 + a.chunk);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int VE = 16 / (int)sizeof(T), UN = 16 / VE;
  if (t == 0.f) {
    float v = kNegInf;
    int idx = -1;
    bool odd = false;  // (a comparison with NaN is false)
    auto one = [&](int i, float x) {
      odd |= !(x < INFINITY);
      if (x > v || (x == v && i < idx)) {
        v = x;
        idx = i;
      }
    };
    for_row<T, UN>(row, i0, i1, one, [&](int i, const float* x, int n) {
      float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int k = 0; k < UN * VE; ++k) {
        odd |= !(x[k] < INFINITY);
        if (k >= 4) t4[k & 3] = fmaxf(t4[k & 3], x[k]);
      }
      const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      if (top > v) {  // (seldom, after the first steps) rising indices: the first of equals
        v = top;
#pragma unroll
        for (int k = UN * VE - 1; k >= 0; --k)
          if (x[k] == top) idx = i + k / VE * (VT * VE) + k % VE;
      }
    });
    if (odd) idx = kOdd;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      best_logit(v, idx, __shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, idx, o));
    if (lane == 0) {
      sm[warp] = v;
      si[warp] = idx;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < VT / 32; ++w) best_logit(v, idx, sm[w], si[w]);
      *out = make_float2(v, __int_as_float(idx));
    }
    return;
  }
  const float c = 1.4426950408889634f / t;
  // one maximum and one rescaling for all values of a step; a NaN stays in l, and so does
  // +infinity (as infinity - infinity); without anything above -infinity nothing is added
  float m = kNegInf, l = 0.f;
  auto one = [&](int, float x) {
    const float nm = fmaxf(m, x), base = nm > kNegInf ? nm : 0.f;
    l = l * ex2((m - base) * c) + ex2((x - base) * c);
    m = nm;
  };
  for_row<T, UN>(row, i0, i1, one, [&](int, const float* x, int) {
    float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int k = 4; k < UN * VE; ++k) t4[k & 3] = fmaxf(t4[k & 3], x[k]);
    const float nm = fmaxf(m, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
    const float base = nm > kNegInf ? nm : 0.f;
    if (nm > m) l *= ex2((m - base) * c);
    m = nm;
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < UN * VE; ++k) s4[k & 3] += ex2((x[k] - base) * c);
    l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    join(m, l, m2, l2, c);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < VT / 32; ++w) join(m, l, sm[w], sl[w], c);
    *out = make_float2(m, l);
  }
}

// One CTA per (row, chunk): rows b * (2S + 1) + s, s <= S the target's, then the
// draft's.
template <typename TX, typename TY>
__global__ void __launch_bounds__(VT) verify_stats(VArgs a) {
  pdl_trigger();
  pdl_wait();
  const int chunk = blockIdx.x % a.nchunk, r = blockIdx.x / a.nchunk;
  const int per = a.y ? 2 * a.S + 1 : a.S + 1;
  const int b = r / per, s = r % per;
  if (s == 0 && chunk == 0 && threadIdx.x == 0) a.tickets[b] = 0;
  const float t = a.temp ? a.temp[b] : 1.f;
  const int nd = a.n_draft ? a.n_draft[b] : a.S;
  if (!temp_ok(t)) return;
  float2* out = a.stats + ((size_t)b * (2 * a.S + 1) + s) * a.nchunk + chunk;
  if (s <= a.S) {
    if (s > nd) return;
    stats_cta<TX>(a, static_cast<const TX*>(a.x) + ((size_t)b * (a.S + 1) + s) * a.x_ld, t, chunk, out);
  } else {
    if (t == 0.f || s - a.S - 1 >= nd) return;
    stats_cta<TY>(a, static_cast<const TY*>(a.y) + ((size_t)b * a.S + s - a.S - 1) * a.y_ld, t, chunk, out);
  }
}

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
  const __nv_bfloat16* t = reinterpret_cast<const __nv_bfloat16*>(&x);
  v[0] = to_f(t[0]), v[1] = to_f(t[1]), v[2] = to_f(t[2]), v[3] = to_f(t[3]);
}

// u q < p by logarithms, for a p that 32 bits hold badly or not at all (a draft far below the
// largest logit, a small T): x, y the draft's logits, mp, lp and mq, lq the rows' statistics. A
// logit of -infinity has the probability 0, every other one more.
__device__ __noinline__ bool accepts_small(float u, float x, float mp, float lp, bool sampled, float y, float mq, float lq,
                                           float t) {
  if (!(x > kNegInf)) return false;
  if (u == 0.f || (sampled && y == kNegInf)) return true;
  const double c = 1.4426950408889634 / t;
  const double q = sampled ? ((double)y - mq) * c - log2((double)lq) : 0.0;
  return log2((double)u) + q < ((double)x - mp) * c - log2((double)lp);
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(VT) verify_race(VArgs a) {
  __shared__ float sm[2 * VMAXS + 1], sl[2 * VMAXS + 1];
  __shared__ int s_stop, s_bad, s_last;
  __shared__ float2 red[VT / 32];
  pdl_trigger();
  pdl_wait();
  // the last requests first: their logits may still be in the L2
  const int chunk = blockIdx.x % a.nrchunk, b = a.B - 1 - blockIdx.x / a.nrchunk;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, S = a.S;
  const float t = a.temp ? a.temp[b] : 1.f;
  const int nd = a.n_draft ? a.n_draft[b] : S;
  const bool range_ok = temp_ok(t) && nd >= 0 && nd <= S;
  const bool cold = t == 0.f;
  const float c = cold ? 0.f : 1.4426950408889634f / t;
  // the drafts, their logits and the slots' random numbers: on their way while the
  // statistics are joined (warp 0, lane = slot)
  const bool has = warp == 0 && range_ok && lane < nd;
  int d = 0;
  float xv = 0.f, yv = 0.f, uv = 0.f;
  if (has) d = a.tok[(size_t)b * S + lane];
  const bool names = d >= 0 && d < a.V;
  if (has && names && !cold) {
    uv = a.u[(size_t)b * S + lane];
    xv = to_f(static_cast<const TX*>(a.x)[((size_t)b * (S + 1) + lane) * a.x_ld + d]);
    if (a.y) yv = to_f(static_cast<const TY*>(a.y)[((size_t)b * S + lane) * a.y_ld + d]);
  }
  if (range_ok) {
    for (int r = warp; r < 2 * S + 1; r += VT / 32) {
      if (r <= S ? r > nd : (cold || !a.y || r - S - 1 >= nd)) continue;
      const float2* st = a.stats + ((size_t)b * (2 * S + 1) + r) * a.nchunk;
      float m = kNegInf, l = 0.f;
      int idx = -1;
      for (int k = lane; k < a.nchunk; k += 32) {
        const float2 v = __ldcg(&st[k]);
        if (cold)
          best_logit(m, idx, v.x, __float_as_int(v.y));
        else
          join(m, l, v.x, v.y, c);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        if (cold)
          best_logit(m, idx, m2, __shfl_xor_sync(0xffffffffu, idx, o));
        else
          join(m, l, m2, __shfl_xor_sync(0xffffffffu, l, o), c);
      }
      if (lane == 0) {
        sm[r] = m;
        sl[r] = cold ? __int_as_float(idx) : l;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    // lane s tests slot s; the first that fails is the stop slot
    bool bad = !range_ok, pass = false, row_bad = false;
    if (!bad && lane <= nd) {
      if (!names) {
        row_bad = true;
      } else if (cold) {
        const int idx = __float_as_int(sl[lane]);
        row_bad = idx < 0;
        pass = has && idx == d;
      } else {
        row_bad = !(sl[lane] > 0.f && sl[lane] < INFINITY);
        float q = 1.f, mq = 0.f, lq = 1.f;
        if (has && a.y) {
          mq = sm[S + 1 + lane];
          lq = sl[S + 1 + lane];
          row_bad = row_bad || !(lq > 0.f && lq < INFINITY);
          q = ex2((yv - mq) * c) / lq;
        }
        if (has && !row_bad) {
          const float p = ex2((xv - sm[lane]) * c) / sl[lane];
          pass = p > 1e-30f ? uv * q < p : accepts_small(uv, xv, sm[lane], sl[lane], a.y != nullptr, yv, mq, lq, t);
        }
      }
    }
    const unsigned fails = ~__ballot_sync(0xffffffffu, pass);
    const unsigned bads = __ballot_sync(0xffffffffu, row_bad);
    // a draft that names no token is refused wherever it stands
    const int stop = __ffs(fails) - 1;
    bool tok_bad = has && !names;
    tok_bad = __any_sync(0xffffffffu, tok_bad);
    if (lane == 0) {
      s_stop = stop;
      s_bad = bad || tok_bad || (stop < 32 && ((bads >> stop) & 1));
    }
  }
  __syncthreads();
  const int stop = s_stop;
  int32_t* out = a.out + (size_t)b * (S + 1);
  if (s_bad || cold) {  // uniform in the request: no race
    if (chunk == 0 && tid <= S) {
      int v = -1;
      if (!s_bad) v = tid < stop ? a.tok[(size_t)b * S + tid] : tid == stop ? __float_as_int(sl[stop]) : -1;
      out[tid] = v;
      if (tid == 0) {
        a.n_acc[b] = s_bad ? 0 : stop + 1;
        if (s_bad && a.status) atomicOr(a.status, HF_S_BAD);
      }
    }
    return;
  }

  // the race over this chunk of the stop slot's rows
  const TX* x = static_cast<const TX*>(a.x) + ((size_t)b * (S + 1) + stop) * a.x_ld;
  const bool residual = stop < nd;
  const TY* y = residual && a.y ? static_cast<const TY*>(a.y) + ((size_t)b * S + stop) * a.y_ld : nullptr;
  const int dtok = residual && !a.y ? a.tok[(size_t)b * S + stop] : -1;
  const float* e = a.e + (size_t)b * a.e_ld;
  const float mp = sm[stop], ip = 1.f / sl[stop];
  const float mq = y ? sm[S + 1 + stop] : 0.f, iq = y ? 1.f / sl[S + 1 + stop] : 0.f;
  const int i0 = chunk * a.rchunk, i1 = min(a.V, i0 + a.rchunk);
  float vw = 0.f;
  int iw = -1;
  // an entry's score (indices rise: the first of equals stays). The quotient is the fast one,
  // within 2 ulp: two scores that near change places with a probability of about 2^-21.
  auto run = [&](int i, float xv, float yv, float n) {
    float w = ex2((xv - mp) * c) * ip;
    if (y) w -= ex2((yv - mq) * c) * iq;
    if (i == dtok) w = 0.f;
    const float s = __fdividef(w, n);
    if (w > 0.f && (iw < 0 ? s == s : s > vw)) {
      vw = s;
      iw = i;
    }
  };
  // four neighbouring entries at a time where the three rows allow it
  auto off = [](const void* q, int n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
  const bool fours = !off(x + i0, 4 * sizeof(TX)) && !(y && off(y + i0, 4 * sizeof(TY))) && !off(e + i0, 16);
  const int i4 = fours ? i0 + (i1 - i0) / 4 * 4 : i0;
#pragma unroll 2
  for (int i = i0 + 4 * tid; i < i4; i += 4 * VT) {
    float xv[4], yv[4] = {};
    load4(x + i, xv);
    if (y) load4(y + i, yv);
    const float4 n = __ldcs(reinterpret_cast<const float4*>(e + i));
    run(i, xv[0], yv[0], n.x);
    run(i + 1, xv[1], yv[1], n.y);
    run(i + 2, xv[2], yv[2], n.z);
    run(i + 3, xv[3], yv[3], n.w);
  }
  for (int i = i4 + tid; i < i1; i += VT) run(i, to_f(x[i]), y ? to_f(y[i]) : 0.f, __ldcg(&e[i]));
  auto cta_best = [&]() {  // of the CTA's threads, in warp 0
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      best(vw, iw, __shfl_xor_sync(0xffffffffu, vw, o), __shfl_xor_sync(0xffffffffu, iw, o));
    __syncthreads();  // red has been read
    if (lane == 0) red[warp] = make_float2(vw, __int_as_float(iw));
    __syncthreads();
    for (int w = 0; w < VT / 32; ++w) best(vw, iw, red[w].x, __float_as_int(red[w].y));
  };
  cta_best();
  if (tid == 0) {
    a.race[(size_t)b * a.nrchunk + chunk] = make_float2(vw, __int_as_float(iw));
    __threadfence();
    s_last = atomicAdd(&a.tickets[b], 1) == a.nrchunk - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  vw = 0.f;
  iw = -1;
  for (int k = tid; k < a.nrchunk; k += VT) {
    const float2 v = __ldcg(&a.race[(size_t)b * a.nrchunk + k]);
    best(vw, iw, v.x, __float_as_int(v.y));
  }
  cta_best();
  if (iw < 0 && residual) {  // p - q nowhere positive (rare): p itself, by this CTA alone
    for (int i = tid; i < a.V; i += VT) {
      const float p = ex2((to_f(x[i]) - mp) * c) * ip, s = __fdividef(p, __ldcg(&e[i]));
      if (p > 0.f && (iw < 0 ? s == s : s > vw)) {
        vw = s;
        iw = i;
      }
    }
    cta_best();
  }
  if (warp != 0) return;
  const int next = iw;
  if (lane <= S) out[lane] = next < 0 ? -1 : lane < stop ? a.tok[(size_t)b * S + lane] : lane == stop ? next : -1;
  if (lane == 0) {
    a.n_acc[b] = next < 0 ? 0 : stop + 1;
    if (next < 0 && a.status) atomicOr(a.status, HF_S_BAD);
  }
}

// Chunk of the vocabulary per CTA: about `per_sm` CTAs per SM in all, at least `least`
// entries each. Both kernels' CTAs begin with a chain of dependent loads (in the race 4 us:
// the request's statistics are joined), so few long ones are faster: 64 x 7 drafts of 100352
// tokens took 82, 69 and 65 us with 32, 16 and 6 for the statistics, 73, 69 and 72 us with 12,
// 4 and 3 for the race.
int chunk_for(long long rows, int V, int least, int per_sm) {
  const long long want = (152 * per_sm + rows - 1) / rows;  // CTAs per row
  const long long c = (V + want - 1) / want;
  return (int)std::max<long long>(least, std::min<long long>((c + 1023) / 1024 * 1024, 65536));
}

struct VPlan {
  int chunk, nchunk, rchunk, nrchunk;
  size_t stats, race, tickets, total;
};

VPlan plan_for(int B, int S, int V) {
  VPlan p{};
  p.chunk = chunk_for((long long)B * (S + 1), V, 2048, 6);
  p.nchunk = (V + p.chunk - 1) / p.chunk;
  p.rchunk = chunk_for(B, V, 1024, 4);
  p.nrchunk = (V + p.rchunk - 1) / p.rchunk;
  p.stats = 0;
  p.race = (p.stats + (size_t)B * (2 * S + 1) * p.nchunk * sizeof(float2) + 15) / 16 * 16;
  p.tickets = p.race + (size_t)B * p.nrchunk * sizeof(float2);
  p.total = (p.tickets + (size_t)B * sizeof(int) + 15) / 16 * 16;
  return p;
}

const char* sizes_bad(int batch, int block, int vocab) {
  if (batch < 0 || batch > (1 << 20)) return "batch must be 0..1048576";
  if (block < 1 || block > VMAXS) return "block must be 1..16";
  if (vocab < 1 || vocab > (1 << 28)) return "vocab must be 1..268435456";
  const VPlan p = plan_for(std::max(batch, 1), block, vocab);
  if ((long long)batch * (2 * block + 1) * p.nchunk > 0x7fffffffLL || (long long)batch * p.nrchunk > 0x7fffffffLL)
    return "batch * block * vocab is too large for one launch";
  return nullptr;
}

template <typename TX, typename TY>
cudaError_t launch(const VArgs& a, cudaStream_t st) {
  const int per = a.y ? 2 * a.S + 1 : a.S + 1;
  cudaError_t e = launch_pdl(verify_stats<TX, TY>, dim3((unsigned)(a.B * per * a.nchunk)), dim3(VT), 0, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(verify_race<TX, TY>, dim3((unsigned)(a.B * a.nrchunk)), dim3(VT), 0, st, a);
  return e;
}

}  // namespace
}  // namespace hf

extern "C" size_t hf_verify_workspace(int32_t batch, int32_t block, int32_t vocab) {
  if (hf::sizes_bad(batch, block, vocab)) return 0;
  return hf::plan_for(std::max(batch, 1), block, vocab).total;
}

extern "C" hf_status hf_verify_tokens(int32_t target_dtype, const void* target_logits, int64_t target_ld,
                                      int32_t draft_dtype, const void* draft_logits, int64_t draft_ld,
                                      const int32_t* draft_tokens, const int32_t* n_draft, const float* u,
                                      const float* noise, int64_t noise_ld, const float* temperature,
                                      int32_t batch, int32_t block, int32_t vocab, int32_t* n_accepted,
                                      int32_t* tokens, void* workspace, size_t workspace_bytes,
                                      int32_t* status, void* stream) {
  using namespace hf;
  auto bad = [](const char* m) {
    set_thread_error(m);
    return HF_EINVAL;
  };
  if (target_dtype != HF_F32 && target_dtype != HF_BF16) return bad("target_dtype must be HF_F32 or HF_BF16");
  if (draft_logits && draft_dtype != HF_F32 && draft_dtype != HF_BF16)
    return bad("draft_dtype must be HF_F32 or HF_BF16");
  if (const char* m = sizes_bad(batch, block, vocab)) return bad(m);
  if (target_ld < vocab || noise_ld < vocab || (draft_logits && draft_ld < vocab))
    return bad("target_ld, draft_ld and noise_ld must be >= vocab");
  if (batch == 0) return HF_OK;
  if (!target_logits || !draft_tokens || !u || !noise || !n_accepted || !tokens || !workspace)
    return bad("NULL buffer");
  auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(target_logits, target_dtype == HF_F32 ? 4 : 2) ||
      (draft_logits && off(draft_logits, draft_dtype == HF_F32 ? 4 : 2)) || off(draft_tokens, 4) ||
      off(n_draft, 4) || off(u, 4) || off(noise, 4) || off(temperature, 4) || off(n_accepted, 4) ||
      off(tokens, 4) || off(status, 4))
    return bad("a buffer is not aligned to its element type");
  if (off(workspace, 16)) return bad("workspace must be 16-byte aligned");
  const VPlan p = plan_for(batch, block, vocab);
  if (workspace_bytes < p.total) {
    char m[120];
    snprintf(m, sizeof m, "workspace has %zu bytes, hf_verify_workspace asks for %zu", workspace_bytes, p.total);
    return bad(m);
  }
  VArgs a{};
  a.x = target_logits;
  a.y = draft_logits;
  a.x_ld = target_ld;
  a.y_ld = draft_ld;
  a.e_ld = noise_ld;
  a.tok = draft_tokens;
  a.n_draft = n_draft;
  a.u = u;
  a.e = noise;
  a.temp = temperature;
  a.B = batch;
  a.S = block;
  a.V = vocab;
  a.chunk = p.chunk;
  a.nchunk = p.nchunk;
  a.rchunk = p.rchunk;
  a.nrchunk = p.nrchunk;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.stats = reinterpret_cast<float2*>(w + p.stats);
  a.race = reinterpret_cast<float2*>(w + p.race);
  a.tickets = reinterpret_cast<int*>(w + p.tickets);
  a.n_acc = n_accepted;
  a.out = tokens;
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
  const bool xf = target_dtype == HF_F32, yf = !draft_logits || draft_dtype == HF_F32;
  const cudaError_t e = xf ? (yf ? launch<float, float>(a, st) : launch<float, bf>(a, st))
                           : (yf ? launch<bf, float>(a, st) : launch<bf, bf>(a, st));
  if (e != cudaSuccess) {
    set_thread_error(cudaGetErrorString(e));
    return HF_ECUDA;
  }
  return HF_OK;
}
