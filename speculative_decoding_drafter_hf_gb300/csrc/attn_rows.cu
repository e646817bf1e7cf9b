// Attention of query rows on CUDA cores, and the entry points hf_attention_prompt
// and hf_attention_pages.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(s_ij - m_i),  s_ij = qscale q_i.k_j
// over the keys j < limit_i, in one pass over the keys: a tile's scores raise the
// running maximum m_i, and what was summed so far is scaled by 2^(old m - new m).
//
// A CTA takes 8 RPT rows of one KV head and walks its keys in tiles of 64: 8 x 16
// threads, RPT x 4 scores each, then the same rows times the value columns 4 tx + 64 c.
// Everything is fp32 in shared memory and registers: this is the variant for fp32 inputs
// and for head dims that the tensor-core kernels do not take; bound by the fp32
// multiply-adds and the shared-memory reads that feed them (RPT = 4: 64 multiply-adds
// for 8 reads), which go in pairs, two to an instruction. K and V have one place each,
// refilled in turn while the other is used: that leaves room for three or four CTAs per SM
// (8 prompts of 100 to 1201 tokens, heads of 64: 65 us with RPT = 4, 73 us with 8; before
// the pairs two places each and two CTAs per SM took 103 us, one place each 75). A prompt's
// rows are few for the GPU and their keys many: a cluster of four CTAs shares a tile of rows,
// each walking every fourth tile of keys, and joins the parts through distributed shared
// memory (clusters of two: 71 us). What bounds that call is latency: a scheduler has four
// warps and issues in 42% of the cycles. Over a paged cache, RPT goes by the rows of a
// request (8 requests of 8 rows x 2 heads: 17.9 us with 2, 20.8 us with 4; of 8 rows x 8
// heads over 1424 tokens each, the first 1024 in common: 28.9 us with 4, 26.8 us with 8, but 64
// such requests 121 and 133 us, and 8 of one KV head of 32 17.5 and 23.4 us: no 8).
//
// Masked keys: scores are selected, never added to a mask value, so whatever K
// holds there cannot matter; V's non-finite values in a tile that any row masks
// are taken as zero (0 * NaN would reach every row) and added back at the end to
// the rows that do see them.
#include <cooperative_groups.h>

#include <cmath>
#include <cstdio>
#include <mutex>

#include "attn.cuh"
#include "e4m3.cuh"
#include "pages.cuh"

namespace hf {
namespace {

namespace cg = cooperative_groups;

constexpr int BN = 64, RT = 128;
constexpr int PLD = BN + 4;
constexpr int CLUSTER = 4;  // CTAs that share a prompt's tile of rows
enum { PROMPT = 0, PAGED = 1 };

__host__ __device__ inline size_t rows_smem(int dh, int bm) {
  return ((size_t)(bm + 2 * BN) * (dh + 4) + (size_t)bm * PLD) * sizeof(float);
}

// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void copy16(float* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 r = __ldcg(reinterpret_cast<const uint2*>(p));
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Four codes (bits of x.x) times a scale (x.y): turned once all loads are under way.
__device__ __forceinline__ float4 values4(const float4& x) {
  const uint32_t c = __float_as_uint(x.x);
  const float scale = held_scale(x.y);
  const float2 a = from_e4m3x2(c & 0xffff), b = from_e4m3x2(c >> 16);
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

__device__ __forceinline__ bool odd_value(float x) { return !(fabsf(x) < INFINITY); }

// Element offset of key j's row of KV head g in K (kind 0) or V; -1: no such page. block: its page
// and head, where the scales of an 8-bit cache lie.
template <int MODE>
__device__ __forceinline__ long long key_at(const AttnRows& a, int start, const int32_t* tab, int g, int j, int kv,
                                            long long* block = nullptr) {
  if (MODE == PROMPT) return (long long)(start + j) * (kv ? a.v_ld : a.k_ld) + (long long)g * a.dh;
  const int shift = 31 - __clz(a.page);  // (a power of two)
  const int id = tab[j >> shift];
  if (id < 0 || id >= a.n_pages) return -1;
  const long long b = (long long)id * a.Hkv + g;
  if (block) *block = b;
  return ((b << shift) + (j & (a.page - 1))) * a.dh;
}

// DHT: the head dim, or 0 for any up to 64 * MAXC. Paged: the first pre_x CTAs work on the
// prefix, those up to all_x on the entries' own keys, the others compare the entries' prefixes.
// KV: the type of the keys and values, T or an 8-bit cache's codes (paged), which become
// values as they come in.
template <typename T, typename KV, int MODE, int MAXC, int DHT, int RPT>
__global__ void __launch_bounds__(RT) rows_kernel(AttnRows a, int pre_x, int all_x) {
  extern __shared__ __align__(16) float smf[];
  constexpr bool F32 = sizeof(T) == 4, KV32 = sizeof(KV) == 4;
  constexpr int BM = 8 * RPT;
  const int dh = DHT ? DHT : a.dh, ldq = dh + 4, c4 = dh / 4;
  float* sq = smf;
  float* sk = sq + BM * ldq;
  float* sv = sk + BN * ldq;
  float* sp = sv + BN * ldq;
  __shared__ int s_odd, s_low;
  __shared__ float2 s_ml[BM];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  constexpr int CL = MODE == PROMPT ? CLUSTER : 1;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  if (tid == 0) s_low = 0x7fffffff;
  pdl_trigger();
  pdl_wait();
  if (MODE == PAGED && (int)blockIdx.x >= all_x) {
    if (blockIdx.y == 0) check_prefixes(a, 1 + (int)blockIdx.x - all_x, (int)gridDim.x - all_x, tid, RT);
    return;
  }
  bool bad = false;  // (reported by an entry's first CTA)
  // the item: rows [row0, row0 + nrows) of KV head g, keys [j0, j1)
  const int g = blockIdx.y;
  int row0, nrows, j0 = 0, j1, start = 0, entry = 0, piece = 0, len = 0;
  const int32_t* tab = nullptr;
  const bool pre = MODE == PAGED && (int)blockIdx.x < pre_x;
  if (MODE == PROMPT) {
    if (blockIdx.x == 0 && g == 0) check_offsets(a, tid, RT);
    const PromptTile t = prompt_tile(a, (int)((gridDim.x - 1 - blockIdx.x) / CL), BM, a.G);
    if (!t.ok) return;  // (all CTAs of the cluster)
    start = t.start;
    row0 = t.tile * BM;
    nrows = (int)min((long long)BM, (long long)t.len * a.G - row0);
    j1 = (row0 + nrows - 1) / a.G + 1;
  } else if (pre) {
    piece = blockIdx.x % a.npre;
    row0 = blockIdx.x / a.npre * BM;
    nrows = min(BM, a.n * a.rows * a.G - row0);
    j0 = piece * a.pre_keys;
    j1 = min(a.shared, j0 + a.pre_keys);
    if (attn_len(a, 0, bad) == 0)  // nothing is shared then: every row is empty
      j1 = j0;
    else
      tab = attn_table(a, 0);
  } else {
    const int x = blockIdx.x - pre_x, blocks = (a.rows * a.G + BM - 1) / BM;
    piece = x % a.nown;
    entry = x / a.nown / blocks;
    row0 = x / a.nown % blocks * BM;
    nrows = min(BM, a.rows * a.G - row0);
    len = attn_len(a, entry, bad);
    if (piece == 0 && row0 == 0 && g == 0 && tid == 0) {
      a.eff[entry] = len;  // for the join
      if (bad && a.status) atomicOr(a.status, HF_S_BAD);
    }
    j0 = a.shared + piece * a.own_keys;
    j1 = min(len, j0 + a.own_keys);
    if (piece > 0 && j0 >= j1) return;  // piece 0 always reports (a direct call has no other)
    if (len > 0) tab = attn_table(a, entry);
  }
  // token row of q and out of the item's row rr, and its query head
  auto token = [&](int rr) { return (size_t)(MODE == PROMPT ? start : pre ? 0 : entry * a.rows) + rr / a.G; };
  auto head = [&](int rr) { return g * a.G + rr % a.G; };

  // K (kv = 0) or V of the keys from jt on. K of the next tile comes in while this one's
  // values are summed, V while the next one's scores are formed.
  auto load = [&](int kv, int jt) {
    constexpr int U = 8;
    float* to = kv ? sv : sk;
    const KV* from = static_cast<const KV*>(kv ? a.v : a.k);
    for (int e0 = tid; jt < j1 && e0 < BN * c4; e0 += RT * U) {
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * RT, j = e / c4, c = (e % c4) * 4;
        if (e >= BN * c4) continue;
        long long block = 0;
        const long long at = jt + j < j1 ? key_at<MODE>(a, start, tab, g, jt + j, kv, &block) : -2;
        if (at == -1 && a.status) atomicOr(a.status, HF_S_BAD);
        const KV* src = from + (at < 0 ? 0 : at + c);
        if constexpr (KV32)
          copy16(&to[j * ldq + c], src, at >= 0);
        else if constexpr (sizeof(KV) == 1)
          x[u] = at >= 0 ? make_float4(__uint_as_float(__ldcg(reinterpret_cast<const uint32_t*>(src))),
                                       __ldcg(&(kv ? a.v_scale : a.k_scale)[block]), 0.f, 0.f)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        else
          x[u] = at >= 0 ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if constexpr (!KV32) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int e = e0 + u * RT;
          if constexpr (sizeof(KV) == 1) x[u] = values4(x[u]);
          if (e < BN * c4) *reinterpret_cast<float4*>(&to[e / c4 * ldq + (e % c4) * 4]) = x[u];
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int first = j0 + rank * BN;
  for (int e = tid; e < BM * c4; e += RT) {  // q comes with the first K
    const int r = e / c4, c = (e % c4) * 4;
    const T* src = static_cast<const T*>(a.q) + c;
    if (r < nrows) src += token(row0 + r) * a.q_ld + (size_t)head(row0 + r) * dh;
    if constexpr (F32)
      copy16(&sq[r * ldq + c], src, r < nrows);
    else
      *reinterpret_cast<float4*>(&sq[r * ldq + c]) = r < nrows ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  load(0, first);
  load(1, first);

  // this thread's rows: the keys they see
  int limit[RPT];
  if (tid == 0) s_odd = j1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    limit[i] = 0;
    if (ty * RPT + i >= nrows) continue;
    const int t = (row0 + ty * RPT + i) / a.G;
    bool dead = false;
    if (MODE == PROMPT) {
      limit[i] = t + 1;
    } else if (pre) {
      const int l = attn_len(a, t / a.rows, bad);
      dead = l == 0;
      limit[i] = max(0, min(a.shared, l - a.rows + t % a.rows + 1));
    } else {
      limit[i] = max(0, len - a.rows + t + 1);
    }
    if (tx == 0 && !dead) atomicMin(&s_low, limit[i]);
  }
  float m[RPT], l[RPT];
  uint64_t o2[RPT][MAXC * 2];  // pairs of neighbouring columns
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < MAXC * 2; ++c) o2[i][c] = 0;
  }

  for (int jt = first; jt < j1; jt += CL * BN) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // K; V may still be on its way
    __syncthreads();
    float s[RPT][4];
    {
      uint64_t s2[RPT][4];  // sums over the even and the odd dimensions
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 8
      for (int d = 0; d < dh; d += 4) {
        ulonglong2 kv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(&sk[(tx + 16 * j) * ldq + d]);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(&sq[(ty * RPT + i) * ldq + d]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s2[i][j] = fma2(qv.y, kv[j].y, fma2(qv.x, kv[j].x, s2[i][j]));
        }
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpair(s2[i][j]);
          s[i][j] = (x.x + x.y) * a.qscale;
        }
    }
    __syncthreads();  // K has been read
    load(0, jt + CL * BN);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int lim = min(limit[i], j1);
      float t = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (jt + tx + 16 * j >= lim) s[i][j] = -INFINITY;
        t = fmaxf(t, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, w));
      const float nm = fmaxf(m[i], t);
      const float base = nm > -INFINITY ? nm : 0.f;  // a row that has seen nothing: all terms 2^-inf = 0
      const float f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - base);
        sum += e;
        sp[(ty * RPT + i) * PLD + tx + 16 * j] = e;
      }
      l[i] = l[i] * f + sum;  // this thread's columns; joined at the end
      m[i] = nm;
#pragma unroll
      for (int c = 0; c < MAXC * 2; ++c) o2[i][c] = mul2(o2[i][c], pair(f, f));
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // V
    __syncthreads();
    // some row masks keys of this tile: the odd values of V there are set aside
    const int low = s_low;
    if (low < min(jt + BN, j1)) {
      const int k0 = max(0, low - jt);
      for (int e = tid; e < (BN - k0) * dh; e += RT) {
        float* x = &sv[(k0 + e / dh) * ldq + e % dh];
        if (odd_value(*x)) {
          *x = 0.f;
          atomicMin(&s_odd, jt);
        }
      }
      __syncthreads();
    }
#pragma unroll 4
    for (int j = 0; j < BN; j += 4) {
      float4 p[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) p[i] = *reinterpret_cast<const float4*>(&sp[(ty * RPT + i) * PLD + j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
          if (tx * 4 + 64 * c >= dh) continue;
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sv[(j + jj) * ldq + tx * 4 + 64 * c]);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
            o2[i][2 * c] = fma2(pair(w, w), x.x, o2[i][2 * c]);
            o2[i][2 * c + 1] = fma2(pair(w, w), x.y, o2[i][2 * c + 1]);
          }
        }
    }
    __syncthreads();  // V has been read
    load(1, jt + CL * BN);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // (q, where there was no tile)
  __syncthreads();
  float o[RPT][MAXC * 4];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int c = 0; c < MAXC * 2; ++c) {
      const float2 x = unpair(o2[i][c]);
      o[i][2 * c] = x.x;
      o[i][2 * c + 1] = x.y;
    }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);

  int odd_from = s_odd;
  if constexpr (CL > 1) {
    // each CTA shows its sums where its tiles were, and joins a quarter of the rows: those
    // with i % 4 = its rank
    cg::cluster_group cluster = cg::this_cluster();
    float* so = sk;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      if (tx == 0) s_ml[ty * RPT + i] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < MAXC; ++c)
        if (tx * 4 + 64 * c < dh)
          *reinterpret_cast<float4*>(&so[(ty * RPT + i) * ldq + tx * 4 + 64 * c]) =
              make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
    }
    cluster.sync();
#pragma unroll
    for (int k = 0; k < CL; ++k) odd_from = min(odd_from, *cluster.map_shared_rank(&s_odd, k));
#pragma unroll
    for (int i0 = 0; i0 < RPT; i0 += CL) {
      const int r = ty * RPT + i0 + rank;
      float2 ml[CL];
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        ml[k] = *cluster.map_shared_rank(&s_ml[r], k);
        top = fmaxf(top, ml[k].x);
      }
      const float base = top > -INFINITY ? top : 0.f;
      float sum = 0.f, v[MAXC * 4];
#pragma unroll
      for (int c = 0; c < MAXC * 4; ++c) v[c] = 0.f;
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        if (ml[k].y == 0.f) continue;
        const float w = exp2f(ml[k].x - base);
        sum += ml[k].y * w;
        const float* src = cluster.map_shared_rank(so, k);
#pragma unroll
        for (int c = 0; c < MAXC; ++c)
          if (tx * 4 + 64 * c < dh) {
            const float4 x = *reinterpret_cast<const float4*>(&src[r * ldq + tx * 4 + 64 * c]);
            v[4 * c] += w * x.x;
            v[4 * c + 1] += w * x.y;
            v[4 * c + 2] += w * x.z;
            v[4 * c + 3] += w * x.w;
          }
      }
#pragma unroll
      for (int i = i0; i < i0 + CL; ++i)
        if (i - i0 == rank) {
          m[i] = top;
          l[i] = sum;
#pragma unroll
          for (int c = 0; c < MAXC * 4; ++c) o[i][c] = v[c];
        }
    }
    cluster.sync();  // read by all before a CTA of the cluster ends
  }
  const bool direct = MODE == PROMPT || attn_direct(a);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int rr = row0 + ty * RPT + i;
    if (ty * RPT + i >= nrows || (CL > 1 && i % CL != rank)) continue;
    if (odd_from < j1)  // rows that see an odd value of V get it after all
      for (int j = odd_from; j < min(limit[i], j1); ++j) {
        const long long at = key_at<MODE>(a, start, tab, g, j, 1);
        if (at < 0) continue;
#pragma unroll
        for (int c = 0; c < MAXC * 4; ++c) {
          const int d = tx * 4 + 64 * (c / 4) + c % 4;
          if (d >= dh) continue;
          float x;
          if constexpr (sizeof(KV) == 1)
            x = from_e4m3(static_cast<const KV*>(a.v)[at + d]);  // (NaN is NaN at any scale)
          else
            x = to_f(static_cast<const KV*>(a.v)[at + d]);
          if (odd_value(x)) o[i][c] += x;
        }
      }
    if (direct) {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      T* dst = static_cast<T*>(a.out) + token(rr) * a.out_ld + (size_t)head(rr) * dh;
#pragma unroll
      for (int c = 0; c < MAXC; ++c) {
        const int d = tx * 4 + 64 * c;
        if (d >= dh) continue;
        if constexpr (F32)
          *reinterpret_cast<float4*>(dst + d) =
              make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
        else
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[d + k] = from_f<T>(o[i][4 * c + k] * inv);
      }
    } else {
      const PartAt at = pre ? part_prefix(a, piece, g, rr / a.G, rr % a.G)
                            : part_own_rows(a, entry, piece, g, rr / a.G, rr % a.G);
      if (tx == 0) a.part_ml[at.first + at.row] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < MAXC; ++c) {
        const int d = tx * 4 + 64 * c;
        if (d < dh)
          *reinterpret_cast<float4*>(&a.part_o[at.first * dh + ((size_t)(d / 8) * at.region + at.row) * 8 + d % 8]) =
              make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
      }
    }
  }
}

// Warps of a CTA: four leave few idle ones in the last round (64 x 8 rows over a prefix of
// 8192, all: 103.7 us, with eight 104.2).
constexpr int join_warps(int wpr) { return wpr > 4 ? wpr : 4; }

// A row's pieces weighted by 2^(m - max m). A warp takes four neighbouring rows of an
// entry, lane = (8 columns, row): its loads are whole lines. WPR warps of a CTA share
// the rows, each joining every WPR-th piece; the CTA's last step joins the warps. SEGS:
// groups of 64 columns of a warp, all of them where warps share rows (24 x 40 rows over a
// prefix of 32768, all: 50.6 us, by 64 columns 52.1), else one, with four pieces in flight
// (64 x 8 rows over 8192, all: 101.4 us, all columns 102.9). Pieces that saw nothing
// hold no values: what lies there is read, and left out. Bound by the latency of the look-ups
// and the reads of the pieces.
template <typename T, int WPR, int SEGS>
__global__ void __launch_bounds__(32 * join_warps(WPR)) join_kernel(AttnRows a) {
  constexpr int WARPS = join_warps(WPR);
  constexpr int BATCH = SEGS == 1 ? 4 : SEGS == 2 ? 2 : 1;  // pieces in flight per warp
  __shared__ float s_acc[WPR > 1 ? WARPS : 1][WPR > 1 ? SEGS * 8 : 1][WPR > 1 ? 33 : 1];
  __shared__ float2 s_ml[WARPS][4];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR, dh = a.dh;
  const int per = a.rows * a.Hq, fours = (per + 3) / 4;
  const long long unit = (long long)blockIdx.x * (WARPS / WPR) + warp / WPR;
  const int entry = (int)(unit / fours), lr = (int)(unit % fours) * 4 + (lane & 3);
  const int col = blockIdx.y * 64 * SEGS + (lane >> 2) * 8;
  bool on = entry < a.n && lr < per && col < dh;
  const int g = on ? lr / (a.rows * a.G) : 0, t = on ? lr / a.G % a.rows : 0, i = on ? lr % a.G : 0;
  // (all of them at once: small calls are bound by the chain of dependent loads)
  const int len = on ? __ldcg(&a.eff[entry]) : 0;
  int t0 = 0, t1 = 0;
  int4 ln = {};
  if (a.line && on) {
    ln = __ldcg(reinterpret_cast<const int4*>(a.line));
    t0 = __ldcg(&a.tile0[entry]);
    t1 = __ldcg(&a.tile0[entry + 1]);
  }
  // the entry's own pieces: `own` of them from number `first` on
  int own = 0, first = 0, slot = 0;
  if (len > 0 && a.line) {
    const AttnLine line = {ln.x, ln.y, ln.z, ln.w};
    const int u = unit_of(a, g, t);
    if (t1 > t0) {
      first = line.cta(u * line.tiles + t0 + a.item_start);
      own = line.cta(u * line.tiles + t1 - 1) - first + 1;
    }
    slot = u * a.n + entry;
    if (a.npre == 0 && own == 1) on = false;  // written already
  } else if (len > 0) {
    own = max(1, (max(0, len - a.shared) + a.own_keys - 1) / a.own_keys);
  }
  const int pieces = on && len > 0 ? a.npre + own : 0;
  float m = -INFINITY, l = 0.f, acc[SEGS][8] = {};
  for (int p0 = sub; p0 < pieces; p0 += BATCH * WPR) {
    float2 ml[BATCH];
    float4 x[BATCH][SEGS][2];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int p = p0 + k * WPR;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (p >= pieces) continue;
      const int k_own = first + p - a.npre;
      const PartAt at = p < a.npre ? part_prefix(a, p, g, entry * a.rows + t, i)
                        : a.line   ? part_own_unit(a, slot + k_own, g, t, i)
                                   : part_own_rows(a, entry, k_own, g, t, i);
      ml[k] = __ldcg(&a.part_ml[at.first + at.row]);
#pragma unroll
      for (int s = 0; s < SEGS; ++s)
        if (col + 64 * s < dh) {
          const float4* src =
              reinterpret_cast<const float4*>(&a.part_o[at.first * dh + ((size_t)(col / 8 + 8 * s) * at.region + at.row) * 8]);
          x[k][s][0] = __ldcg(src);
          x[k][s][1] = __ldcg(src + 1);
        }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (ml[k].y == 0.f) continue;
      const float nm = fmaxf(m, ml[k].x), base = nm > -INFINITY ? nm : 0.f;
      const float f = exp2f(m - base), w = exp2f(ml[k].x - base);
      m = nm;
      l = l * f + ml[k].y * w;
#pragma unroll
      for (int s = 0; s < SEGS; ++s)
        if (col + 64 * s < dh) {
          const float* v = reinterpret_cast<const float*>(x[k][s]);
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[s][c] = acc[s][c] * f + w * v[c];
        }
    }
  }
  if (WPR > 1) {
#pragma unroll
    for (int s = 0; s < SEGS; ++s)
#pragma unroll
      for (int c = 0; c < 8; ++c) s_acc[warp][s * 8 + c][lane] = acc[s][c];
    if (lane < 4) s_ml[warp][lane & 3] = make_float2(m, l);
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float2 ml = s_ml[warp + k][lane & 3];
      if (ml.y == 0.f) continue;
      const float nm = fmaxf(m, ml.x), base = nm > -INFINITY ? nm : 0.f;
      const float f = exp2f(m - base), w = exp2f(ml.x - base);
      m = nm;
      l = l * f + ml.y * w;
#pragma unroll
      for (int s = 0; s < SEGS; ++s)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[s][c] = acc[s][c] * f + w * s_acc[warp + k][s * 8 + c][lane];
    }
  }
  if (!on) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = static_cast<T*>(a.out) + ((size_t)entry * a.rows + t) * a.out_ld + (size_t)(g * a.G + i) * dh + col;
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    if (col + 64 * s >= dh) continue;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        reinterpret_cast<float4*>(dst + 64 * s)[h] = make_float4(acc[s][4 * h] * inv, acc[s][4 * h + 1] * inv,
                                                                 acc[s][4 * h + 2] * inv, acc[s][4 * h + 3] * inv);
    } else {
      uint4 y;
      __nv_bfloat162* y2 = reinterpret_cast<__nv_bfloat162*>(&y);
#pragma unroll
      for (int h = 0; h < 4; ++h) y2[h] = __floats2bfloat162_rn(acc[s][2 * h] * inv, acc[s][2 * h + 1] * inv);
      *reinterpret_cast<uint4*>(dst + 64 * s) = y;
    }
  }
}

constexpr int kMaxDev = 64;
std::mutex g_mu;
bool g_set[kMaxDev][2][3][5][2] = {};

template <typename T, typename KV, int MODE, int MAXC, int DHT, int RPT>
cudaError_t launch_one(const AttnRows& a, int pre_x, int all_x, dim3 grid, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* kern = rows_kernel<T, KV, MODE, MAXC, DHT, RPT>;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_set[dev & (kMaxDev - 1)][sizeof(T) == 4][sizeof(KV) == 1 ? 2 : MODE][DHT ? 3 + (DHT == 128) : MAXC / 2][RPT / 4];
    if (!set || dev >= kMaxDev) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)rows_smem(DHT ? DHT : 64 * MAXC, 8 * RPT));
      if (e != cudaSuccess) return e;
      set = true;
    }
  }
  const size_t smem = rows_smem(a.dh, 8 * RPT);
  if (MODE != PROMPT) return launch_pdl(kern, grid, dim3(RT), smem, st, a, pre_x, all_x);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(RT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CLUSTER;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, pre_x, all_x);
}

template <typename T, typename KV, int MODE, int RPT>
cudaError_t launch_dh(const AttnRows& a, int pre_x, int all_x, dim3 grid, cudaStream_t st) {
  constexpr bool F32 = sizeof(T) == 4;
  if (F32 && a.dh == 64) return launch_one<T, KV, MODE, 1, F32 ? 64 : 0, RPT>(a, pre_x, all_x, grid, st);
  if (F32 && a.dh == 128) return launch_one<T, KV, MODE, 2, F32 ? 128 : 0, RPT>(a, pre_x, all_x, grid, st);
  if (a.dh <= 64) return launch_one<T, KV, MODE, 1, 0, RPT>(a, pre_x, all_x, grid, st);
  if (a.dh <= 128) return launch_one<T, KV, MODE, 2, 0, RPT>(a, pre_x, all_x, grid, st);
  return launch_one<T, KV, MODE, 4, 0, RPT>(a, pre_x, all_x, grid, st);
}

template <int MODE, int RPT>
cudaError_t launch_mode(int dtype, const AttnRows& a, int pre_x, int all_x, dim3 grid, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if constexpr (MODE == PAGED)
    if (a.k_scale)
      return dtype == HF_F32 ? launch_dh<float, uint8_t, MODE, RPT>(a, pre_x, all_x, grid, st)
                             : launch_dh<bf, uint8_t, MODE, RPT>(a, pre_x, all_x, grid, st);
  return dtype == HF_F32 ? launch_dh<float, float, MODE, RPT>(a, pre_x, all_x, grid, st)
                         : launch_dh<bf, bf, MODE, RPT>(a, pre_x, all_x, grid, st);
}

// Rows of a thread, over a paged cache: by the rows of a request.
constexpr int kPromptRpt = 4;
int paged_rpt(const AttnRows& a) { return a.rows * a.G <= 16 ? 2 : 4; }

}  // namespace

cudaError_t launch_attn_rows_prompt(int dtype, const AttnRows& a, cudaStream_t st) {
  const long long slots = prompt_slots(a.total, a.n_seq, a.G, 8 * kPromptRpt) * CLUSTER;
  if (slots > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_mode<PROMPT, kPromptRpt>(dtype, a, 0, 0, dim3((unsigned)slots, a.Hkv), st);
}
cudaError_t launch_attn_rows_pages(int dtype, const AttnRows& a, cudaStream_t st) {
  const int rpt = paged_rpt(a), bm = 8 * rpt;
  const long long rows = (long long)a.n * a.rows * a.G;
  const long long pre_x = (rows + bm - 1) / bm * a.npre;
  const long long own_x = (long long)a.n * ((a.rows * a.G + bm - 1) / bm) * a.nown;
  const long long all_x = pre_x + own_x, checks = a.shared > 0 && a.status ? std::min(a.n, 152) : 0;
  if (all_x + checks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(all_x + checks), a.Hkv);
  return rpt == 4 ? launch_mode<PAGED, 4>(dtype, a, (int)pre_x, (int)all_x, grid, st)
                  : launch_mode<PAGED, 2>(dtype, a, (int)pre_x, (int)all_x, grid, st);
}

namespace {
// Warps that share a row's pieces: eight, which read them side by side, where there are few
// rows, else one; more rows the more pieces they have. Whole calls in a graph, us with eight /
// one, by the fours of rows. Tensor cores, a prefix: 240 (24 rows over 32768 tokens) 64.8 / 87.1,
// 512 46.9 / 55.7, 768 80.7 / 78.5, 1024 50.2 / 46.2, 1536 67.3 / 59.3, 4096 135 / 115; no prefix:
// 8 (one request, 32768 tokens) 40.5 / 54.5, 64 36.4 / 39.3, 240 50.5 / 51.1, 320 110.4 / 110.1,
// 512 (64 requests of 1000) 56.4 / 54.4, 640 44.1 / 41.2. CUDA cores, whose pieces are shorter:
// 128 15.2 / 16.3, 512 46.7 / 49.4, 1024 105.5 / 108.9. (Two were best nowhere by more than 1%.)
template <typename T, int SEGS>
cudaError_t join(const AttnRows& a, cudaStream_t st) {
  const long long units = (long long)a.n * ((a.rows * a.Hq + 3) / 4);
  const int wpr = units >= (!a.line ? 1216 : a.npre > 0 ? 608 : 304) ? 1 : 8;
  const int warps = join_warps(wpr);
  const dim3 grid((unsigned)((units * wpr + warps - 1) / warps), wpr == 1 ? (a.dh + 63) / 64 : 1);
  return launch_pdl(wpr == 8 ? join_kernel<T, 8, SEGS> : join_kernel<T, 1, 1>, grid, dim3(32 * warps), 0, st, a);
}
}  // namespace

cudaError_t launch_attn_join(int dtype, const AttnRows& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (dtype == HF_F32)
    return a.dh <= 64 ? join<float, 1>(a, st) : a.dh <= 128 ? join<float, 2>(a, st) : join<float, 4>(a, st);
  return a.dh <= 64 ? join<bf, 1>(a, st) : a.dh <= 128 ? join<bf, 2>(a, st) : join<bf, 4>(a, st);
}

namespace {

hf_status refuse(const char* m) {
  set_thread_error(m);
  return HF_EINVAL;
}
hf_status done(cudaError_t e) {
  if (e == cudaSuccess) return HF_OK;
  set_thread_error(cudaGetErrorString(e));
  return HF_ECUDA;
}
bool off(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

const char* heads_bad(int hq, int hkv, int dh, float scale) {
  if (hq < 1 || hkv < 1 || hkv > 1024 || hq % hkv) return "n_kv_heads must be 1..1024 and divide n_q_heads";
  if (hq / hkv > 64) return "n_q_heads / n_kv_heads must be <= 64";
  if (dh < 8 || dh % 8 || dh > 256) return "head_dim must be a multiple of 8, <= 256";
  if (!(scale >= 0.f) || !(scale <= 1e38f)) return "scale must be in 0..1e38 (0: 1/sqrt(head_dim))";
  return nullptr;
}
const char* ld_bad(int64_t ld, long long least, int esize, const void* p) {
  if (ld < least || ld > (1LL << 36)) return "a row stride is smaller than heads * head_dim, or above 2^36";
  if (ld * esize % 16 || off(p, 16)) return "q, k, v and out must be 16-byte aligned, their strides multiples of 16 bytes";
  return nullptr;
}
float base2_scale(float scale, int dh) {
  return (float)(1.4426950408889634 * (scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)dh)));
}

// Pieces of the key axis on CUDA cores: as many as give every SM eight CTAs of four warps,
// of a tile of keys at least. A request's own pieces go by its table's reach, not by
// its length, which only the device knows.
void plan_pieces(AttnRows& a) {
  auto split = [](long long keys, long long tiles, int& count, int& each) {
    const long long want = (152 * 8 + tiles - 1) / std::max<long long>(tiles, 1);
    const long long c = std::max<long long>(1, std::min<long long>({want, (keys + BN - 1) / BN, 64}));
    each = (int)std::max<long long>(((keys + c - 1) / c + BN - 1) / BN * BN, BN);  // (no keys: no pieces)
    count = (int)((keys + each - 1) / each);
  };
  const int bm = 8 * paged_rpt(a);
  split(a.shared, ((long long)a.n * a.rows * a.G + bm - 1) / bm * a.Hkv, a.npre, a.pre_keys);
  split((long long)a.table_ld * a.page - a.shared, (long long)a.n * a.Hkv * ((a.rows * a.G + bm - 1) / bm), a.nown,
        a.own_keys);
  a.nown = std::max(a.nown, 1);  // it also writes the empty rows of a direct call
}

// Sizes and workspace of a call.
struct PagesPlan {
  bool tc, dense;                       // dense: an 8-bit cache's prefix as bf16 rows
  int pre_items;                        // tensor cores: items of the prefix
  size_t eff, tile0, ml, o, plan, k, v, total; // offsets in the workspace (the line is at 0)
};
// Where very many rows share a long prefix, it is turned into bf16 rows once (a power of two as the scale:
// exactly) and taken by the kernel for those, 256 rows at a time, instead of as codes, 64 or 128 at a time.
// Worth it by the work that it saves: KV heads x rows of a head, beyond what codes take as fast, x tokens. Whole calls
// in a graph, us, as codes / as rows, heads of 128: 1 KV head, 384 rows of it over 8192 tokens 28 / 45, 1536 46 / 51, over 131072
// 256 80 / 99, 384 133 / 112; 2, 768 over 8192 48 / 48, 1024 57 / 50; 4, 384 48 / 48, 512 56 / 49; 8, 192 48 / 56, 256 56 / 56,
// 384 76 / 60, 1536 231 / 114, over 2048 512 48 / 48, 1024 86 / 63; 10, 256 62 / 65, 384 85 / 70. Heads of 64: 2, 512 over 8192 36 / 36;
// 4, 256 36 / 34; 8, 192 44 / 39. (268 shapes: 1.7% behind the better of the two on average, 36% at most.)
constexpr int kDenseRows = 180;
constexpr long long kDenseWork = 10 << 20;
PagesPlan plan_call(AttnRows& a, int dtype) {
  PagesPlan w{};
  w.tc = attn_tc_ok(dtype, a.dh);
  const size_t N = (size_t)a.n * a.rows * a.Hq;
  size_t rows;
  const long long shared_rows = (long long)a.n * a.rows * a.G;
  const bool e4m3 = a.tile != kTileRows;
  w.dense = w.tc && e4m3 && a.Hkv * (shared_rows - kDenseRows) * a.shared > kDenseWork;
  if (w.tc) {
    if (e4m3) {
      // rows that need two tiles and more are spread evenly over them (32 x 16 rows of 4
      // heads over 4096 tokens 118 us, as 48 and 16 rows 157);
      // an entry's own as well, or all in one tile
      const long long most = a.tile / a.G;
      auto even = [&](long long tokens) {
        const long long pairs = (tokens + 2 * most - 1) / (2 * most);
        return tokens <= most ? tokens : (tokens + 2 * pairs - 1) / (2 * pairs);
      };
      const long long own = even(a.rows), all = w.dense || a.shared == 0 ? own : even((long long)a.n * a.rows);
      a.tile = (int)std::max(own, all) * a.G;
    }
    if (e4m3 && (w.dense || a.shared == 0)) a.item_start = kItemStart8;
    long long slots;
    int pre = 0;
    if (w.dense) {
      AttnRows b = a;
      b.tile = kTileRows;
      attn_tc_sizes(b, w.pre_items, slots);
      attn_tc_sizes(a, pre, slots);
      a.npre = b.npre;
      a.pre_keys = b.pre_keys;
    } else {
      attn_tc_sizes(a, w.pre_items, slots);
    }
    rows = a.npre * N + (size_t)slots * a.unit_rows;
  } else {
    plan_pieces(a);
    rows = attn_direct(a) ? 0 : (a.npre + a.nown) * N;
  }
  w.eff = 16;
  w.tile0 = w.eff + (size_t)a.n * sizeof(int);
  w.ml = (w.tile0 + ((size_t)a.n + 1) * sizeof(int) + 15) / 16 * 16;
  w.o = (w.ml + rows * sizeof(float2) + 31) / 32 * 32;
  w.total = w.o + rows * a.dh * sizeof(float) + 16;  // (the rows start on 32 bytes)
  if (w.dense) {
    const size_t values = (size_t)a.shared * a.Hkv * a.dh * 2;
    w.plan = (w.total + 15) / 16 * 16;  // the prefix's own line, lengths and places
    w.k = (w.plan + 16 + (2 * (size_t)a.n + 1) * sizeof(int) + 15) / 16 * 16;
    w.v = w.k + values;
    w.total = w.v + values;
  }
  return w;
}

// A cache of either kind: its descriptor, the scales of an 8-bit one and the type of q and out.
struct AnyPages {
  const hf_pages* p;
  bool e4m3;
  PageScales s;
  int dtype;
};
AnyPages any_pages(const hf_pages* p) { return {p, false, {}, p ? p->dtype : 0}; }
AnyPages any_pages(const hf_pages8* p) {
  return p ? AnyPages{&p->pages, true, {p->k_scale, p->v_scale}, p->rows} : AnyPages{nullptr, true, {}, 0};
}

const char* pages_args(const AnyPages& c, bool buffers, int n, int rows, int hq, int shared, AttnRows& a) {
  const hf_pages* p = c.p;
  if (const char* m = pages_bad(p, buffers, c.e4m3)) return m;
  if (const char* m = heads_bad(hq, p->n_kv_heads, p->head_dim, 0.f)) return m;
  if (n < 0 || n > (1 << 20)) return "n must be 0..1048576";
  if (rows < 1 || rows > 64) return "rows must be 1..64";
  if (shared < 0 || shared % p->page || shared > (long long)p->table_ld * p->page)
    return "shared must be a multiple of page, at most table_ld * page";
  // (places and units of a line are int: with row tiles of 48 rows there are up to 1.3 times as many as counted here)
  if ((long long)n * rows * hq > 0x7fffffffLL / 4 ||
      ((long long)p->table_ld * p->page / kKeyTile + 1 + (c.e4m3 ? kItemStart8 : kItemStart)) * n * ((long long)rows * hq / (c.e4m3 ? kTileRows8 : kTileRows) + p->n_kv_heads) > 0x3fffffffLL)
    return "n * rows * n_q_heads, or that times the table's reach, is too large";
  a.Hq = hq;
  a.Hkv = p->n_kv_heads;
  a.G = hq / p->n_kv_heads;
  a.dh = p->head_dim;
  a.esize = pages_esize(c.dtype);
  a.tile = c.e4m3 ? tile_rows8(a.G) : kTileRows;
  a.item_start = kItemStart;
  a.table = p->table;
  a.lens = p->lens;
  a.status = p->status;
  a.n = n;
  a.rows = rows;
  a.page = p->page;
  a.n_pages = p->n_pages;
  a.n_requests = p->n_requests;
  a.table_ld = p->table_ld;
  a.shared = shared;
  return nullptr;
}


size_t attend_workspace(const AnyPages& c, int n, int rows, int hq, int shared) {
  AttnRows a{};
  if (pages_args(c, false, std::max(n, 1), rows, hq, shared, a)) return 0;
  return plan_call(a, c.dtype).total;
}

hf_status attend(const AnyPages& c, int32_t layer, int32_t n, int32_t rows, int32_t n_q_heads, const void* q,
                 int64_t q_ld, const int32_t* requests, int32_t shared, float scale, void* out, int64_t out_ld,
                 void* workspace, size_t workspace_bytes, cudaStream_t st) {
  const hf_pages* p = c.p;
  AttnRows a{};
  if (const char* m = pages_args(c, true, n, rows, n_q_heads, shared, a)) return refuse(m);
  if (const char* m = heads_bad(n_q_heads, p->n_kv_heads, p->head_dim, scale)) return refuse(m);
  if (layer < 0 || layer >= p->n_layers) return refuse("layer must be a layer of the cache");
  if (!requests && n > p->n_requests) return refuse("n must be <= n_requests without a list of requests");
  if (n == 0) return HF_OK;
  if (!q || !out || !workspace) return refuse("NULL buffer");
  for (const char* m : {ld_bad(q_ld, (long long)n_q_heads * p->head_dim, a.esize, q),
                        ld_bad(out_ld, (long long)n_q_heads * p->head_dim, a.esize, out)})
    if (m) return refuse(m);
  if (off(requests, 4)) return refuse("requests must be 4-byte aligned");
  const PagesPlan w = plan_call(a, c.dtype);
  if (off(workspace, 16) || workspace_bytes < w.total) {
    char m[160];
    snprintf(m, sizeof m, "workspace must be 16-byte aligned and hold %zu bytes (hf_attention_pages%s_workspace), got %zu",
             w.total, c.e4m3 ? "8" : "", workspace_bytes);
    return refuse(m);
  }
  const size_t layer_bytes = (size_t)p->n_pages * pages_block(p) * pages_esize(p->dtype);
  a.qscale = base2_scale(scale, p->head_dim);
  a.q = q;
  a.q_ld = q_ld;
  a.out = out;
  a.out_ld = out_ld;
  a.k = static_cast<const uint8_t*>(p->k) + layer * layer_bytes;
  a.v = static_cast<const uint8_t*>(p->v) + layer * layer_bytes;
  if (c.e4m3) {
    a.k_scale = c.s.k + (size_t)layer * p->n_pages * p->n_kv_heads;
    a.v_scale = c.s.v + (size_t)layer * p->n_pages * p->n_kv_heads;
  }
  a.req = requests;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.eff = reinterpret_cast<int*>(ws + w.eff);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws + w.o) + 31) / 32 * 32);
  cudaError_t e;
  if (w.tc) {
    a.line = reinterpret_cast<int*>(ws);
    a.tile0 = reinterpret_cast<int*>(ws + w.tile0);
    if (w.dense) {
      AttnRows b = a;
      b.dense = 1;
      b.tile = kTileRows;
      b.tb = kTileRows / a.G;
      b.units = 0;  // no keys of the entries' own
      b.k = ws + w.k;
      b.v = ws + w.v;
      b.k_ld = b.v_ld = (long long)a.Hkv * a.dh;
      b.line = reinterpret_cast<int*>(ws + w.plan);
      b.eff = b.line + 4;
      b.tile0 = b.eff + a.n;
      // SMs that the prefix leaves free begin with the entries' own keys, and take that much more of them: a place
      // of theirs takes 1.6 us, the prefix 1.56 us a tile and 5 an item
      const int ctas = std::min(w.pre_items, 152), rounds = (w.pre_items + ctas - 1) / ctas;
      const int busy = a.n <= kSmall && ctas < 152 ? ctas : 0, places = rounds * (a.pre_keys / kKeyTile + 3);
      e = launch_prefix_values(*p, c.s, layer, requests, a.shared, ws + w.k, ws + w.v, st);
      if (e == cudaSuccess) e = launch_attn_tc_pages(b, w.pre_items, st);
      if (e == cudaSuccess) e = launch_attn_tc8_pages(a, 0, busy, places, st);
    } else {
      e = c.e4m3 ? launch_attn_tc8_pages(a, w.pre_items, 0, 0, st) : launch_attn_tc_pages(a, w.pre_items, st);
    }
  } else {
    e = launch_attn_rows_pages(c.dtype, a, st);
  }
  if (e == cudaSuccess && (w.tc || !attn_direct(a))) e = launch_attn_join(c.dtype, a, st);
  return done(e);
}

}  // namespace
}  // namespace hf

extern "C" hf_status hf_attention_prompt(int32_t dtype, int32_t n_seq, int32_t total, int32_t n_q_heads,
                                         int32_t n_kv_heads, int32_t head_dim, const void* q, int64_t q_ld,
                                         const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                                         const int32_t* offsets, float scale, void* out, int64_t out_ld,
                                         int32_t* status, void* stream) {
  using namespace hf;
  if (dtype != HF_F32 && dtype != HF_BF16) return refuse("dtype must be HF_F32 or HF_BF16");
  if (n_seq < 0 || n_seq > (1 << 24) || total < 0) return refuse("n_seq must be 0..16777216 and total >= 0");
  if (const char* m = heads_bad(n_q_heads, n_kv_heads, head_dim, scale)) return refuse(m);
  // (CTAs: at most a slot per 2 tokens and one per sequence, for each KV head, times four)
  if (((long long)total * (n_q_heads / n_kv_heads) / 32 + total / 4 + n_seq) * n_kv_heads > 0x7fffffffLL / 4)
    return refuse("total * n_q_heads, or n_seq * n_kv_heads, is too large");
  if (n_seq == 0 || total == 0) return HF_OK;
  if (!q || !k || !v || !offsets || !out) return refuse("NULL buffer");
  const int esize = dtype == HF_F32 ? 4 : 2;
  const long long qd = (long long)n_q_heads * head_dim, kd = (long long)n_kv_heads * head_dim;
  for (const char* m : {ld_bad(q_ld, qd, esize, q), ld_bad(k_ld, kd, esize, k), ld_bad(v_ld, kd, esize, v),
                        ld_bad(out_ld, qd, esize, out)})
    if (m) return refuse(m);
  if (off(offsets, 4) || off(status, 4)) return refuse("offsets and status must be 4-byte aligned");
  AttnRows a{};
  a.Hq = n_q_heads;
  a.Hkv = n_kv_heads;
  a.G = n_q_heads / n_kv_heads;
  a.dh = head_dim;
  a.esize = esize;
  a.qscale = base2_scale(scale, head_dim);
  a.q = q;
  a.q_ld = q_ld;
  a.k = k;
  a.k_ld = k_ld;
  a.v = v;
  a.v_ld = v_ld;
  a.out = out;
  a.out_ld = out_ld;
  a.off = offsets;
  a.n_seq = n_seq;
  a.total = total;
  a.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  return done(attn_tc_ok(dtype, head_dim) ? launch_attn_tc_prompt(a, st) : launch_attn_rows_prompt(dtype, a, st));
}

extern "C" size_t hf_attention_pages_workspace(const hf_pages* p, int32_t n, int32_t rows, int32_t n_q_heads,
                                               int32_t shared) {
  return hf::attend_workspace(hf::any_pages(p), n, rows, n_q_heads, shared);
}

extern "C" hf_status hf_attention_pages(const hf_pages* p, int32_t layer, int32_t n, int32_t rows,
                                        int32_t n_q_heads, const void* q, int64_t q_ld, const int32_t* requests,
                                        int32_t shared, float scale, void* out, int64_t out_ld, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return hf::attend(hf::any_pages(p), layer, n, rows, n_q_heads, q, q_ld, requests, shared, scale, out, out_ld,
                    workspace, workspace_bytes, (cudaStream_t)stream);
}

extern "C" size_t hf_attention_pages8_workspace(const hf_pages8* p, int32_t n, int32_t rows, int32_t n_q_heads,
                                                int32_t shared) {
  if (hf::pages8_bad(p, false)) return 0;
  return hf::attend_workspace(hf::any_pages(p), n, rows, n_q_heads, shared);
}

extern "C" hf_status hf_attention_pages8(const hf_pages8* p, int32_t layer, int32_t n, int32_t rows,
                                         int32_t n_q_heads, const void* q, int64_t q_ld, const int32_t* requests,
                                         int32_t shared, float scale, void* out, int64_t out_ld, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  if (const char* m = hf::pages8_bad(p, true)) return hf::refuse(m);
  return hf::attend(hf::any_pages(p), layer, n, rows, n_q_heads, q, q_ld, requests, shared, scale, out, out_ld,
                    workspace, workspace_bytes, (cudaStream_t)stream);
}
