// Attention of many query rows on the tensor cores (bf16, head dim 64 or 128):
// whole prompts, and the common prefix of a paged cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(qscale s_ij - m_i),  s_ij = q_i.k_j
// in one pass over key tiles of 128 with a running m_i. A CTA has two tiles of 128
// rows of one KV head (rows are token * G + head in the group, so the group's
// heads share every key tile). tcgen05 forms S = Q K^T into TMEM; one thread per row
// reads its 128 scores, writes the weights back over them as bf16, and tcgen05 adds
// P V to the row's sums in TMEM, with P read from TMEM and V straight from its
// row-major tile (the transposed operand form). m_i is raised only when a tile's
// maximum passes it by more than 2^8 (in the exponent): until then weights stay
// below 2^8 and nothing is rescaled, so the sums in TMEM are touched by the tensor
// cores alone for most tiles.
//
// While the softmax threads of one row tile work, the tensor cores work for the
// other: warp 0 loads (TMA), warp 1 issues the products, warps 4-7 and 8-11 are the
// two softmax groups. Per key tile the two products of both row tiles take 4 x 512
// tensor cycles, and each group's 128 x 128 exponentials and conversions have to fit
// beside them.
//
// Masked keys: scores are selected by position. V's non-finite values in a tile that
// some row masks are set to zero in shared memory (0 * NaN would reach every row) and
// added back at the end to the rows that see them.
#include <mutex>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace hf {
namespace {

constexpr int BN = 128;        // keys per tile
constexpr int TCT = 384;       // threads
enum { PROMPT = 0, PREFIX = 1 };

template <int DH>
struct Tc {
  static constexpr int TILE = BN * DH * 2;            // bytes of a K, V or Q tile
  static constexpr int SLOTS = DH == 128 ? 5 : 10;    // ring of K and V tiles
  static constexpr int O_COL = 256;                   // TMEM: S0 | S1 | O0 | O1
  static constexpr size_t smem() { return 1024 + (size_t)(2 + SLOTS) * TILE + (2 * SLOTS + 8) * 8 + 64; }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Products issued by a whole warp in uniform control flow: every lane computes the
// same operands (they stay in uniform registers), `lead` is set in one lane.
// Descriptors come as their low words; the high words are constants.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
// A row-major [keys][64] tile read along its rows (the operand's N runs along a row, its
// K over the rows): the next 64 columns are a tile of BN rows further.
__device__ __forceinline__ uint32_t desc_lo_rows(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFu) | ((uint32_t)(BN * 128) >> 4) << 16;
}
// D (+)= A B, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%2, %6};\n\tmov.b64 y, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], x, y, %4, p;\n\t}\n" ::"r"(lead),
      "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi));
}
// The same with A in TMEM (bf16 pairs along a lane's columns).
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], y, %4, p;\n\t}\n" ::"r"(lead),
      "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}\n" ::"r"(lead),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}

__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The loads have arrived; the values pass through, so that nothing uses them earlier.
__device__ __forceinline__ void tmem_hold32(float* v) {
  asm volatile(""
               : "+f"(v[0]),"+f"(v[1]),"+f"(v[2]),"+f"(v[3]),"+f"(v[4]),"+f"(v[5]),"+f"(v[6]),"+f"(v[7]),
                 "+f"(v[8]),"+f"(v[9]),"+f"(v[10]),"+f"(v[11]),"+f"(v[12]),"+f"(v[13]),"+f"(v[14]),"+f"(v[15]),
                 "+f"(v[16]),"+f"(v[17]),"+f"(v[18]),"+f"(v[19]),"+f"(v[20]),"+f"(v[21]),"+f"(v[22]),"+f"(v[23]),
                 "+f"(v[24]),"+f"(v[25]),"+f"(v[26]),"+f"(v[27]),"+f"(v[28]),"+f"(v[29]),"+f"(v[30]),"+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(t)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool odd_half(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }

// Bounded wait of a whole warp; the answer is the same in every lane.
__device__ __forceinline__ bool try_wait_addr(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  for (;;) {
    if (try_wait_addr(bar, parity)) return true;
    if (__any_sync(0xffffffffu, clock64() - t0 > kWaitCycles)) return false;
  }
}
__device__ __forceinline__ bool wait_uniform(uint32_t bar, uint32_t parity) {
  return try_wait_addr(bar, parity) || wait_slow(bar, parity);
}

struct TcArgs {
  AttnRows a;
  int tb;          // tokens per row tile: 128 / G
  int items;       // row blocks (prompt: slots) of 2 tb tokens
  int box_rows;    // rows of a K / V box (prompt: 128, paged: the page)
};

template <int MODE>
__device__ __forceinline__ long long v_at(const AttnRows& a, int start, const int32_t* tab, int g, int j) {
  if (MODE == PROMPT) return (long long)(start + j) * a.v_ld + (long long)g * a.dh;
  const int id = __ldg(&tab[j / a.page]);
  if (id < 0 || id >= a.n_pages) return -1;
  return (((long long)id * a.Hkv + g) * a.page + j % a.page) * a.dh;
}

// What row `o[32]` (columns d0 ..) gets from V's non-finite values at keys [j0, j1).
template <int MODE>
__device__ __noinline__ float odd_sum(const AttnRows& a, int start, const int32_t* tab, int g, int j0, int j1, int d) {
  float s = 0.f;
  for (int j = j0; j < j1; ++j) {
    const long long at = v_at<MODE>(a, start, tab, g, j);
    if (at < 0) continue;
    const float x = to_f(static_cast<const __nv_bfloat16*>(a.v)[at + d]);
    if (!(fabsf(x) < INFINITY)) s += x;
  }
  return s;
}

template <int DH, int MODE>
__global__ void __launch_bounds__(TCT, 1)
tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv, const TcArgs c) {
  using L = Tc<DH>;
  constexpr int NS = L::SLOTS, HALVES = DH / 64, HALF = BN * 128;
  const AttnRows& a = c.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * L::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + (size_t)NS * L::TILE);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;
  uint64_t* s_full = q_full + 1;  // [2]
  uint64_t* p_full = s_full + 2;  // [2]
  uint64_t* o_full = p_full + 2;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* odd_from = reinterpret_cast<int*>(tmem_slot + 2);
  int* low = odd_from + 1;  // [2] least limit of a group's rows
  int* issued = low + 2;    // tiles that the loader has asked for

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&o_full[g], 1);
    }
    *abort_flag = 0;
    *odd_from = 0x7fffffff;
    low[0] = low[1] = 0x7fffffff;
    *issued = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // the item: tokens [t0, t0 + ntok) of KV head g, keys [j0, j1)
  const int g = blockIdx.x % a.Hkv, block = blockIdx.x / a.Hkv;
  int start = 0, t0, ntok, j0 = 0, j1, piece = 0;
  const int32_t* tab = nullptr;
  bool work = true;
  if (MODE == PROMPT) {
    if (blockIdx.x == 0) check_offsets(a);
    const PromptTile t = prompt_tile(a, c.items - 1 - block, 2 * c.tb, 1);
    work = t.ok;
    start = t.start;
    t0 = t.tile * 2 * c.tb;
    ntok = min(2 * c.tb, t.len - t0);
    j1 = t0 + ntok;
  } else {
    t0 = block * 2 * c.tb;
    ntok = min(2 * c.tb, a.n * a.rows - t0);
    piece = blockIdx.y;
    j0 = piece * a.pre_keys;
    j1 = min(a.shared, j0 + a.pre_keys);
    bool bad = false;
    if (attn_raw_len(a, 0, bad) == 0)
      j1 = j0;
    else
      tab = attn_table(a, 0);
  }
  const int nt = work ? (j1 - j0 + BN - 1) / BN : 0;
  // prompt: the first row tile ends earlier
  const int nt0 = MODE == PROMPT ? min(nt, (min(j1, t0 + c.tb) + BN - 1) / BN) : nt;
  const int nt1 = ntok > c.tb ? nt : 0;  // no second row tile

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && nt > 0) {
      // ---- loads: Q, then K(0), V(0), K(1), ... through the ring
      if (lane == 0) {
        const uint32_t rows = (uint32_t)(c.tb * a.G);
        mbar_expect_tx(q_full, (nt1 > 0 ? 2u : 1u) * HALVES * rows * 128u);
        for (int r = 0; r < (nt1 > 0 ? 2 : 1); ++r)
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(sQ + r * L::TILE + h * HALF, &mq, q_full, h * 64, g * a.G, start + t0 + r * c.tb);
      }
      const int nbox = HALVES * (BN / c.box_rows);
      int i = 0;
      for (; i < 2 * nt; ++i) {
        const int s = i % NS;
        bool ok = true;
        if (lane == 0) {
          if (i >= NS) ok = mbar_wait(&empty[s], ((uint32_t)(i / NS) & 1u) ^ 1u);
          if (ok && !*abort_flag)
            mbar_expect_tx(&full[s], L::TILE);
          else
            ok = false;
        }
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
          *abort_flag = 1;
          break;
        }
        if (lane < nbox) {
          const int h = lane % HALVES, b = lane / HALVES;
          const int j = j0 + (i >> 1) * BN + b * c.box_rows;
          uint8_t* dst = sKV + (size_t)s * L::TILE + h * HALF + b * c.box_rows * 128;
          if (MODE == PROMPT) {
            tma_load_3d(dst, (i & 1) ? &mv : &mk, &full[s], h * 64, g, start + j);
          } else {
            int z = a.n_pages * a.Hkv;  // behind the pool: reads zeros
            if (j < j1) {
              const int id = __ldg(&tab[j / a.page]);
              if (id >= 0 && id < a.n_pages)
                z = id * a.Hkv + g;
              else if (a.status)
                atomicOr(a.status, HF_S_BAD);
            }
            tma_load_3d(dst, (i & 1) ? &mv : &mk, &full[s], h * 64, 0, z);
          }
        }
      }
      if (lane == 0) *issued = i;
    } else if (warp == 1 && nt > 0) {
      // ---- products: S0(0), S1(0), then PV0(j), S0(j+1), PV1(j), S1(j+1)
      constexpr uint32_t id_s = idesc_bf16(BN);
      constexpr uint32_t id_o = idesc_bf16(DH) | (1u << 16);
      const uint32_t lead = elect_one();
      const int un = __shfl_sync(0xffffffffu, nt, 0), un0 = __shfl_sync(0xffffffffu, nt0, 0),
                un1 = __shfl_sync(0xffffffffu, nt1, 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t aq = desc_lo(smem_u32(sQ)), ak = desc_lo(smem_u32(sKV)), av = desc_lo_rows(smem_u32(sKV));
      const uint32_t b_full = smem_u32(full), b_empty = smem_u32(empty), b_s = smem_u32(s_full), b_p = smem_u32(p_full),
                     b_o = smem_u32(o_full);
      auto score = [&](int r, int slot) {
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint32_t step = (uint32_t)((k / 4) * (HALF >> 4) + (k % 4) * 2);
          mma_ss(lead, tm + r * BN, aq + r * (L::TILE >> 4) + step, ak + slot * (L::TILE >> 4) + step, id_s, k > 0);
        }
        mma_commit(lead, b_s + 8 * r);
      };
      bool ok = wait_uniform(smem_u32(q_full), 0) && wait_uniform(b_full, 0);
      if (ok) {
        tc_fence_after();
        score(0, 0);
        if (un1 > 0) score(1, 0);
        mma_commit(lead, b_empty);
      }
      int vs = 1 % NS, ks = 2 % NS;    // slots of V(j), K(j+1) and the parity of their fill
      uint32_t vph = 0, kph = 0;
      for (int j = 0; j < un && ok; ++j) {
        const bool more = j + 1 < un;
        ok = wait_uniform(b_full + 8 * vs, vph) && (!more || wait_uniform(b_full + 8 * ks, kph));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int mine = r ? un1 : un0;
          if (!ok || j >= mine) continue;
          ok = wait_uniform(b_p + 8 * r, (uint32_t)j & 1u);
          if (!ok) continue;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts(lead, tm + L::O_COL + r * DH, tm + r * BN + k * 8, av + vs * (L::TILE >> 4) + k * (2048 >> 4), id_o,
                   j > 0 || k > 0);
          mma_commit(lead, b_o + 8 * r);
          if (j + 1 < mine) score(r, ks);
        }
        if (ok) {
          mma_commit(lead, b_empty + 8 * vs);
          if (more) mma_commit(lead, b_empty + 8 * ks);
        }
        vs += 2;
        if (vs >= NS) {
          vs -= NS;
          vph ^= 1u;
        }
        ks += 2;
        if (ks >= NS) {
          ks -= NS;
          kph ^= 1u;
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- softmax: one thread per row
    const int r = warp >= 8, quad = warp & 3, row = quad * 32 + lane;
    const int mine = r ? nt1 : nt0;
    const int tl = r * c.tb + row / a.G;  // token within the item
    const bool valid = row < c.tb * a.G && tl < ntok && mine > 0;
    const int head = g * a.G + row % a.G;
    int limit = 0x7fffffff;  // keys below it are seen (rows without a token: all, and dropped)
    bool dead = false;       // an entry without tokens
    const size_t orow = (size_t)start + t0 + tl;
    if (valid) {
      if (MODE == PROMPT) {
        limit = t0 + tl + 1;
      } else {
        bool bad = false;
        const int t = t0 + tl, len = attn_len(a, t / a.rows, bad);
        dead = len == 0;
        if (!dead) limit = max(0, len - a.rows + t % a.rows + 1);
      }
    }
    if (valid && !dead) atomicMin(&low[r], limit);
    asm volatile("bar.sync %0, 128;" ::"r"(1 + r) : "memory");
    const int glow = *(volatile int*)&low[r];
    const int wlow = __reduce_min_sync(0xffffffffu, min(limit, j1));
    const int lim = min(limit, j1);
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + r * BN, to = tmem + lanes + L::O_COL + r * DH;
    float mb = -INFINITY, l = 0.f;  // maximum in use, times qscale; sum of the weights
    bool ok = true;
    for (int j = 0; j < mine; ++j) {
      const int jt = j0 + j * BN;
      ok = mbar_wait(&s_full[r], (uint32_t)j & 1u);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float s[BN];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s + q * 32);
      tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_hold32(s + q * 32);
      if (jt + BN > wlow) {
#pragma unroll
        for (int q = 0; q < BN; ++q)
          if (jt + q >= lim) s[q] = -INFINITY;
      }
      float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int q = 4; q < BN; ++q) t4[q & 3] = fmaxf(t4[q & 3], s[q]);
      const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * a.qscale;
      bool lift = top > mb + 8.f;
      if (__any_sync(0xffffffffu, lift)) {
        // (mb = -infinity: the sums are zero, or not written yet)
        const float nm = lift ? top : mb;
        const float f = mb > -INFINITY ? ex2(mb - nm) : 1.f;
        if (j > 0 && __any_sync(0xffffffffu, lift && mb > -INFINITY)) {
          ok = mbar_wait(&o_full[r], (uint32_t)(j - 1) & 1u);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < DH; q += 32) {
            float o[32];
            tmem_ld32(to + q, o);
            tmem_wait_ld();
            tmem_hold32(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f;
            tmem_st32(to + q, reinterpret_cast<uint32_t*>(o));
          }
          tmem_wait_st();
        }
        l *= f;
        mb = nm;
      }
      const float base = mb > -INFINITY ? mb : 0.f;
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[32];
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          const float e0 = ex2(fmaf(s[h * 64 + 2 * q], a.qscale, -base));
          const float e1 = ex2(fmaf(s[h * 64 + 2 * q + 1], a.qscale, -base));
          l4[q & 1] += e0;
          l4[2 + (q & 1)] += e1;
          p[q] = pack_bf16(e0, e1);
        }
        tmem_st32(ts + h * 32, p);
      }
      l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      tmem_wait_st();
      if (glow < (MODE == PROMPT ? jt + BN : min(jt + BN, j1))) {
        // some row of the group masks keys of this tile
        const int vi = 2 * j + 1, vs = vi % NS;
        ok = mbar_wait(&full[vs], (uint32_t)(vi / NS) & 1u);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint4* v = reinterpret_cast<uint4*>(sKV + (size_t)vs * L::TILE);
        for (int q = row; q < L::TILE / 16; q += 128) {
          uint4 x = v[q];
          uint32_t* w = reinterpret_cast<uint32_t*>(&x);
          bool odd = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (odd_half(w[k])) {
              w[k] &= 0xffff0000u;
              odd = true;
            }
            if (odd_half(w[k] >> 16)) {
              w[k] &= 0x0000ffffu;
              odd = true;
            }
          }
          if (odd) {
            atomicMin(odd_from, jt);
            __threadfence_block();
            v[q] = x;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[r]);
    }
    // ---- epilogue
    ok = __all_sync(0xffffffffu, ok);
    if (ok && mine > 0) {
      ok = mbar_wait(&o_full[r], (uint32_t)(mine - 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (!ok) {
      *abort_flag = 1;
    } else if (work) {
      const bool direct = MODE == PROMPT || attn_direct(a);
      const float inv = l == 0.f || dead ? 0.f : 1.f / l;
      const int from = *(volatile int*)odd_from;
      const size_t N = (size_t)a.n * a.rows * a.Hq;
      const bool mine_row = row < c.tb * a.G && tl < ntok;  // also where there was no key at all
      const size_t pr = piece * N + orow * a.Hq + head;
#pragma unroll 1
      for (int q = 0; q < DH; q += 32) {
        float o[32];
        if (mine > 0) {
          tmem_ld32(to + q, o);
          tmem_wait_ld();
          tmem_hold32(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (valid && !dead && from < lim)
          for (int k = 0; k < 32; ++k) o[k] += odd_sum<MODE>(a, start, tab, g, from, lim, q + k);
        if (!mine_row) continue;
        if (direct) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * a.out_ld +
                                                (size_t)head * DH + q);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = dead ? 0u : pack_bf16(o[8 * k + 2 * x] * inv, o[8 * k + 2 * x + 1] * inv);
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (mine > 0) {
          float4* dst = reinterpret_cast<float4*>(&a.part_o[pr * DH + q]);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (!direct && mine_row) {
        a.part_ml[pr] = dead || mine == 0 ? make_float2(-INFINITY, 0.f) : make_float2(mb, l);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {
    if (tid == 0) {
      if (a.status) atomicOr(a.status, HF_S_TIMEOUT);
      if (nt > 0) mbar_wait(q_full, 0);
      // the copies still in flight land before the CTA's shared memory goes
      for (int i = max(0, *issued - NS); i < *issued; ++i) mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDev = 64;
std::mutex g_mu;
bool g_set[kMaxDev][2][2] = {};

template <int DH, int MODE>
cudaError_t launch_one(const TcArgs& c, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       dim3 grid, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_set[dev & (kMaxDev - 1)][DH == 128][MODE];
    if (!set || dev >= kMaxDev) {
      e = cudaFuncSetAttribute(tc_kernel<DH, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)Tc<DH>::smem());
      if (e != cudaSuccess) return e;
      set = true;
    }
  }
  return launch_pdl(tc_kernel<DH, MODE>, grid, dim3(TCT), Tc<DH>::smem(), st, mq, mk, mv, c);
}

template <int MODE>
cudaError_t launch_mode(const AttnRows& a, cudaStream_t st) {
  TcArgs c{};
  c.a = a;
  c.tb = 128 / a.G;
  const long long tokens = MODE == PROMPT ? a.total : (long long)a.n * a.rows;
  c.items = (int)(MODE == PROMPT ? prompt_slots(a.total, a.n_seq, 1, 2 * c.tb) : (tokens + 2 * c.tb - 1) / (2 * c.tb));
  c.box_rows = MODE == PROMPT ? BN : a.page;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_map_3d(&mq, a.q, a.dh, a.Hq, tokens, a.dh, a.q_ld, a.G, c.tb);
  if (MODE == PROMPT) {
    if (e == cudaSuccess) e = make_map_3d(&mk, a.k, a.dh, a.Hkv, a.total, a.dh, a.k_ld, 1, BN);
    if (e == cudaSuccess) e = make_map_3d(&mv, a.v, a.dh, a.Hkv, a.total, a.dh, a.v_ld, 1, BN);
  } else {
    const long long block = (long long)a.page * a.dh;
    if (e == cudaSuccess) e = make_map_3d(&mk, a.k, a.dh, a.page, (long long)a.n_pages * a.Hkv, a.dh, block, a.page, 1);
    if (e == cudaSuccess) e = make_map_3d(&mv, a.v, a.dh, a.page, (long long)a.n_pages * a.Hkv, a.dh, block, a.page, 1);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)c.items * a.Hkv), MODE == PROMPT ? 1 : a.npre);
  return a.dh == 128 ? launch_one<128, MODE>(c, mq, mk, mv, grid, st) : launch_one<64, MODE>(c, mq, mk, mv, grid, st);
}

}  // namespace

bool attn_tc_ok(int dtype, const AttnRows& a) {
  return dtype == HF_BF16 && (a.dh == 64 || a.dh == 128);
}
cudaError_t launch_attn_tc_prompt(const AttnRows& a, cudaStream_t st) { return launch_mode<PROMPT>(a, st); }
cudaError_t launch_attn_tc_prefix(const AttnRows& a, cudaStream_t st) { return launch_mode<PREFIX>(a, st); }

}  // namespace hf
