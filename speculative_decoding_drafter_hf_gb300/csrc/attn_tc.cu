// Attention on the tensor cores (bf16, head dim 64 or 128): whole prompts, and the
// newest rows of requests over a paged cache, its common prefix read once for all.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(qscale s_ij - m_i),  s_ij = q_i.k_j
// in one pass over key tiles of 128 with a running m_i. A CTA works on two tiles of 128
// rows (rows are token * G + head in the group, so the group's heads share every key
// tile). tcgen05 forms S = Q K^T into TMEM; one thread per row reads its 128 scores and
// writes the weights back over them as bf16, and tcgen05 adds P V to the row's sums in
// TMEM, with P read from TMEM and V straight from its row-major tile. m_i is raised only
// when a tile's maximum passes it by more than 8 (a factor 2^8): until then nothing is
// rescaled, so for most tiles only the tensor cores touch the sums.
//
// While the softmax threads of one row tile work, the tensor cores work for the other.
// The two row tiles use the same keys (prompts, a prefix that more rows share than fit
// one tile), or, where one tile holds all rows, belong to two KV heads and have keys of
// their own. Warp 0 loads (TMA), warp 1 issues the products, warp 2 hands out items,
// warps 4-7 and 8-11 are the softmax groups; CTAs stay and take item after item, so that
// the next item's loads and first product run beside the last one's end. Prompt items are
// the launch's own CTAs, taken over from the ones not started yet, heaviest first (16
// prompts of 1 to 1969 tokens: in the order of the pack 15% more). Over a cache the
// prefix's items go round the CTAs, and what each has of the requests' own tiles is a
// stretch of one line (AttnLine).
//
// Bound by the chain scores - softmax - values of a row tile, of which two take turns on
// the tensor cores: about 2700 cycles for two row tiles and 128 keys, where the products
// alone take 2048 and the exponentials 1024. A prompt of 8192 tokens, 32 heads of 128 over
// 8: 367 us in a stream of calls on new inputs (1.50 PFLOP/s), 340 replayed on the same; heads
// of 64: 286, the softmax threads alone. Over a cache, by the reads: 64 requests of 4096
// tokens 165 to 172 us (6.2 to 6.5 TB/s), with pages of 16 tokens 215 us (5.0: a copy brings
// 4 KB).
//
// Masked keys: scores are selected by position. V's non-finite values in a tile that
// some row masks are set to zero in shared memory (0 * NaN would reach every row) and
// added back at the end to the rows that see them.
#include <atomic>
#include <mutex>

#include "attn_tc.cuh"

namespace hf {
namespace {

enum { PROMPT = 0, PAGED = 1 };

template <int DH>
struct Tc {
  static constexpr int TILE = BN * DH * 2;            // bytes of a K, V or Q tile
  static constexpr int SLOTS = DH == 128 ? 5 : 10;    // ring of K and V tiles
  static constexpr int O_COL = 256;                   // TMEM: S0 | S1 | O0 | O1
  static constexpr int BARS = 2 * SLOTS + 16;  // (an even number: 16 bytes for what comes behind)
  static constexpr size_t smem() { return (size_t)(2 + SLOTS) * TILE + BARS * 8 + 16 + 2 * 80 + 48 + (2 * kSmall + 2) * 4; }
};

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
__device__ __forceinline__ void take_next_cta(uint4* answer, uint64_t* bar) {
  mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// The index of the CTA taken over, or -1: all have started.
__device__ __forceinline__ int taken_cta(const uint4* answer) {
  int x = -1;
  uint32_t got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.b32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}\n"
      : "=&r"(x), "=&r"(got)
      : "r"(smem_u32(answer))
      : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return got ? x : -1;
}

// Prompts of a call with few sequences, in the order of their tiles' work: all last tiles
// of the longest, then those one tile shorter, and so on (a long sequence's tiles would
// else come wherever it stands in the pack). One warp; lane = sequence. Indices mostly
// come in rising order, so the search goes on from the last one.
constexpr int kSorted = 128;  // sequences
struct TileOrder {
  int start[kSorted / 32], len[kSorted / 32], tiles[kSorted / 32];
  int top, p, before;  // highest position; `before` tiles are at positions above p

  __device__ __forceinline__ void init(const AttnRows& a, int tokens) {
    int most = 0;
#pragma unroll
    for (int k = 0; k < kSorted / 32; ++k) {
      const int s = (threadIdx.x & 31) + 32 * k;
      const int s0 = s < a.n_seq ? a.off[s] : 0, s1 = s < a.n_seq ? a.off[s + 1] : 0;
      const bool ok = s0 >= 0 && s0 <= s1 && s1 <= a.total;
      start[k] = s0;
      len[k] = ok ? s1 - s0 : 0;
      tiles[k] = (len[k] + tokens - 1) / tokens;
      most = max(most, tiles[k]);
    }
    p = top = __reduce_max_sync(0xffffffffu, most) - 1;
    before = 0;
  }
  // Tile number i, ok = false behind the last one.
  __device__ __forceinline__ PromptTile at(int i) {
    PromptTile t{};
    if (i < before) {
      p = top;
      before = 0;
    }
    while (p >= 0) {
      uint32_t has[kSorted / 32];
      int count = 0;
#pragma unroll
      for (int k = 0; k < kSorted / 32; ++k) {
        has[k] = __ballot_sync(0xffffffffu, tiles[k] > p);
        count += __popc(has[k]);
      }
      int j = i - before;
      if (j >= count) {
        before += count;
        --p;
        continue;
      }
#pragma unroll
      for (int k = 0; k < kSorted / 32; ++k) {
        const int n = __popc(has[k]);
        if (j >= 0 && j < n) {
          const int lane = __fns(has[k], 0, j + 1);
          t.start = __shfl_sync(0xffffffffu, start[k], lane);
          t.len = __shfl_sync(0xffffffffu, len[k], lane);
        }
        j -= n;
      }
      t.tile = p;
      t.ok = true;
      return t;
    }
    return t;
  }
};

// The item of tile t, if there is one.
__device__ __forceinline__ bool make_prompt(const TcArgs& c, int idx, Item& it, const PromptTile& t) {
  const AttnRows& a = c.a;
  it.split = 0;
  it.start = it.entry = it.len = it.part = 0;
  it.odd[0] = it.odd[1] = kNone;
  if (!t.ok) return false;
  it.kind = 0;
  it.g = idx % a.Hkv;
  it.t0 = t.tile * 2 * c.tb;
  it.start = t.start;
  it.tok0 = t.start + it.t0;
  it.ntok = min(2 * c.tb, t.len - it.t0);
  it.j0 = 0;
  it.j1 = it.t0 + it.ntok;
  it.direct = 1;
  it.low = it.t0 + 1;
  it.hold = kNone;
  const int nt = (it.j1 + BN - 1) / BN;
  // the first row tile ends earlier
  it.nt[0] = min(nt, (min(it.j1, it.t0 + c.tb) + BN - 1) / BN);
  it.nt[1] = it.ntok > c.tb ? nt : 0;
  return true;
}

// Element offset in V of key j's row of KV head g.
template <int MODE>
__device__ __forceinline__ long long v_at(const AttnRows& a, const Item& it, int g, int j) {
  if (MODE == PROMPT || a.dense) return (long long)(it.start + j) * a.v_ld + (long long)g * a.dh;
  const int id = attn_table(a, it.entry)[j / a.page];
  if (id < 0 || id >= a.n_pages) return -1;
  return (((long long)id * a.Hkv + g) * a.page + j % a.page) * a.dh;
}

// What a row's column d gets from V's non-finite values at keys [j0, j1).
template <int MODE>
__device__ __noinline__ float odd_sum(const AttnRows& a, const Item& it, int g, int j0, int j1, int d) {
  float s = 0.f;
  for (int j = j0; j < j1; ++j) {
    const long long at = v_at<MODE>(a, it, g, j);
    if (at < 0) continue;
    const float x = to_f(static_cast<const __nv_bfloat16*>(a.v)[at + d]);
    if (!(fabsf(x) < INFINITY)) s += x;
  }
  return s;
}

template <int DH, int MODE>
__global__ void __launch_bounds__(TCT, 1)
tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv, const __grid_constant__ TcArgs c) {
  using L = Tc<DH>;
  constexpr int NS = L::SLOTS, HALVES = DH / 64, HALF = BN * 128;
  const AttnRows& a = c.a;
  // (no other shared memory in this kernel: the tiles start at the alignment that their swizzle needs)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * L::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + (size_t)NS * L::TILE);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;   // [2]
  uint64_t* p_full = q_full + 4;   // [2]
  uint64_t* o_full = q_full + 6;   // [2]
  uint64_t* i_full = q_full + 8;   // [2] items
  uint64_t* i_empty = q_full + 10; // [2]
  uint64_t* n_full = q_full + 12;  // the next CTA's index has come
  uint64_t* drained = q_full + 13; // after a wait that ran out: the products have ended
  uint4* answer = reinterpret_cast<uint4*>(full + L::BARS);
  Item* items = reinterpret_cast<Item*>(answer + 1);  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(items + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;  // [0] tiles, [1] row-tile loads that the loader has asked for
  int* s_eff = const_cast<int*>(issued) + 2;  // small calls: [kSmall] lengths, [kSmall + 1] places on the line
  int* s_tile0 = s_eff + kSmall;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool beside = MODE == PAGED && a.dense;
  if (!beside) pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(n_full, 1);
    mbar_init(drained, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&o_full[g], 1);
      mbar_init(&i_full[g], 1);
      mbar_init(&i_empty[g], 10);  // the loader, the products, eight softmax warps
    }
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (tid >= 64 && tid < 67) {  // (the first copies would wait for them)
    const CUtensorMap* map = tid == 64 ? &mq : tid == 65 ? &mk : &mv;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // The launch directly behind a dense prefix reads the cache and the rows before it waits (attn_tc8.cu, c.busy): it comes
  // once all CTAs are here, so when what ran before them has ended and its writes are in memory. It relies on this order.
  if (beside) pdl_trigger();
  if (MODE == PROMPT && blockIdx.x == 0) check_offsets(a, tid, TCT);
  __syncwarp();  // (its lanes' loops end apart, and the next instruction wants the warp together)

  if (c.wait == 0) {
    *abort_flag = 1;
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---- loads: a stream's K(0), the rows, then V(j), K(j+1) through the ring
      int ri = 0, qn = 0;  // tiles, row-tile loads so far
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item& it = items[n & 1];
        ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!ok || it.kind < 0) break;
        const int nt0 = it.nt[0], nt1 = it.nt[1], nt = max(nt0, nt1), j1 = it.j1, split = it.split, g = it.g;
        const int32_t* tab = MODE == PROMPT ? nullptr : attn_table(a, it.entry);
        const int nbox = HALVES * (BN / c.box_rows);
        auto tile = [&](int j, int r, bool is_v) {  // tile j of stream r
          if (!ok) return;
          const int s = ri % NS;
          if (ri >= NS) ok = wait_uniform(smem_u32(&empty[s]), ((uint32_t)(ri / NS) & 1u) ^ 1u);
          if (!ok || *abort_flag) {
            ok = false;
            return;
          }
          if (lane == 0) mbar_expect_tx(&full[s], L::TILE);
          __syncwarp();
          if (lane < nbox) {
            const int h = lane % HALVES, b = lane / HALVES;
            const int key = it.j0 + j * BN + b * c.box_rows;
            uint8_t* dst = sKV + (size_t)s * L::TILE + h * HALF + b * c.box_rows * 128;
            if (MODE == PROMPT || a.dense) {
              tma_load_3d(dst, is_v ? &mv : &mk, &full[s], h * 64, g + r, it.start + key);
            } else {
              int z = a.n_pages * a.Hkv;  // behind the pool: reads zeros
              if (key < j1) {
                const int id = tab[key / a.page];
                if (id >= 0 && id < a.n_pages)
                  z = id * a.Hkv + g + r;
                else if (a.status)
                  atomicOr(a.status, HF_S_BAD);
              }
              tma_load_3d(dst, is_v ? &mv : &mk, &full[s], h * 64, 0, z);
            }
          }
          ++ri;
        };
        if (nt > 0) {
          tile(0, 0, false);
          if (split && nt1 > 0) tile(0, 1, false);
          if (ok && qn > 0) ok = wait_uniform(smem_u32(q_empty), (uint32_t)(qn - 1) & 1u);
          if (ok && lane == 0) {
            const int tiles = nt1 > 0 ? 2 : 1;
            mbar_expect_tx(q_full, (uint32_t)(tiles * HALVES * c.tb * a.G) * 128u);
            for (int r = 0; r < tiles; ++r)
              for (int h = 0; h < HALVES; ++h)
                tma_load_3d(sQ + r * L::TILE + h * HALF, &mq, q_full, h * 64, (g + (split ? r : 0)) * a.G,
                            it.tok0 + (split ? 0 : r * c.tb));
          }
          if (ok) ++qn;
          for (int j = 0; j < nt && ok; ++j) {
            const int streams = split && nt1 > 0 ? 2 : 1;
            for (int r = 0; r < streams; ++r) {
              tile(j, r, true);
              if (j + 1 < nt) tile(j + 1, r, false);
            }
          }
        }
        if (lane == 0) mbar_arrive(&i_empty[n & 1]);
      }
      if (lane == 0) {
        issued[0] = ri;
        issued[1] = qn;
        if (!ok) *abort_flag = 1;
      }
    } else if (warp == 1) {
      // ---- products: S_r(0), then P V_r(j), S_r(j+1) for r = 0, 1 in turn
      constexpr uint32_t id_s = idesc_bf16(BN);
      constexpr uint32_t id_o = idesc_bf16(DH) | (1u << 16);
      const uint32_t lead = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t aq = desc_lo(smem_u32(sQ)), ak = desc_lo(smem_u32(sKV)), av = desc_lo_rows(smem_u32(sKV));
      const uint32_t b_full = smem_u32(full), b_empty = smem_u32(empty), b_s = smem_u32(s_full), b_p = smem_u32(p_full),
                     b_o = smem_u32(o_full);
      int at = 0;           // next slot of the ring, and the parity of its fill
      uint32_t ph = 0, qph = 0, pph[2] = {0, 0};
      bool ok = true;
      auto next = [&]() {  // waits for the next slot of the ring
        const int s = at;
        ok = ok && wait_uniform(b_full + 8 * s, ph);
        if (++at == NS) {
          at = 0;
          ph ^= 1u;
        }
        return s;
      };
      auto score = [&](int r, int slot) {
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint32_t step = (uint32_t)((k / 4) * (HALF >> 4) + (k % 4) * 2);
          mma_ss(lead, tm + r * BN, aq + r * (L::TILE >> 4) + step, ak + slot * (L::TILE >> 4) + step, id_s, k > 0);
        }
        mma_commit(lead, b_s + 8 * r);
      };
      for (int n = 0; ok; ++n) {
        const Item& it = items[n & 1];
        ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!ok || __shfl_sync(0xffffffffu, it.kind, 0) < 0) break;
        const int nt0 = __shfl_sync(0xffffffffu, it.nt[0], 0), nt1 = __shfl_sync(0xffffffffu, it.nt[1], 0);
        const bool two = MODE == PAGED && __shfl_sync(0xffffffffu, it.split, 0) && nt1 > 0;  // two streams of keys
        const int nt = max(nt0, nt1);
        if (nt > 0) {
          int ks = next();
          int ks1 = two ? next() : ks;
          ok = ok && wait_uniform(smem_u32(q_full), qph);
          qph ^= 1u;
          if (ok) {
            tc_fence_after();
            score(0, ks);
            if (two) mma_commit(lead, b_empty + 8 * ks);
            if (nt1 > 0) score(1, ks1);
            mma_commit(lead, b_empty + 8 * ks1);
            if (nt == 1) mma_commit(lead, smem_u32(q_empty));
          }
          int vs = 0;
          // from tile `look` on the softmax groups look V over before they hand their weights
          // on; where both have the tile, each looks at half of it
          const int look = __shfl_sync(0xffffffffu, it.first_cut(), 0);
          for (int j = 0; j < nt && ok; ++j) {
            const bool more = j + 1 < nt;
            if (!two) {
              vs = next();
              if (more) ks = next();
            }
            const bool both = !two && j >= look && j < nt0 && j < nt1;
            if (both) ok = ok && wait_uniform(b_p, pph[0]) && wait_uniform(b_p + 8, pph[1]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int mine = r ? nt1 : nt0;
              if (!ok || j >= mine) continue;
              if (two) vs = next();
              if (!both) ok = ok && wait_uniform(b_p + 8 * r, pph[r]);
              pph[r] ^= 1u;
              if (!ok) continue;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < BN / 16; ++k)
                mma_ts(lead, tm + L::O_COL + r * DH, tm + r * BN + k * 8, av + vs * (L::TILE >> 4) + k * (2048 >> 4),
                       id_o, j > 0 || k > 0);
              mma_commit(lead, b_o + 8 * r);
              if (two) mma_commit(lead, b_empty + 8 * vs);
              if (j + 1 < mine) {
                if (two) ks = next();
                if (!ok) continue;
                tc_fence_after();
                score(r, ks);
                if (two) mma_commit(lead, b_empty + 8 * ks);
              }
            }
            if (ok) {
              if (!two) {
                mma_commit(lead, b_empty + 8 * vs);
                if (more) mma_commit(lead, b_empty + 8 * ks);
              }
              if (j + 2 == nt) mma_commit(lead, smem_u32(q_empty));  // the last scores are on their way
            }
          }
        }
        if (lane == 0) mbar_arrive(&i_empty[n & 1]);
      }
      if (!ok) *abort_flag = 1;
    } else if (warp == 2) {
      // ---- items
      bool ok = true;
      int n = 0;
      auto put = [&](const Item& it) {
        if (n >= 2) ok = wait_uniform(smem_u32(&i_empty[n & 1]), ((uint32_t)(n >> 1) & 1u) ^ 1u);
        if (!ok) return;
        if (lane == 0) {
          items[n & 1] = it;
          mbar_arrive(&i_full[n & 1]);
        }
        ++n;
      };
      Item it;
      if (MODE == PROMPT) {
        int idx = blockIdx.x, taken = 0;
        TileOrder order;
        if (a.n_seq <= kSorted) order.init(a, 2 * c.tb);
        while (ok && idx >= 0) {
          if (lane == 0) take_next_cta(answer, n_full);
          const PromptTile t = a.n_seq <= kSorted ? order.at(idx / a.Hkv)
                                                  : prompt_tile(a, c.blocks - 1 - idx / a.Hkv, 2 * c.tb, 1);
          if (make_prompt(c, idx, it, t)) put(it);
          // (also after a failure: the answer asked for lands before the CTA goes)
          const bool came = wait_uniform(smem_u32(n_full), (uint32_t)taken & 1u);
          ++taken;
          idx = came ? taken_cta(answer) : -1;
          ok = ok && came;
          if (idx == 0) check_offsets(a, lane, 32);  // (CTA 0 never starts then)
          __syncwarp();
        }
      } else {
        const int me = blockIdx.x, all = gridDim.x;
        const int *eff = a.eff, *tile0 = a.tile0;
        if (c.small) {
          bool bad = false;
          for (int i = lane; i < a.n; i += 32) {
            s_eff[i] = attn_len(a, i, bad);
            if (me == 0) a.eff[i] = s_eff[i];
          }
          if (bad && a.status && me == 0) atomicOr(a.status, HF_S_BAD);
          eff = s_eff;
          tile0 = s_tile0;
          __syncwarp();
        }
        for (int idx = me; ok && idx < c.pre_items; idx += all) {
          make_prefix(c, idx, it, eff);
          put(it);
        }
        const int heavy = c.pre_items % all;
        AttnLine line;
        if (c.small) {
          line = make_line(scan_tiles(a, s_eff, s_tile0), a.units, all, heavy, prefix_places(a));
          if (me == 0) {
            for (int i = lane; i <= a.n; i += 32) a.tile0[i] = s_tile0[i];
            if (lane == 0) *reinterpret_cast<AttnLine*>(a.line) = line;
          }
        } else {
          line = *reinterpret_cast<const AttnLine*>(a.line);
        }
        const int cta = (me - heavy + all) % all, end = min(line.start(cta + 1), line.tiles * a.units);
        for (int pos = line.start(cta); ok && pos < end;) {
          bool some;
          pos += make_own(c, line, cta, pos, end, it, some, eff, tile0);
          if (some) put(it);
        }
      }
      it.kind = -1;
      if (ok) put(it);
      if (!ok) *abort_flag = 1;
    } else if (MODE == PAGED && c.small) {
      check_prefixes(a, 1 + blockIdx.x, gridDim.x, lane, 32);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- softmax: one thread per row
    const int r = warp >= 8, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + r * BN, to = tmem + lanes + L::O_COL + r * DH;
    const uint32_t b_s = smem_u32(&s_full[r]), b_o = smem_u32(&o_full[r]);
    const int row_tok = row / c.a.G, row_head = row % c.a.G;
    int tiles = 0;  // key tiles of this row tile so far, and all tiles of the ring
    int ring = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      Item& it = items[n & 1];
      ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
      if (!ok || it.kind < 0) break;
      const int split = it.split, mine = it.nt[r], j0 = it.j0, j1 = it.j1;
      const int g = it.g + (split ? r : 0);
      const int tl = (split ? 0 : r * c.tb) + row_tok;  // token within the item
      // a row of its own in out (also where there is no key at all)
      const bool valid = row < c.tb * a.G && tl < it.ntok && g < a.Hkv;
      const size_t orow = (size_t)it.tok0 + tl;
      const int head = g * a.G + row_head;
      int limit = kNone;   // keys below it are seen (rows without a token: all, and dropped)
      bool dead = false;   // an entry without tokens
      if (valid) {
        if (MODE == PROMPT) {
          limit = it.t0 + tl + 1;
        } else {
          const int t = it.t0 + tl;
          const int len = it.kind == 1 ? (c.small ? s_eff[t / a.rows] : __ldcg(&a.eff[t / a.rows])) : it.len;
          dead = len == 0;
          if (!dead) limit = max(0, len - a.rows + (it.kind == 1 ? t % a.rows : t) + 1);
        }
      }
      const bool any = __any_sync(0xffffffffu, valid);
      const int lim = min(limit, j1), wlow = __reduce_min_sync(0xffffffffu, lim);
      const int streams = split && it.nt[1] > 0 ? 2 : 1, look = it.first_cut();
      float mb = -INFINITY, l = 0.f;  // maximum in use, times qscale; sum of the weights
      for (int j = 0; j < mine; ++j) {
        const int jt = j0 + j * BN;
        ok = wait_uniform(b_s, (uint32_t)(tiles + j) & 1u);
        if (!ok) break;
        tc_fence_after();
        if (any) {
          float s[BN];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s + q * 32);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_hold32(s + q * 32);
          if (jt + BN > wlow) {
            const int seen = lim - jt;  // keys of this tile
#pragma unroll
            for (int h = 0; h < BN; h += 32) {
              // bits rather than comparisons: a register of them becomes predicates at once
              const uint32_t bits = seen >= h + 32 ? 0xffffffffu : seen <= h ? 0u : (1u << (seen - h)) - 1u;
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (!(bits >> q & 1)) s[h + q] = -INFINITY;
            }
          }
          float t8[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) t8[q] = fmaxf(s[q], s[q + 8]);
#pragma unroll
          for (int q = 16; q < BN; q += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) t8[k] = max3(t8[k], s[q + k], s[q + k + 8]);
          const float top = max3(max3(t8[0], t8[1], t8[2]), max3(t8[3], t8[4], t8[5]), fmaxf(t8[6], t8[7])) * a.qscale;
          const bool lift = top > mb + 8.f;
          if (__any_sync(0xffffffffu, lift)) {
            // (mb = -infinity: the sums are zero, or not written yet)
            const float nm = lift ? top : mb;
            const float f = mb > -INFINITY ? ex2(mb - nm) : 1.f;
            if (j > 0 && __any_sync(0xffffffffu, lift && mb > -INFINITY)) {
              ok = wait_uniform(b_o, (uint32_t)(tiles + j - 1) & 1u);
              if (!ok) break;
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
          const uint64_t qs2 = pair(a.qscale, a.qscale), base2 = pair(-base, -base);
          uint64_t l2[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              float2 e = unpair(fma2(pair(s[h * 64 + 2 * q], s[h * 64 + 2 * q + 1]), qs2, base2));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              l2[q & 1] = add2(l2[q & 1], pair(e.x, e.y));
              p[q] = pack_bf16(e.x, e.y);
            }
            tmem_st32(ts + h * 32, p);
          }
          const float2 la = unpair(l2[0]), lb = unpair(l2[1]);
          l += (la.x + la.y) + (lb.x + lb.y);
          tmem_wait_st();
        }
        if (j >= look) {
          // some row masks keys that the tile holds
          const int nt = max(it.nt[0], it.nt[1]);
          const int vi = ring + (streams == 1 ? 1 + 2 * j : 2 + 4 * j + (j + 1 < nt ? 2 * r : r)), vs = vi % NS;
          ok = wait_uniform(smem_u32(&full[vs]), (uint32_t)(vi / NS) & 1u);
          if (!ok) break;
          uint4* v = reinterpret_cast<uint4*>(sKV + (size_t)vs * L::TILE);
          // rows (keys) k0 .. k1 - 1 of the tile, a half of 64 columns after the other
          const int k0 = max(0, min(it.low, j1) - jt), k1 = min(BN, it.hold - jt), per = (k1 - k0) * 8;
          const bool both = streams == 1 && j < it.nt[0] && j < it.nt[1];
          const int step = both ? 256 : 128;
          for (int q0 = both ? r * 128 + row : row; q0 < per * HALVES; q0 += 4 * step) {
            uint4 x[4];
            auto at = [&](int u) {
              const int q = q0 + u * step, h = q >= per;
              return v + h * (HALF / 16) + k0 * 8 + (q - h * per);
            };
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = q0 + u * step < per * HALVES ? *at(u) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t* w = reinterpret_cast<uint32_t*>(&x[u]);
              // an exponent of all ones carries into its half's top bit
              uint32_t hit[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) hit[k] = ((w[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
              if (hit[0] | hit[1] | hit[2] | hit[3]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] &= ~((hit[k] >> 15) * 0xffffu);
                atomicMin(&it.odd[streams == 1 ? 0 : r], jt);
                *at(u) = x[u];
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[r]);
      }
      if (!ok) break;
      // ---- the item's end
      if (mine > 0) {
        ok = wait_uniform(b_o, (uint32_t)(tiles + mine - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
      }
      tiles += mine;
      ring += 2 * max(it.nt[0], it.nt[1]) * streams;
      if (any) {
        const bool direct = it.direct;
        const float inv = l == 0.f || dead ? 0.f : 1.f / l;
        const int from = *(volatile int*)&it.odd[streams == 1 ? 0 : r];
        PartAt at{};
        if (MODE == PAGED)
          at = it.kind == 1 ? part_prefix(a, it.part, g, it.t0 + tl, row_head)
                            : part_own_unit(a, it.part, g, it.t0 + tl, row_head);
#pragma unroll 1
        for (int q = 0; q < DH; q += 32) {
          __syncwarp();  // (lanes without a row come back early: the load wants the warp together)
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
#pragma unroll 1
            for (int k = 0; k < 32; ++k) {
              const float x = odd_sum<MODE>(a, it, g, from, lim, q + k);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = i == k ? o[i] + x : o[i];
            }
          if (!valid) continue;
          if (direct) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + orow * a.out_ld + (size_t)head * DH + q;
            uint32_t w[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) w[x] = dead ? 0u : pack_bf16(o[2 * x] * inv, o[2 * x + 1] * inv);
            if (c.wide) {
              store8(dst, w);
              store8(dst + 16, w + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                reinterpret_cast<uint4*>(dst)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
          } else if (mine > 0) {
            float* dst = a.part_o + at.first * DH + ((size_t)(q / 8) * at.region + at.row) * 8;
#pragma unroll
            for (int k = 0; k < 4; ++k) store8(dst + (size_t)k * at.region * 8, reinterpret_cast<uint32_t*>(o) + 8 * k);
          }
        }
        if (!direct && valid)
          a.part_ml[at.first + at.row] = dead || mine == 0 ? make_float2(-INFINITY, 0.f) : make_float2(mb, l);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[n & 1]);
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {
    // the lengths and the line that the join reads may be missing: it takes entries without
    // tokens for empty, and looks at nothing else of them
    if (MODE == PAGED && c.small && blockIdx.x == 0)
      for (int i = tid; i < a.n; i += TCT) a.eff[i] = 0;
    if (warp == 1) {  // the products still in flight end before their operands and TMEM go
      mma_commit(elect_one(), smem_u32(drained));  // (the lane that issued them)
      wait_uniform(smem_u32(drained), 0);
    }
    if (tid == 0) {
      if (a.status) atomicOr(a.status, HF_S_TIMEOUT);
      // the copies still in flight land before the CTA's shared memory goes
      if (issued[1] > 0) mbar_wait(q_full, (uint32_t)(issued[1] - 1) & 1u);
      for (int i = max(0, issued[0] - NS); i < issued[0]; ++i) mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Which entries the call sees, and the line of their tiles: one CTA for the lengths and
// the places on the line, the others compare the entries' prefixes.
__global__ void __launch_bounds__(1024) plan_kernel(AttnRows a, int ctas, int heavy) {
  __shared__ int s_scan[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x > 0) {
    check_prefixes(a, blockIdx.x, gridDim.x - 1, tid, 1024);
    return;
  }
  bool bad = false;
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += 1024) {
    const int i = i0 + tid;
    int t = 0;
    if (i < a.n) {
      const int len = attn_len(a, i, bad);
      a.eff[i] = len;
      t = entry_places(a, len - a.shared);
    }
    int x = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int before = carry, sum = carry;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_scan[w];
      sum += s_scan[w];
    }
    if (i < a.n) a.tile0[i] = before + x - t;
    carry = sum;
  }
  if (bad && a.status) atomicOr(a.status, HF_S_BAD);
  if (tid == 0) {
    a.tile0[a.n] = carry;
    *reinterpret_cast<AttnLine*>(a.line) = make_line(carry, a.units, ctas, heavy, prefix_places(a));
  }
}

constexpr int kMaxDev = 64;
std::mutex g_mu;
bool g_set[kMaxDev][2][2] = {};
std::atomic<long long> g_wait{kWaitCycles};

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

}  // namespace

void set_target_wait_limit(long long cycles) { g_wait.store(cycles); }
bool attn_gives_up() { return g_wait.load() <= 0; }

bool attn_tc_ok(int dtype, int dh) { return dtype == HF_BF16 && (dh == 64 || dh == 128); }

namespace {
int wide_rows(const AttnRows& a) { return reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_ld % 16 == 0; }
}  // namespace

cudaError_t launch_attn_tc_prompt(const AttnRows& a, cudaStream_t st) {
  TcArgs c{};
  c.a = a;
  c.wide = wide_rows(a);
  c.wait = !attn_gives_up();
  c.tb = kTileRows / a.G;
  c.blocks = (int)prompt_slots(a.total, a.n_seq, 1, 2 * c.tb);
  c.box_rows = BN;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_map_3d(&mq, a.q, a.dh, a.Hq, a.total, a.dh, a.q_ld, a.G, c.tb);
  if (e == cudaSuccess) e = make_map_3d(&mk, a.k, a.dh, a.Hkv, a.total, a.dh, a.k_ld, 1, BN);
  if (e == cudaSuccess) e = make_map_3d(&mv, a.v, a.dh, a.Hkv, a.total, a.dh, a.v_ld, 1, BN);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)c.blocks * a.Hkv));
  return a.dh == 128 ? launch_one<128, PROMPT>(c, mq, mk, mv, grid, st)
                     : launch_one<64, PROMPT>(c, mq, mk, mv, grid, st);
}

cudaError_t launch_attn_plan(const AttnRows& a, int ctas, int heavy, cudaStream_t st) {
  const int checks = a.shared > 0 && a.status ? std::min(a.n, 151) : 0;
  return launch_pdl(plan_kernel, dim3(1 + checks), dim3(1024), 0, st, a, ctas, heavy);
}

void attn_tc_sizes(AttnRows& a, int& pre_items, long long& slots) {
  const int tb = a.tile / a.G, heads = (a.Hkv + 1) / 2;
  const long long tokens = (long long)a.n * a.rows;
  const long long blocks = (tokens + 2 * tb - 1) / (2 * tb);
  const long long per = tokens <= tb ? heads : blocks * a.Hkv;  // items of one piece of the prefix
  a.tb = tb;
  a.units = a.rows <= tb ? heads : (a.rows + 2 * tb - 1) / (2 * tb) * a.Hkv;
  a.unit_rows = (a.rows <= tb ? 2 * a.rows : 2 * tb) * a.G;
  a.npre = 0;
  a.pre_keys = BN;
  if (a.shared > 0) {
    // pieces of the prefix: the least of (rounds of items over the SMs) * (tiles of a piece,
    // an item's start and end) plus what a piece costs to write and join
    const int tiles = (a.shared + BN - 1) / BN;
    double best = 1e30;
    for (int p = 1; p <= 64 && p <= tiles; ++p) {
      const int each = (tiles + p - 1) / p;
      const double rounds = (double)((per * p + 151) / 152);
      const double cost = rounds * (each + 2) + 0.02 * (double)p * (double)tokens * a.Hq * a.dh / (152 * 4096.0);
      if (cost < best) {
        best = cost;
        a.npre = (tiles + each - 1) / each;
        a.pre_keys = each * BN;
      }
    }
  }
  pre_items = (int)(per * a.npre);
  slots = (long long)a.units * a.n + 152;
}

cudaError_t launch_attn_tc_pages(const AttnRows& a, int pre_items, cudaStream_t st) {
  TcArgs c{};
  c.a = a;
  c.tb = a.tb;
  const long long tokens = (long long)a.n * a.rows, block = (long long)a.page * a.dh;
  c.blocks = (int)((tokens + 2 * c.tb - 1) / (2 * c.tb));
  c.box_rows = a.dense ? BN : a.page;
  c.wide = wide_rows(a);
  c.wait = !attn_gives_up();
  c.pre_items = pre_items;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_map_3d(&mq, a.q, a.dh, a.Hq, tokens, a.dh, a.q_ld, a.G, c.tb);
  if (a.dense) {
    if (e == cudaSuccess) e = make_map_3d(&mk, a.k, a.dh, a.Hkv, a.shared, a.dh, a.k_ld, 1, BN);
    if (e == cudaSuccess) e = make_map_3d(&mv, a.v, a.dh, a.Hkv, a.shared, a.dh, a.v_ld, 1, BN);
  } else {
    if (e == cudaSuccess) e = make_map_3d(&mk, a.k, a.dh, a.page, (long long)a.n_pages * a.Hkv, a.dh, block, a.page, 1);
    if (e == cudaSuccess) e = make_map_3d(&mv, a.v, a.dh, a.page, (long long)a.n_pages * a.Hkv, a.dh, block, a.page, 1);
  }
  if (e != cudaSuccess) return e;
  // (the line is at most as long as all tables reach)
  const long long reach = (((long long)a.table_ld * a.page - a.shared + BN - 1) / BN + a.item_start) * a.n * a.units;
  const int grid = (int)std::min<long long>(std::max<long long>(pre_items + reach, 1), 152);
  c.small = a.n <= kSmall;
  if (!c.small) e = launch_attn_plan(a, grid, pre_items % grid, st);
  if (e != cudaSuccess) return e;
  return a.dh == 128 ? launch_one<128, PAGED>(c, mq, mk, mv, dim3(grid), st)
                     : launch_one<64, PAGED>(c, mq, mk, mv, dim3(grid), st);
}

}  // namespace hf
