// Tensor-core attention (attn_tc.cu, attn_tc8.cu): what its kernels share. Instructions, bounded
// waits, and the items of a call over a paged cache.
#pragma once

#include "attn.cuh"
#include "tcgen05.cuh"

namespace hf {

constexpr int BN = kKeyTile;   // keys per tile
constexpr int TCT = 384;       // threads
constexpr int kNone = 0x7fffffff;

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

// 32 bytes at once: whole sectors of the L2.
__device__ __forceinline__ void store8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

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
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity) {
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
  int tb;          // tokens per row tile: its rows / G
  int blocks;      // prompt: slots of 2 tb tokens; paged: blocks of the prefix rows
  int box_rows;    // rows of a K / V box (prompt: 128, paged: the page)
  int pre_items;   // paged: items of the prefix
  int wide;        // rows of out start on 32 bytes
  int small;       // paged: every CTA plans for itself
  int busy, places; // 8-bit cache: launch_attn_tc8_pages
  int wait;        // 0: every wait gives up before it begins (set by a test)
};

// What a CTA works on at a time, written by warp 2. Tile r's rows are tokens
// tok0 + (split ? 0 : r tb) .. of KV head g + (split ? r : 0).
struct Item {
  int kind;        // 0 prompt, 1 prefix, 2 own keys, -1 the end
  int g, split;    // split: two KV heads with keys of their own; else the same keys
  int nt[2];       // key tiles of each row tile
  int j0, j1;      // keys
  int tok0, ntok;  // first row of q and out, tokens
  int t0;          // prompt, own: position of tok0 in its sequence or entry
  int start;       // prompt: row of key 0
  int entry, len;  // own: the entry and its tokens
  int direct;      // rows go to out
  int part;        // else: the prefix's piece, the own pieces' slot
  int low, hold;   // least number of keys that a row sees; keys behind `hold` read as zeros
  int odd[2];      // first key of a tile whose odd values of V were taken as zero
  // first key tile that holds keys which some row masks (so does every later one)
  __device__ __forceinline__ int first_cut() const {
    const int m = min(low, j1);
    return m < hold ? max(0, m - j0) / BN : kNone;
  }
};
static_assert(sizeof(Item) <= 80, "item slots");

// Item idx of the prefix.
__device__ __forceinline__ void make_prefix(const TcArgs& c, int idx, Item& it, const int* eff) {
  const AttnRows& a = c.a;
  it.split = 0;
  it.start = it.entry = it.len = it.part = 0;
  it.odd[0] = it.odd[1] = kNone;
  const int heads = (a.Hkv + 1) / 2;  // split: pairs of heads
  const int tokens = a.n * a.rows;
  it.kind = 1;
  it.split = tokens <= c.tb;
  if (it.split) {
    it.g = 2 * (idx % heads);
    it.part = idx / heads;
    it.t0 = 0;
  } else {
    it.t0 = idx % c.blocks * 2 * c.tb;
    it.g = idx / c.blocks % a.Hkv;
    it.part = idx / c.blocks / a.Hkv;
  }
  it.tok0 = it.t0;
  it.ntok = min(it.split ? c.tb : 2 * c.tb, tokens - it.t0);
  it.j0 = it.part * a.pre_keys;
  it.j1 = eff[0] ? min(a.shared, it.j0 + a.pre_keys) : it.j0;  // entry 0 empty: so is every row
  it.direct = 0;
  it.hold = it.j1;  // (whole pages)
  int low = kNone;  // an entry's first row sees least
  for (int e = it.t0 / a.rows + (threadIdx.x & 31); e * a.rows < it.t0 + it.ntok; e += 32) {
    const int row = max(e * a.rows, it.t0) - e * a.rows;
    if (eff[e] > 0) low = min(low, max(0, eff[e] - a.rows + row + 1));
  }
  it.low = __reduce_min_sync(0xffffffffu, low);
  const int nt = it.nt[0] = (it.j1 - it.j0 + BN - 1) / BN;
  it.nt[1] = (it.split ? it.g + 1 < a.Hkv : it.ntok > c.tb) ? nt : 0;
}

// The item at pos of the line, in the stretch [pos, end) of its CTA `cta`, if a tile lies
// there; the places that it takes are returned. eff, tile0: in shared memory or the
// workspace.
__device__ __forceinline__ int make_own(const TcArgs& c, const AttnLine& line, int cta, int pos, int end, Item& it,
                                        bool& some, const int* eff, const int* tile0) {
  const AttnRows& a = c.a;
  const int u = pos / line.tiles, at = pos - u * line.tiles;
  int lo = 0, hi = a.n;  // the last entry that starts at or before `at`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile0[mid] <= at)
      lo = mid;
    else
      hi = mid;
  }
  const int first = tile0[lo] + a.item_start, last = tile0[lo + 1], skip = max(0, first - at);
  const int take = min(end - pos, last - at) - skip, from = at + skip;
  some = take > 0;
  if (!some) return min(end - pos, skip);
  it.kind = 2;
  it.entry = lo;
  it.len = eff[lo];
  it.start = 0;
  it.odd[0] = it.odd[1] = kNone;
  it.split = a.rows <= c.tb;
  if (it.split) {
    it.g = 2 * u;
    it.t0 = 0;
  } else {
    it.g = u % a.Hkv;
    it.t0 = u / a.Hkv * 2 * c.tb;
  }
  it.tok0 = lo * a.rows + it.t0;
  it.ntok = min(it.split ? c.tb : 2 * c.tb, a.rows - it.t0);
  it.j0 = a.shared + (from - first) * BN;
  it.j1 = min(it.len, it.j0 + take * BN);
  it.low = max(0, it.len - a.rows + it.t0 + 1);
  it.hold = (it.j1 + a.page - 1) / a.page * a.page;
  it.direct = a.npre == 0 && line.cta(u * line.tiles + first) == line.cta(u * line.tiles + last - 1);
  it.part = u * a.n + lo + cta;
  it.nt[0] = take;
  it.nt[1] = (it.split ? it.g + 1 < a.Hkv : it.ntok > c.tb) ? take : 0;
  return skip + take;
}

// An item of the prefix, in tiles of own keys: its two row tiles share their keys (measured
// 1.56 us a tile), or are two heads with keys of their own (2.9 us), and end with more rows.
__device__ __forceinline__ int prefix_places(const AttnRows& a) {
  const int tiles = a.pre_keys / BN;
  return (a.n * a.rows <= a.tb ? tiles * 5 / 4 : tiles * 9 / 16) + 2;
}

// One warp: where the entries start on the line, from their lengths; all places returned.
__device__ __forceinline__ int scan_tiles(const AttnRows& a, const int* eff, int* tile0) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += 32) {
    const int i = i0 + lane;
    const int t = i < a.n ? entry_places(a, eff[i] - a.shared) : 0;
    int x = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (i < a.n) tile0[i] = carry + x - t;
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) tile0[a.n] = carry;
  __syncwarp();
  return carry;
}

cudaError_t launch_attn_plan(const AttnRows& a, int ctas, int heavy, cudaStream_t st);

}  // namespace hf
