// Attention of the newest rows over the 8-bit cache on the tensor cores (bf16 rows, head dim 64 or
// 128), its common prefix read once for all.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  s_ij = c_i ks_j (q_i . k_j),  p_ij = 2^s_ij
// with k_j, v_j codes, ks_j, vs_j the scales of their pages, q_i a row in units of its own scale. The
// codes are operands of the tensor cores as they come from memory (kind::f8f6f4): nothing turns them into a
// wider type. The products are formed the other way round, keys along the 128 lanes of TMEM:
//   S' = K Q'  (128 keys x rows),   O' += V' W  (head dim x rows),   w_ij = p_ij vs_j 2^-M_i
// so that a tile's work goes by its rows (4 of a decoded token, 32 of 8 verified ones) and not by 128, and
// a softmax thread has a key: one scale of K, one of V, one position to compare, for all rows.
//
// Rows and weights have more bits than a code. A row goes in as two codes, hi = its nearest, lo = the
// nearest of 16 times the rest, side by side as columns of one product; of the two columns of the result the
// second counts a sixteenth: a bf16 row exactly, down to 2^-22 of its largest value.
//
// A weight goes in as three e5m2 codes of 3 bits, each 8 times finer than the one before:
// 9 bits down to 2^-14, and what is below 2^-23 is lost. The room below the largest weight matters: where
// one key holds most of a row's sum, the others' weights, though thousands of them make up the output, are
// 2^-10 to 2^-25 of it (two e4m3 codes, which end at 2^-15 of the largest weight, were off by 0.03 to 0.6 of such
// outputs; V as 16-bit floats in shared memory against 16-bit weights is exact as well, but moves four times
// V's bytes through it: 64 x 1 row over 4096 tokens 106 us). M_i is set by an item's first tile, to where the largest weight
// is 2^10, and raised to there when one passes 2^15 (that needs the maximum over the 128 threads, so most tiles only vote on
// it; to 2^8 64 x 8 rows over 4096 tokens take 119 us, to 2^10 121, to 2^12 127): weights keep 9 bits down to 2^-24 of the item's
// largest one at least, and end at 2^-33 of it. Sums, maxima and TMEM are fp32; the sum of p_ij is kept per thread, as w_ij / vs_j before it is rounded, and joined at an item's end.
//
// The CTA's warps, items, the line of own tiles and the parts are those of attn_tc.cu: warp 0 loads
// (TMA; the scales by 4-byte copies beside V's pages), warp 1 issues the products, warp 2 hands out
// items, warps 4-7 and 8-11 are the softmax groups of two row tiles of up to 48 rows (heads of more than 48 to a KV
// head: 64, whose scores share TMEM, so that the groups take turns). While an item is worked
// on, warp 3 turns the next one's rows into codes, if a row tile has 16 at most (one warp took longer than
// an item for more: 64 x 8 rows over 4096 tokens 136 us), or fetches them, if 32; else the groups do it when they
// come to it. Row tiles of two KV heads read pages that lie side by
// side: one copy brings both, eight rows of one, eight of the other (4 KB for a page of 16 tokens; 64 x 1
// rows over 4096 tokens with such pages 105 us instead of 125, and 96 now).
//
// Bound by the reads where requests are long: 64 requests of 2048 to 32768 tokens, one row of 40 heads over 10 each,
// 285 us (6.6 TB/s, as a copy). Shorter ones by what an item costs beside its
// tiles (about 17000 cycles for 32 rows, 8000 for 5: codes, waits, joining the sums, storing; the first of a CTA twice
// that, as its instructions come from the L2) and tiles by their chain (64 x 8 rows over 4096 tokens 121 us, 4.5
// TB/s; 4 us of them for the third code of a weight). Heads of 64, 64 x 1 rows over 4096 tokens: 74 us (3.6 TB/s), 65 with two
// codes; there neither a longer ring, nor a second loading warp made it faster.
#include <cudaTypedefs.h>

#include <mutex>

#include "attn_tc.cuh"
#include "e4m3.cuh"

namespace hf {
namespace {

constexpr float kLift = 15.f, kLifted = 10.f;
constexpr float kFine = 16.f;       // a row's lo is held times this
constexpr float kFinerW = 8.f;      // a weight's second code times this, its third times the square

constexpr int kItems = 160;  // bytes of two items: what comes behind them starts on 16 bytes
static_assert(2 * sizeof(Item) <= kItems, "item slots");

// NM: sixteens of rows of the largest row tile.
template <int DH, int NM>
struct Tc8 {
  static constexpr int NR = NM * 16;                  // rows of a row tile
  static constexpr int TILE = BN * DH;                // bytes of a K or V tile
  static constexpr int Q = 2 * NM * 16 * DH;          // bytes of a row tile's codes
  static constexpr bool AHEAD = NM == 1;              // warp 3 makes the codes, of two items at a time
  static constexpr int QN = AHEAD ? 2 : 1;
  static constexpr int RAW = NM == 2 ? 2 * 32 * DH * 2 : 0;  // rows as warp 3 fetches them
  static constexpr int W = BN * 3 * NM * 16;          // bytes of a tile's weights
  // TMEM: the scores and the sums of both row tiles; of four sixteens the scores of one at a time
  static constexpr bool TURNS = NM == 4;
  static constexpr int S_COL = 2 * NM * 16, O_COL = TURNS ? S_COL : 2 * S_COL, O_STEP = 3 * NM * 16;
  static_assert(O_COL + 2 * O_STEP <= 512, "TMEM");
  static constexpr size_t small(int slots) {          // what comes behind the tiles
    return (size_t)(2 * slots + 16) * 8 + kItems + 16 + slots * 32 * 4 + 4 * NR * 16 + 2 * NR * 16 + (2 * kSmall + 2) * 4;
  }
  static constexpr size_t with(int slots) { return (size_t)slots * TILE + 2 * QN * Q + RAW + 2 * W + small(slots); }
  // ring of K and V tiles; an even number: the two tiles of a copy lie side by side
  static constexpr int most() {
    int n = 16;
    while (with(n) > 232448) n -= 2;
    return n;
  }
  static constexpr int SLOTS = most();
  static constexpr size_t smem() { return with(SLOTS); }
};

// High words of the operands' descriptors. K and the rows along their bytes, V across its keys: rows of DH
// bytes, swizzled by 128 or 64 bytes, groups of 8 rows one after the other.
template <int DH>
constexpr uint32_t kHi = ((uint32_t)(8 * DH) >> 4) | (1u << 14) | ((DH == 128 ? 2u : 4u) << 29);
// The same with the groups of two heads in turn.
template <int DH>
constexpr uint32_t kHiPair = ((uint32_t)(16 * DH) >> 4) | (1u << 14) | ((DH == 128 ? 2u : 4u) << 29);
// Weights, across their keys, not swizzled: pieces of 16 rows x 8 keys (128 bytes), the next 8 keys
// 128 bytes further (low word), the next 16 rows 2048.
constexpr uint32_t kHiW = (2048u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_keys(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
// V as an operand of 128 rows: for heads of 64 the other 64 are whatever lies 512 bytes on (inside the CTA's shared
// memory), lanes 64 .. 127 of the sums are not read.
__device__ __forceinline__ uint32_t desc_values(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | ((512u >> 4) << 16); }
__device__ __forceinline__ uint32_t desc_weights(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | ((128u >> 4) << 16); }

// e4m3 x e4m3 -> fp32, 128 x n, along the bytes of both.
__device__ __forceinline__ uint32_t idesc_scores(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }
// e4m3 x e5m2 (bit 10) -> fp32, 128 x n, across the rows of both (bits 15, 16).
__device__ __forceinline__ uint32_t idesc_values(int n) { return idesc_scores(n) | (1u << 10) | (3u << 15); }

__device__ __forceinline__ void mma8(uint32_t lead, uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                     uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%2, %6};\n\tmov.b64 y, {%3, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%1], x, y, %4, p;\n\t}\n" ::"r"(lead),
      "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(a_hi), "r"(b_hi));
}

__device__ __forceinline__ void tmem_ld16_async(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_hold16(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}

// Barrier of a softmax group; true if some thread says so.
__device__ __forceinline__ bool group_any(int r, bool x) {
  uint32_t y;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(y)
      : "r"((uint32_t)x), "r"(1 + r)
      : "memory");
  return y != 0;
}

__device__ __forceinline__ void copy4(float* dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
// The barrier counts this thread once its copies have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Two values (magnitude up to 448, or NaN) as two codes each. In 16 bits: a code is exact there, and so is
// the rest of a value of 11 bits, 2^-12 of it being nothing beside lo's own rounding.
__device__ __forceinline__ void split_codes(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = to_e4m3x2(x, y);
  uint32_t r;
  asm("{\n\t.reg .b32 a, b, c;\n\t.reg .b16 l;\n\t"
      "cvt.rn.f16x2.f32 a, %3, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, %1;\n\t"
      "mov.b32 c, 0x4c004c00;\n\t"        // 16
      "sub.rn.f16x2 a, a, b;\n\t"
      "mul.rn.f16x2 a, a, c;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, a;\n\t"
      "cvt.u32.u16 %0, l;\n\t}\n"
      : "=r"(r)
      : "h"((uint16_t)hi), "f"(x), "f"(y));
  lo = r;
}

// Four weights (0 .. 2^15) as three e5m2 codes each, w = a + b / 8 + c / 64 to 9 bits. An e5m2 code is the upper byte of
// a 16-bit float: w as one (11 bits), cut after its upper byte, leaves 8 bits, those cut again 5, exactly; the last
// code is rounded. (NaN may become anything: the sum of a row that has one is NaN.)
__device__ __forceinline__ void split_weights(const float* w, uint32_t& a, uint32_t& b, uint32_t& c) {
  uint32_t x[2], y[2], z[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("{\n\t.reg .b32 e, t;\n\t"
        "mov.b32 e, 0x48004800;\n\t"         // 8
        "cvt.rn.f16x2.f32 %0, %4, %3;\n\t"
        "and.b32 t, %0, 0xff00ff00;\n\t"
        "sub.rn.f16x2 t, %0, t;\n\t"
        "mul.rn.f16x2 %1, t, e;\n\t"
        "and.b32 t, %1, 0xff00ff00;\n\t"
        "sub.rn.f16x2 t, %1, t;\n\t"
        "mul.rn.f16x2 t, t, e;\n\t"
        "add.u32 %2, t, 0x00800080;\n\t}\n"
        : "=&r"(x[i]), "=&r"(y[i]), "=&r"(z[i])
        : "f"(w[2 * i]), "f"(w[2 * i + 1]));
  }
  a = __byte_perm(x[0], x[1], 0x7531);
  b = __byte_perm(y[0], y[1], 0x7531);
  c = __byte_perm(z[0], z[1], 0x7531);
}

__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %3, %2, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

// What a softmax group has in shared memory for its row tile's rows.
template <int NR>
struct GroupRows {
  float4 cm[NR / 2];  // two rows' factors of the scores (base 2), and their -M
  int lim[NR];        // keys below it are seen
  float red[NR];      // maxima, sums or factors being joined
};
template <int NR>
__device__ __forceinline__ float& row_factor(GroupRows<NR>& R, int n) { return reinterpret_cast<float*>(R.cm)[(n >> 1) * 4 + (n & 1)]; }
template <int NR>
__device__ __forceinline__ float& row_minus_m(GroupRows<NR>& R, int n) { return reinterpret_cast<float*>(R.cm)[(n >> 1) * 4 + 2 + (n & 1)]; }
static_assert(sizeof(GroupRows<64>) == 64 * 16, "size in Tc8::smem");

template <int NR>
struct Group {
  const TcArgs& c;
  Item& it;
  uint8_t* sKV;
  uint8_t* sW;
  uint64_t* full;
  const float* sc;  // [slot][K, V][page of the tile]
  GroupRows<NR>* rows;
  float* red;       // [4][NR]
  uint32_t b_s, b_o;
  uint64_t* p_full;
  uint32_t ts, to;
  int r, quad, lane;
  const int* s_eff;
};

// Maxima or sums of 16 columns over a warp's lanes: the one of column (lane >> 1 & 15) in every lane.
template <bool SUM>
__device__ __forceinline__ float warp_columns(float* v, int lane) {
  auto join = [](float a, float b) { return SUM ? a + b : fmaxf(a, b); };
#pragma unroll
  for (int o = 16, n = 8; n >= 1; o >>= 1, n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], o);
      v[i] = join(up ? v[i + n] : v[i], other);
    }
  }
  return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

template <int DH>
__device__ __noinline__ float odd_sum8(const AttnRows& a, const Item& it, int g, int j0, int j1, int d) {
  for (int j = j0; j < j1; ++j) {
    const int id = attn_table(a, it.entry)[j / a.page];
    if (id < 0 || id >= a.n_pages) continue;
    const size_t at = (((size_t)id * a.Hkv + g) * a.page + j % a.page) * DH + d;
    if ((static_cast<const uint8_t*>(a.v)[at] & 0x7f) == 0x7f) return NAN;
  }
  return 0.f;
}

// n / G of n < 64, G <= 64
struct ByGroup {
  uint32_t by;
  __device__ __forceinline__ explicit ByGroup(int G) : by((65535u + G) / G) {}
  __device__ __forceinline__ int operator()(int n) const { return (int)(n * by >> 16); }
};

// Tokens of row tile r of an item, from its first one on.
__device__ __forceinline__ int tile_tokens(const TcArgs& c, const Item& it, int r) {
  if (it.split) return it.g + r < c.a.Hkv ? it.ntok : 0;
  return max(0, min(c.tb, it.ntok - r * c.tb));
}

// The rows of row tile r of an item as codes, their factors and limits, by T threads. N: rows of a row tile; rows
// without a token have no codes, and a factor of zero. raw: the rows in shared memory, or NULL: where they lie.
template <int DH, int N, int T, int NR>
__device__ __forceinline__ void make_rows(const TcArgs& c, const Item& it, int r, uint8_t* to, const uint8_t* raw,
                                          GroupRows<NR>& R, const int* s_eff, int tid) {
  const AttnRows& a = c.a;
  const ByGroup token_of(a.G);
  constexpr int PER = DH / 8, WIDE = T / PER;  // threads of a row, 8 values each; rows at a time
  const int part = tid % PER;
  const int heads = tile_tokens(c, it, r) * a.G, tl0 = it.split ? 0 : r * c.tb, g = it.g + (it.split ? r : 0);
  for (int n = tid; n < N; n += T) {
    int limit = kNone;  // (rows without a token, entries without tokens: all, and dropped)
    if (n < heads) {
      const int t = it.t0 + tl0 + token_of(n);
      const int len = it.kind == 1 ? (c.small ? s_eff[t / a.rows] : __ldcg(&a.eff[t / a.rows])) : it.len;
      if (len > 0) limit = max(0, len - a.rows + (it.kind == 1 ? t % a.rows : t) + 1);
    }
    R.lim[n] = limit;
    row_minus_m(R, n) = 0.f;
    if (n >= heads) row_factor(R, n) = 0.f;
  }
  auto values = [&](int n) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (n < heads) {
      const int t = token_of(n);
      x = raw ? *reinterpret_cast<const uint4*>(raw + (n * PER + part) * 16)
              : *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (size_t)(it.tok0 + tl0 + t) * a.q_ld +
                                                (size_t)(g * a.G + n - t * a.G) * DH + part * 8);
    }
    return x;
  };
  // (not unrolled: an item's first tile waits for this, and a kernel's first item for its instructions)
  uint4 x = values(tid / PER);
#pragma unroll 1
  for (int first = 0; first < heads; first += WIDE) {
    const int n = first + tid / PER;
    const uint4 then = values(n + WIDE);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8], top = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]) < INFINITY ? fabsf(v[k]) : 0.f);
#pragma unroll
    for (int o = PER / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // as scale_for, for every bf16 value
    const int bits = __float_as_int(top);
    const int e = max((bits >> 23) - 135 + ((bits & 0x7fffff) > 0x600000), -126);
    const float inv = pow2f(-e);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) split_codes(no_inf(v[2 * k]) * inv, no_inf(v[2 * k + 1]) * inv, hi[k], lo[k]);
    // 16-byte pieces of a row change places by the row's number, as the copies of K do it
    auto at = [&](int q) {
      const int piece = (part >> 1) ^ (DH == 128 ? q & 7 : (q >> 1) & 3);
      return reinterpret_cast<uint2*>(to + q * DH + piece * 16 + (part & 1) * 8);
    };
    if (n < heads) {
      *at(n) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *at(N + n) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      if (part == 0) row_factor(R, n) = a.qscale * pow2f(e);
    }
    x = then;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// The rows of an item to shared memory, by one warp.
template <int DH>
__device__ __forceinline__ void fetch_rows(const TcArgs& c, const Item& it, uint8_t* raw) {
  const AttnRows& a = c.a;
  const ByGroup token_of(a.G);
  constexpr int PER = DH / 8;
  for (int r = 0; r < 2; ++r) {
    const int heads = tile_tokens(c, it, r) * a.G, tl0 = it.split ? 0 : r * c.tb, g = it.g + (it.split ? r : 0);
    for (int i = threadIdx.x & 31; i < heads * PER; i += 32) {
      const int n = i / PER, t = token_of(n);
      const void* src = static_cast<const __nv_bfloat16*>(a.q) + (size_t)(it.tok0 + tl0 + t) * a.q_ld +
                        (size_t)(g * a.G + n - t * a.G) * DH + i % PER * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(raw + (r * 32 * PER + i) * 16)), "l"(src) : "memory");
    }
  }
}

// An item's softmax by one group, its rows in NC sixteens. tiles: key tiles of this group so far;
// ring: tiles of the ring so far; fail: a wait has run out in this warp. False: a wait ran out (the same answer in all of the group's threads).
template <int DH, int NC, int NS, int NR>
__device__ __forceinline__ bool soft_item(const Group<NR>& G, int tiles, int ring, bool fail) {
  constexpr int N = NC * 16, TILE = BN * DH;
  const AttnRows& a = G.c.a;
  Item& it = G.it;
  const int r = G.r, lane = G.lane, row = G.quad * 32 + lane;
  const int split = it.split, mine = it.nt[r], j0 = it.j0, j1 = it.j1, g = it.g + (split ? r : 0);
  const int tl0 = split ? 0 : r * G.c.tb;  // first token within the item
  GroupRows<NR>& R = *G.rows;
  const ByGroup token_of(a.G);

  const int streams = split && it.nt[1] > 0 ? 2 : 1, look = it.first_cut();
  const int shift = 31 - __clz(a.page);
  uint64_t l2[N / 2];  // sums of two rows each
#pragma unroll
  for (int n = 0; n < N / 2; ++n) l2[n] = 0;
  for (int j = 0; j < mine; ++j) {
    const int jt = j0 + j * BN, key = jt + row;
    const int vi = ring + (streams == 1 ? 1 + 2 * j : 2 + 4 * j), vs = vi % NS, turn = vi / NS;  // V's place
    // The scales of an item's first tile behind its scores: all tiles before this one have been worked on by then. A group
    // that had no part in the item before would else come several turns of the ring early, where a parity says nothing.
    if (j == 0) fail = fail || !wait_uniform(G.b_s, (uint32_t)tiles & 1u);
    fail = fail || !wait_uniform(smem_u32(&G.full[vs]), (uint32_t)turn & 1u);
    const float* sc = G.sc + (vs + (streams == 1 ? 0 : r)) * 32 + (row >> shift);
    const float ks = held_scale(sc[0]), vscale = held_scale(sc[16]);
    const float lv = (float)((__float_as_int(vscale) >> 23) - 127), rv = 1.f / vscale;
    const uint64_t ks2 = pair(ks, ks), lv2 = pair(lv, lv), rv2 = pair(rv, rv), fine2 = pair(1.f / kFine, 1.f / kFine);
    if (j > 0) fail = fail || !wait_uniform(G.b_s, (uint32_t)(tiles + j) & 1u);
    tc_fence_after();
    const bool cut = jt + BN > min(it.low, j1);
    uint8_t* w = G.sW + row * 16;
    // 32 rows at a time: the exponents of more do not fit the registers beside the sums
#pragma unroll
    for (int h0 = 0; h0 < NC; h0 += 2) {
      constexpr int HB = NC < 2 ? NC : 2;
      const int hb = NC - h0 < HB ? NC - h0 : HB;
      float z[HB * 16];  // exponents of the weights
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      float t[HB * 16];
#pragma unroll
      for (int i = 0; i < HB; ++i)
        if (i < hb) {
          tmem_ld16_async(G.ts + (h0 + i) * 16, z + i * 16);
          tmem_ld16_async(G.ts + N + (h0 + i) * 16, t + i * 16);
        }
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        if (i >= hb) continue;
        const int h = h0 + i;
        tmem_hold16(z + i * 16);
        tmem_hold16(t + i * 16);
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          const int m = i * 16 + n;
          const float4 cm = R.cm[h * 8 + n / 2];
          const uint64_t s2 = fma2(pair(t[m], t[m + 1]), fine2, pair(z[m], z[m + 1]));
          const float2 e = unpair(fma2(s2, mul2(pair(cm.x, cm.y), ks2), add2(pair(cm.z, cm.w), lv2)));
          z[m] = e.x;
          z[m + 1] = e.y;
        }
        if (cut) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (key >= min(R.lim[h * 16 + n], j1)) z[i * 16 + n] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) top[n & 3] = max3(top[n & 3], z[i * 16 + n], z[i * 16 + 8 + n]);
      }
      // a vote on a raise
      if (group_any(r, fail || fmaxf(max3(top[0], top[1], top[2]), top[3]) > kLift) || j == 0) {
        // the maximum of every row over the 128 keys
#pragma unroll
        for (int i = 0; i < HB; ++i) {
          if (i >= hb) continue;
          const int h = h0 + i;
          float v[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) v[n] = z[i * 16 + n];
          const float m = warp_columns<false>(v, lane);
          if (!(lane & 1)) G.red[G.quad * NR + h * 16 + (lane >> 1)] = m;
        }
        if (j > 0) fail = fail || !wait_uniform(G.b_o, (uint32_t)(tiles + j - 1) & 1u);
        if (group_any(r, fail)) return false;
        tc_fence_after();
        if (row >= h0 * 16 && row < (h0 + hb) * 16) {
          const float m = fmaxf(fmaxf(G.red[row], G.red[NR + row]), fmaxf(G.red[2 * NR + row], G.red[3 * NR + row]));
          // (a row that sees nothing of the first tile sees nothing of the item)
          const float down = (j == 0 ? m > -INFINITY : m > kLift) ? kLifted - m : 0.f;
          R.red[row] = down;
          G.red[row] = j == 0 ? 1.f : ex2(down);  // (the column's maxima have been read, by this thread alone)
          row_minus_m(R, row) += down;
        }
        group_any(r, false);
        if (j > 0) {
#pragma unroll 1
          for (int i = 0; i < hb; ++i) {
            const float4* f4 = reinterpret_cast<const float4*>(G.red + (h0 + i) * 16);
            const float4 f[4] = {f4[0], f4[1], f4[2], f4[3]};
            const float* factor = reinterpret_cast<const float*>(f);
            bool same = true;  // (mostly one row of many is raised)
#pragma unroll
            for (int n = 0; n < 16; ++n) same = same && factor[n] == 1.f;
            if (same) continue;
#pragma unroll 1
            for (int h = h0 + i; h < 3 * NC; h += NC) {
              float o[16];
              tmem_ld16_async(G.to + h * 16, o);
              tmem_wait_ld();
              tmem_hold16(o);
#pragma unroll
              for (int n = 0; n < 16; ++n) o[n] *= factor[n];
              tmem_st16(G.to + h * 16, o);
            }
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int n = 0; n < HB * 16; n += 2) {
          if (n >= hb * 16) continue;
          const float2 down = *reinterpret_cast<const float2*>(&R.red[h0 * 16 + n]);
          l2[h0 * 8 + n / 2] = mul2(l2[h0 * 8 + n / 2], *reinterpret_cast<const uint64_t*>(&G.red[h0 * 16 + n]));
          z[n] += down.x;
          z[n + 1] += down.y;
        }
      }
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        if (i >= hb) continue;
        const int h = h0 + i;
        uint32_t c0[4], c1[4], c2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = ex2(z[i * 16 + q * 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; k += 2)
            l2[h * 8 + q * 2 + k / 2] = fma2(pair(x[k], x[k + 1]), rv2, l2[h * 8 + q * 2 + k / 2]);
          split_weights(x, c0[q], c1[q], c2[q]);
        }
        *reinterpret_cast<uint4*>(w + h * 2048) = make_uint4(c0[0], c0[1], c0[2], c0[3]);
        *reinterpret_cast<uint4*>(w + (NC + h) * 2048) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
        *reinterpret_cast<uint4*>(w + (2 * NC + h) * 2048) = make_uint4(c2[0], c2[1], c2[2], c2[3]);
      }
    }
    if (j >= look) {
      // some row masks keys that the tile holds: NaN codes of V there are set aside
      uint8_t* v = G.sKV + (size_t)vs * TILE;
      const int k0 = max(0, min(it.low, j1) - jt), k1 = min(BN, it.hold - jt);
      const bool both = streams == 1 && j < it.nt[0] && j < it.nt[1];
      const int step = both ? 256 : 128;
      for (int q = k0 * (DH / 16) + (both ? r * 128 + row : row); q < k1 * (DH / 16); q += step) {
        // (groups of eight rows; of two heads in turn)
        uint4* at = reinterpret_cast<uint4*>(v) + (streams == 1 ? q : q + (q / (DH / 2) + r) * (DH / 2));
        uint4 x = *at;
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
        uint32_t hit[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) hit[k] = ((xw[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        if (hit[0] | hit[1] | hit[2] | hit[3]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) xw[k] &= ~((hit[k] >> 7) * 0xffu);
          atomicMin(&it.odd[streams == 1 ? 0 : r], jt);
          *at = x;
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(G.p_full);
  }

  // ---- the item's end: the sums over the threads, then the rows
  if (mine > 0) fail = fail || !wait_uniform(G.b_o, (uint32_t)(tiles + mine - 1) & 1u);
  tc_fence_after();
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    float t[16];
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      const float2 x = unpair(l2[h * 8 + n / 2]);
      t[n] = x.x;
      t[n + 1] = x.y;
    }
    const float x = warp_columns<true>(t, lane);
    if (!(lane & 1)) G.red[G.quad * NR + h * 16 + (lane >> 1)] = x;
  }
  if (group_any(r, fail)) return false;
  const bool direct = it.direct;
  const int heads = tile_tokens(G.c, it, r) * a.G;  // rows with a token
  PartAt at{};
  if (heads > 0) at = it.kind == 1 ? part_prefix(a, it.part, g, it.t0 + tl0, 0) : part_own_unit(a, it.part, g, it.t0 + tl0, 0);
  if (row < N) {
    const float sum = G.red[row] + G.red[NR + row] + (G.red[2 * NR + row] + G.red[3 * NR + row]);
    bool dead = false;
    if (row < heads && it.kind == 1) {
      const int e = (it.t0 + tl0 + token_of(row)) / a.rows;
      dead = (G.c.small ? G.s_eff[e] : __ldcg(&a.eff[e])) == 0;
    }
    R.red[row] = sum == 0.f || dead ? 0.f : 1.f / sum;
    if (!direct && row < heads)
      a.part_ml[at.first + at.row + row] = dead || mine == 0 ? make_float2(-INFINITY, 0.f) : make_float2(-row_minus_m(R, row), sum);
  }
  group_any(r, false);
  const int from = *(volatile int*)&it.odd[streams == 1 ? 0 : r];
#pragma unroll 1
  for (int h = 0; h < NC; ++h) {
    if (h * 16 >= heads) break;
    __syncwarp();
    float o[16], t[16], u[16];
    if (mine > 0) {
      tmem_ld16_async(G.to + h * 16, o);
      tmem_ld16_async(G.to + N + h * 16, t);
      tmem_ld16_async(G.to + 2 * N + h * 16, u);
      tmem_wait_ld();
      tmem_hold16(o);
      tmem_hold16(t);
      tmem_hold16(u);
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n] = mine > 0 ? fmaf(fmaf(u[n], 1.f / kFinerW, t[n]), 1.f / kFinerW, o[n]) : 0.f;
    if (row >= DH) continue;
    if (from < j1) {
#pragma unroll 1
      for (int n = 0; n < 16; ++n) {
        if (h * 16 + n >= heads) break;
        const int lim = R.lim[h * 16 + n];
        if (lim == kNone || from >= min(lim, j1)) continue;
        const float x = odd_sum8<DH>(a, it, g, from, min(lim, j1), row);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = i == n ? o[i] + x : o[i];
      }
    }
    if (direct) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int m = h * 16 + n, t = token_of(m);
        if (m >= heads) break;
        const float inv = R.red[m];
        static_cast<__nv_bfloat16*>(a.out)[((size_t)it.tok0 + tl0 + t) * a.out_ld + (size_t)(g * a.G + m - t * a.G) * DH + row] =
            __float2bfloat16_rn(inv == 0.f ? 0.f : o[n] * inv);
      }
    } else if (mine > 0) {
      float* dst = a.part_o + at.first * DH + ((size_t)(row / 8) * at.region + at.row + h * 16) * 8 + row % 8;
#pragma unroll
      for (int n = 0; n < 16; ++n)
        if (h * 16 + n < heads) dst[n * 8] = o[n];
    }
  }
  tc_fence_before();
  return true;
}

// NO, NP: sixteens of rows of a row tile, of an entry's own keys and of the prefix (0: none). One pair a
// kernel: a softmax loop for every number of rows in one kernel spills its registers.
template <int DH, int NO, int NP>
__global__ void __launch_bounds__(TCT, 1)
tc8_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mk2, const __grid_constant__ CUtensorMap mv2, const __grid_constant__ TcArgs c) {
  constexpr int NM = NO > NP ? NO : NP;
  using L = Tc8<DH, NM>;
  constexpr int NS = L::SLOTS, NR = L::NR;
  const AttnRows& a = c.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                                        // [QN][2]
  uint8_t* sRaw = smem + 2 * L::QN * L::Q;                   // [2]
  uint8_t* sKV = sRaw + L::RAW;
  uint8_t* sW = sKV + (size_t)NS * L::TILE;                  // [2]
  uint64_t* full = reinterpret_cast<uint64_t*>(sW + 2 * L::W);
  uint64_t* empty = full + NS;
  uint64_t* r_full = empty + NS;   // [2] an item's rows as codes
  uint64_t* s_full = r_full + 2;   // [2]
  uint64_t* p_full = r_full + 4;   // [2]
  uint64_t* o_full = r_full + 6;   // [2]
  uint64_t* i_full = r_full + 8;   // [2] items
  uint64_t* i_empty = r_full + 10; // [2]
  uint64_t* drained = r_full + 12; // after a wait that ran out: the products have ended
  uint64_t* f_full = r_full + 13;  // rows fetched
  uint64_t* f_empty = r_full + 14;
  Item* items = reinterpret_cast<Item*>(r_full + 16);        // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(items) + kItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;  // tiles that the loader has asked for
  float* s_sc = reinterpret_cast<float*>(tmem_slot + 4);     // [NS][2][16]
  GroupRows<NR>* s_rows = reinterpret_cast<GroupRows<NR>*>(s_sc + NS * 32);  // [2 items][2]
  float* s_red = reinterpret_cast<float*>(s_rows + 4);       // [2][4][NR]
  int* s_eff = reinterpret_cast<int*>(s_red + 2 * 4 * NR);   // small calls: [kSmall] lengths, [kSmall + 1] places
  int* s_tile0 = s_eff + kSmall;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 33);  // the tile's bytes, and the scales of 32 lanes
      mbar_init(&empty[s], 1);
    }
    mbar_init(drained, 1);
    mbar_init(f_full, 32);
    mbar_init(f_empty, 8);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&r_full[g], L::AHEAD ? 1 : 8);  // warp 3, or eight softmax warps
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&o_full[g], 1);
      mbar_init(&i_full[g], 1);
      mbar_init(&i_empty[g], 11);  // the loader, the products, the rows, eight softmax warps
    }
    *abort_flag = 0;
    *issued = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (tid >= 64 && tid < 68) {  // (the first copies would wait for them)
    const CUtensorMap* map = tid == 64 ? &mk : tid == 65 ? &mv : tid == 66 ? &mk2 : &mv2;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Beside a dense prefix the wait comes at the end: that launch, directly before this one, triggers behind its own wait
  // only, when all launches before it have ended, and nothing that it writes is read here.
  if (c.busy == 0) pdl_wait();
  __syncwarp();

  if (c.wait == 0) {
    *abort_flag = 1;
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---- loads: K(0), then V(j), K(j+1) through the ring; of two heads a place and the next one at a time
      int ri = 0;  // places so far
      bool ok = true;
      const int nbox = BN / a.page, shift = 31 - __clz(a.page), box = lane & (nbox - 1);
      for (int n = 0; ok; ++n) {
        const Item& it = items[n & 1];
        ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!ok || it.kind < 0) break;
        const int nt = max(it.nt[0], it.nt[1]), j1 = it.j1, g = it.g;
        const bool two = it.split && it.nt[1] > 0;
        const int32_t* tab = attn_table(a, it.entry);
        // The item's pages, 32 at a time and 32 ahead: a look-up for every tile, though made a tile ahead, held the copies
        // up (64 x 1 rows over 4096 tokens, heads of 64, with weights of two codes: 80 us, so 73).
        const int first = it.j0 >> shift, pages = j1 > it.j0 ? ((j1 - 1) >> shift) - first + 1 : 0;
        auto look_up = [&](int batch) { return batch * 32 + lane < pages ? tab[first + batch * 32 + lane] : 0; };
        int batch = 0, now = look_up(0), then = look_up(1);
        // Waits for the next place of the ring, of two heads for two: a lane looks at one of them.
        auto place = [&](int count) {
          const int s = ri % NS;
          if (ri >= NS) ok = wait_uniform(smem_u32(&empty[s + (lane & (count - 1))]), ((uint32_t)(ri / NS) & 1u) ^ 1u);
          ok = ok && !*abort_flag;
          return s;
        };
        // (few instructions a tile: this warp's were the limit where tiles are short; the same call 73 us before, then 65)
        auto tile = [&](int j, bool is_v) {
          const int at = j * nbox, id = __shfl_sync(0xffffffffu, (at >> 5) == batch ? now : then, (at + box) & 31);
          const int s = place(two ? 2 : 1);
          if (!ok) return;
          if (lane < (two ? 2 : 1)) mbar_expect_tx(&full[s + lane], lane ? 0 : two ? 2 * L::TILE : L::TILE);
          __syncwarp();
          const bool mine = at + box < pages, on = mine && id >= 0 && id < a.n_pages;
          if (lane < nbox) {
            if (mine && !on && a.status) atomicOr(a.status, HF_S_BAD);
            tma_load_page(sKV + (size_t)s * L::TILE + lane * a.page * (two ? 2 * DH : DH), two ? (is_v ? &mv2 : &mk2) : is_v ? &mv : &mk,
                          &full[s], g, on ? id : a.n_pages);  // behind the pool: reads zeros
          }
          if (is_v)  // all scales, one a lane: V's places stay until the weights are there
            for (int i = lane; i < (two ? 4 : 2) * nbox; i += 32) {
              const int q = i >> (7 - shift), head = q >> 1;  // (nbox = 128 >> shift)
              copy4(s_sc + (s + head) * 32 + (q & 1) * 16 + box,
                    (q & 1 ? a.v_scale : a.k_scale) + (on ? (size_t)id * a.Hkv + g + head : 0), on);
            }
          copies_arrive(&full[s]);
          if (two) copies_arrive(&full[s + 1]);
          ri += two ? 2 : 1;
        };
        if (nt > 0) {
          if (two && (ri & 1)) {  // two places lie side by side from an even one on: this one stays empty
            const int s = place(1);
            if (ok) {
              if (lane == 0) mbar_arrive(&full[s]);
              copies_arrive(&full[s]);
              ++ri;
            }
          }
          tile(0, false);
          for (int j = 0; j < nt && ok; ++j) {
            tile(j, true);
            if (ok && j + 1 < nt) tile(j + 1, false);
            if (((j + 1) * nbox & 31) == 0) {
              now = then;
              then = look_up(++batch + 1);
            }
          }
        }
        if (lane == 0) mbar_arrive(&i_empty[n & 1]);
      }
      if (lane == 0) {
        *issued = ri;
        if (!ok) *abort_flag = 1;
      }
    } else if (warp == 1) {
      // ---- products: S_r(0), then V_r(j) W, S_r(j+1) for r = 0, 1 in turn; where the row tiles take turns with their
      // scores, S_0(0), then S_1(j), V_0(j) W, V_1(j) W, S_0(j+1)
      const uint32_t lead = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t dq = desc_keys(smem_u32(sQ)), dk = desc_keys(smem_u32(sKV)), dv = desc_values(smem_u32(sKV)),
                     dw = desc_weights(smem_u32(sW));
      const uint32_t b_full = smem_u32(full), b_empty = smem_u32(empty), b_s = smem_u32(s_full), b_p = smem_u32(p_full),
                     b_o = smem_u32(o_full);
      int ri = 0;  // places so far
      uint32_t pph[2] = {0, 0};
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item& it = items[n & 1];
        ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!ok || __shfl_sync(0xffffffffu, it.kind, 0) < 0) break;
        const int nt0 = __shfl_sync(0xffffffffu, it.nt[0], 0), nt1 = __shfl_sync(0xffffffffu, it.nt[1], 0);
        const bool two = __shfl_sync(0xffffffffu, it.split, 0) && nt1 > 0;  // keys of two heads
        const int nt = max(nt0, nt1);
        const int cols = 16 * (NP > 0 && __shfl_sync(0xffffffffu, it.kind, 0) == 1 ? NP : NO);
        const uint32_t id_s = idesc_scores(2 * cols), id_o = idesc_values(3 * cols);
        const uint32_t hi = two ? kHiPair<DH> : kHi<DH>, pair_r = two ? 8 * DH >> 4 : 0, groups = two ? 2 : 1;
        const uint32_t q = dq + (n % L::QN) * (2 * L::Q >> 4);
        auto next = [&]() {  // waits for the next tile
          const int s = ri % NS;
          ok = ok && wait_uniform(b_full + 8 * s, (uint32_t)(ri / NS) & 1u);
          if (two) ok = ok && wait_uniform(b_full + 8 * (s + 1), (uint32_t)(ri / NS) & 1u);
          ri += two ? 2 : 1;
          return s;
        };
        auto done = [&](int s) {  // its places are free once the products so far have ended
          mma_commit(lead, b_empty + 8 * s);
          if (two) mma_commit(lead, b_empty + 8 * (s + 1));
        };
        auto score = [&](int r, int slot) {
#pragma unroll
          for (int k = 0; k < DH / 32; ++k)
            mma8(lead, tm + (L::TURNS ? 0 : r * L::S_COL), dk + slot * (L::TILE >> 4) + r * pair_r + 2 * k, hi, q + r * (L::Q >> 4) + 2 * k, kHi<DH>,
                 id_s, k > 0);
          mma_commit(lead, b_s + 8 * r);
        };
        if (nt > 0) {
          if (two && (ri & 1)) {
            const int s = ri % NS;
            ok = ok && wait_uniform(b_full + 8 * s, (uint32_t)(ri / NS) & 1u);
            if (ok) mma_commit(lead, b_empty + 8 * s);
            ++ri;
          }
          int ks = next(), vs = 0;
          ok = ok && wait_uniform(smem_u32(&r_full[n & 1]), (uint32_t)(n >> 1) & 1u);
          if (ok) {
            tc_fence_after();
            score(0, ks);
            if (nt1 > 0 && !L::TURNS) score(1, ks);
            if (nt1 == 0 || !L::TURNS) done(ks);
          }
          // from tile `look` on the softmax groups look V over before they hand their weights
          // on; where both have the tile, each looks at half of it
          const int look = __shfl_sync(0xffffffffu, it.first_cut(), 0);
          auto weights = [&](int r) {  // waits for a row tile's weights
            ok = ok && wait_uniform(b_p + 8 * r, pph[r]);
            pph[r] ^= 1u;
            if (ok) tc_fence_after();
          };
          auto values = [&](int r, int j) {
#pragma unroll
            for (int k = 0; k < BN / 32; ++k)
              mma8(lead, tm + L::O_COL + r * L::O_STEP, dv + vs * (L::TILE >> 4) + r * pair_r + k * groups * (32 * DH >> 4), hi,
                   dw + r * (L::W >> 4) + k * (512 >> 4), kHiW, id_o, j > 0 || k > 0);
            mma_commit(lead, b_o + 8 * r);
          };
          for (int j = 0; j < nt && ok; ++j) {
            const bool more = j + 1 < nt;
            const int k0 = ks;
            vs = next();
            if (more) ks = next();
            const bool both = !two && j >= look && j < nt0 && j < nt1;
            if constexpr (L::TURNS) {
              weights(0);
              if (ok && nt1 > 0) {
                score(1, k0);
                done(k0);
              }
              if (both) weights(1);
              if (ok) values(0, j);
              if (nt1 > 0) {
                if (!both) weights(1);
                if (ok) values(1, j);
              }
              if (ok && more) score(0, ks);
            } else {
              if (both) {
                weights(0);
                weights(1);
              }
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int mine = r ? nt1 : nt0;
                if (!ok || j >= mine) continue;
                if (!both) weights(r);
                if (!ok) continue;
                values(r, j);
                if (j + 1 < mine) score(r, ks);
              }
            }
            if (ok) {
              done(vs);
              if (more && (!L::TURNS || nt1 == 0)) done(ks);
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
      for (int idx = me; NP > 0 && ok && idx < c.pre_items; idx += all) {
        make_prefix(c, idx, it, eff);
        put(it);
      }
      // (beside another launch the first CTAs are those that found an SM free)
      const int heavy = c.busy ? c.busy : c.pre_items % all;
      AttnLine line;
      if (c.small) {
        line = make_line(scan_tiles(a, s_eff, s_tile0), a.units, all, heavy, c.busy ? c.places : prefix_places(a));
        if (me == 0) {
          for (int i = lane; i <= a.n; i += 32) a.tile0[i] = s_tile0[i];
          if (lane == 0) *reinterpret_cast<AttnLine*>(a.line) = line;
        }
      } else {
        line = *reinterpret_cast<const AttnLine*>(a.line);
      }
      const int cta = c.busy ? me : (me - heavy + all) % all, end = min(line.start(cta + 1), line.tiles * a.units);
      for (int pos = line.start(cta); ok && pos < end;) {
        bool some;
        pos += make_own(c, line, cta, pos, end, it, some, eff, tile0);
        if (some) put(it);
      }
      it.kind = -1;
      if (ok) put(it);
      if (!ok) *abort_flag = 1;
    } else {
      // ---- rows
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item& it = items[n & 1];
        // (a place of items is free once all have done with what it held, and so are its codes)
        ok = wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!ok || it.kind < 0) break;
        if constexpr (L::AHEAD) {
          for (int r = 0; r < 2; ++r)
            make_rows<DH, 16, 32>(c, it, r, sQ + ((n & 1) * 2 + r) * L::Q, nullptr, s_rows[2 * (n & 1) + r], s_eff, lane);
          if (lane == 0) mbar_arrive(&r_full[n & 1]);
        } else if constexpr (L::RAW > 0) {
          if (n > 0) ok = wait_uniform(smem_u32(f_empty), (uint32_t)(n - 1) & 1u);
          if (!ok) break;
          fetch_rows<DH>(c, it, sRaw);
          copies_arrive(f_full);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[n & 1]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok) *abort_flag = 1;
      if (c.small) check_prefixes(a, 1 + blockIdx.x, gridDim.x, lane, 32);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int r = warp >= 8, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    int tiles = 0, ring = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      Item& it = items[n & 1];
      // (the group's warps go on together: a wait that ran out in one ends it in all)
      ok = !group_any(r, !wait_uniform(smem_u32(&i_full[n & 1]), (uint32_t)(n >> 1) & 1u));
      if (!ok || it.kind < 0) break;
      const bool two = it.split && it.nt[1] > 0;
      const int nt = max(it.nt[0], it.nt[1]);
      if (two) ring += ring & 1;
      const Group<NR> G{c, it, sKV, sW + r * L::W, full, s_sc, s_rows + 2 * (n & 1) + r, s_red + r * 4 * NR,
                    smem_u32(&s_full[r]), smem_u32(&o_full[r]), &p_full[r],
                    tmem + lanes + (L::TURNS ? 0 : r * L::S_COL), tmem + lanes + L::O_COL + r * L::O_STEP, r, quad, lane, s_eff};
      bool fail = false;
      if constexpr (L::AHEAD) {
        fail = !wait_uniform(smem_u32(&r_full[n & 1]), (uint32_t)(n >> 1) & 1u);
      } else {
        // (the codes of the item before have been read: its last scores came to this group)
        const uint8_t* raw = L::RAW ? sRaw + r * (L::RAW / 2) : nullptr;
        if (L::RAW) fail = !wait_uniform(smem_u32(f_full), (uint32_t)n & 1u);
        GroupRows<NR>& R = s_rows[2 * (n & 1) + r];
        if (NP > 0 && it.kind == 1)
          make_rows<DH, NP == 0 ? 16 : NP * 16, 128>(c, it, r, sQ + r * L::Q, raw, R, s_eff, tid & 127);
        else
          make_rows<DH, NO * 16, 128>(c, it, r, sQ + r * L::Q, raw, R, s_eff, tid & 127);
        if (L::RAW && lane == 0) mbar_arrive(f_empty);
        if (lane == 0) mbar_arrive(&r_full[n & 1]);
        ok = !group_any(r, fail);  // the factors and limits are there
        if (!ok) break;
      }
      if (NP > 0 && it.kind == 1)
        ok = soft_item<DH, NP == 0 ? 1 : NP, NS>(G, tiles, ring, fail);
      else
        ok = soft_item<DH, NO, NS>(G, tiles, ring, fail);
      if (!ok) break;
      tiles += it.nt[r];
      ring += 2 * nt * (two ? 2 : 1);
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
    if (c.small && blockIdx.x == 0)
      for (int i = tid; i < a.n; i += TCT) a.eff[i] = 0;
    if (warp == 1) {  // the products still in flight end before their operands and TMEM go
      mma_commit(elect_one(), smem_u32(drained));  // (the lane that issued them)
      wait_uniform(smem_u32(drained), 0);
    }
    if (tid == 0) {
      if (a.status) atomicOr(a.status, HF_S_TIMEOUT);
      // the copies still in flight land before the CTA's shared memory goes
      for (int i = max(0, *issued - NS); i < *issued; ++i) mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (c.busy) pdl_wait();  // this launch has ended only when the one that it ran beside has: the join waits for both
}

// Pages of the cache, bytes [n_pages][hkv][page][dh]: a box is one page of `heads` neighbouring KV heads, in shared
// memory eight rows of the first head, eight of the second, the next eight of the first, .., swizzled by its
// rows of dh bytes.
cudaError_t make_map_pages8(CUtensorMap* map, const void* base, int dh, int page, int hkv, long long n_pages, int heads) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  static cudaError_t found = cudaSuccess;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (found == cudaSuccess && (q != cudaDriverEntryPointSuccess || !fn)) found = cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (found != cudaSuccess) return found;
  const cuuint64_t row = dh, block = row * page;
  const cuuint64_t dims[5] = {row, 8u, (cuuint64_t)hkv, (cuuint64_t)page / 8, (cuuint64_t)n_pages};
  const cuuint64_t strides[4] = {row, block, 8 * row, block * hkv};
  const cuuint32_t box[5] = {(cuuint32_t)dh, 8u, (cuuint32_t)heads, (cuuint32_t)page / 8, 1u}, step[5] = {1u, 1u, 1u, 1u, 1u};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, dh == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kMaxDev = 64;
std::mutex g_mu;
bool g_set[kMaxDev][2][4][5] = {};

template <int DH, int NO, int NP>
cudaError_t launch_one(const TcArgs& c, const CUtensorMap* m, dim3 grid, cudaStream_t st) {
  using L = Tc8<DH, (NO > NP ? NO : NP)>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_set[dev & (kMaxDev - 1)][DH == 128][NO - 1][NP];
    if (!set || dev >= kMaxDev) {
      e = cudaFuncSetAttribute(tc8_kernel<DH, NO, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::smem());
      if (e != cudaSuccess) return e;
      set = true;
    }
  }
  return launch_pdl(tc8_kernel<DH, NO, NP>, grid, dim3(TCT), L::smem(), st, m[0], m[1], m[2], m[3], c);
}

// By the rows of a row tile, of an entry and of the prefix (at least as many): 1, 2, 3, 4 sixteens, and none or these.
// (4 x 2 rows of 4 heads over 8192 tokens, all: 23.9 us with two sixteens for the prefix, 25.8 with three.)
template <int DH>
cudaError_t launch_rows(const TcArgs& c, const CUtensorMap* m, dim3 grid, cudaStream_t st) {
  const auto sixteens = [&](long long tokens) { return (int)((std::min<long long>(tokens, c.tb) * c.a.G + 15) / 16); };
  const int own = sixteens(c.a.rows), pre = c.pre_items > 0 ? sixteens((long long)c.a.n * c.a.rows) : 0;
  switch (own) {
    case 1:
      if (pre == 0) return launch_one<DH, 1, 0>(c, m, grid, st);
      if (pre == 1) return launch_one<DH, 1, 1>(c, m, grid, st);
      if (pre == 2) return launch_one<DH, 1, 2>(c, m, grid, st);
      return launch_one<DH, 1, 3>(c, m, grid, st);
    case 2:
      if (pre == 0) return launch_one<DH, 2, 0>(c, m, grid, st);
      if (pre == 2) return launch_one<DH, 2, 2>(c, m, grid, st);
      return launch_one<DH, 2, 3>(c, m, grid, st);
    case 3: return pre == 0 ? launch_one<DH, 3, 0>(c, m, grid, st) : launch_one<DH, 3, 3>(c, m, grid, st);
    default: return pre == 0 ? launch_one<DH, 4, 0>(c, m, grid, st) : launch_one<DH, 4, 4>(c, m, grid, st);
  }
}

}  // namespace

cudaError_t launch_attn_tc8_pages(const AttnRows& a, int pre_items, int busy, int places, cudaStream_t st) {
  TcArgs c{};
  c.a = a;
  c.tb = a.tb;
  c.blocks = (int)(((long long)a.n * a.rows + 2 * c.tb - 1) / (2 * c.tb));
  c.box_rows = a.page;
  c.wait = !attn_gives_up();
  c.pre_items = pre_items;
  c.busy = busy;
  c.places = places;
  CUtensorMap m[4];  // K, V of one head, of two
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = make_map_pages8(&m[i], i & 1 ? a.v : a.k, a.dh, a.page, a.Hkv, a.n_pages, 1 + i / 2);
  if (e != cudaSuccess) return e;
  // (the line is at most as long as all tables reach)
  const long long reach = (((long long)a.table_ld * a.page - a.shared + BN - 1) / BN + a.item_start) * a.n * a.units;
  const int grid = busy ? 152 : (int)std::min<long long>(std::max<long long>(pre_items + reach, 1), 152);
  c.small = a.n <= kSmall;
  if (!c.small) e = launch_attn_plan(a, grid, pre_items % grid, st);
  if (e != cudaSuccess) return e;
  return a.dh == 128 ? launch_rows<128>(c, m, dim3(grid), st) : launch_rows<64>(c, m, dim3(grid), st);
}

}  // namespace hf
