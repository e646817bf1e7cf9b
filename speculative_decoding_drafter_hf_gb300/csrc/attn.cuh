// Attention of query rows over packed prompts or a paged cache: what its variants
// (attn_rows.cu on CUDA cores, attn_tc.cu on tensor cores) share.
//
// Rows that use one KV head are numbered token * G + (query head in its group), so
// that a tile of rows always shares its keys, whatever the group size G is.
#pragma once

#include "common.cuh"

namespace hf {

// Two floats a 64-bit register: one instruction for two multiply-adds, sums or products.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct AttnRows {
  int Hq, Hkv, G, dh, esize;
  float qscale;  // scale * log2(e): scores are kept in the base-2 domain
  const void* q;
  long long q_ld;  // elements
  void* out;
  long long out_ld;
  int32_t* status;
  // prompts
  const void* k;  // packed: [total, k_ld]; paged: the layer's pool
  const void* v;
  long long k_ld, v_ld;
  const int32_t* off;
  int n_seq, total;
  // paged cache
  const int32_t* table;
  const int32_t* lens;
  const int32_t* req;
  int n, rows, page, n_pages, n_requests, table_ld;
  int shared;      // tokens of the common prefix
  // 8-bit cache: the layer's scales [n_pages, Hkv]; NULL of any other
  const float* k_scale;
  const float* v_scale;
  int dense;       // tensor cores: the prefix lies in rows k, v (k_ld, v_ld), only its pieces are computed
  // pieces of the key axis: npre of the prefix (pre_keys keys each), then each
  // entry's own tokens: on CUDA cores nown pieces of own_keys each (unused ones
  // among them), on tensor cores wherever the line of all tiles is cut (AttnLine). Rows
  // of one piece in all are written straight to out; the others' parts go to part_o /
  // part_ml and attn_join joins them. part_o holds 8 columns of all rows of a piece,
  // then the next 8: a warp with a row per lane writes whole lines. PartAt says where.
  int npre, pre_keys, nown, own_keys;
  float* part_o;   // [...][dh / 8][rows of the piece][8], not normalised
  float2* part_ml; // the same rows: maximum (base 2), sum
  // written on the device before the pieces are read
  int* eff;        // [n] tokens of each entry, 0 for those that break a rule
  int* line;       // tensor cores: an AttnLine
  int* tile0;      // [n + 1] where each entry starts on the line
  int tile;        // tensor cores: rows of a row tile
  int item_start;  // places before an entry's tiles
  int tb, units, unit_rows;  // tokens of a row tile; units of an entry's rows
};

__host__ __device__ inline bool attn_direct(const AttnRows& a) { return a.npre + a.nown == 1; }

constexpr int kKeyTile = 128;  // keys of a tile (tensor cores)

// Where the part of one row of one piece lies.
struct PartAt {
  size_t first;  // rows before the piece
  int region;    // rows of the piece
  int row;       // in the piece
};
__device__ __forceinline__ PartAt part_prefix(const AttnRows& a, int piece, int g, int t, int i) {
  const int N = a.n * a.rows * a.Hq;
  return {(size_t)piece * N, N, (g * a.n * a.rows + t) * a.G + i};
}
__device__ __forceinline__ PartAt part_own_rows(const AttnRows& a, int entry, int piece, int g, int t, int i) {
  const int N = a.rows * a.Hq;
  return {(size_t)a.npre * a.n * N + ((size_t)entry * a.nown + piece) * N, N, (g * a.rows + t) * a.G + i};
}
// unit: a pair of KV heads with all rows, or 2 tb tokens of one head (where all rows
// are more than a tile); slots are numbered along the line.
__device__ __forceinline__ PartAt part_own_unit(const AttnRows& a, int slot, int g, int t, int i) {
  const int row = a.rows <= a.tb ? ((g & 1) * a.rows + t) * a.G + i : t % (2 * a.tb) * a.G + i;
  return {(size_t)a.npre * a.n * a.rows * a.Hq + (size_t)slot * a.unit_rows, a.unit_rows, row};
}
__device__ __forceinline__ int unit_of(const AttnRows& a, int g, int t) {
  return a.rows <= a.tb ? g / 2 : t / (2 * a.tb) * a.Hkv + g;
}

// The entries' own key tiles, entry after entry, once per unit, laid out on one line
// that is cut into a stretch per CTA: the first `light` CTAs get `more` places each, the
// others `less`. A piece is what a CTA has of one entry and unit. An entry with tiles
// first has item_start empty places: what an item costs beside its tiles (measured, 64 x 8
// rows: about 2.2 us a tile, 1.7 us an item; of an 8-bit cache without items of the prefix, whose tiles are
// shorter, 1.6 and 5: all of 64 x 8 rows over 8192 shared and 8 to 4096 own tokens 141 us with three places, 165 with one, over
// 2048 shared 74 and 83; 32 x 16 rows over 4096 own tokens 119 either way).
constexpr int kItemStart = 1, kItemStart8 = 3;
__device__ __forceinline__ int entry_places(const AttnRows& a, int keys) {
  return keys > 0 ? (keys + kKeyTile - 1) / kKeyTile + a.item_start : 0;
}
struct AttnLine {
  int tiles;  // places of all entries (times units: the line's length)
  int light, more, less;
  __device__ __forceinline__ int cta(int pos) const {  // whose stretch pos lies in
    const int head = light * more;
    return pos < head ? pos / more : light + (pos - head) / max(less, 1);
  }
  __device__ __forceinline__ int start(int c) const { return c <= light ? c * more : light * more + (c - light) * less; }
};
// heavy: CTAs that have an item of the prefix more, as long as `pre` tiles, than the others.
__device__ __forceinline__ AttnLine make_line(int tiles, int units, int ctas, int heavy, int pre) {
  AttnLine l{tiles, ctas, 0, 0};
  const int all = tiles * units;
  if (heavy > 0) {
    l.light = ctas - heavy;
    const int rest = all - l.light * pre;  // what is left once all have as much to do
    l.less = rest > 0 ? (rest + ctas - 1) / ctas : 0;
    l.more = rest > 0 ? l.less + pre : (all + l.light - 1) / l.light;
  } else {
    l.more = (all + ctas - 1) / ctas;
  }
  l.more = max(l.more, 1);
  return l;
}

// Lengths, tables, lists, offsets and, on CUDA cores, the rows themselves come from
// calls that may still be running when a CTA starts (programmatic launches): they are read
// after pdl_wait and never through the non-coherent path, which is for data that nobody
// writes while the kernel lives. Many CTAs look the same lengths, bounds and ids up: they
// go through the L1 (8 fp32 prompts 66.8 us, past it 68.7).

// Length of entry i as the call takes it: 0 for entries that break a rule (bad set).
__device__ __forceinline__ int attn_raw_len(const AttnRows& a, int i, bool& bad) {
  const int r = a.req ? a.req[i] : i;
  if (r < 0 || r >= a.n_requests) {
    bad = true;
    return 0;
  }
  const int len = a.lens[r];
  if (len < 0 || len > (long long)a.table_ld * a.page || (len > 0 && len < a.shared)) {
    bad = true;
    return 0;
  }
  return len;
}
__device__ __forceinline__ int attn_len(const AttnRows& a, int i, bool& bad) {
  const int len = attn_raw_len(a, i, bad);
  if (len > 0 && a.shared > 0 && i > 0 && attn_raw_len(a, 0, bad) == 0) {
    bad = true;
    return 0;
  }
  return len;
}

__device__ __forceinline__ const int32_t* attn_table(const AttnRows& a, int i) {
  const int r = a.req ? a.req[i] : i;
  return a.table + (size_t)r * a.table_ld;
}

// Whether the entries from first on, every step-th, have entry 0's pages before `shared`;
// by one CTA or warp (tid of threads).
__device__ __forceinline__ void check_prefixes(const AttnRows& a, int first, int step, int tid, int threads) {
  if (a.shared == 0 || !a.status) return;
  bool bad = false, skip = false;
  if (attn_raw_len(a, 0, skip) == 0) return;
  const int32_t* t0 = attn_table(a, 0);
  for (int i = first; i < a.n; i += step) {
    if (attn_raw_len(a, i, skip) == 0) continue;
    const int32_t* t = attn_table(a, i);
    for (int j = tid; j < a.shared / a.page; j += threads) bad = bad || t[j] != t0[j];
  }
  if (bad) atomicOr(a.status, HF_S_BAD);
}

// Slot of a prompt tile -> sequence and tile within it: a sequence of rows
// [off_s, off_e) owns the slots [floor(off_s G / BM) + s, floor(off_e G / BM) + s + 1),
// at least as many as it has tiles, so no prefix sum over the sequences is needed.
__host__ __device__ inline long long prompt_slots(long long total, int n_seq, int G, int BM) {
  return total * G / BM + n_seq;
}
struct PromptTile {
  int start, len, tile;  // first row and length of the sequence, tile in it
  bool ok;
};
__device__ __forceinline__ PromptTile prompt_tile(const AttnRows& a, int slot, int BM, int G) {
  int lo = 0, hi = a.n_seq;  // the last sequence whose first slot is at or before `slot`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const long long first = (long long)max(0, min(a.off[mid], a.total)) * G / BM + mid;
    if (first <= slot)
      lo = mid;
    else
      hi = mid;
  }
  PromptTile t{};
  const int s0 = a.off[lo], s1 = a.off[lo + 1];
  t.ok = s0 >= 0 && s0 <= s1 && s1 <= a.total;
  if (!t.ok) return t;
  t.start = s0;
  t.len = s1 - s0;
  t.tile = slot - (int)((long long)s0 * G / BM + lo);
  t.ok = t.tile >= 0 && (long long)t.tile * BM < (long long)t.len * G;
  return t;
}

// Check of the whole list of sequence bounds, by one CTA or warp (tid of threads).
__device__ __forceinline__ void check_offsets(const AttnRows& a, int tid, int threads) {
  if (!a.status) return;
  bool bad = false;
  for (int s = tid; s <= a.n_seq; s += threads) {
    const int x = a.off[s];
    bad = bad || x < 0 || x > a.total || (s > 0 && x < a.off[s - 1]);
  }
  if (bad) atomicOr(a.status, HF_S_BAD);
}

// Tensor-core variants (attn_tc.cu; an 8-bit cache: attn_tc8.cu), where attn_tc_ok.
bool attn_tc_ok(int dtype, int dh);
constexpr int kTileRows = 128, kTileRows8 = 64;
// Rows of a row tile over an 8-bit cache: as many as TMEM holds the scores and sums of two row tiles for; more only where a
// KV head has more heads.
inline int tile_rows8(int G) { return G > 48 ? kTileRows8 : 48; }
constexpr int kSmall = 256;    // entries of a call that every CTA plans for itself
// busy: CTAs of the launch directly before it (attn_tc_pages of a dense prefix) that this one runs beside, each as long
// as `places` of an entry's; 0: it waits for that launch. Beside it, this launch reads the cache and the rows before its own
// wait (as a commit's early reads do): the launch directly before it triggers only behind its own wait, when all launches before
// that have ended and their writes are in memory. Not with more than kSmall entries: their plan would be between.
cudaError_t launch_attn_tc8_pages(const AttnRows& a, int pre_items, int busy, int places, cudaStream_t st);
bool attn_gives_up();  // a test made every wait give up before it begins
cudaError_t launch_attn_tc_prompt(const AttnRows& a, cudaStream_t st);
// Over a paged cache: the prefix's pieces and the rows' units (fields of a), items of the
// prefix and slots of own pieces.
void attn_tc_sizes(AttnRows& a, int& pre_items, long long& slots);
cudaError_t launch_attn_tc_pages(const AttnRows& a, int pre_items, cudaStream_t st);
cudaError_t launch_attn_rows_prompt(int dtype, const AttnRows& a, cudaStream_t st);
cudaError_t launch_attn_rows_pages(int dtype, const AttnRows& a, cudaStream_t st);
cudaError_t launch_attn_join(int dtype, const AttnRows& a, cudaStream_t st);

}  // namespace hf
