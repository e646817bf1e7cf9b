// Attention of query rows over packed prompts or a paged cache: what its variants
// (attn_rows.cu on CUDA cores, attn_tc.cu on tensor cores) share.
//
// Rows that use one KV head are numbered token * G + (query head in its group), so
// that a tile of rows always shares its keys, whatever the group size G is.
#pragma once

#include "common.cuh"

namespace hf {

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
  // pieces of the key axis: npre of the prefix (pre_keys keys each), then each
  // entry's own tokens: on CUDA cores nown pieces of own_keys each (unused ones
  // among them), on tensor cores as many as the plan gives it. An entry of one
  // piece in all has its rows written straight to out; the others' go to part_o /
  // part_ml and attn_join joins them: the prefix's pieces of n * rows * Hq rows each,
  // then the entries' of rows * Hq. Within a piece rows are ordered (KV head, token,
  // head in its group), and part_o holds 8 columns of all rows, then the next 8: a
  // warp with a row per lane writes whole lines.
  int npre, pre_keys, nown, own_keys;
  float* part_o;   // [...][dh / 8][rows of the piece][8], not normalised
  float2* part_ml; // the same rows: maximum (base 2), sum
  // written on the device before the pieces are read
  int* eff;        // [n] tokens of each entry, 0 for those that break a rule
  int* plan;       // tensor cores: [0] item counter, [1] keys per piece, [2] pieces
  int* base;       // [n + 1] first piece of each entry
  int* piece_of;   // entry of each piece
};

__host__ __device__ inline bool attn_direct(const AttnRows& a) { return a.npre + a.nown == 1; }

// Rows before piece p of the prefix or, own, before a piece of an entry, and the row
// of (KV head g, token t of `tokens`, head i in the group) within it.
__device__ __forceinline__ size_t part_first(const AttnRows& a, bool own, int p) {
  const size_t N = (size_t)a.n * a.rows * a.Hq;
  return own ? a.npre * N + (size_t)p * a.rows * a.Hq : p * N;
}
__device__ __forceinline__ int part_row(const AttnRows& a, bool own, int g, int t, int i) {
  return (g * (own ? a.rows : a.n * a.rows) + t) * a.G + i;
}

// First piece of entry i's own tokens, and how many there are.
__device__ __forceinline__ int attn_pieces(const AttnRows& a, int i, int& count) {
  if (a.plan) {
    const int b = __ldcg(&a.base[i]);
    count = __ldcg(&a.base[i + 1]) - b;
    return b;
  }
  count = max(1, (max(0, __ldcg(&a.eff[i]) - a.shared) + a.own_keys - 1) / a.own_keys);
  return i * a.nown;
}

// Length of entry i as the call takes it: 0 for entries that break a rule (bad set).
__device__ __forceinline__ int attn_raw_len(const AttnRows& a, int i, bool& bad) {
  const int r = a.req ? __ldg(&a.req[i]) : i;
  if (r < 0 || r >= a.n_requests) {
    bad = true;
    return 0;
  }
  const int len = __ldg(&a.lens[r]);
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
  const int r = a.req ? __ldg(&a.req[i]) : i;
  return a.table + (size_t)r * a.table_ld;
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
    const long long first = (long long)max(0, min(__ldg(&a.off[mid]), a.total)) * G / BM + mid;
    if (first <= slot)
      lo = mid;
    else
      hi = mid;
  }
  PromptTile t{};
  const int s0 = __ldg(&a.off[lo]), s1 = __ldg(&a.off[lo + 1]);
  t.ok = s0 >= 0 && s0 <= s1 && s1 <= a.total;
  if (!t.ok) return t;
  t.start = s0;
  t.len = s1 - s0;
  t.tile = slot - (int)((long long)s0 * G / BM + lo);
  t.ok = t.tile >= 0 && (long long)t.tile * BM < (long long)t.len * G;
  return t;
}

// One CTA's check of the whole list of sequence bounds.
__device__ __forceinline__ void check_offsets(const AttnRows& a) {
  if (!a.status) return;
  bool bad = false;
  for (int s = threadIdx.x; s <= a.n_seq; s += blockDim.x) {
    const int x = __ldg(&a.off[s]);
    bad = bad || x < 0 || x > a.total || (s > 0 && x < __ldg(&a.off[s - 1]));
  }
  if (bad) atomicOr(a.status, HF_S_BAD);
}

// Tensor-core variants (attn_tc.cu), where attn_tc_ok.
bool attn_tc_ok(int dtype, int dh);
cudaError_t launch_attn_tc_prompt(const AttnRows& a, cudaStream_t st);
// Over a paged cache: items of one piece of the prefix and of one piece of an entry,
// and how many pieces of the entries there are at most beside n (a.npre, a.pre_keys set).
void attn_tc_sizes(AttnRows& a, int& pre_items, int& units, int& budget);
cudaError_t launch_attn_tc_pages(const AttnRows& a, int pre_items, int units, int budget, cudaStream_t st);
// Entries' lengths and status checks; with budget > 0 the pieces of the entries.
cudaError_t launch_attn_plan(const AttnRows& a, int budget, int units, int first, int pre_items, cudaStream_t st);

cudaError_t launch_attn_rows_prompt(int dtype, const AttnRows& a, cudaStream_t st);
cudaError_t launch_attn_rows_prefix(int dtype, const AttnRows& a, cudaStream_t st);
cudaError_t launch_attn_rows_own(int dtype, const AttnRows& a, cudaStream_t st);
// `pieces`: about how many a row has (how many warps share a row).
cudaError_t launch_attn_join(int dtype, const AttnRows& a, int pieces, cudaStream_t st);

}  // namespace hf
