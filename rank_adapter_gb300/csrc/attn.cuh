// Shared pieces of the attention calls (lora_prepare_seqs, lora_kv_write,
// lora_attn_prompt, lora_attn_paged): the plan that the kernels walk, what they
// read of their operands, and the launchers.
#pragma once

#include "common.cuh"

namespace ra {

constexpr int kKeyBlock = 128;  // keys that the plan counts in, and a tensor-core tile takes

// Bits of the plan's error word.
constexpr int kErrAttn = 1;     // a kernel gave up waiting on its pipeline
constexpr int kErrBadPage = 2;  // a page id outside the cache was met

// How one geometry is cut into work: rows of a unit are (token, query head of one
// key-value head's group), token-major.
struct AttnShape {
  int dtype, Hq, Hkv, G, D, causal;
  bool tc;           // on the tensor cores
  int few;           // rows of a unit of few rows (attn_few.cu), 0: units of up to two tiles (attn_tc.cu)
  int tile_tokens;   // tokens whose rows share one 128-row tile (tensor cores)
  int unit_tokens;   // most tokens of a unit
  int slot_rows;     // rows of a partial result
  int ctas;          // CTAs the work is cut for
  int min_cost;      // least cost of a piece of a split unit
  float piece_cost, join_cost;  // what a piece, and joining, take besides
  float alone;       // time of a piece that runs when few others do
  int max_slots;     // partial results of one key-value head, at most
  float scale_log2;  // score scale times log2(e)
};

// The plan, int32 words: a header, the sequences as checked {first row, rows, keys, 0}
// (rows 0 for one that was refused), a running count of their units, their first rows in
// rising order, the units in the order in which the kernels take them, and the groups of
// units that have to be joined.
struct AttnPlan {
  static constexpr int kHeader = 16;
  static constexpr int kUnits = 0, kGroups = 1, kErr = 2, kBad = 3;  // words of the header
  static constexpr int kUnit = 8, kGroup = 4;                        // words of a record
  int max_seqs, max_units, max_groups;
  __host__ __device__ int seqs() const { return kHeader; }
  __host__ __device__ int cum() const { return seqs() + 4 * max_seqs; }  // and start(): max_seqs words each
  __host__ __device__ int start() const { return cum() + max_seqs; }
  __host__ __device__ int64_t units() const { return start() + ((2 * max_seqs + 3) & ~3) - max_seqs; }
  __host__ __device__ int64_t groups() const { return units() + (int64_t)kUnit * max_units; }
  __host__ __device__ int64_t words() const { return groups() + (int64_t)kGroup * max_groups; }
};

// A unit as stored: the rows of `tokens` tokens from row0 of one key-value head against
// keys [kb0, kb1) in blocks of kKeyBlock. pos0: position of row0 among the sequence's
// keys (negative where there are fewer keys than rows). slot: its partial result, or -1
// where it covers all keys its rows see.
struct AttnUnit {
  int seq, row0, tokens, kb0, kb1, kv_len, pos0, slot;
};
// Partial results of one unit's rows: slots [slot, slot + pieces).
struct AttnGroup {
  int row0, tokens, slot, pieces;
};

// Keys that the row at position `pos` sees.
__device__ __forceinline__ int visible_keys(int pos, int kv_len, int causal) {
  return causal ? max(0, min(kv_len, pos + 1)) : kv_len;
}

// Where keys and values are: rows of a packed matrix (page_size 0), or pages of a cache.
struct AttnKv {
  const void *k, *v;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;  // strides in elements
  int page_size, num_pages, max_pages;
  int log2_page;
  const int32_t *table;
  int64_t ld_table;
};

struct AttnArgs {
  AttnShape s;
  AttnPlan p;
  const int32_t *plan;
  int *err;
  const void *q;
  int64_t ldq;
  AttnKv kv;
  void *out;
  int64_t ldo;
  float *lse;     // or null
  float *ws;      // partial results
  int num_tokens;
};

// Partial results: for every (slot, key-value head) slot_rows rows of D unnormalised fp32
// outputs, then slot_rows pairs {maximum of the scaled scores in log2 units, sum}.
__host__ __device__ inline int64_t slot_floats(const AttnShape &s) { return (int64_t)s.slot_rows * (s.D + 2); }

AttnShape attn_shape(const lora_seqs &q);
AttnPlan attn_plan(const AttnShape &s, int num_seqs, int num_tokens);
int64_t attn_slot_rows(const lora_seqs &q);  // rows of partial results of one key-value head, likewise
size_t attn_plan_bytes(const lora_seqs &q);  // enough for up to so many sequences and rows, however units are cut
bool attn_may_split(const AttnShape &s, int64_t max_kv);

cudaError_t launch_prepare_seqs(const lora_seqs &q, cudaStream_t st);
cudaError_t launch_kv_write(const lora_seqs &q, const lora_kv_cache &c, const void *k, int64_t ldk, const void *v,
                            int64_t ldv, cudaStream_t st);
bool attn_tc_takes(const AttnShape &s);
cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t st);       // tensor cores (attn_tc.cu)
cudaError_t launch_attn_few(const AttnArgs &a, cudaStream_t st);      // the same, units of few rows (attn_few.cu)
cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t st);     // CUDA cores (attn_rows.cu)
cudaError_t launch_attn_combine(const AttnArgs &a, cudaStream_t st);  // joins the partial results

// Errors of the calling thread, as lora_last_cuda_error reports them (lora_abi.cu).
void clear_stale_error();
int cuda_status(cudaError_t e);

}  // namespace ra
