// Launch interface of the chunk attention kernel (internal to libmxa).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "mxa.h"
#include "mxa_launch.h"

namespace mxa {

struct alignas(64) PrefillMaps {
  TmapPair kv;     // the caches: boxes of box_tokens keys of one head, or of one chunk of 8 of them
  CUtensorMap q;   // the packed queries: boxes of {64 elements, G heads, TQ tokens}
};

// A unit whose first block lies in an earlier CTA's range, as the merge needs it.
struct PieceDesc {
  int q0, h, t0, tokens;   // the row's first packed token, KV head, the unit's first token and its tokens
  int c_first, n_pieces;   // the CTAs that hold its pieces; n_pieces 0: no such unit
  int pad[2];
};

struct PrefillArgs {
  const int32_t *cu_q;         // [B + 1]
  const int32_t *seqlens;      // [B]
  const int32_t *block_table;  // [B, mpps], or null (contiguous)
  void *out;                   // [total_q, Hq, D]
  float *lse;                  // [Hq, total_q] or null
  PieceDesc *pieces;           // [grid]: each CTA's head piece
  float *lse_part;             // [grid][2][tiles * 128]
  float *o_part;               // [grid][2][tiles * 128][D]
  int *err;
  int B, Hq, Hkv, G, TQ;       // TQ: tokens of a 128-row tile
  int total_q, max_q;
  int page_size, num_pages, mpps, contiguous, box_tokens;
  int grouped;                 // boxes of whole keys (rows at multiples of 8 tokens), else of one chunk
  int max_seqlen_k;
  int causal, window, sinks;
  int wide_out;                // out lies at a multiple of 32 bytes
  int unit_cost;               // fixed cost of a unit, in KV blocks
  int max_positions;           // what total_q tokens make at most on one KV head
  float scale_log2;
};

struct PrefillPlan {
  int grid, unit_cost;
  size_t lse_off, o_off, workspace_bytes;
};
// Upper bound on the positions that the work of a call is laid out on.
long long prefill_positions(const mxa_decode_params_t &p, int total_q);
PrefillPlan plan_prefill(const mxa_decode_params_t &p, int total_q, int sm_count);

struct PrefillLaunch {
  const void *q, *k_cache, *v_cache;
  const int32_t *cu_q, *block_table, *seqlens;
  int total_q;
  void *out;
  float *lse;
  void *workspace;
  mxa_decode_params_t p;
  PrefillPlan plan;
  float scale;
  int causal, window, sinks;
};
mxa_status_t launch_prefill(const PrefillLaunch &L, cudaStream_t stream);

}  // namespace mxa
