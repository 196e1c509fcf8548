// Shared by the kernels of bsa_prefix_attn: the call's parameters, the requests' ranges, and the
// partial results that the merge kernel joins.
#pragma once

#include "bsa_common.cuh"

namespace bsa {

constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PrefixParams {
  const void *q, *k, *v;  // q [T, Hq, d] with token stride q_stride; pools [P, Hk, page, d]
  long long q_stride;     // elements
  int T, B, Hq, Hk, G, page_shift, num_pages;
  const int* table;  // [B, table_ld] pages of each request's own tokens
  int table_ld;
  const int* lens;    // [B] own tokens, the new ones included
  const int* ptable;  // pages of the prefix
  int prefix_len;
  const int* cu_q;  // [B + 1] or null: one new token per request
  int max_q;
  void* o;
  float* lse;
  // Partial results: slots [0, ns1) hold the pieces of the prefix, [ns1, ns1 + ns2) those of the
  // own tokens; part_o [slot][T * Hq][d] unnormalised, part_ml [slot][T * Hq] = (row maximum in
  // log2 units, row sum).  A row without keys in a piece has sum 0 and no part_o.
  float* part_o;
  float2* part_ml;
  int ns1, ns2;
  // Pieces of prefix_attn_rows: item = kv head of the prefix (the first prefix_items), then request *
  // Hk + kv head; item_cta[item] = first and last CTA that worked on it; the piece of CTA c is slot
  // item + c of item_o [slot][item_rows][d] and item_ml [slot][item_rows].
  int2* item_cta;
  float* item_o;
  float2* item_ml;
  int item_rows, item_ctas, prefix_items;  // item_ctas = 0: no items
};

// Request b: its first new token, how many it has, its own tokens.  Values that would reach
// outside the call's arrays are cut.
struct PaRequest {
  int t0, nq, len;
};
__device__ __forceinline__ PaRequest pa_request(const PrefixParams& p, int b) {
  PaRequest r;
  if (p.cu_q) {
    r.t0 = min(max(p.cu_q[b], 0), p.T);
    r.nq = min(max(p.cu_q[b + 1], r.t0), p.T) - r.t0;
  } else {
    r.t0 = b;
    r.nq = 1;
  }
  r.len = min(max(p.lens[b], 0), p.table_ld << p.page_shift);
  return r;
}
// Own keys of a request that any of its new tokens sees.
__device__ __forceinline__ int pa_own_keys(const PrefixParams& p, const PaRequest& r) {
  return r.nq > 0 ? max(0, r.len - r.nq + min(r.nq, p.max_q)) : 0;
}
// New tokens in all: rows at or after this are left as they were.
__device__ __forceinline__ int pa_tokens(const PrefixParams& p) {
  return p.cu_q ? min(max(p.cu_q[p.B], 0), p.T) : p.B;
}

// prefix_attn_tc.cu
bsa_status prefix_attn_tc(const PrefixParams& p, int d, int tiles1, int tiles2, bool fused,
                          bool direct, int* status, cudaStream_t st);

// prefix_attn_rows.cu
bsa_status prefix_attn_rows(const PrefixParams& p, int d, bool prefix, int* status,
                            cudaStream_t st);

}  // namespace bsa
