// Shared by the kernels of bsa_prefix_attn: the call's parameters, the requests' ranges, and the
// partial results that the merge kernel joins.
#pragma once

#include <atomic>

#include "tc_common.cuh"

namespace bsa {

constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PrefixParams {
  const void *q, *k, *v;  // q [T, Hq, d] with token stride q_stride; pools [P, Hk, page, d]
  long long q_stride;     // elements
  int T, B, Hq, Hk, G, g_shift, page_shift, num_pages;  // G = Hq / Hk = 1 << g_shift
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
  // Pieces of prefix_attn_rows: items are the prefix_items = Hk * groups of packed rows x prefix, then
  // request * Hk + kv head; item_cta[item] = first and last CTA that worked on it; the piece of CTA
  // c is slot item + c, of prefix_rows rows for a prefix item and own_rows for another (pa_item_row).
  int2* item_cta;
  float* item_o;    // [row][d]
  float2* item_ml;  // [row]
  int prefix_rows, own_rows, item_ctas, prefix_items;  // item_ctas = 0: no items
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
// First row of the piece that CTA c has of an item.
__device__ __forceinline__ long long pa_item_row(const PrefixParams& p, int item, int c) {
  if (item < p.prefix_items) return (long long)(item + c) * p.prefix_rows;
  return (long long)(p.prefix_items ? p.prefix_items + p.item_ctas : 0) * p.prefix_rows +
         (long long)(item - p.prefix_items + c) * p.own_rows;
}
// New tokens in all: rows at or after this are left as they were.
__device__ __forceinline__ int pa_tokens(const PrefixParams& p) {
  return p.cu_q ? min(max(p.cu_q[p.B], 0), p.T) : p.B;
}

// The call's kernels are launched as programmatic dependents, so that one's launch and prologue run
// while the one before drains.  pdl_wait: everything queued before is complete and visible.
// pdl_trigger: the next kernel may start once every CTA has said so (or left).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Args>
bool launch_pdl(void (*kern)(Args...), int grid, int threads, int smem, cudaStream_t st,
                const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return true;
  (void)cudaGetLastError();
  return false;
}

// Dynamic shared memory above 48 KB, asked for once per device (`done`: one bit each).
template <typename Kern>
bool allow_smem(Kern kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// prefix_attn_tc.cu
// Tensor maps: `rows` packed query rows of one kv head per box (a (d, G, Hk, T) view of q: a box is
// rows t0 * G .. of token-major, head-minor rows), and boxes of 1 << box_shift rows of a pool.
bool prefix_q_map(CUtensorMap* m, const PrefixParams& p, int d, int rows);
bool prefix_kv_map(CUtensorMap* m, const void* pool, const PrefixParams& p, int d, int box_shift);
__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, int col, int h,
                                           int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(0), "r"(h), "r"(token),
      "r"(smem_u32(bar))
      : "memory");
}
bsa_status prefix_attn_tc(const PrefixParams& p, int d, int tiles1, int tiles2, bool fused,
                          bool direct, int* status, cudaStream_t st);

// prefix_attn_rows.cu
bsa_status prefix_attn_rows(const PrefixParams& p, int d, int mt, int groups, bool after_tc,
                            int* status, cudaStream_t st);

}  // namespace bsa
