// Shared by the kernels of bsa_prefix_attn: the call's parameters, the requests' ranges, and the
// partial results that the merge kernel joins.
#pragma once

#include "launch.cuh"
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
  const int* slots;  // [num_slots] or null: the places of the new tokens (pa_placed)
  int num_slots;
  int give_up;  // self-test: the roles of a CTA act as if their first wait had run out
  void* o;
  float* lse;
  // Partial results: slots [0, ns1) hold the pieces of the prefix, [ns1, ns1 + ns2) those of the
  // own tokens; part_o [slot][T * Hq][d] unnormalised, part_ml [slot][T * Hq] = (row maximum in
  // log2 units, row sum).  A row without keys in a piece has sum 0 and no part_o.
  float* part_o;
  float2* part_ml;
  int ns1, ns2;
  // Pieces of prefix_attn_rows: an item is a kv head and a group of packed rows (prefix) or a
  // request (own keys); *_cta[item] = first and last CTA that worked on it, and CTA c's piece of it
  // is a run of prefix_rows / own_rows rows of item_o [row][d] and item_ml [row] (pa_piece_row).
  int groups;       // row groups of the prefix, 0: the prefix is not among the items
  int2* item_cta;   // [Hk * groups] prefix items, then [B * Hk] own ones
  float* item_o;
  float2* item_ml;
  int prefix_rows, own_rows;
  int item_ctas;  // CTAs that share the items, 0: no items
  int cluster;    // they are one cluster per kv head, which also joins its pieces
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
__device__ __forceinline__ int2* pa_item_cta(const PrefixParams& p, bool prefix, int h, int i) {
  return p.item_cta + (prefix ? (size_t)h * p.groups + i
                              : (size_t)p.Hk * p.groups + (size_t)i * p.Hk + h);
}
// First row of CTA c's piece of an item: kv head h, group or request i.  CTAs and items both only
// grow along the order in which the items' tiles are dealt out, so item + CTA is a place of its
// own; with a cluster per head, the order is within the head.
__device__ __forceinline__ long long pa_piece_row(const PrefixParams& p, bool prefix, int h, int i,
                                                  int c) {
  const long long before =  // pieces of the prefix
      p.groups == 0 ? 0
      : p.cluster   ? (long long)p.Hk * (p.groups + p.item_ctas)
                    : (long long)p.Hk * p.groups + p.item_ctas;
  if (prefix)
    return (p.cluster ? (long long)h * (p.groups + p.item_ctas) + i : (long long)h * p.groups + i) *
               p.prefix_rows + (long long)c * p.prefix_rows;
  return before * p.prefix_rows +
         (p.cluster ? (long long)h * (p.B + p.item_ctas) + i : (long long)i * p.Hk + h) *
             p.own_rows + (long long)c * p.own_rows;
}
// Row tiles of the requests, 1 << shift rows each, as places in a row: request b's start at (its
// first packed row >> shift) + b, which leaves room for a last, partly filled one each, so (T * G
// >> shift) + B places hold them all however the tokens are spread.
inline long long pa_places(int T, int B, int G, int shift) {
  return ((long long)T * G >> shift) + B;
}
// The request of a place and the tile of it (b = -1: none); all lanes of a warp take part.
__device__ __forceinline__ int2 pa_place(const PrefixParams& p, int place, int shift) {
  auto start = [&](int b) {
    return ((min(max(p.cu_q ? p.cu_q[b] : b, 0), p.T) << p.g_shift) >> shift) + b;
  };
  int n = 0;
#pragma unroll 4
  for (int i = 0; i < p.B; i += 32) {
    const int b = i + (threadIdx.x & 31);
    n += __popc(__ballot_sync(0xffffffffu, b < p.B && start(b) <= place));
  }
  return n ? make_int2(n - 1, place - start(n - 1)) : make_int2(-1, 0);
}
// bf16 pairs: the sign bit of each half that holds an infinity or NaN
__device__ __forceinline__ uint32_t pa_nonfinite(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// New tokens in all: rows at or after this are left as they were.
__device__ __forceinline__ int pa_tokens(const PrefixParams& p) {
  return p.cu_q ? min(max(p.cu_q[p.B], 0), p.T) : p.B;
}

// Whether token t has a place in the cache.  One without (its request was refused pages, or no slot
// was left for it) has no position either: where it would stand by its request's length, another
// token is.
__device__ __forceinline__ bool pa_placed(const int* slots, int num_slots, int places, int t) {
  return !slots || (t < num_slots && (unsigned)slots[t] < (unsigned)places);
}
__device__ __forceinline__ bool pa_placed(const PrefixParams& p, int t) {
  return pa_placed(p.slots, p.num_slots, p.num_pages << p.page_shift, t);
}

// Joins the pieces of row (token t, query head hq) and writes o and lse: a warp, d / 32 columns per
// lane.  t is a token of a request.
template <typename T, int D>
__device__ __forceinline__ void pa_join_row(const PrefixParams& p, int t, int hq, int lane) {
  constexpr int C = D / 32;
  const long long rows = (long long)p.T * p.Hq, row = (long long)t * p.Hq + hq;
  int b = t;
  if (p.cu_q) {
    // the request of the token: how many requests end at or before it
    b = 0;
    for (int i = 0; i < p.B; i += 32) {
      const bool before = i + lane < p.B && p.cu_q[i + lane + 1] <= t;
      b += __popc(__ballot_sync(0xffffffffu, before));
    }
    // tokens before the first request and beyond max_q of their own were not attended
    if (b >= p.B || t < p.cu_q[b] || t - p.cu_q[b] >= p.max_q) return;
  }
  // the row's pieces: dense ones, then up to two runs of item slots (first row, rows from one to
  // the next, how many)
  long long first0 = 0, first1 = 0;
  int count0 = 0, count1 = 0;
  if (p.item_ctas) {
    const int h = hq >> p.g_shift, g = hq & (p.G - 1);
    auto pieces = [&](bool prefix, int i, int r, long long& first, int& count) {
      const int2 c = *pa_item_cta(p, prefix, h, i);  // cut, should lengths change under the call
      const int c0 = min(max(c.x, 0), p.item_ctas - 1), c1 = min(max(c.y, c0), p.item_ctas - 1);
      first = pa_piece_row(p, prefix, h, i, c0) + r;
      count = c1 - c0 + 1;
    };
    if (p.groups) {
      const int r = (t << p.g_shift) + g, i = r / p.prefix_rows;  // its group
      pieces(true, i, r - i * p.prefix_rows, first0, count0);
    }
    const PaRequest r = pa_request(p, b);
    if (pa_own_keys(p, r) > 0) pieces(false, b, ((t - r.t0) << p.g_shift) + g, first1, count1);
  }
  const int ns = p.ns1 + p.ns2, n = pa_placed(p, t) ? ns + count0 + count1 : 0;
  auto piece = [&](int s, const float2*& ml, const float*& o) {
    if (s < ns) {
      const long long i = s * rows + row;
      ml = p.part_ml + i;
      o = p.part_o + i * D;
    } else {
      const int e = s - ns;
      const long long i = e < count0 ? first0 + (long long)e * p.prefix_rows
                                     : first1 + (long long)(e - count0) * p.own_rows;
      ml = p.item_ml + i;
      o = p.item_o + i * D;
    }
  };
  // running maximum and sum over the pieces, kAhead of them loaded together
  constexpr int kAhead = 8;
  float top = -INFINITY, l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  for (int s0 = 0; s0 < n; s0 += kAhead) {
    float2 ml[kAhead];
    float x[kAhead][C];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      ml[e] = make_float2(-INFINITY, 0.f);
      if (s0 + e < n) {
        const float2* mp;
        const float* op;
        piece(s0 + e, mp, op);
        ml[e] = *mp;
        load_vec<float, C>(op + lane * C, x[e]);
      }
    }
    float m = top;
#pragma unroll
    for (int e = 0; e < kAhead; ++e) m = fmaxf(m, ml[e].x);
    const float keep = m == -INFINITY ? 1.f : exp2f(top - m);
    top = m;
    l *= keep;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= keep;
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (ml[e].y == 0.f) continue;  // no key in the piece: its o was not written
      const float w = exp2f(ml[e].x - top);
      l += ml[e].y * w;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += x[e][c] * w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // no key at all: o = 0
  T* op = static_cast<T*>(p.o) + row * D + lane * C;
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 w[C / 2];
#pragma unroll
    for (int c = 0; c < C; c += 2) w[c / 2] = __floats2bfloat162_rn(acc[c] * inv, acc[c + 1] * inv);
    if constexpr (C == 4) *reinterpret_cast<uint2*>(op) = *reinterpret_cast<uint2*>(w);
    else *reinterpret_cast<uint32_t*>(op) = *reinterpret_cast<uint32_t*>(w);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2)
      *reinterpret_cast<float2*>(op + c) = make_float2(acc[c] * inv, acc[c + 1] * inv);
  }
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kPaLn2;
}

// The call's kernels are launched as programmatic dependents, so that one's launch and prologue run
// while the one before drains.  pdl_wait: everything queued before is complete and visible.
// pdl_trigger: the next kernel may start once every CTA has said so (or left).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Args>
bool launch_pdl(void (*kern)(Args...), int grid, int cluster, int threads, int smem,
                cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return true;
  (void)cudaGetLastError();
  return false;
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
bsa_status prefix_attn_rows(const PrefixParams& p, int d, int mt, bool after_tc, int* status,
                            cudaStream_t st);

}  // namespace bsa
