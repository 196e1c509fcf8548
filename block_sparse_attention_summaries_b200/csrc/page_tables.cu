// Page tables, slot maps and the write of new tokens into a paged K/V cache.
//
// A paged cache keeps K and V as [num_pages, Hk, page, d]; a request's own tokens lie in the pages
// its table row lists, in order.  Free pages wait in a ring: free = {head, avail} says that
// ring[(head + i) mod N], i < avail, are free (N = num_pages = the ring's length).
//
// page_tables_kernel.  One step moves every request from lens[b] to new_lens[b] tokens.  With
// have = ceil(lens / page), want = ceil(new_lens / page), grow = max(0, want - have) and the
// inclusive sum G_b of grow over requests, request b is served iff grow_b = 0 or G_b <= avail (so a
// pool that runs dry refuses whole requests, in order, never half of one), and takes ring entries
// G_b - grow_b .. G_b - 1 behind head.  A shrinking request's pages go to the ring's end in request
// order.  Token t of the packed new tokens belongs to the request whose range of the exclusive sum
// of new tokens holds it, found by a binary search in shared memory unless the 128 tokens of a warp
// step all belong to the request before; a page that moves finds its request the same way.  All
// integer work on a few KB: what bounds it is latency (the lengths' load, a block scan, the
// dependent page-id load), so it is ONE launch: a cluster of up to 16 CTAs, each of which scans all
// requests for itself (one load and a scan are cheaper than a second launch or a grid-wide
// exchange) and then handles its share of the requests' pages and of the tokens.  The cluster
// barrier between reading lens / free and writing lens_out / free_out lets the caller pass the same
// arrays (a state advanced in place). Measured: 5.3 us for a tick of 64 requests, of which 4 are
// the launch and two dependent loads; 14.7 us for 1024 requests with a quarter million new tokens
// (2.3 MB), whose instructions 16 SMs issue.  (With outputs that are none of the inputs nothing needs
// the barrier: what is read behind it -- table entries that stay or leave, ring places head .. head +
// taken -- is disjoint from what is written.  A grid over all SMs could then do such a step.)
//
// paged_append_kernel.  A copy bound by HBM: one 16-byte chunk of K and of V per thread and step,
// neighbouring threads on neighbouring chunks of a head's row (256 B at d = 128 bf16), so reads
// and writes are whole 32-byte sectors whatever the slots' order.
// Measured: 16,384 tokens of 8 x 128 bf16 (134 MB) in 23.3 us, 5.8 TB/s; 64 tokens in 1.9 us.
#include <cooperative_groups.h>

#include "bsa_common.cuh"
#include "launch.cuh"

namespace bsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kPtThreads = 1024;
constexpr int kPtMaxB = 8192;      // requests of a step (shared memory: five ints each)
constexpr int kPtCluster = 16;     // CTAs of a large step
// Up to this many requests + new tokens one CTA does it all: above, its 1024 threads would take
// more than a few rounds.
constexpr int kPtOneCta = 4096;

struct PageTablesParams {
  int B, page_shift, ld, N, max_tokens, pos_offset;
  bool vec4;  // slots and positions start on 16-byte boundaries
  const int *lens, *new_lens;
  int *table, *ring;
  const int* free_in;
  int *lens_out, *free_out, *cu_new, *slots, *positions, *status;
};

struct Sum3 {
  long long grow, drop, add;
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return {a.grow + b.grow, a.drop + b.drop, a.add + b.add};
}
__device__ __forceinline__ Sum3 shfl_up3(const Sum3& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.grow, o), __shfl_up_sync(0xffffffffu, a.drop, o),
          __shfl_up_sync(0xffffffffu, a.add, o)};
}

// What a request asks for; a request whose lengths are impossible asks for nothing.
struct Ask {
  int have, want, add;
  bool bad;
};
__device__ __forceinline__ Ask ask(const PageTablesParams& p, int len, int new_len) {
  Ask a;
  const int top = (1 << p.page_shift) - 1;
  const long long cap = (long long)p.ld << p.page_shift;
  a.bad = len < 0 || new_len < 0 || len > cap || new_len > cap;
  a.have = a.bad ? 0 : (int)(((long long)len + top) >> p.page_shift);
  a.want = a.bad ? 0 : (int)(((long long)new_len + top) >> p.page_shift);
  a.add = a.bad ? 0 : max(0, new_len - len);
  return a;
}

// ring index of a place `off` < N behind head
__device__ __forceinline__ int ring_at(int head, int off, int N) {
  const int i = head + off;  // < 2 N <= 2^28
  return i >= N ? i - N : i;
}

__global__ void __launch_bounds__(kPtThreads, 1) page_tables_kernel(const PageTablesParams p) {
  extern __shared__ int sm[];
  int* s_cu = sm;                  // [B + 1] first new token of the request
  int* s_len = s_cu + p.B + 1;     // [B] tokens before; -1: not served, its tokens get no slot
  int* s_new = s_len + p.B;        // [B] tokens to have
  int* s_take = s_new + p.B;       // [B] ring entries taken by the requests before it
  int* s_drop = s_take + p.B;      // [B] pages freed by the requests before it
  __shared__ Sum3 s_warp[32];
  __shared__ long long s_taken, s_freed;
  __shared__ int s_bits;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int threads = blockDim.x, warps = threads >> 5;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + threads - 1) / threads;  // consecutive requests of a thread
  if (tid == 0) {
    s_taken = 0;
    s_bits = 0;
  }
  // the ring's state, made sane: head in [0, N), avail in [0, N]
  int head = p.free_in[0];
  if (head < 0 || head >= p.N) head = (int)((((long long)head % p.N) + p.N) % p.N);
  const int avail = min(max(p.free_in[1], 0), p.N);

  Sum3 mine = {0, 0, 0};
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b >= p.B) break;
    const int len = p.lens[b], new_len = p.new_lens[b];
    const Ask a = ask(p, len, new_len);
    s_len[b] = len;
    s_new[b] = new_len;
    mine = mine + Sum3{max(0, a.want - a.have), max(0, a.have - a.want), a.add};
  }
  Sum3 upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum3 t = shfl_up3(upto, o);
    if (lane >= o) upto = upto + t;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    Sum3 w = lane < warps ? s_warp[lane] : Sum3{0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sum3 t = shfl_up3(w, o);
      if (lane >= o) w = w + t;
    }
    s_warp[lane] = w;
    if (lane == 31) s_freed = w.drop;
  }
  __syncthreads();
  Sum3 at = upto;  // exclusive sums of the thread's first request
  if (warp > 0) at = at + s_warp[warp - 1];
  at = {at.grow - mine.grow, at.drop - mine.drop, at.add - mine.add};

  int bits = 0;
  long long taken = 0;
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b >= p.B) break;
    const int len = s_len[b];
    const Ask a = ask(p, len, s_new[b]);
    const int grow = max(0, a.want - a.have);
    const bool served = !a.bad && (grow == 0 || at.grow + grow <= avail);
    if (a.bad) bits |= BSA_PAGES_BAD_LENGTH;
    else if (!served) bits |= BSA_PAGES_EXHAUSTED;
    if (served && grow > 0) taken = at.grow + grow;
    s_cu[b] = (int)min(at.add, (long long)INT_MAX);
    s_take[b] = (int)min(at.grow, (long long)INT_MAX);
    s_drop[b] = (int)min(at.drop, (long long)INT_MAX);
    if (!served) {
      s_new[b] = len;  // what it keeps
      s_len[b] = -1;
    }
    at = at + Sum3{grow, max(0, a.have - a.want), a.add};
  }
  if (tid == threads - 1) {  // its exclusive sum over all requests
    s_cu[p.B] = (int)min(at.add, (long long)INT_MAX);
    if (at.add > p.max_tokens) bits |= BSA_PAGES_TOKENS;
  }
  if (taken > 0) atomicMax((unsigned long long*)&s_taken, (unsigned long long)taken);
  if (bits) atomicOr(&s_bits, bits);
  if (ranks > 1) cluster.sync();  // every CTA has read lens, new_lens and free
  else __syncthreads();
  const int freed = (int)min(s_freed, (long long)(p.N - avail));
  if (tid == 0 && s_freed > freed) atomicOr(&s_bits, BSA_PAGES_RING);

  const int all = ranks * threads, me = rank * threads + tid;
  for (int b = me; b < p.B; b += all) {
    p.cu_new[b] = s_cu[b];
    p.lens_out[b] = s_new[b];
  }
  // the last entry of s[0 .. B) that is at most x (s ascends, s[0] = 0): of the requests whose
  // ranges start there, the last is the one that has any
  auto owner = [&](const int* s, int lo, int x) {
    int hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  // pages that join and pages that leave, one after another over all threads
  const int page_mask = (1 << p.page_shift) - 1;
  auto pages_of = [&](int n) { return (int)(((long long)n + page_mask) >> p.page_shift); };
  for (int i = me; i < (int)s_taken; i += all) {
    const int b = owner(s_take, 0, i);
    p.table[(size_t)b * p.ld + pages_of(s_len[b]) + (i - s_take[b])] = p.ring[ring_at(head, i, p.N)];
  }
  for (int i = me; i < freed; i += all) {
    const int b = owner(s_drop, 0, i);
    p.ring[ring_at(head, avail + i, p.N)] =
        p.table[(size_t)b * p.ld + pages_of(s_new[b]) + (i - s_drop[b])];
  }

  // slots and positions of the new tokens: a run of consecutive tokens per warp, 128 at a time,
  // four a lane: they share the search for their request and, as a rule, the page id, and issuing
  // instructions is what a large step takes its time for
  const int gwarp = rank * warps + warp, gwarps = ranks * warps;
  const int total = s_cu[p.B];
  const long long run = (((long long)p.max_tokens + gwarps - 1) / gwarps + 127) / 128 * 128;
  const int t_end = (int)min((long long)p.max_tokens, (gwarp + 1) * run);
  auto page_id = [&](int b, int len, int c) {
    const int have = pages_of(len);
    return c < have ? p.table[(size_t)b * p.ld + c]
                    : p.ring[ring_at(head, s_take[b] + (c - have), p.N)];
  };
  int lo = 0;  // a request whose range starts at or before the warp's tokens
  for (int w0 = (int)min((long long)p.max_tokens, gwarp * run); w0 < t_end; w0 += 128) {
    const int t0 = w0 + 4 * lane;
    int slot[4] = {-1, -1, -1, -1}, pos[4] = {-1, -1, -1, -1};
    if (w0 >= total) {
      // no tokens (nor, without requests, an s_cu[1])
    } else if (w0 + 128 <= s_cu[lo + 1]) {  // all in the request of the tokens before
      const int len = s_len[lo];
      if (len >= 0) {
        const int own = len + (t0 - s_cu[lo]);
        const int c = own >> p.page_shift, c3 = (own + 3) >> p.page_shift;
        int id = page_id(lo, len, c);
        const int id3 = c3 == c ? id : page_id(lo, len, c3);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (own + e) >> p.page_shift == c ? id : id3;
          const bool there = i >= 0 && i < p.N;
          if (!there && t0 + e < p.max_tokens) atomicOr(&s_bits, BSA_PAGES_BAD_ID);
          slot[e] = there ? (i << p.page_shift) + ((own + e) & page_mask) : -1;
          pos[e] = own + e + p.pos_offset;
        }
      }
    } else {
      int b = owner(s_cu, lo, min(t0, total - 1));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        if (t >= total) continue;
        while (s_cu[b + 1] <= t) ++b;
        const int len = s_len[b];
        if (len < 0) continue;
        const int own = len + (t - s_cu[b]);
        const int i = page_id(b, len, own >> p.page_shift);
        const bool there = i >= 0 && i < p.N;
        if (!there && t < p.max_tokens) atomicOr(&s_bits, BSA_PAGES_BAD_ID);
        slot[e] = there ? (i << p.page_shift) + (own & page_mask) : -1;
        pos[e] = own + p.pos_offset;
      }
      lo = __shfl_sync(0xffffffffu, b, 31);
    }
    if (p.vec4 && t0 + 4 <= p.max_tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (p.positions)
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (t0 + e >= p.max_tokens) break;
        p.slots[t0 + e] = slot[e];
        if (p.positions) p.positions[t0 + e] = pos[e];
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (rank == 0) {
      p.cu_new[p.B] = total;
      p.free_out[0] = ring_at(head, (int)s_taken, p.N);
      p.free_out[1] = (int)(avail - s_taken + freed);
    }
    if (s_bits && p.status) atomicOr(p.status, s_bits);
  }
}

// K and V rows of new tokens to their slots; V is the chunk type (16 bytes, or one element when a
// row does not start on a 16-byte boundary).
template <typename V>
__global__ void __launch_bounds__(256) paged_append_kernel(
    const unsigned char* __restrict__ k, const unsigned char* __restrict__ v, long long k_stride,
    long long v_stride, const int* __restrict__ slots, int T, int Hk, int row_shift,
    int page_shift, int num_pages, V* __restrict__ kp, V* __restrict__ vp) {
  // chunk c of head h of token t; a head's row has 1 << row_shift chunks
  const int chunks = Hk << row_shift;
  const long long n = (long long)T * chunks;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n;
       i += (long long)gridDim.x * 256) {
    const int t = (int)(i / chunks), hc = (int)(i - (long long)t * chunks);
    const int slot = slots[t];
    const V a = reinterpret_cast<const V*>(k + t * k_stride)[hc];
    const V b = reinterpret_cast<const V*>(v + t * v_stride)[hc];
    const int id = slot >> page_shift;
    if (slot < 0 || id >= num_pages) continue;
    const int h = hc >> row_shift, c = hc & ((1 << row_shift) - 1);
    const long long row =
        (((long long)id * Hk + h) << page_shift) + (slot & ((1 << page_shift) - 1));
    kp[(row << row_shift) + c] = a;
    vp[(row << row_shift) + c] = b;
  }
}

template <typename V>
void launch_append(const void* k, const void* v, long long ks, long long vs, const int* slots,
                   int T, int Hk, int row_bytes, int page_shift, int num_pages, void* kp, void* vp,
                   cudaStream_t st) {
  int row_shift = 0;
  while ((int)sizeof(V) << row_shift < row_bytes) ++row_shift;
  const long long n = (long long)T * (Hk << row_shift);
  const int grid = (int)std::min<long long>((n + 255) / 256, 8LL * kSMs * 4);
  paged_append_kernel<V><<<grid, 256, 0, st>>>(
      static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v), ks, vs, slots, T,
      Hk, row_shift, page_shift, num_pages, static_cast<V*>(kp), static_cast<V*>(vp));
}

int page_shift_of(int page) {
  for (int s = 4; s <= 7; ++s)
    if (page == 1 << s) return s;
  return -1;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" bsa_status bsa_page_tables(int B, int page, const int* lens, const int* new_lens,
                                      int* table, int table_ld, int* ring, int num_pages,
                                      const int* free_in, int* lens_out, int* free_out,
                                      int* cu_new, int* slots, int* positions, int max_tokens,
                                      int pos_offset, int* status, void* stream) {
  BSA_REQUIRE(B >= 0 && max_tokens >= 0 && table_ld >= 0 && page > 0 && num_pages >= 1,
              BSA_ERR_ARG);
  BSA_REQUIRE(free_in && free_out && cu_new && ring, BSA_ERR_ARG);
  BSA_REQUIRE(B == 0 || (lens && new_lens && lens_out && (table || table_ld == 0)), BSA_ERR_ARG);
  BSA_REQUIRE(slots || max_tokens == 0, BSA_ERR_ARG);
  const int shift = page_shift_of(page);
  BSA_REQUIRE(shift > 0 && B <= kPtMaxB, BSA_ERR_UNSUPPORTED);
  // slots and a row's tokens are 32-bit
  BSA_REQUIRE((long long)num_pages << shift <= INT_MAX && (long long)table_ld << shift <= INT_MAX,
              BSA_ERR_UNSUPPORTED);
  BSA_REQUIRE(pos_offset >= 0 && (long long)pos_offset + ((long long)table_ld << shift) <= INT_MAX,
              BSA_ERR_ARG);
  BSA_REQUIRE(max_tokens <= INT_MAX - kPtCluster * kPtThreads * 4, BSA_ERR_UNSUPPORTED);
  PageTablesParams p = {B,        shift,    table_ld, num_pages, max_tokens, pos_offset,
                        all_aligned16(slots, positions),
                        lens,     new_lens, table,    ring,      free_in,    lens_out,
                        free_out, cu_new,   slots,    positions, status};
  const int smem = (5 * B + 1) * (int)sizeof(int);
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(page_tables_kernel, (5 * kPtMaxB + 1) * (int)sizeof(int), done, true))
    return BSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const long long work = (long long)B + max_tokens;
  // One CTA to an SM (48 registers a thread).  With 8 CTAs 263K tokens of 1024 requests took 20.0 us,
  // with 16 14.7; 2.2M tokens of 8192 requests 111 and 67 us.
  const unsigned ctas = work <= kPtOneCta ? 1u : kPtCluster;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  // a small step needs no more threads than it has items; fewer warps meet faster at the barriers
  cfg.blockDim = dim3(work <= 256 ? 256 : kPtThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, page_tables_kernel, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return BSA_ERR_CUDA;
  }
  return BSA_OK;
}

extern "C" bsa_status bsa_paged_append(const void* k, const void* v, bsa_dtype dt, int T, int Hk,
                                       int d, long long k_stride, long long v_stride,
                                       const int* slots, int page, int num_pages, void* k_pages,
                                       void* v_pages, void* stream) {
  BSA_REQUIRE(T >= 0 && Hk > 0 && d > 0 && page > 0 && num_pages >= 1, BSA_ERR_ARG);
  BSA_REQUIRE(dtype_ok(dt), BSA_ERR_DTYPE);
  BSA_REQUIRE(T == 0 || (k && v && slots && k_pages && v_pages), BSA_ERR_ARG);
  const int shift = page_shift_of(page);
  BSA_REQUIRE(head_dim_ok(d) && shift > 0, BSA_ERR_UNSUPPORTED);
  BSA_REQUIRE((long long)num_pages << shift <= INT_MAX && Hk <= 4096, BSA_ERR_UNSUPPORTED);
  BSA_REQUIRE(T <= 1 || (k_stride >= (long long)Hk * d && v_stride >= (long long)Hk * d),
              BSA_ERR_SHAPE);
  BSA_REQUIRE(all_aligned16(k_pages, v_pages), BSA_ERR_ARG);
  if (T == 0) return BSA_OK;
  const int es = dt == BSA_BF16 ? 2 : 4;
  BSA_REQUIRE(((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & (es - 1)) == 0,
              BSA_ERR_ARG);
  const long long ks = k_stride * es, vs = v_stride * es;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (all_aligned16(k, v) && (T == 1 || (ks % 16 == 0 && vs % 16 == 0)))
    launch_append<uint4>(k, v, ks, vs, slots, T, Hk, d * es, shift, num_pages, k_pages, v_pages,
                         st);
  else if (es == 2)
    launch_append<uint16_t>(k, v, ks, vs, slots, T, Hk, d * es, shift, num_pages, k_pages, v_pages,
                            st);
  else
    launch_append<uint32_t>(k, v, ks, vs, slots, T, Hk, d * es, shift, num_pages, k_pages, v_pages,
                            st);
  BSA_LAUNCH_CHECK();
  return BSA_OK;
}
