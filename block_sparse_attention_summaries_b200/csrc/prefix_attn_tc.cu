// bsa_prefix_attn on the tensor cores (bf16): 128-row query tiles, tcgen05 with S, P and O in TMEM.
//
// A unit is up to 256 rows of one kv head (row = token * G + head of the group, so one TMA box over
// a (d, G, Hk, T) view of q is a query tile) and a piece of their keys, in tiles of 128.  Rows are
//   packed:  the tokens of ALL requests one after another, against the prefix: its keys are read
//            once per 256 rows whatever the number of requests;
//   request: one request's tokens against its own pages (causal) or, when a request fills tiles by
//            itself, against prefix and own pages in one pass, with nothing to merge.
// One CTA per SM runs two softmax streams, each with its own S / P / O in TMEM (128 + D columns)
// and a warpgroup: while one stream's softmax runs, the tensor cores do the other's products.
//   wide (more than 128 rows):  stream s owns rows 128 s ..; both read every key tile;
//   deep (up to 128 rows):      both own the same rows and take alternate key tiles; the two halves
//                               are joined at the end.  Keys in flight and softmax rate stay the same.
// A tile of 128 x 128 scores needs 16,384 exponentials (1,024 clocks of the SM's 16 per clock) and,
// at d = 128, 1,024 clocks of tensor work.  A step of both streams takes about 3,400 clocks: in it
// a stream waits 900 for its products, 300 for its scores and 450 for their maximum, while the
// other works.  Batches of up to about 256 packed rows are bound by HBM as much as by that.
// Measured at 32 / 8 heads: 7,492 prompt tokens behind 8,192 (1.13 TFLOP) in 0.93 ms, 1,210
// TFLOP/s, 73 % of the cuBLAS burst rate (1.05 ms when run back to back under the power limit, 76 %
// of the sustained rate); 64 decode tokens behind 32K (134 MB, 34 GFLOP) in 39 us; 32 tokens of 16
// single-key heads, d = 64, behind 64K (268 MB) in 55 us, 4.9 TB/s.
//   warps 0-3, 4-7: softmax of stream 0, 1 (a thread owns a row: TMEM lane = row)
//   warp 8: TMA producer; lane i loads box i (a page, or 128 rows of one) of K and V into a ring.  It
//           mends tiles of V that hold what a row must not see, because 0 x NaN would reach it: rows
//           behind the last key, infinities and NaNs of tiles on the diagonal
//   warp 9: MMA issuer (one elected lane)
//   warp 10: adds such infinities and NaNs in the end to the rows that do see them
//   warp 11: none (it completes the helper warpgroup, whose registers the softmax takes)
// P is written over S in TMEM and read from there as the A operand.  S_s of step i + 1 is issued
// behind P V_s of step i, so its completion also says that O_s may be rescaled (lazily: only when a
// row's maximum rises by more than 2^8, else the old maximum stays and P just exceeds 1).
// Every mbarrier wait is bounded; a role whose wait runs out stops, the CTA reaches its last
// barrier, its unit's rows get NaN (of a piece: sum NaN), and it frees TMEM.
#include <cudaTypedefs.h>

#include <mutex>

#include "prefix_attn.cuh"

namespace bsa {
namespace {

constexpr int kXThreads = 384;
// registers: 168 a thread at launch, moved from the helper warpgroup to the softmax warpgroups,
// which hold a row of 128 scores (2 x 216 + 72 = 3 x 168)
constexpr int kXRegsSoftmax = 216, kXRegsHelper = 72;
constexpr int kXKeys = 128;
constexpr float kXRescale = 8.f;  // log2 units
// P goes to the tensor cores in two parts: the product with V of the first kXFirst keys runs while
// the last exponentials are computed
constexpr int kXFirst = 64;
constexpr int kXMend = 8;         // mended tiles under way: more than the ring holds
constexpr int kXMasks = 8;        // key tiles whose page masks are kept: more than the ring holds

template <int D>
struct TcSmem {
  static constexpr int kTile = 128 * D * 2;  // 128 rows: [D / 64][128 x 128 B], 128-byte swizzle
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kTotal = kRing + kSlots * kTile;
};

struct TcGrid {
  int units1;   // CTAs over packed rows
  int tiles1;   // 256-row tiles of the packed rows
  int tiles2;   // places of request tiles (pa_place)
  int fused;    // request units take the prefix too
  int direct;   // one piece in all: o and lse are written here
  int boxes;    // boxes of a key tile (128 / rows of a box)
  int box_shift;
  int* status;
};

// Issue by a warp in step: `leader` is nonzero in the one lane that issues.  The operands are the
// same in all lanes and the warp does not branch, so they stay in uniform registers, which the
// instruction reads; built inside a one-lane branch they are moved there one by one, and 16
// products a step then cost the issuing warp more than the tensor cores (2.6 us a step and unit of
// 256 x 128 scores instead of 1.4).  A descriptor is a constant high word and a low word, start
// address / 16 and the leading offset.
__device__ __forceinline__ int elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return (int)r;
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // rows of 8 x 128 B, swizzled
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, uint32_t lbo_bytes) {
  return (smem_addr >> 4) | ((lbo_bytes >> 4) << 16);
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(int leader, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, c;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.s32 e, %0, 0;\n\tsetp.ne.b32 c, %6, 0;\n\t"
      "mov.b64 a, {%2, %5};\n\tmov.b64 b, {%3, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, c;\n\t}" ::"r"(leader),
      "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "n"(ACC ? 1 : 0)
      : "memory");
}
// the same with A in TMEM
__device__ __forceinline__ void mma_ts(int leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, c;\n\t.reg .b64 b;\n\t"
      "setp.ne.s32 e, %0, 0;\n\tsetp.ne.b32 c, %6, 0;\n\t"
      "mov.b64 b, {%3, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, c;\n\t}" ::"r"(leader),
      "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_one(int leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.s32 e, %0, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(
          leader),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Infinities and NaNs of a tile of V ([halves][128 x 128 B]) to zero; whether there were any.
__device__ __forceinline__ bool clean_tile(unsigned char* vt, int halves, int lane) {
  // a multiply by zero keeps them and nothing else
  __nv_bfloat162 found = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 zero = found;
  const int n = halves * 128 * 8;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const uint4 v = reinterpret_cast<const uint4*>(vt)[i];
    found = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), zero, found);
    found = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), zero, found);
    found = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), zero, found);
    found = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), zero, found);
  }
  const bool dirty = pa_nonfinite(*reinterpret_cast<const uint32_t*>(&found)) != 0;
  if (!__any_sync(0xffffffffu, dirty)) return false;
  for (int i = lane; i < 4 * n; i += 32) {
    uint32_t* w = reinterpret_cast<uint32_t*>(vt) + i;
    *w &= ~((pa_nonfinite(*w) >> 15) * 0xffffu);
  }
  return true;
}

// What a CTA works on.
struct Unit {
  int t0, r0;        // first token; first row among the packed rows (t0 * G)
  int nrows, h, slot;
  int n0, n1;        // keys of the prefix and of the request's own pages
  int tiles0;        // key tiles of the prefix; the own ones follow
  const int* own;    // own pages
  int first_pos;     // row r sees own keys j <= first_pos + r / G
  int tile0, tile1;  // the piece
};

__device__ __forceinline__ Unit unit_of(const PrefixParams& p, const TcGrid& g) {
  Unit u;
  int i = blockIdx.x, piece, pieces;
  if (i < g.units1) {
    piece = i % p.ns1;
    i /= p.ns1;
    const int tile = i % g.tiles1;
    u.h = i / g.tiles1;
    u.r0 = tile * 256;
    u.t0 = u.r0 >> p.g_shift;
    u.nrows = min(256, pa_tokens(p) * p.G - u.r0);
    u.n0 = p.prefix_len;
    u.n1 = 0;
    u.own = nullptr;
    u.first_pos = -1;
    u.slot = piece;
    pieces = p.ns1;
  } else {
    // kv head slowest: the CTAs that run together read the same keys
    i -= g.units1;
    piece = i % p.ns2;
    i /= p.ns2;
    const int2 place = pa_place(p, i % g.tiles2, 8);
    const int b = max(place.x, 0), tile = place.y;
    u.h = i / g.tiles2;
    const PaRequest r = pa_request(p, b);
    u.t0 = r.t0 + tile * (256 >> p.g_shift);
    u.r0 = u.t0 * p.G;
    u.nrows = place.x < 0 || tile < 0 ? 0 : min(256, min(r.nq, p.max_q) * p.G - tile * 256);
    u.first_pos = r.len - r.nq + tile * (256 >> p.g_shift);
    u.n0 = g.fused ? p.prefix_len : 0;
    u.n1 = max(0, min(r.len, u.first_pos + ((u.nrows - 1) >> p.g_shift) + 1));
    u.own = p.table + (size_t)b * p.table_ld;
    u.slot = p.ns1 + piece;
    pieces = p.ns2;
  }
  u.tiles0 = (u.n0 + kXKeys - 1) / kXKeys;
  const int tiles = u.tiles0 + (u.n1 + kXKeys - 1) / kXKeys;
  const int per = (tiles + pieces - 1) / pieces;
  u.tile0 = min(piece * per, tiles);
  u.tile1 = min(u.tile0 + per, tiles);
  return u;
}

// Adds the infinities and NaNs of V at own keys [j0, n) to the results (o, or else part) of the
// rows that see them: a warp.  Not inline and by value, so that it takes no register of the other
// roles.  o is final: rows of tokens without a place keep their 0.
template <int D>
__device__ __noinline__ void add_cleaned(const __nv_bfloat16* v, const int* pages, int num_pages,
                                         int page_shift, int Hk, int h, int j0, int n,
                                         int first_pos, int r0, int nrows, int g_shift, int Hq,
                                         __nv_bfloat16* o, float* part, const int* slots,
                                         int num_slots) {
  for (int i = threadIdx.x & 31; i < nrows * D; i += 32) {
    const int row = i / D, c = i % D, rr = r0 + row;
    if (o && !pa_placed(slots, num_slots, num_pages << page_shift, rr >> g_shift)) continue;
    const int end = min(n, first_pos + (row >> g_shift) + 1);
    float add = 0.f;
    for (int j = j0; j < end; ++j) {
      const int pg = pages[j >> page_shift];
      if (pg < 0 || pg >= num_pages) continue;
      const float f = __bfloat162float(
          v[((((long long)pg * Hk + h) << page_shift) + (j & ((1 << page_shift) - 1))) * D + c]);
      if (!isfinite(f)) add += f;
    }
    if (add == 0.f) continue;
    const long long at = ((long long)(rr >> g_shift) * Hq + (h << g_shift) +
                          (rr & ((1 << g_shift) - 1))) * D + c;
    if (o) o[at] = __float2bfloat16_rn(__bfloat162float(o[at]) + add);
    else part[at] += add;
  }
}

// The end of a CTA that gave up: its unit's rows get NaN (a piece's: sum NaN), whatever the softmax
// warps wrote of tiles that were not there.  Not inline, and the unit is worked out again: nothing is
// kept for this in the registers of the usual way.
template <int D>
__device__ __noinline__ void give_up(const PrefixParams& p, const TcGrid& g) {
  const Unit u = unit_of(p, g);
  if (threadIdx.x == 0) report_timeout(g.status, 5);
  for (int r = threadIdx.x; r < u.nrows; r += kXThreads) {
    const int rr = u.r0 + r;
    const long long id = (long long)(rr >> p.g_shift) * p.Hq + u.h * p.G + (rr & (p.G - 1));
    if (!g.direct) {
      p.part_ml[(long long)u.slot * p.T * p.Hq + id] = make_float2(0.f, NAN);
      continue;
    }
    if (p.lse) p.lse[id] = NAN;
    for (int c = 0; c < D; ++c)
      static_cast<__nv_bfloat16*>(p.o)[id * D + c] = __float2bfloat16_rn(NAN);
  }
}

template <int D>
__global__ void __launch_bounds__(kXThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmq,
                     const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ PrefixParams p, const __grid_constant__ TcGrid g) {
  using L = TcSmem<D>;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_align1024(smem_raw);
  __shared__ __align__(8) uint64_t bars[2 * L::kSlots + kXMasks + 10 + kXMend];
  uint64_t* full = bars;
  uint64_t* empty = full + L::kSlots;
  uint64_t* mask_full = empty + L::kSlots;  // page mask of a key tile written
  uint64_t* q_full = mask_full + kXMasks;
  uint64_t* s_full = q_full + 1;  // [2]
  uint64_t* p_full = s_full + 2;  // [stream][part]
  uint64_t* o_done = p_full + 4;  // [2]
  uint64_t* fin = o_done + 2;     // every product issued is complete
  uint64_t* mended = fin + 1;     // V of a tile is fit for its product
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_dirty;  // first own key of a tile of V that was cleaned
  __shared__ uint32_t s_mask[kXMasks];  // boxes of the key tile that are on pages of the pool

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  pdl_wait();
  pdl_trigger();
  const Unit u = unit_of(p, g);
  if (u.nrows <= 0) return;
  const long long rows = (long long)p.T * p.Hq;
  auto row_id = [&](int r) {
    const int rr = u.r0 + r;
    return (long long)(rr >> p.g_shift) * p.Hq + u.h * p.G + (rr & (p.G - 1));
  };
  if (u.tile0 >= u.tile1) {  // no key: rows of sum 0
    for (int r = tid; r < u.nrows; r += kXThreads) {
      if (g.direct) {
        if (p.lse) p.lse[row_id(r)] = -INFINITY;
        uint4* op = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + row_id(r) * D);
        for (int c = 0; c < D / 8; ++c) op[c] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        p.part_ml[u.slot * rows + row_id(r)] = make_float2(-INFINITY, 0.f);
      }
    }
    return;
  }
  const bool wide = u.nrows > 128;
  const int nt = u.tile1 - u.tile0;
  // steps of stream s and the tile of a step
  auto steps = [&](int s) { return wide ? nt : (nt - s + 1) >> 1; };
  auto tile_at = [&](int s, int i) { return wide ? i : 2 * i + s; };

  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kXMasks; ++i) mbar_init(&mask_full[i], 1);
    for (int i = 0; i < kXMend; ++i) mbar_init(&mended[i], 1);
    mbar_init(q_full, 1);
    mbar_init(fin, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[2 * s], 4);
      mbar_init(&p_full[2 * s + 1], 4);
      mbar_init(&o_done[s], 1);
    }
    fence_mbar_init();
    s_abort = 0;
    s_dirty = INT_MAX;
  }
  if (warp == 9) {
    tc::tmem_alloc(&s_tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tc::prefetch_tmap(&tmq);
    tc::prefetch_tmap(&tmk);
    tc::prefetch_tmap(&tmv);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  auto s_col = [&](int s) { return tmem + (uint32_t)(s * 128); };
  auto o_col = [&](int s) { return tmem + 256u + (uint32_t)(s * 128); };
  auto slot_at = [&](int i) { return smem + L::kRing + i * L::kTile; };
  // Tile ti of the piece needs its V mended before a product: rows without a key (the rest of a
  // last tile, pages outside the pool), or keys that some row does not see.
  auto j0_at = [&](int ti) {  // its first key
    const int t = u.tile0 + ti;
    return (t >= u.tiles0 ? t - u.tiles0 : t) * kXKeys;
  };
  auto left_at = [&](int ti) {  // keys from there on
    return (u.tile0 + ti >= u.tiles0 ? u.n1 : u.n0) - j0_at(ti);
  };
  auto partly = [&](int ti) {
    return u.tile0 + ti >= u.tiles0 && j0_at(ti) + min(left_at(ti), kXKeys) - 1 > u.first_pos;
  };
  auto mends = [&](int ti) {
    return left_at(ti) < kXKeys || s_mask[ti % kXMasks] != (1u << g.boxes) - 1u || partly(ti);
  };
  const uint32_t all_boxes = (1u << g.boxes) - 1u;

  if (warp >= 8) {  // the helper roles
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kXRegsHelper));
  if (warp == 8) {
    // ------------------------------------------------------------------------- producer
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, (wide ? 2 : 1) * L::kTile);
      for (int s = 0; s < (wide ? 2 : 1); ++s)
        for (int hf = 0; hf < kHalves; ++hf)
          tma_load_q(smem + L::kQ + s * L::kTile + hf * 16384, &tmq, hf * 64, u.h,
                     u.t0 + s * (128 >> p.g_shift), q_full);
    }
    // the page of lane's box in tile t, -1: nothing to load
    auto page_of = [&](int t) -> int {
      if (t >= u.tile1 || lane >= g.boxes) return -1;
      const bool own = t >= u.tiles0;
      const int j = (own ? t - u.tiles0 : t) * kXKeys + (lane << g.box_shift);
      if (j >= (own ? u.n1 : u.n0)) return -1;
      const int id = (own ? u.own : p.ptable)[j >> p.page_shift];
      return id >= 0 && id < p.num_pages ? id : -1;
    };
    const uint32_t box_bytes = (uint32_t)(128 << g.box_shift);  // of one 64-column half
    int next = page_of(u.tile0);
    int k = 0, nmend = 0;  // ring position, mended tiles
    bool ok = true;
    for (int i = 0; i < nt && ok; ++i) {
      const int t = u.tile0 + i, id = next;
      next = page_of(t + 1);
      const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
      // a box is one page: a page never exceeds the tile's 128 rows
      const int y = ((id * p.Hk + u.h) << p.page_shift);
      if (lane == 0) {
        s_mask[i % kXMasks] = have;
        mbar_arrive(&mask_full[i % kXMasks]);
      }
      for (int kv = 0; kv < 2; ++kv, ++k) {
        const int sl = k % L::kSlots;
        if (k >= L::kSlots)
          ok = !p.give_up && mbar_wait_bounded(&empty[sl], ((k / L::kSlots) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&full[sl], (uint32_t)__popc(have) * box_bytes * kHalves);
        __syncwarp();
        if (id >= 0)
          for (int hf = 0; hf < kHalves; ++hf)
            tc::tma_load_2d(slot_at(sl) + hf * 16384 + lane * box_bytes, kv ? &tmv : &tmk, hf * 64,
                            y, &full[sl]);
      }
      if (!ok || !mends(i)) continue;
      // the tile's V, once it is there
      const int kv = k - 1, sl = kv % L::kSlots;
      ok = !p.give_up;
      ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&full[sl], (kv / L::kSlots) & 1));
      if (!ok) break;
      unsigned char* vt = slot_at(sl);
      const int j0 = j0_at(i), left = left_at(i);
      for (int r = lane; r < kXKeys; r += 32) {
        if (r < left && ((have >> (r >> g.box_shift)) & 1)) continue;
        for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(vt + hf * 16384 + r * 128 + c * 16) =
                make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
      // an infinity or NaN behind a row's position must not reach it as 0 x NaN: it is zeroed here,
      // and added in the end to the rows that do see it
      if (partly(i) && clean_tile(vt, kHalves, lane) && lane == 0) s_dirty = min(s_dirty, j0);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&mended[nmend % kXMend]);
      ++nmend;
    }
    if (!ok && lane == 0) s_abort = 1;
    // copies still in flight land before the CTA leaves, whatever the other roles do
    (void)mbar_wait_bounded(q_full, 0);
    for (int j = max(0, k - L::kSlots); j < k; ++j)
      (void)mbar_wait_bounded(&full[j % L::kSlots], (j / L::kSlots) & 1);
  } else if (warp == 9) {
    // ----------------------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = tc::idesc_bf16(128, 128, false, false);
    constexpr uint32_t idO = tc::idesc_bf16(128, D, false, true);
    const int leader = elect_one();
    const uint32_t ring = smem_u32(smem + L::kRing), empty0 = smem_u32(empty);
    const uint32_t q_lo = desc_lo(smem_u32(smem + L::kQ), 16);
    const uint32_t q_next = wide ? L::kTile >> 4 : 0;  // to the second stream's queries
    auto ready = [&](int k) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(&full[k % L::kSlots], (k / L::kSlots) & 1));
    };
    // S_s of the stream's step i
    auto issue_s = [&](int s, int i) -> bool {
      const int k = 2 * tile_at(s, i), sl = k % L::kSlots;
      if (!ready(k)) return false;
      tc::fence_after_sync();
      const uint32_t a = q_lo + (s ? q_next : 0), b = desc_lo(ring + sl * L::kTile, 16);
      const uint32_t d = s_col(s);
      mma_ss<false>(leader, d, a, b, idS);
#pragma unroll
      for (int kk = 1; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        mma_ss<true>(leader, d, a + at, b + at, idS);
      }
      commit_one(leader, smem_u32(&s_full[s]));
      if (!wide || s == 1) commit_one(leader, empty0 + 8 * sl);
      return true;
    };
    bool ok = __all_sync(0xffffffffu, !p.give_up && mbar_wait_bounded(q_full, 0));
    int nmend = 0;
    bool any = false;  // products issued
    for (int s = 0; s < 2 && ok; ++s)
      if (steps(s) > 0) any |= (ok = issue_s(s, 0));
    for (int i = 0; i < steps(0) && ok; ++i) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok || i >= steps(s)) continue;
        const int ti = tile_at(s, i), k = 2 * ti + 1, sl = k % L::kSlots;
        ok = ready(k);
        if (!ok) continue;
        // a tile of V that the producer mends first, once per tile
        if ((!wide || s == 0) && mends(ti)) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&mended[nmend % kXMend],
                                                         (nmend / kXMend) & 1));
          ++nmend;
          if (!ok) continue;
        }
        const uint32_t b = desc_lo(ring + sl * L::kTile, 16384);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&p_full[2 * s + part], i & 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int kk = part ? kXFirst / 16 : 0; kk < (part ? kXKeys : kXFirst) / 16; ++kk)
            mma_ts(leader, o_col(s), s_col(s) + kk * 8, b + kk * (2048 >> 4), idO, i + kk > 0);
        }
        if (!ok) continue;
        if (!wide || s == 1) commit_one(leader, empty0 + 8 * sl);
        if (i + 1 == steps(s)) commit_one(leader, smem_u32(&o_done[s]));
        else ok = issue_s(s, i + 1);
      }
    }
    // Every product issued is complete, and every arrival that waits for one is made, before TMEM
    // and shared memory are given up: an arrival behind the CTA's end would hit the next CTA's
    // barriers.
    if (any) {
      commit_one(leader, smem_u32(fin));
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(fin, 0)) && ok;
    }
    if (!ok && lane == 0) s_abort = 1;
  } else if (warp == 10) {
    // ------------------------------------- adds what was cleaned to the rows that do see it
    asm volatile("bar.sync 2, 288;" ::: "memory");  // the results are written
    const int j0 = *(volatile int*)&s_dirty;
    if (j0 < INT_MAX)
      add_cleaned<D>(static_cast<const __nv_bfloat16*>(p.v), u.own, p.num_pages, p.page_shift, p.Hk,
                     u.h, j0, min(u.n1, (u.tile1 - u.tiles0) * kXKeys), u.first_pos, u.r0, u.nrows,
                     p.g_shift, p.Hq, g.direct ? static_cast<__nv_bfloat16*>(p.o) : nullptr,
                     p.part_o + (size_t)u.slot * rows * D, p.slots, p.num_slots);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kXRegsSoftmax));
    // ---------------------------------------------------------------- softmax of stream s
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;  // row of the stream's tile
    const int row = r + (wide ? 128 * s : 0);             // row of the unit
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float scale = rsqrtf((float)D) * kPaLog2e;
    const int pos = u.first_pos + (row >> p.g_shift);
    bool ok = !p.give_up;
    const int ns = ok ? steps(s) : 0;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < ns; ++i) {
      const int ti = tile_at(s, i), t = u.tile0 + ti;
      ok = mbar_wait_bounded(&mask_full[ti % kXMasks], (ti / kXMasks) & 1) &&
           mbar_wait_bounded(&s_full[s], i & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t have = s_mask[ti % kXMasks];
      float x[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) tc::tmem_ld32(s_col(s) + lanes + c, x + c);
      tc::tmem_wait_ld();
      tc::reg_fence(x);
      // columns of the tile the row sees: [0, hi), on pages of the pool
      const bool own = t >= u.tiles0;
      const int j0 = (own ? t - u.tiles0 : t) * kXKeys;
      const int hi =
          (own ? min(u.n1, pos + 1) : u.n0) - j0;
      if (!__all_sync(0xffffffffu, hi >= kXKeys && have == all_boxes)) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int left = hi - 32 * w;
          uint32_t keep = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
          if (have != all_boxes) {
            uint32_t on = 0;
            for (int c = 0; c < 32; c += 16)
              if ((have >> ((32 * w + c) >> g.box_shift)) & 1) on |= 0xffffu << c;
            keep &= on;
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * w + c] = (keep >> c) & 1 ? x[32 * w + c] : -INFINITY;
        }
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < 124; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[c + e], x[c + 4 + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
      const float m_new = fmaxf(m, fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale);
      const bool rescale = m != -INFINITY && m_new > m + kXRescale;
      float corr = 1.f;
      if (rescale) corr = tc::ex2_approx(m - m_new);
      if (rescale || m == -INFINITY) m = m_new;
      if (i > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          tc::tmem_ld32(o_col(s) + lanes + c, ov);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] *= corr;
          tc::tmem_st32(o_col(s) + lanes + c, ov);
        }
      }
      const float neg_m = m == -INFINITY ? 0.f : -m;  // hidden keys give 2^-inf = 0
      const uint64_t sc2 = tc::pack_f2(scale, scale), nm2 = tc::pack_f2(neg_m, neg_m);
      uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c = 0; c < kXKeys; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a0, a1;
          tc::unpack_f2(tc::fma_f2(tc::pack_f2(x[c + e], x[c + e + 1]), sc2, nm2), a0, a1);
          const float p0 = tc::ex2_approx(a0), p1 = tc::ex2_approx(a1);
          sum2[(e >> 1) & 3] = tc::add_f2(sum2[(e >> 1) & 3], tc::pack_f2(p0, p1));
          // weights are rounded to bf16 for the product with V; their sum is not
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
          pk[e / 2] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        tmem_st16(s_col(s) + lanes + c / 2, pk);
        if (c + 32 == kXFirst) {
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * s]);
        }
      }
      float sl[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) tc::unpack_f2(sum2[e], sl[2 * e], sl[2 * e + 1]);
      l = l * corr + (((sl[0] + sl[1]) + (sl[2] + sl[3])) + ((sl[4] + sl[5]) + (sl[6] + sl[7])));
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * s + 1]);
    }
    if (ok && ns > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&o_done[s], 0));
    if (!ok) s_abort = 1;
    tc::fence_after_sync();
    // O to memory through shared memory, so that a warp writes whole rows (a thread writing its own
    // row 16 bytes at a time took 4.4 us a unit).  A deep unit's streams join their halves: TMEM
    // lanes are the rows for both, so each stream's warps read both O and write half the columns.
    float w0 = 1.f, w1 = 0.f;
    unsigned char* stage = smem + L::kQ + s * L::kTile + (warp & 3) * (L::kTile / 4);
    if (!wide) {
      float2* ml = reinterpret_cast<float2*>(smem + L::kQ + L::kTile);  // no second query tile
      ml[s * 128 + r] = make_float2(m, l);
      tc::fence_before_sync();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc::fence_after_sync();
      const float2 a = ml[r], b = ml[128 + r];
      m = fmaxf(a.x, b.x);
      const float base = m == -INFINITY ? 0.f : m;
      w0 = tc::ex2_approx(a.x - base);
      w1 = tc::ex2_approx(b.x - base);
      l = a.y * w0 + b.y * w1;
      stage = smem + L::kRing + warp * (L::kTile / 4);  // both streams have read the ring
    }
    const bool live = row < u.nrows;
    if (g.direct && live && !pa_placed(p, (u.r0 + row) >> p.g_shift)) l = 0.f;  // as without keys
    if (live && (wide || s == 0)) {
      const long long id = row_id(row);
      if (!g.direct) p.part_ml[u.slot * rows + id] = make_float2(m, l);
      else if (p.lse) p.lse[id] = l == 0.f ? -INFINITY : (m + log2f(l)) * kPaLn2;
    }
    if (g.direct) {
      const float inv = 1.f / l;  // a row without a key is set to 0 below
      w0 *= inv;
      w1 *= inv;
    }
    constexpr int PC = D / 2;  // columns of a pass: 32 rows of them fill the warp's share of a tile
    const int row0 = (warp & 3) * 32 + (wide ? 128 * s : 0);  // the warp's first row
    for (int pass = 0; pass < (wide ? 2 : 1); ++pass) {
      const int col = (wide ? pass : s) * PC;
#pragma unroll
      for (int c = 0; c < PC; c += 32) {
        float ov[32];
        tc::tmem_ld32(o_col(wide ? s : 0) + lanes + col + c, ov);
        tc::tmem_wait_ld();
        tc::reg_fence(ov);
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] *= w0;
        if (!wide && nt > 1) {
          float o1[32];
          tc::tmem_ld32(o_col(1) + lanes + col + c, o1);
          tc::tmem_wait_ld();
          tc::reg_fence(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = fmaf(o1[e], w1, ov[e]);
        }
        if (l == 0.f)
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(stage + lane * (PC * 4) +
                                     ((((c + e) >> 2) ^ (lane & (PC / 4 - 1))) << 4)) =
              make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
      }
      __syncwarp();
      constexpr int LR = PC / 4;  // lanes of a row, 16 bytes each
#pragma unroll 4
      for (int i = 0; i < 32; i += 32 / LR) {
        const int rr = i + lane / LR, ch = lane % LR;
        const float4 v = *reinterpret_cast<const float4*>(stage + rr * (PC * 4) +
                                                          ((ch ^ (rr & (LR - 1))) << 4));
        if (row0 + rr >= u.nrows) continue;
        const long long id = row_id(row0 + rr);
        if (g.direct) {
          __nv_bfloat162 b2[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + id * D + col + 4 * ch) =
              *reinterpret_cast<uint2*>(b2);
        } else {
          *reinterpret_cast<float4*>(p.part_o + (u.slot * rows + id) * D + col + 4 * ch) = v;
        }
      }
      __syncwarp();
    }
    asm volatile("bar.arrive 2, 288;" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  if (s_abort) give_up<D>(p, g);
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    else
      (void)cudaGetLastError();
  });
  return fn;
}

template <int D>
bsa_status launch_tc(const PrefixParams& p, const TcGrid& g, int grid, cudaStream_t st) {
  CUtensorMap tmq, tmk, tmv;
  if (!prefix_q_map(&tmq, p, D, 128) || !prefix_kv_map(&tmk, p.k, p, D, g.box_shift) ||
      !prefix_kv_map(&tmv, p.v, p, D, g.box_shift))
    return BSA_ERR_CUDA;
  const int smem = TcSmem<D>::kTotal + 1024;  // + alignment slack
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(prefix_tc_kernel<D>, smem, done) ||
      !launch_pdl(prefix_tc_kernel<D>, grid, 1, kXThreads, smem, st, tmq, tmk, tmv, p, g))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

}  // namespace

bool prefix_q_map(CUtensorMap* m, const PrefixParams& p, int d, int rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)p.G, (cuuint64_t)p.Hk, (cuuint64_t)p.T};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)p.G * d * 2,
                                 (cuuint64_t)p.q_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)p.G, 1, (cuuint32_t)(rows >> p.g_shift)};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.q), dims, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool prefix_kv_map(CUtensorMap* m, const void* pool, const PrefixParams& p, int d, int box_shift) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t ones[2] = {1, 1};
  const cuuint64_t dims[2] = {(cuuint64_t)d, ((cuuint64_t)p.num_pages * p.Hk) << p.page_shift};
  const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)1 << box_shift};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The units of a plan on the tensor cores: packed rows x prefix (tiles1 > 0, p.ns1 pieces) and
// requests x own keys (tiles2 > 0 places, p.ns2 pieces; `fused`: prefix and own keys).
bsa_status prefix_attn_tc(const PrefixParams& p, int d, int tiles1, int tiles2, bool fused,
                          bool direct, int* status, cudaStream_t st) {
  TcGrid g;
  const long long units1 = (long long)tiles1 * p.Hk * p.ns1;
  const long long units2 = (long long)tiles2 * p.Hk * p.ns2;
  if (units1 + units2 > INT_MAX) return BSA_ERR_UNSUPPORTED;
  if (units1 + units2 == 0) return BSA_OK;
  g.units1 = (int)units1;
  g.tiles1 = tiles1;
  g.tiles2 = tiles2;
  g.fused = fused;
  g.direct = direct;
  g.box_shift = p.page_shift;
  g.boxes = kXKeys >> p.page_shift;
  g.status = status;
  const int grid = (int)(units1 + units2);
  return d == 64 ? launch_tc<64>(p, g, grid, st) : launch_tc<128>(p, g, grid, st);
}

}  // namespace bsa
