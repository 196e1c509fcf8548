// bsa_prefix_attn for few query rows per key (bf16): a request's own keys in decode or with a few
// drafted tokens (up to 64 rows) and, where they are few, the prefix.  Such rows read each key once
// for at most 64 rows: HBM-bound, so the kernel is a stream of keys with as much of it in flight as
// fits.
//
// An item is (request, kv head) -- or (prefix, kv head, group of packed rows) -- and its keys in
// tiles of 64 (d = 128) or 128 (d = 64).  The tiles of all items, one after another, are cut into
// equal runs, one per CTA (two CTAs per SM), whatever the requests' lengths: a CTA's producer warp
// walks its run without stopping at item borders, so the ring of tiles stays full while the
// consumers change rows.  An item is then cut into at most the pieces that its CTAs saw; piece
// (item, CTA) is stored at slot item + CTA, unique because both only grow along the run, and the
// merge kernel joins an item's slots.  In a small call a cluster of CTAs does this per kv head and
// joins the pieces itself behind a cluster barrier.
//   warps 0-3: per tile, S of 16 or 32 keys each for MT tiles of 16 rows (mma.sync m16n8k16: an M = 128
//              tcgen05 tile would be padding for half its rows or more, and HBM bounds the rate far
//              below either); the row maxima meet in shared memory, each warp exponentiates its
//              keys, P meets in shared memory, then each warp multiplies all keys into its d / 4 output
//              columns, so no accumulator is joined across warps
//   warp 4:    TMA producer; lane i loads box i (a page, or a tile's rows of one) of K and V, and with a
//              piece's first tile its query rows.  Its lanes hold the ranges of the next 32
//              requests, and page ids are read a tile ahead, so that an item border costs it no
//              wait for memory (items of one tile took 5 us each before, 64 x 64 tokens x 8 heads
//              15.8 us in all, now 11.2 us)
// V rows without a key are masked to zero in the registers that feed the products.
// Measured at 32 / 8 heads, d = 128: 512 requests of 1024 own tokens (2.15 GB) in 343 us, 6.3 TB/s;
// 64 of up to 1024 (144 MB) in 26 us.
#include <cooperative_groups.h>

#include "prefix_attn.cuh"

namespace bsa {
namespace {

constexpr int kRThreads = 160;
constexpr float kRRescale = 8.f;  // log2 units: O is rescaled when a row's maximum rises by more

template <int D, int MT>
struct RowsSmem {
  // keys of a tile: 32 KB of K and V; the barriers and shuffles of a tile cost the same at d = 64
  // as at d = 128 (64-key tiles at d = 64: 117 us where this takes 70)
  static constexpr int kKeys = 8192 / D;
  static constexpr int kHalf = kKeys * 128;       // rows x 128 B, 128-byte swizzle
  static constexpr int kTile = (D / 64) * kHalf;  // K or V
  // K and V tiles alternate in the ring; two CTAs share the SM's 227 KB
  static constexpr int kSlots = MT == 1 ? 6 : MT == 2 ? 5 : 4;
  static constexpr int kPHalf = MT * 2048;        // [16 MT x 64] bf16
  static constexpr int kPTile = kPHalf * kKeys / 64;
  static constexpr int kQHalf = MT * 2048;        // 16 MT query rows x 128 B
  static constexpr int kQTile = (D / 64) * kQHalf;
  static constexpr int kQBufs = MT == 4 ? 1 : 2;              // of successive pieces
  static constexpr int kP = kSlots * kTile;                   // two buffers
  static constexpr int kQ = kP + 2 * kPTile;
  static constexpr int kTotal = kQ + kQBufs * kQTile;
};

// What the producer tells the consumers about a tile.
struct TileInfo {
  int prefix, h, i;  // item: of the prefix or not, kv head, group or request
  int nrows, first_pos;
  int j0, n;      // its first key; keys of the item
  uint32_t have;  // boxes on pages of the pool | first tile of the run's piece << 16 | last << 17
                  // | query buffer << 18
};

constexpr uint32_t kFirst = 1u << 16, kLast = 1u << 17;

struct RowsGrid {
  int box_shift;     // rows of a box
  int after_tc;      // a kernel of the same call runs before: its results are not read here
  int* status;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Adds the infinities and NaNs of V at own keys [j0, n), D / 4 columns from col, to the rows that
// see them: a warp, which has written those columns.  Not inline: it runs for bad values only.
template <int D>
__device__ __noinline__ void add_cleaned(const __nv_bfloat16* v, const int* pages, int num_pages,
                                         int page_shift, int Hk, int h, int j0, int n,
                                         int first_pos, int nrows, int g_shift, float* out,
                                         int col) {
  for (int i = threadIdx.x & 31; i < nrows * (D / 4); i += 32) {
    const int row = i / (D / 4), c = col + i % (D / 4);
    const int end = min(n, first_pos + (row >> g_shift) + 1);
    float add = 0.f;
    for (int j = j0; j < end; ++j) {
      const int pg = pages[j >> page_shift];
      if (pg < 0 || pg >= num_pages) continue;
      const float f = __bfloat162float(
          v[((((long long)pg * Hk + h) << page_shift) + (j & ((1 << page_shift) - 1))) * D + c]);
      if (!isfinite(f)) add += f;
    }
    if (add != 0.f) out[row * D + c] += add;
  }
}

// The pieces of a CTA that gave up: the tiles [f0, f1) of the call (of the cluster's head), in the
// order in which they are dealt out.  Their rows get sum NaN, whatever was written of them, so that the
// join cannot take what an earlier call left in the workspace for their results.  A warp; not inline,
// as it runs after a timeout only.
__device__ __noinline__ void give_up(const PrefixParams& p, int keys, int group_rows, long long f0,
                                     long long f1) {
  const int heads = p.cluster ? 1 : p.Hk, head0 = p.cluster ? blockIdx.x / p.item_ctas : 0;
  const int me = p.cluster ? blockIdx.x % p.item_ctas : blockIdx.x;
  const int lane = threadIdx.x & 31;
  long long at = 0;  // the item's first tile
  auto item = [&](bool prefix, int h, int i, int n, int nrows) {
    const int tiles = (n + keys - 1) / keys;
    if (at < f1 && at + tiles > f0) {
      if (lane == 0) {
        if (at >= f0) pa_item_cta(p, prefix, h, i)->x = me;
        if (at + tiles <= f1) pa_item_cta(p, prefix, h, i)->y = me;
      }
      const long long row = pa_piece_row(p, prefix, h, i, me);
      for (int r = lane; r < nrows; r += 32) p.item_ml[row + r] = make_float2(0.f, NAN);
    }
    at += tiles;
  };
  for (int h = 0; h < heads; ++h)
    for (int i = 0; i < p.groups; ++i)
      item(true, head0 + h, i, p.prefix_len,
           min((pa_tokens(p) << p.g_shift) - i * group_rows, group_rows));
  for (int b = 0; b < p.B; ++b) {
    const PaRequest r = pa_request(p, b);
    for (int h = 0; h < heads; ++h)
      item(false, head0 + h, b, pa_own_keys(p, r), min(r.nq, p.max_q) << p.g_shift);
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(kRThreads, 2)
    prefix_rows_kernel(const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ PrefixParams p, const RowsGrid g) {
  using L = RowsSmem<D, MT>;
  constexpr int kRKeys = L::kKeys;
  constexpr int NT = D / 32;                   // 8-column output tiles of a warp
  constexpr int NS = kRKeys / 32;              // 8-key score tiles of a warp
  constexpr int kInfos = (L::kSlots + 1) / 2;  // tiles that the ring can hold, a started one included
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_align1024(smem_raw);
  __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], q_free[2];
  __shared__ TileInfo s_info[kInfos + 1];
  __shared__ long long s_sum[kRThreads];
  __shared__ float s_max[2][4][16 * MT], s_l[2][4][16 * MT];
  __shared__ int s_abort, s_stop;
  __shared__ long long s_run[2];  // the CTA's tiles
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // Behind the tensor-core kernel the inputs are already there: it has waited for them before it
  // let this one start.  The fence is so that this SM's L1 holds nothing older than that.  Its own
  // results are only the merge's concern, which waits for this kernel.
  if (g.after_tc) __threadfence();
  else pdl_wait();
  pdl_trigger();

  // tiles of all requests, a run of consecutive requests per thread
  const int per = (p.B + kRThreads - 1) / kRThreads;
  long long mine = 0;
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b)
    mine += (pa_own_keys(p, pa_request(p, b)) + kRKeys - 1) / kRKeys;
  s_sum[tid] = mine;
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    mbar_init(&q_free[0], 4);
    mbar_init(&q_free[1], 4);
    fence_mbar_init();
    s_abort = s_stop = 0;
  }
  __syncthreads();
  if (warp == 0) {  // inclusive sums
    long long carry = 0;
    for (int i = 0; i < kRThreads; i += 32) {
      long long x = s_sum[i + lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x += carry;
      s_sum[i + lane] = x;
      carry = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int ptiles = p.groups ? (p.prefix_len + kRKeys - 1) / kRKeys : 0;
  // the heads whose tiles are dealt out: all, or the cluster's
  const int heads = p.cluster ? 1 : p.Hk, head0 = p.cluster ? blockIdx.x / p.item_ctas : 0;
  const int me = p.cluster ? blockIdx.x % p.item_ctas : blockIdx.x;
  const int pitems = heads * p.groups;
  const long long total = (long long)pitems * ptiles + (long long)heads * s_sum[kRThreads - 1];
  // no CTA within a run of pieces may be without one: at most as many CTAs work as there are tiles
  const long long ctas = min((long long)p.item_ctas, total);
  const long long f0 = me < ctas ? total * me / ctas : 0;
  const int count = me < ctas ? (int)(total * (me + 1) / ctas - f0) : 0;
  if (tid == 0) {
    s_run[0] = f0;
    s_run[1] = f0 + count;
  }

  if (count == 0) {
    // nothing to attend
  } else if (warp == 4) {
    // ------------------------------------------------------------------------- producer
    // where the run is: request (-1: the prefix), head of the run's (prefix: head * groups +
    // group), tile of the item
    struct Place {
      int b, h, tile, tiles, n, t0, nrows, first_pos;
    } c;
    // the ranges of requests base .. base + 31, one per lane
    int base = -64;
    PaRequest mine_r = {};
    auto enter = [&](Place& x, int b) {
      if (b >= base + 32) {
        base = b;
        mine_r = pa_request(p, min(b + lane, p.B - 1));
      }
      PaRequest r;
      r.t0 = __shfl_sync(0xffffffffu, mine_r.t0, b - base);
      r.nq = __shfl_sync(0xffffffffu, mine_r.nq, b - base);
      r.len = __shfl_sync(0xffffffffu, mine_r.len, b - base);
      x.b = b;
      x.n = pa_own_keys(p, r);
      x.tiles = (x.n + kRKeys - 1) / kRKeys;
      x.t0 = r.t0;
      x.nrows = min(r.nq, p.max_q) << p.g_shift;
      x.first_pos = r.len - r.nq;
    };
    const int prefix_rows = p.groups ? pa_tokens(p) << p.g_shift : 0;
    auto enter_prefix = [&](Place& x, int h) {
      const int r0 = h % p.groups * 16 * MT;
      x.b = -1;
      x.h = h;
      x.tiles = ptiles;
      x.n = x.first_pos = p.prefix_len;
      x.t0 = r0 >> p.g_shift;
      x.nrows = min(prefix_rows - r0, 16 * MT);
    };
    if (f0 < (long long)pitems * ptiles) {
      enter_prefix(c, (int)(f0 / ptiles));
      c.tile = (int)(f0 - (long long)c.h * ptiles);
    } else {
      const long long f = f0 - (long long)pitems * ptiles;
      int th = 0;
      while ((long long)heads * s_sum[th] <= f) ++th;
      long long before = th ? s_sum[th - 1] : 0;
      enter(c, th * per);
      while ((long long)heads * (before + c.tiles) <= f) {
        before += c.tiles;
        enter(c, c.b + 1);
      }
      const int rest = (int)(f - (long long)heads * before);
      c.h = rest / c.tiles;
      c.tile = rest - c.h * c.tiles;
    }
    const int boxes = kRKeys >> g.box_shift;
    const uint32_t box_bytes = (uint32_t)(128 << g.box_shift);
    const uint64_t pol = l2_evict_first();
    // the page of the lane's box at a place, -1: nothing to load
    auto page_at = [&](const Place& x) {
      const int j = x.tile * kRKeys + (lane << g.box_shift);
      if (lane >= boxes || j >= x.n) return -1;
      const int id = (x.b < 0 ? p.ptable : p.table + (size_t)x.b * p.table_ld)[j >> p.page_shift];
      return id < p.num_pages ? id : -1;
    };
    bool ok = true, first = true;
    int done = 0, piece = 0;
    int id = page_at(c);
    int k = 0;  // loads issued: ring position
    for (; done < count; ++done) {
      const bool ends = c.tile + 1 == c.tiles;
      // the next place, and its pages on their way
      Place nx = c;
      if (!ends) {
        ++nx.tile;
      } else if (done + 1 < count) {
        nx.tile = 0;
        ++nx.h;
        if (nx.b < 0 && nx.h < pitems) {
          enter_prefix(nx, nx.h);
        } else if (nx.b < 0 || nx.h == heads) {
          nx.h = 0;
          do {
            ok = nx.b + 1 < p.B;  // holds unless the lengths change under the call
            if (ok) enter(nx, nx.b + 1);
          } while (ok && nx.tiles == 0);
          if (!ok) break;
        }
      }
      const int next_id = done + 1 < count ? page_at(nx) : -1;
      const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
      const bool last = ends || done + 1 == count;
      const int kh = head0 + (c.b < 0 ? c.h / p.groups : c.h);
      const int qb = piece % L::kQBufs;
      // a page of 128 holds two boxes
      const int j = c.tile * kRKeys + (lane << g.box_shift);
      const int y = ((id * p.Hk + kh) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int sl = k % L::kSlots;
        if (k >= L::kSlots)
          ok = !p.give_up && mbar_wait_bounded(&empty[sl], ((k / L::kSlots) - 1) & 1);
        const bool queries = first && kv == 0;
        if (queries && piece >= L::kQBufs)
          ok = ok && mbar_wait_bounded(&q_free[qb], ((piece / L::kQBufs) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          if (kv == 0) {
            TileInfo t;
            t.prefix = c.b < 0;
            t.h = kh;
            t.i = c.b < 0 ? c.h % p.groups : c.b;
            t.nrows = c.nrows;
            t.first_pos = c.first_pos;
            t.j0 = c.tile * kRKeys;
            t.n = c.n;
            t.have = have | (first ? kFirst : 0u) | (last ? kLast : 0u) | (uint32_t)qb << 18;
            s_info[done % (kInfos + 1)] = t;
            if (c.tile == 0) pa_item_cta(p, c.b < 0, kh, t.i)->x = me;
            if (ends) pa_item_cta(p, c.b < 0, kh, t.i)->y = me;
          }
          mbar_arrive_expect_tx(&full[sl], (uint32_t)__popc(have) * box_bytes * (D / 64) +
                                               (queries ? (uint32_t)L::kQTile : 0u));
          if (queries)
            for (int hf = 0; hf < D / 64; ++hf)
              tma_load_q(smem + L::kQ + qb * L::kQTile + hf * L::kQHalf, &tmq, hf * 64, kh, c.t0,
                         &full[sl]);
        }
        __syncwarp();
        if (id >= 0)
          for (int hf = 0; hf < D / 64; ++hf)
            tc::tma_load_2d_hint(smem + sl * L::kTile + hf * L::kHalf + lane * box_bytes,
                                 kv ? &tmv : &tmk, hf * 64, y, &full[sl], pol);
        ++k;
      }
      if (!ok) break;
      if (last) ++piece;
      first = last;
      c = nx;
      id = next_id;
    }
    if (!ok && lane == 0) s_abort = 1;
    // copies still in flight land before the CTA leaves, whatever the consumers do
    for (int i = max(0, k - L::kSlots); i < k; ++i)
      (void)mbar_wait_bounded(&full[i % L::kSlots], (i / L::kSlots) & 1);
  } else {
    // ------------------------------------------------------------------------ consumers
    const float scale = rsqrtf((float)D) * kPaLog2e;
    const int qr = lane >> 2, qc = (lane & 3) * 2;  // row (and row + 8), first column of a pair
    const int mat = lane >> 3, mrow = lane & 7;
    const uint32_t base = smem_u32(smem);
    // one row tile keeps its queries in registers; more read them from shared memory for each tile
    uint32_t q[MT == 1 ? D / 16 : 1][4];
    float acc[MT][NT][4], m[MT][2], l[MT][2];
    int dirty = INT_MAX;  // first key of a tile whose V was cleaned, in this piece
    int k = 0;
    const int todo = p.give_up ? 0 : count;
    if (p.give_up) s_abort = 1;
    for (int i = 0; i < todo; ++i, k += 2) {
      const int buf = i & 1;
      const int ks = k % L::kSlots, vs = (k + 1) % L::kSlots;
      bool ok = mbar_wait_bounded(&full[ks], (k / L::kSlots) & 1) &&
                mbar_wait_bounded(&full[vs], ((k + 1) / L::kSlots) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        // the consumers stop together, behind the tile's first barrier
        s_stop = s_abort = 1;
        bar_consumers();
        break;
      }
      const TileInfo t = s_info[i % (kInfos + 1)];
      const uint32_t qt = base + L::kQ + ((t.have >> 18) & 1) * L::kQTile;
      auto load_q = [&](uint32_t (&r)[4], int mt, int kk) {
        ldsm4(r, qt + (kk >> 2) * L::kQHalf +
                     tc::sw128_offset(16 * mt + mrow + (mat & 1) * 8, (kk & 3) * 2 + (mat >> 1)));
      };
      if (t.have & kFirst) {  // a new piece
        if constexpr (MT == 1) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) load_q(q[kk], 0, kk);
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_free[(t.have >> 18) & 1]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][c][e] = 0.f;
          m[mt][0] = m[mt][1] = -INFINITY;
          l[mt][0] = l[mt][1] = 0.f;
        }
        dirty = INT_MAX;
      }
      const uint32_t kt = base + ks * L::kTile, vt = base + vs * L::kTile;
      // scores of keys 8 NS warp .. of the tile
      float s[MT][NS][4] = {};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b[NS / 2][4];
#pragma unroll
        for (int c = 0; c < NS / 2; ++c)
          ldsm4(b[c], kt + (kk >> 2) * L::kHalf +
                          tc::sw128_offset(8 * NS * warp + 16 * c + mrow + (mat >> 1) * 8,
                                           (kk & 3) * 2 + (mat & 1)));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          if constexpr (MT > 1) load_q(a, mt, kk);
#pragma unroll
          for (int c = 0; c < NS; ++c) {
            if constexpr (MT == 1) mma16816(s[0][c], q[kk], b[c / 2][c % 2 * 2], b[c / 2][c % 2 * 2 + 1]);
            else mma16816(s[mt][c], a, b[c / 2][c % 2 * 2], b[c / 2][c % 2 * 2 + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty[ks]);
        if (MT > 1 && (t.have & kLast)) mbar_arrive(&q_free[(t.have >> 18) & 1]);
      }
      const int left = t.n - t.j0;  // keys of the tile
      const uint32_t all = (1u << (kRKeys >> g.box_shift)) - 1u;
      const bool part = left < kRKeys || (t.have & all) != all;
      // a key of the tile that exists
      auto is_key = [&](int j) { return j < left && ((t.have >> (j >> g.box_shift)) & 1); };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int pos[2] = {t.first_pos + ((16 * mt + qr) >> p.g_shift) - t.j0,
                            t.first_pos + ((16 * mt + qr + 8) >> p.g_shift) - t.j0};
        if (part || pos[0] < kRKeys - 1) {  // later rows only look further down the tile
#pragma unroll
          for (int c = 0; c < NS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * (NS * warp + c) + qc + (e & 1);
              if (!is_key(j) || j > pos[e >> 1]) s[mt][c][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float top = fmaxf(s[mt][0][2 * a], s[mt][0][2 * a + 1]);
#pragma unroll
          for (int c = 1; c < NS; ++c)
            top = fmaxf(top, fmaxf(s[mt][c][2 * a], s[mt][c][2 * a + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if ((lane & 3) == 0) s_max[buf][warp][16 * mt + qr + 8 * a] = top;
        }
      }
      bar_consumers();
      if (*(volatile int*)&s_stop) break;  // set before this barrier or not at all in this tile
      unsigned char* pb = smem + L::kP + buf * L::kPTile;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        bool move = false;
        float corr[2] = {1.f, 1.f};
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int row = 16 * mt + qr + 8 * a;
          const float x = fmaxf(fmaxf(s_max[buf][0][row], s_max[buf][1][row]),
                                fmaxf(s_max[buf][2][row], s_max[buf][3][row])) * scale;
          float& ma = m[mt][a];
          if (ma == -INFINITY) {
            ma = x;
          } else if (x > ma + kRRescale) {
            corr[a] = tc::ex2_approx(ma - x);
            ma = x;
            move = true;
          }
          const float neg = ma == -INFINITY ? 0.f : -ma;
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < NS; ++c) {
            const float p0 = tc::ex2_approx(fmaf(s[mt][c][2 * a], scale, neg));
            const float p1 = tc::ex2_approx(fmaf(s[mt][c][2 * a + 1], scale, neg));
            sum += p0 + p1;
            // weights are rounded to bf16 for the product with V; their sum is not
            const int ch = NS * warp + c;  // 16-byte chunk of the row: 8 keys
            *reinterpret_cast<uint32_t*>(pb + (ch >> 3) * L::kPHalf +
                                         tc::sw128_offset(row, ch & 7) + qc * 2) =
                pack_bf16(p0, p1);
          }
          l[mt][a] = l[mt][a] * corr[a] + sum;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][c][e] *= corr[e >> 1];
        }
      }
      bar_consumers();
      // some row sees the tile in part: an infinity or NaN behind its position must not reach it as
      // 0 x NaN; it is zeroed here and added at the end to the rows that see it
      if (t.j0 + min(left, kRKeys) - 1 > t.first_pos) {
        uint32_t found = 0;
        constexpr int NC = D / 32;  // 16-byte chunks of the warp's columns
        for (int e = lane; e < kRKeys * NC; e += 32) {
          const int ch = warp * NC + e % NC;
          uint32_t* w = reinterpret_cast<uint32_t*>(smem + vs * L::kTile + (ch >> 3) * L::kHalf +
                                                    tc::sw128_offset(e / NC, ch & 7));
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            // keys that do not exist are masked below
            const uint32_t bad = pa_nonfinite(w[f]);
            if (bad) w[f] &= ~((bad >> 15) * 0xffffu);
            if (is_key(e / NC)) found |= bad;
          }
        }
        fence_proxy_async();  // the next copy into the slot comes after these writes
        if (__any_sync(0xffffffffu, found != 0)) dirty = min(dirty, t.j0);
        __syncwarp();
      }
#pragma unroll
      for (int kk = 0; kk < kRKeys / 16; ++kk) {
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (part)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 16 * kk + 8 * e + qc;
            keep[e] = (is_key(j) ? 0xffffu : 0u) | (is_key(j + 1) ? 0xffff0000u : 0u);
          }
        uint32_t v[NT / 2][4];
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
          const int col = warp * (D / 4) + c * 8;
          ldsm4_t(v[c / 2], vt + (col >> 6) * L::kHalf +
                                tc::sw128_offset(16 * kk + mrow + (mat & 1) * 8,
                                                 ((col & 63) >> 3) + (mat >> 1)));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[c / 2][e] &= keep[e & 1];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          ldsm4(a, smem_u32(pb) + (kk >> 2) * L::kPHalf +
                       tc::sw128_offset(16 * mt + mrow + (mat & 1) * 8,
                                        (kk & 3) * 2 + (mat >> 1)));
#pragma unroll
          for (int c = 0; c < NT; c += 2) {
            mma16816(acc[mt][c], a, v[c / 2][0], v[c / 2][1]);
            mma16816(acc[mt][c + 1], a, v[c / 2][2], v[c / 2][3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[vs]);
      if (t.have & kLast) {  // the piece's last tile
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            float x = l[mt][a];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if ((lane & 3) == 0) s_l[buf][warp][16 * mt + qr + 8 * a] = x;
          }
        bar_consumers();
        const long long slot = pa_piece_row(p, t.prefix, t.h, t.i, me);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int row = 16 * mt + qr + 8 * a;
            if (row >= t.nrows) continue;
            const float sum =
                (s_l[buf][0][row] + s_l[buf][1][row]) + (s_l[buf][2][row] + s_l[buf][3][row]);
            if (warp == 0 && (lane & 3) == 0) p.item_ml[slot + row] = make_float2(m[mt][a], sum);
            float* op = p.item_o + (slot + row) * D + warp * (D / 4) + qc;
#pragma unroll
            for (int c = 0; c < NT; ++c)
              *reinterpret_cast<float2*>(op + 8 * c) =
                  make_float2(acc[mt][c][2 * a], acc[mt][c][2 * a + 1]);
          }
        if (dirty < INT_MAX) {
          __syncwarp();
          add_cleaned<D>(static_cast<const __nv_bfloat16*>(p.v),
                         p.table + (size_t)t.i * p.table_ld, p.num_pages, p.page_shift, p.Hk, t.h,
                         dirty, min(t.n, t.j0 + kRKeys), t.first_pos, t.nrows, p.g_shift,
                         p.item_o + slot * D, warp * (D / 4));
        }
      }
    }
  }
  __syncthreads();
  if (s_abort) {
    if (tid == 0) report_timeout(g.status, 6);
    if (warp == 0) give_up(p, kRKeys, 16 * MT, s_run[0], s_run[1]);
  }
  if (g.after_tc) pdl_wait();  // this kernel is not complete before the one before it
  if (p.cluster) {
    // the head's pieces are all written: join its rows here
    cooperative_groups::this_cluster().sync();
    const int n = pa_tokens(p) << p.g_shift;
    for (int r = me * (kRThreads / 32) + warp; r < n; r += p.item_ctas * (kRThreads / 32))
      pa_join_row<__nv_bfloat16, D>(p, r >> p.g_shift, (head0 << p.g_shift) + (r & (p.G - 1)), lane);
  }
}

template <int D, int MT>
bsa_status launch_rows(const PrefixParams& p, const RowsGrid& g, cudaStream_t st) {
  using L = RowsSmem<D, MT>;
  CUtensorMap tmq, tmk, tmv;
  if (!prefix_q_map(&tmq, p, D, 16 * MT) || !prefix_kv_map(&tmk, p.k, p, D, g.box_shift) ||
      !prefix_kv_map(&tmv, p.v, p, D, g.box_shift))
    return BSA_ERR_CUDA;
  const int smem = L::kTotal + 1024;  // + alignment slack
  static_assert(2 * (L::kTotal + 1024 + 4096 + 1024) <= 228 * 1024, "two CTAs per SM");
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(prefix_rows_kernel<D, MT>, smem, done, true) ||
      !launch_pdl(prefix_rows_kernel<D, MT>, p.item_ctas * (p.cluster ? p.Hk : 1),
                  p.cluster ? p.item_ctas : 1, kRThreads, smem, st, tmq, tmk, tmv, p, g))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

}  // namespace

// Own keys of every request, with up to 16 mt rows each, and the prefix for p.groups groups of as
// many packed rows.
bsa_status prefix_attn_rows(const PrefixParams& p, int d, int mt, bool after_tc, int* status,
                            cudaStream_t st) {
  RowsGrid g;
  g.box_shift = std::min(p.page_shift, d == 64 ? 7 : 6);
  g.after_tc = after_tc;
  g.status = status;
  if (d == 64)
    return mt == 1 ? launch_rows<64, 1>(p, g, st)
         : mt == 2 ? launch_rows<64, 2>(p, g, st) : launch_rows<64, 4>(p, g, st);
  return mt == 1 ? launch_rows<128, 1>(p, g, st)
       : mt == 2 ? launch_rows<128, 2>(p, g, st) : launch_rows<128, 4>(p, g, st);
}

}  // namespace bsa
