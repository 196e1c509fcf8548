// bsa_prefix_attn for few query rows per key (bf16): a request's own keys in decode (G rows, or a
// few drafted tokens' worth, up to 16) and, for the smallest batches, the prefix (all rows of a kv
// head together, up to 16).  Such rows read each key once for at most 16 rows: HBM-bound by a
// factor of ten, so the kernel is a stream of keys with as much of it in flight as fits.
//
// An item is (request, kv head) -- or (prefix, kv head) -- and its keys in tiles of 64.  The tiles of
// all items, one after another, are cut into equal runs, one per CTA (two CTAs per SM), whatever
// the requests' lengths: a CTA's producer warp walks its run without stopping at item borders, so
// the ring of tiles stays full while the consumers change rows.  An item is then cut into at most
// the pieces that its CTAs saw; piece (item, CTA) is stored at slot item + CTA, unique because both
// only grow along the run, and the merge kernel joins an item's slots.
//   warps 0-3: per tile, S of 16 keys each (mma.sync m16n8k16: an M = 128 tcgen05 tile would be
//              padding for 1/8 of its rows or less, and HBM bounds the rate at a tenth of either);
//              the row maxima meet in shared memory, each warp exponentiates its keys, P meets in
//              shared memory, then each warp multiplies all 64 keys into its d / 4 output columns,
//              so no accumulator is joined across warps
//   warp 4:    TMA producer; lane i loads box i (a page, or 64 rows of one) of K and V, and with a
//              piece's first tile its query rows.  Its lanes hold the ranges of the next 32
//              requests, and page ids are read a tile ahead, so that an item border costs it no
//              wait for memory (items of one tile took 5 us each before, 64 x 64 tokens x 8 heads
//              15.8 us in all)
// V rows without a key are masked to zero in the registers that feed the products.
#include "prefix_attn.cuh"

namespace bsa {
namespace {

constexpr int kRThreads = 160;
constexpr int kRKeys = 64;
constexpr float kRRescale = 8.f;  // log2 units: O is rescaled when a row's maximum rises by more

template <int D>
struct RowsSmem {
  static constexpr int kHalf = kRKeys * 128;         // 64 rows x 128 B, 128-byte swizzle
  static constexpr int kTile = (D / 64) * kHalf;     // K or V
  static constexpr int kStages = D == 128 ? 3 : 6;   // 96 KB in flight per CTA
  static constexpr int kP = kStages * 2 * kTile;     // two buffers of [16 x 64] bf16
  static constexpr int kQTile = (D / 64) * 2048;     // 16 query rows: [D / 64][16 x 128 B]
  static constexpr int kQ = kP + 2 * 2048;           // two buffers: of alternate pieces
  static constexpr int kTotal = kQ + 2 * kQTile;
};

// What the producer tells the consumers about a tile.
struct TileInfo {
  int item, nrows, first_pos;
  int j0, n;      // its first key; keys of the item
  uint32_t have;  // boxes on pages of the pool | first tile of the run's piece << 8 | last << 9
                  // | query buffer << 10
};

struct RowsGrid {
  int prefix_items;  // Hk, or 0: the prefix is not this kernel's part
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

template <int D>
__global__ void __launch_bounds__(kRThreads, 2)
    prefix_rows_kernel(const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const PrefixParams p,
                       const RowsGrid g) {
  using L = RowsSmem<D>;
  constexpr int NT = D / 32;  // 8-column output tiles of a warp
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_align1024(smem_raw);
  __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], q_free[2];
  __shared__ TileInfo s_info[L::kStages];
  __shared__ long long s_sum[kRThreads];
  __shared__ float s_max[2][4][16], s_l[2][4][16];
  __shared__ int s_abort, s_stop;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Behind the tensor-core kernel the inputs are already there (it has waited for them before it
  // let this one start); its own results are only the merge's concern, which waits for this kernel.
  if (!g.after_tc) pdl_wait();
  pdl_trigger();

  // tiles of all requests, a run of consecutive requests per thread
  const int per = (p.B + kRThreads - 1) / kRThreads;
  long long mine = 0;
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b)
    mine += (pa_own_keys(p, pa_request(p, b)) + kRKeys - 1) / kRKeys;
  s_sum[tid] = mine;
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
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
  const int ptiles = g.prefix_items ? (p.prefix_len + kRKeys - 1) / kRKeys : 0;
  const long long total = (long long)p.Hk * (ptiles + s_sum[kRThreads - 1]);
  // no CTA within a run of pieces may be without one: at most as many CTAs work as there are tiles
  const long long ctas = min((long long)gridDim.x, total);
  if (blockIdx.x >= ctas) {
    if (g.after_tc) pdl_wait();  // this kernel is not complete before the one before it
    return;
  }
  const long long f0 = total * blockIdx.x / ctas, f1 = total * (blockIdx.x + 1) / ctas;
  const int count = (int)(f1 - f0);

  if (warp == 4) {
    // ------------------------------------------------------------------------- producer
    // where the run is: request (-1: the prefix), kv head, tile of the item
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
    if (f0 < (long long)p.Hk * ptiles) {
      c.b = -1;
      c.h = (int)(f0 / ptiles);
      c.tile = (int)(f0 - (long long)c.h * ptiles);
      c.tiles = ptiles;
      c.n = c.first_pos = p.prefix_len;
      c.t0 = 0;
      c.nrows = pa_tokens(p) << p.g_shift;
    } else {
      const long long f = f0 - (long long)p.Hk * ptiles;
      int th = 0;
      while ((long long)p.Hk * s_sum[th] <= f) ++th;
      long long before = th ? s_sum[th - 1] : 0;
      enter(c, th * per);
      while ((long long)p.Hk * (before + c.tiles) <= f) {
        before += c.tiles;
        enter(c, c.b + 1);
      }
      const int rest = (int)(f - (long long)p.Hk * before);
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
    for (; done < count; ++done) {
      const int st = done % L::kStages;
      const bool ends = c.tile + 1 == c.tiles;
      // the next place, and its pages on their way
      Place nx = c;
      if (!ends) {
        ++nx.tile;
      } else if (done + 1 < count) {
        nx.tile = 0;
        if (++nx.h == p.Hk) {
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
      if (done >= L::kStages) ok = mbar_wait_bounded(&empty[st], ((done / L::kStages) - 1) & 1);
      if (first && piece >= 2)
        ok = ok && mbar_wait_bounded(&q_free[piece & 1], ((piece >> 1) - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        TileInfo t;
        t.item = c.b < 0 ? c.h : g.prefix_items + c.b * p.Hk + c.h;
        t.nrows = c.nrows;
        t.first_pos = c.first_pos;
        t.j0 = c.tile * kRKeys;
        t.n = c.n;
        t.have = have | (first ? 256u : 0u) | (last ? 512u : 0u) | (uint32_t)(piece & 1) << 10;
        s_info[st] = t;
        if (c.tile == 0) p.item_cta[t.item].x = blockIdx.x;
        if (ends) p.item_cta[t.item].y = blockIdx.x;
        mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(have) * box_bytes * (D / 64) * 2 +
                                             (first ? (uint32_t)L::kQTile : 0u));
        if (first)
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_q(smem + L::kQ + (piece & 1) * L::kQTile + hf * 2048, &tmq, hf * 64, c.h, c.t0,
                       &full[st]);
      }
      __syncwarp();
      if (id >= 0) {
        // a page of 128 holds two boxes
        const int j = c.tile * kRKeys + (lane << g.box_shift);
        const int y = ((id * p.Hk + c.h) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        unsigned char* dst = smem + st * 2 * L::kTile + lane * box_bytes;
        for (int hf = 0; hf < D / 64; ++hf)
          tc::tma_load_2d_hint(dst + hf * L::kHalf, &tmk, hf * 64, y, &full[st], pol);
        for (int hf = 0; hf < D / 64; ++hf)
          tc::tma_load_2d_hint(dst + L::kTile + hf * L::kHalf, &tmv, hf * 64, y, &full[st], pol);
      }
      if (last) ++piece;
      first = last;
      c = nx;
      id = next_id;
    }
    if (!ok && lane == 0) s_abort = 1;
    // copies still in flight land before the CTA leaves, whatever the consumers do
    for (int i = max(0, done - L::kStages); i < done; ++i)
      (void)mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1);
  } else {
    // ------------------------------------------------------------------------ consumers
    const float scale = rsqrtf((float)D) * kPaLog2e;
    const int qr = lane >> 2, qc = (lane & 3) * 2;  // row (and row + 8), first column of a pair
    const int mat = lane >> 3, mrow = lane & 7;
    uint32_t q[D / 16][4];
    float acc[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    for (int i = 0; i < count; ++i) {
      const int st = i % L::kStages, buf = i & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[st], (i / L::kStages) & 1));
      if (!ok) {
        // the consumers stop together, behind the tile's first barrier
        s_stop = s_abort = 1;
        bar_consumers();
        break;
      }
      const TileInfo t = s_info[st];
      if (t.have & 256u) {  // a new piece
        const int qb = (t.have >> 10) & 1;
        const uint32_t qt = smem_u32(smem + L::kQ + qb * L::kQTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ldsm4(q[kk], qt + (kk >> 2) * 2048 +
                           tc::sw128_offset(mrow + (mat & 1) * 8, (kk & 3) * 2 + (mat >> 1)));
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_free[qb]);
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }
      const uint32_t kt = smem_u32(smem + st * 2 * L::kTile), vt = kt + L::kTile;
      // scores of keys 16 warp .. of the tile
      float s[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b[4];
        ldsm4(b, kt + (kk >> 2) * L::kHalf +
                     tc::sw128_offset(16 * warp + mrow + (mat >> 1) * 8, (kk & 3) * 2 + (mat & 1)));
        mma16816(s[0], q[kk], b[0], b[1]);
        mma16816(s[1], q[kk], b[2], b[3]);
      }
      const int left = t.n - t.j0;  // keys of the tile
      const uint32_t all = (1u << (kRKeys >> g.box_shift)) - 1u;
      const bool part = left < kRKeys || (t.have & all) != all;
      // a key of the tile that exists
      auto is_key = [&](int j) { return j < left && ((t.have >> (j >> g.box_shift)) & 1); };
      const int pos[2] = {t.first_pos + (qr >> p.g_shift) - t.j0,
                          t.first_pos + ((qr + 8) >> p.g_shift) - t.j0};
      if (part || pos[0] < kRKeys - 1) {  // rows only look further down the tile
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 16 * warp + 8 * c + qc + (e & 1);
            if (!is_key(j) || j > pos[e >> 1]) s[c][e] = -INFINITY;
          }
      }
      float top[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        top[a] = fmaxf(fmaxf(s[0][2 * a], s[0][2 * a + 1]), fmaxf(s[1][2 * a], s[1][2 * a + 1]));
        top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 1));
        top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 2));
        if ((lane & 3) == 0) s_max[buf][warp][qr + 8 * a] = top[a];
      }
      bar_consumers();
      if (*(volatile int*)&s_stop) break;  // set before this barrier or not at all in this tile
      bool move = false;
      float corr[2] = {1.f, 1.f};
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int row = qr + 8 * a;
        const float x = fmaxf(fmaxf(s_max[buf][0][row], s_max[buf][1][row]),
                              fmaxf(s_max[buf][2][row], s_max[buf][3][row])) * scale;
        if (m[a] == -INFINITY) {
          m[a] = x;
        } else if (x > m[a] + kRRescale) {
          corr[a] = tc::ex2_approx(m[a] - x);
          m[a] = x;
          move = true;
        }
        const float neg = m[a] == -INFINITY ? 0.f : -m[a];
        float pe[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          pe[e] = tc::ex2_approx(fmaf(s[e >> 1][2 * a + (e & 1)], scale, neg));
        l[a] = l[a] * corr[a] + ((pe[0] + pe[1]) + (pe[2] + pe[3]));
        // weights are rounded to bf16 for the product with V; their sum is not
        unsigned char* pb = smem + L::kP + buf * 2048;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<uint32_t*>(pb + tc::sw128_offset(row, 2 * warp + c) + qc * 2) =
              pack_bf16(pe[2 * c], pe[2 * c + 1]);
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[c][e] *= corr[e >> 1];
      }
      bar_consumers();
      const uint32_t pb = smem_u32(smem + L::kP + buf * 2048);
#pragma unroll
      for (int ks = 0; ks < kRKeys / 16; ++ks) {
        uint32_t a[4];
        ldsm4(a, pb + tc::sw128_offset(mrow + (mat & 1) * 8, 2 * ks + (mat >> 1)));
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (part)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 16 * ks + 8 * e + qc;
            keep[e] = (is_key(j) ? 0xffffu : 0u) | (is_key(j + 1) ? 0xffff0000u : 0u);
          }
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
          const int col = warp * (D / 4) + c * 8;
          uint32_t b[4];
          ldsm4_t(b, vt + (col >> 6) * L::kHalf +
                         tc::sw128_offset(16 * ks + mrow + (mat & 1) * 8,
                                          ((col & 63) >> 3) + (mat >> 1)));
          mma16816(acc[c], a, b[0] & keep[0], b[1] & keep[1]);
          mma16816(acc[c + 1], a, b[2] & keep[0], b[3] & keep[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (t.have & 512u) {  // the piece's last tile
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float x = l[a];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if ((lane & 3) == 0) s_l[buf][warp][qr + 8 * a] = x;
        }
        bar_consumers();
        const long long slot = (long long)(t.item + (int)blockIdx.x) * p.item_rows;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int row = qr + 8 * a;
          if (row >= t.nrows) continue;
          const float sum =
              (s_l[buf][0][row] + s_l[buf][1][row]) + (s_l[buf][2][row] + s_l[buf][3][row]);
          if (warp == 0 && (lane & 3) == 0) p.item_ml[slot + row] = make_float2(m[a], sum);
          float* op = p.item_o + (slot + row) * D + warp * (D / 4) + qc;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            *reinterpret_cast<float2*>(op + 8 * c) = make_float2(acc[c][2 * a], acc[c][2 * a + 1]);
        }
      }
    }
  }
  __syncthreads();
  if (s_abort && tid == 0) report_timeout(g.status, 6);
  if (g.after_tc) pdl_wait();  // this kernel is not complete before the one before it
}

template <int D>
bsa_status launch_rows(const PrefixParams& p, const RowsGrid& g, cudaStream_t st) {
  CUtensorMap tmq, tmk, tmv;
  if (!prefix_q_map(&tmq, p, D, 16) || !prefix_kv_map(&tmk, p.k, p, D, g.box_shift) ||
      !prefix_kv_map(&tmv, p.v, p, D, g.box_shift))
    return BSA_ERR_CUDA;
  const int smem = RowsSmem<D>::kTotal + 1024;  // + alignment slack
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(prefix_rows_kernel<D>, smem, done) ||
      !launch_pdl(prefix_rows_kernel<D>, p.item_ctas, kRThreads, smem, st, tmq, tmk, tmv, p, g))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

}  // namespace

// Own keys of every request and, with `prefix`, the prefix, for up to 16 rows each.
bsa_status prefix_attn_rows(const PrefixParams& p, int d, bool prefix, bool after_tc, int* status,
                            cudaStream_t st) {
  RowsGrid g;
  g.prefix_items = prefix ? p.Hk : 0;
  g.box_shift = std::min(p.page_shift, 6);
  g.after_tc = after_tc;
  g.status = status;
  return d == 64 ? launch_rows<64>(p, g, st) : launch_rows<128>(p, g, st);
}

}  // namespace bsa
