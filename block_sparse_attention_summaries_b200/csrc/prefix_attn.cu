// Attention of a batch that shares a long prefix, over a paged K/V cache (bsa_prefix_attn).
//
// Token t, the i-th of nq new tokens of request b, sits at own position p = lens[b] - nq + i and
// sees every key of the prefix and its request's own keys j <= p:
//     o = sum_j softmax_j(q . k_j / sqrt(d)) v_j,   lse = log sum_j exp(q . k_j / sqrt(d)).
// A softmax over two sets of keys joins from each set's maximum m, sum l and weighted values a:
//     M = max(m1, m2),  l = l1 2^(m1 - M) + l2 2^(m2 - M),  o = (a1 2^(m1 - M) + a2 2^(m2 - M)) / l
// (log2 units), so the prefix is attended once for the rows of ALL requests -- packed, token after
// token, into full query tiles, whose keys are then read once per tile and not once per request --
// and each request's own keys only for its own rows.  Both parts may be cut into pieces along the
// keys when there are too few tiles to fill the GPU; prefix_merge_kernel joins a row's
// pieces: bound by L2 (2048 rows of 19 pieces, 20 MB, in 5.6 us) and by latency in small calls, so
// a warp loads eight pieces of its row at a time.
//
// prefix_simt_kernel: float32, CUDA cores (its tensor-core formats would round q, k and the
// weights). A CTA of 128 threads takes RG rows (of one kv head, row = token * G + head of the
// group) and a piece of the keys in tiles of 64 (d = 64) or 32: S = Q K^T in registers from shared
// memory, online softmax with the running maximum of each row in registers of the 8 threads that
// share it, P through shared memory, O += P V in registers.  A warp is 4 x 8 threads of 4 rows and
// 8 keys each (RG = 64, d = 64), so that its reads of Q and of K are one shared-memory wavefront
// each: with 2 x 16 threads of 4 x 4 the wavefronts (79 % of their peak) held the FMAs at 50 % (159
// requests of 16 single-key heads behind 46K keys, d = 64: 1.10 ms; now 1.01 ms, 30 TFLOP/s of the
// CUDA cores' 72).  The next tile is copied (cp.async) while one is worked on, its page ids read a
// tile earlier still: with loads in line a tile took 5 us, the time of two dependent trips to
// memory.
#include <cooperative_groups.h>

#include "prefix_attn.cuh"

namespace bsa {
namespace {

constexpr int kPsThreads = 128;
constexpr int kClusterCtas = 16;  // of a kv head in a small call

template <int D, int RG>
struct SimtSmem {
  static constexpr int kKeys = 4096 / D;  // 16 KB of K or V
  static constexpr int kLd = D + 4;       // floats; rows 4 banks apart
  static constexpr int kLdP = kKeys + 4;
  static constexpr int kQ = 0;
  static constexpr int kTile = kKeys * kLd;
  static constexpr int kKV = kQ + RG * kLd;      // two buffers of K and V
  static constexpr int kP = kKV + 4 * kTile;
  static constexpr int kTotal = (kP + RG * kLdP) * (int)sizeof(float);
};

struct SimtGrid {
  int tiles1;  // tiles of the packed rows
  int tiles2;  // of the requests: one each, or places (pa_place)
};

// The rows and keys of a CTA.
struct SimtUnit {
  int h, r0, nrows;  // rows r0 .. r0 + nrows of kv head h
  int n, first_pos;  // keys [0, n) on `pages`; row r sees keys j <= first_pos + r / G
  const int* pages;
  int slot, piece, pieces;
};

// 16 bytes to shared memory behind the back of the thread; `bytes` 0: zeros
__device__ __forceinline__ void cp_async16(float* dst, const float* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

template <int D, int RG>
__device__ __forceinline__ void simt_unit(const PrefixParams& p, const SimtUnit& un, float* smf) {
  using L = SimtSmem<D, RG>;
  constexpr int TM = RG / 16;           // rows of a thread
  constexpr int NE = L::kKeys / 8;      // keys of a thread's scores
  constexpr int DC = D / 32;            // float4 columns of a thread
  constexpr int RPP = kPsThreads / (D / 4);  // key rows copied at a time
  constexpr int NR = L::kKeys / RPP;         // of each thread
  float *sq = smf + L::kQ, *sp = smf + L::kP;
  const int tid = threadIdx.x, ty = tid >> 3, tx = tid & 7;
  const int h = un.h, r0 = un.r0, nrows = un.nrows, n = un.n, first_pos = un.first_pos;
  const int slot = un.slot, piece = un.piece, pieces = un.pieces;
  const int* pages = un.pages;
  if (nrows <= 0) return;
  const int tiles = (n + L::kKeys - 1) / L::kKeys, per = (tiles + pieces - 1) / pieces;
  const int tile0 = min(piece * per, tiles), tile1 = min(tile0 + per, tiles);

  const long long rows = (long long)p.T * p.Hq;
  auto row_id = [&](int r) {  // of the partial results: token * Hq + query head
    const int rr = r0 + r;
    return (long long)(rr >> p.g_shift) * p.Hq + h * p.G + (rr & (p.G - 1));
  };
  float m[TM], l[TM];
  uint64_t acc[TM][DC * 2];  // columns tx * 4 + 32 c .. in pairs
#pragma unroll
  for (int a = 0; a < TM; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int c = 0; c < DC * 2; ++c) acc[a][c] = 0ull;
  }
  // the thread copies 16 bytes (columns 4 cc ..) of rows cr + RPP i of a tile
  const int cr = tid / (D / 4), cc = tid % (D / 4) * 4;
  int ids[NR];  // their pages, -1: no key
  auto read_ids = [&](int tile) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int j = tile * L::kKeys + cr + RPP * i;
      ids[i] = tile < tile1 && j < n ? pages[j >> p.page_shift] : -1;
    }
  };
  auto copy = [&](int tile) {
    float* dst = smf + L::kKV + (tile & 1) * 2 * L::kTile;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int j = tile * L::kKeys + cr + RPP * i;
      const bool is = ids[i] >= 0 && ids[i] < p.num_pages;
      const long long at =
          is ? (((((long long)ids[i] * p.Hk + h) << p.page_shift) +
                 (j & ((1 << p.page_shift) - 1))) * D) + cc
             : 0;
      cp_async16(dst + (cr + RPP * i) * L::kLd + cc, static_cast<const float*>(p.k) + at,
                 is ? 16 : 0);
      cp_async16(dst + L::kTile + (cr + RPP * i) * L::kLd + cc,
                 static_cast<const float*>(p.v) + at, is ? 16 : 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (tile0 < tile1) {
    read_ids(tile0);
    // queries, scaled to log2 units
    const float scale = rsqrtf((float)D) * kPaLog2e;
    for (int i = tid; i < RG * (D / 4); i += kPsThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        const int rr = r0 + r;
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                             (rr >> p.g_shift) * p.q_stride +
                                             (long long)(h * p.G + (rr & (p.G - 1))) * D + c);
      }
      *reinterpret_cast<float4*>(sq + r * L::kLd + c) =
          make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
    }
    copy(tile0);
    read_ids(tile0 + 1);
  }
  for (int tile = tile0; tile < tile1; ++tile) {
    const int j0 = tile * L::kKeys;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the tile is there, the one before is read
    if (tile + 1 < tile1) {
      copy(tile + 1);
      read_ids(tile + 2);
    }
    const float *sk = smf + L::kKV + (tile & 1) * 2 * L::kTile, *sv = sk + L::kTile;
    // keys tx + 8 e of the tile that exist: in range, on a page of the pool
    uint32_t live = 0;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int j = j0 + tx + 8 * e;
      if (j < n) {
        const int id = pages[j >> p.page_shift];
        if (id >= 0 && id < p.num_pages) live |= 1u << e;
      }
    }
    // scores of rows ty + 16 a and keys tx + 8 e, two columns in a packed FMA
    uint64_t s2[TM][NE];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int e = 0; e < NE; ++e) s2[a][e] = 0ull;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      ulonglong2 kk[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e)
        kk[e] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 8 * e) * L::kLd + c);
#pragma unroll
      for (int a = 0; a < TM; ++a) {
        const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(sq + (ty + 16 * a) * L::kLd + c);
#pragma unroll
        for (int e = 0; e < NE; ++e)
          s2[a][e] = tc::fma_f2(qq.y, kk[e].y, tc::fma_f2(qq.x, kk[e].x, s2[a][e]));
      }
    }
    float s[TM][NE];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        float lo, hi;
        tc::unpack_f2(s2[a][e], lo, hi);
        s[a][e] = lo + hi;
      }
    bool hides = false;  // a row of the thread does not see a key of the tile that exists
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      const int last = first_pos + ((ty + 16 * a) >> p.g_shift);
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const bool sees = j0 + tx + 8 * e <= last;
        hides |= !sees && ((live >> e) & 1);
        if (!((live >> e) & 1) || !sees) s[a][e] = -INFINITY;
        top = fmaxf(top, s[a][e]);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m_new = fmaxf(m[a], top);
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float corr = exp2f(m[a] - base);
      m[a] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const float pe = exp2f(s[a][e] - base);
        sp[(ty + 16 * a) * L::kLdP + tx + 8 * e] = pe;
        sum += pe;
      }
      l[a] = l[a] * corr + sum;  // of the thread's keys
#pragma unroll
      for (int c = 0; c < DC * 2; ++c) acc[a][c] = tc::mul_f2(acc[a][c], tc::pack_f2(corr, corr));
    }
    // a row's P is written and read by 8 threads of one warp
    const bool careful = __any_sync(0xffffffffu, hides);
    __syncwarp();
    auto product = [&](auto check) {
#pragma unroll 2
      for (int j = 0; j < L::kKeys; j += 4) {
        float pj[TM][4];
#pragma unroll
        for (int a = 0; a < TM; ++a) {
          const float4 t = *reinterpret_cast<const float4*>(sp + (ty + 16 * a) * L::kLdP + j);
          pj[a][0] = t.x; pj[a][1] = t.y; pj[a][2] = t.z; pj[a][3] = t.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < DC; ++c) {
            const ulonglong2 vv =
                *reinterpret_cast<const ulonglong2*>(sv + (j + e) * L::kLd + tx * 4 + 32 * c);
#pragma unroll
            for (int a = 0; a < TM; ++a) {
              const float w = pj[a][e];
              // a key that the row does not see adds nothing, whatever its value holds
              if (decltype(check)::value && w == 0.f) continue;
              acc[a][2 * c] = tc::fma_f2(tc::pack_f2(w, w), vv.x, acc[a][2 * c]);
              acc[a][2 * c + 1] = tc::fma_f2(tc::pack_f2(w, w), vv.y, acc[a][2 * c + 1]);
            }
          }
      }
    };
    if (careful) product(std::true_type());
    else product(std::false_type());
  }
#pragma unroll
  for (int a = 0; a < TM; ++a) {
    const int r = ty + 16 * a;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], o);
    if (r >= nrows) continue;
    const long long at = (long long)slot * rows + row_id(r);
    if (tx == 0) p.part_ml[at] = make_float2(m[a], l[a]);
    if (l[a] == 0.f) continue;  // no key (scores of NaN leave the maximum at -inf and l at NaN)
#pragma unroll
    for (int c = 0; c < DC; ++c)
      *reinterpret_cast<ulonglong2*>(p.part_o + at * D + tx * 4 + 32 * c) =
          make_ulonglong2(acc[a][2 * c], acc[a][2 * c + 1]);
  }
}

// Unit u of kv head h: the packed rows' tiles x pieces (RG1 rows each) against the prefix, then the
// requests' (RG2 rows) against their own keys.
template <int D, int RG1, int RG2>
__device__ __forceinline__ void simt_unit_of(const PrefixParams& p, const SimtGrid& g, int h, int u,
                                             float* smf) {
  SimtUnit un;
  un.h = h;
  if (u < g.tiles1 * p.ns1) {
    un.piece = u % p.ns1;
    un.r0 = u / p.ns1 * RG1;
    un.nrows = min(RG1, pa_tokens(p) * p.G - un.r0);
    un.pages = p.ptable;
    un.n = p.prefix_len;
    un.first_pos = un.n;
    un.slot = un.piece;
    un.pieces = p.ns1;
    simt_unit<D, RG1>(p, un, smf);
  } else {
    u -= g.tiles1 * p.ns1;
    un.piece = u % p.ns2;
    u /= p.ns2;
    // 16-row tiles are taken when no request has more than 16 rows: one each
    int2 place = make_int2(u, 0);
    if constexpr (RG2 == 64) place = pa_place(p, u, 6);
    const int tile = place.y, b = max(place.x, 0);
    if (place.x < 0 || tile < 0) return;
    const PaRequest r = pa_request(p, b);
    un.r0 = r.t0 * p.G + tile * RG2;
    un.nrows = min(RG2, min(r.nq, p.max_q) * p.G - tile * RG2);
    un.pages = p.table + (size_t)b * p.table_ld;
    // tiles start at whole tokens: G divides RG2
    un.first_pos = r.len - r.nq + tile * (RG2 / p.G);
    un.n = max(0, min(r.len, un.first_pos + ((un.nrows - 1) >> p.g_shift) + 1));
    un.slot = p.ns1 + un.piece;
    un.pieces = p.ns2;
    simt_unit<D, RG2>(p, un, smf);
  }
}

// A unit per CTA; or, in a small call, a cluster of CTAs per kv head, which takes its units in turn and
// joins their pieces behind a cluster barrier.
template <int D, int RG1, int RG2>
__global__ void __launch_bounds__(kPsThreads, 2) prefix_simt_kernel(const PrefixParams p,
                                                                    const SimtGrid g) {
  extern __shared__ __align__(16) float smf[];
  pdl_wait();
  pdl_trigger();
  const int units1 = g.tiles1 * p.ns1, units2 = g.tiles2 * p.ns2;  // of a head
  if (!p.cluster) {
    // the prefix's units, longer as a rule, of all heads first
    int i = blockIdx.x, h;
    if (i < units1 * p.Hk) {
      h = i / units1;
      i -= h * units1;
    } else {
      i -= units1 * p.Hk;
      h = i / units2;
      i += units1 - h * units2;
    }
    simt_unit_of<D, RG1, RG2>(p, g, h, i, smf);
    return;
  }
  const int h = blockIdx.x / kClusterCtas, me = blockIdx.x % kClusterCtas;
  for (int u = me; u < units1 + units2; u += kClusterCtas) {
    if (u != me) __syncthreads();  // the unit before has been read
    simt_unit_of<D, RG1, RG2>(p, g, h, u, smf);
  }
  cooperative_groups::this_cluster().sync();
  const int n = pa_tokens(p) << p.g_shift, warp = threadIdx.x >> 5;
  for (int r = me * (kPsThreads / 32) + warp; r < n; r += kClusterCtas * (kPsThreads / 32))
    pa_join_row<float, D>(p, r >> p.g_shift, (h << p.g_shift) + (r & (p.G - 1)),
                          threadIdx.x & 31);
}

// Joins the pieces of a row, a warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const PrefixParams p) {
  pdl_wait();
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.T * p.Hq) return;
  const int t = (int)(row / p.Hq);
  if (t < pa_tokens(p))
    pa_join_row<T, D>(p, t, (int)(row - (long long)t * p.Hq), threadIdx.x & 31);
}

// How the keys are cut: enough pieces that `units` CTAs a piece fill `ctas`, none of fewer than
// `least` tiles.
int pieces_for(long long units, long long ctas, long long tiles, int least) {
  const long long want = ctas / std::max(1LL, units);
  return (int)std::max(1LL, std::min(std::min(want, (tiles + least - 1) / least), 64LL));
}

constexpr int kRowsCtas = 2 * kSMs;  // of the few-rows kernel: two per SM
constexpr int kRowsMax = 64;         // its rows
// Key tiles of a kv head up to which a call is small: of the few-rows kernel, of the CUDA cores (a
// tile takes those 2 us: with up to 8 a CTA 10 requests of 500 keys took 57 us instead of 45; with up
// to 2 a call from Python takes 24.4 us instead of 26.2 (4 requests behind 500), while the device,
// which the host keeps waiting, is at it for 16.6 us instead of 12.3)
constexpr long long kClusterTiles = 4 * kClusterCtas, kClusterTiles2 = 2 * kClusterCtas;
// Key tiles of 32 KB (over all heads and row groups) up to which the few-rows kernel takes the
// prefix of more rows: four a CTA.
constexpr long long kPrefixTiles = 4 * kRowsCtas;

// Which kernel does which part.
struct PrefixPlan {
  int rg1, rg2;            // rows of a CUDA-core tile: packed (prefix), of a request (own keys)
  int simt1, simt2;        // such tiles, and places of such tiles (pa_place); 0: not its part
  int tc1, tc2;            // 256-row tiles on the tensor cores, the same way
  bool fused, direct;      // request tiles take the prefix too; one piece in all, no merge
  bool cluster;            // a cluster per kv head, which joins the pieces itself (one launch)
  int mt, groups;          // few-rows kernel: 16-row tiles (0: not used), row groups of the prefix
  int ns1, ns2, prefix_rows, own_rows, item_ctas;
  long long items;
  size_t ml_bytes, o_bytes, cta_bytes, item_ml_bytes, item_o_bytes;
  size_t bytes() const { return ml_bytes + o_bytes + cta_bytes + item_ml_bytes + item_o_bytes; }
};

PrefixPlan plan_of(bsa_dtype dt, int T, int B, int Hq, int Hk, int d, int page, int table_ld,
                   int prefix_len, int max_q) {
  PrefixPlan w = {};
  const int G = Hq / Hk;
  const long long rows = (long long)T * G, rows_q = (long long)max_q * G;
  const long long keys2 = (long long)table_ld * page;
  auto tiles = [](long long n, int of) { return (int)((n + of - 1) / of); };  // of a length
  auto mt_of = [](long long n) { return n <= 16 ? 1 : n <= 32 ? 2 : 4; };
  // 33 to 64 rows a request: its own tensor-core tile costs about 6 us to start and 1 us per 128
  // keys, on 148 SMs; the few-rows kernel 5 us per 32 KB tile, on 296 CTAs (64 requests of 1000 keys
  // and 56 rows: 108 against 131 us; 142 of 13 keys and 36 rows: 105 against 59 us).
  const long long own = (long long)B * Hk;
  const bool few = rows_q <= 32 || (rows_q <= kRowsMax &&
                                    5 * ((own * tiles(keys2, 8192 / d) + kRowsCtas - 1) /
                                         kRowsCtas) <=
                                        (own + kSMs - 1) / kSMs * (6 + tiles(keys2, 128)));
  if (dt == BSA_BF16 && !few) {
    // More: 128-row tiles on the tensor cores.  Requests that fill half a tile on average keep
    // their rows to themselves: prefix and own keys in one pass.  Below that the padding would cost
    // more than the merge.
    w.fused = rows >= 64LL * B;
    w.tc2 = (int)pa_places(T, B, G, 8);
    if (!w.fused && prefix_len) w.tc1 = tiles(rows, 256);
  } else if (dt == BSA_BF16) {
    // The few-rows kernel.  It takes the prefix too where all rows of a kv head fit 16, or where
    // reading the prefix once per row group is cheap; else the rows of all requests fill 128-row
    // tiles (32 rows of d = 64 behind 64K keys: 80 us there, 87 us with 32-row tiles here, whose
    // warps wait for one another more than for HBM).
    w.mt = mt_of(rows_q);
    const int groups = prefix_len ? tiles(rows, 16 * w.mt) : 0;
    if ((groups <= 1 && w.mt == 1) ||
        (long long)groups * Hk * tiles(prefix_len, 8192 / d) <= kPrefixTiles)
      w.groups = groups;
    else
      w.tc1 = tiles(rows, 256);
    w.prefix_rows = 16 * w.mt;
    w.own_rows = (int)rows_q;
    w.items = ((long long)w.groups + B) * Hk;
    // A small call is one launch: a cluster per kv head (4 requests behind 1000 tokens: 11.3 us on
    // the device and 24.5 us a call from Python, as two launches 11.7 and 26.2). With fewer CTAs
    // than the GPU holds it loses that again once each has several tiles.
    w.cluster = !w.tc1 && (long long)w.groups * tiles(prefix_len, 8192 / d) +
                                  (long long)B * tiles(keys2, 8192 / d) <= kClusterTiles;
    w.item_ctas = w.cluster ? kClusterCtas : kRowsCtas;
  } else {
    w.rg2 = rows_q <= 16 ? 16 : 64;
    w.rg1 = w.rg2 == 64 || rows > 32 ? 64 : rows > 16 ? 32 : 16;
    w.simt1 = prefix_len ? tiles(rows, w.rg1) : 0;
    w.simt2 = keys2 ? (w.rg2 == 64 ? (int)pa_places(T, B, G, 6) : B) : 0;
  }
  if (w.tc1) w.ns1 = pieces_for((long long)w.tc1 * Hk, kSMs, (prefix_len + 127) / 128, 4);
  if (w.simt1 || w.simt2) {
    const int t1 = tiles(prefix_len, 4096 / d), t2 = tiles(keys2, 4096 / d);  // of 16 KB
    const long long all = (long long)w.simt1 * t1 + (long long)w.simt2 * t2;
    w.cluster = all <= kClusterTiles2;
    if (w.cluster) {
      const int len = std::max(2, tiles(all, kClusterCtas));  // key tiles of a piece
      w.ns1 = w.simt1 ? tiles(t1, len) : 0;
      w.ns2 = w.simt2 ? tiles(t2, len) : 0;
    } else {
      // Two CTAs per SM: half for the prefix, unless the own keys fill the GPU by themselves.
      const long long own2 = (long long)w.simt2 * Hk;
      if (w.simt1)
        w.ns1 = pieces_for((long long)w.simt1 * Hk, own2 > 2 * kSMs ? 2 * kSMs : kSMs, t1, 2);
      if (w.simt2) w.ns2 = pieces_for(own2, kSMs, t2, 2);
    }
  }
  if (w.tc2)
    w.ns2 = pieces_for((rows + 255) / 256 * Hk, kSMs,
                       (keys2 + (w.fused ? prefix_len : 0) + 127) / 128, 4);
  w.direct = w.tc2 && !w.tc1 && w.ns2 == 1;
  const long long all = w.direct ? 0 : (long long)T * Hq * (w.ns1 + w.ns2);
  w.ml_bytes = align_up((size_t)all * sizeof(float2), 256);
  w.o_bytes = align_up((size_t)all * d * sizeof(float), 256);
  if (w.mt) {
    const size_t ctas = (size_t)w.item_ctas * (w.cluster ? Hk : 1);
    const size_t n = (w.groups ? ((size_t)w.groups * Hk + ctas) * w.prefix_rows : 0) +
                     ((size_t)B * Hk + ctas) * w.own_rows;
    w.cta_bytes = align_up((size_t)w.items * sizeof(int2), 256);
    w.item_ml_bytes = align_up(n * sizeof(float2), 256);
    w.item_o_bytes = n * d * sizeof(float);
  }
  return w;
}

template <int D, int RG1, int RG2>
bsa_status launch_simt(const PrefixParams& p, const PrefixPlan& w, cudaStream_t st) {
  const long long units1 = (long long)w.simt1 * p.Hk * p.ns1;
  const long long units2 = (long long)w.simt2 * p.Hk * p.ns2;
  if (units1 + units2 > INT_MAX) return BSA_ERR_UNSUPPORTED;
  if (units1 + units2 == 0) return BSA_OK;
  const int smem = std::max(SimtSmem<D, RG1>::kTotal, SimtSmem<D, RG2>::kTotal);
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(prefix_simt_kernel<D, RG1, RG2>, smem, done, true) ||
      !launch_pdl(prefix_simt_kernel<D, RG1, RG2>,
                  w.cluster ? kClusterCtas * p.Hk : (int)(units1 + units2),
                  w.cluster ? kClusterCtas : 1, kPsThreads, smem, st, p,
                  SimtGrid{w.simt1, w.simt2}))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

template <typename T, int D>
bsa_status launch_parts(const PrefixParams& p, const PrefixPlan& w, int* status, cudaStream_t st) {
  bsa_status rc = BSA_OK;
  if constexpr (sizeof(T) == 2) {
    rc = prefix_attn_tc(p, D, w.tc1, w.tc2, w.fused, w.direct, status, st);
    if (rc != BSA_OK || w.direct) return rc;
    if (w.mt) rc = prefix_attn_rows(p, D, w.mt, w.tc1 > 0, status, st);
  } else {
    rc = w.rg2 == 64   ? launch_simt<D, 64, 64>(p, w, st)
         : w.rg1 == 64 ? launch_simt<D, 64, 16>(p, w, st)
         : w.rg1 == 32 ? launch_simt<D, 32, 16>(p, w, st)
                       : launch_simt<D, 16, 16>(p, w, st);
  }
  if (rc != BSA_OK || w.cluster) return rc;
  const long long rows = (long long)p.T * p.Hq;
  return launch_pdl(prefix_merge_kernel<T, D>, (int)((rows + 7) / 8), 1, 256, 0, st, p)
             ? BSA_OK
             : BSA_ERR_CUDA;
}

thread_local int t_give_up = 0;  // set by the self-test alone

constexpr int kMaxKeys = INT_MAX - 1024;  // room to round up to tiles

bool sizes_ok(int T, int B, int Hq, int Hk, int d, int page, int table_ld, int prefix_len,
              int max_q) {
  return T >= 0 && B >= 0 && Hq > 0 && Hk > 0 && d > 0 && page > 0 && table_ld >= 0 &&
         prefix_len >= 0 && max_q > 0;
}
bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
int page_shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" size_t bsa_prefix_attn_workspace_bytes(bsa_dtype dt, int T, int B, int Hq, int Hk,
                                                  int d, int page, int table_ld, int prefix_len,
                                                  int max_q) {
  if (!dtype_ok(dt) || !sizes_ok(T, B, Hq, Hk, d, page, table_ld, prefix_len, max_q) ||
      !head_dim_ok(d) || !group_ok(Hq, Hk) || !page_ok(page))
    return 0;
  const PrefixPlan w = plan_of(dt, T, B, Hq, Hk, d, page, table_ld, prefix_len, max_q);
  return w.bytes();
}

extern "C" bsa_status bsa_prefix_attn_slots(
    const void* q, long long q_stride, const void* k_pages, const void* v_pages, bsa_dtype dt, int T,
    int B, int Hq, int Hk, int d, int page, int num_pages, const int* table, int table_ld,
    const int* lens, const int* prefix_table, int prefix_len, const int* cu_q, int max_q,
    const int* slots, int num_slots, void* o, float* lse, int* status, void* workspace,
    size_t workspace_bytes, void* stream) {
  BSA_REQUIRE(sizes_ok(T, B, Hq, Hk, d, page, table_ld, prefix_len, max_q) && num_pages >= 1,
              BSA_ERR_ARG);
  BSA_REQUIRE(num_slots >= 0, BSA_ERR_ARG);
  BSA_REQUIRE(dtype_ok(dt), BSA_ERR_DTYPE);
  BSA_REQUIRE(T == 0 || B == 0 || (q && k_pages && v_pages && lens && o), BSA_ERR_ARG);
  BSA_REQUIRE(prefix_len == 0 || prefix_table, BSA_ERR_ARG);
  BSA_REQUIRE(table_ld == 0 || B == 0 || table, BSA_ERR_ARG);
  BSA_REQUIRE(Hq % Hk == 0, BSA_ERR_SHAPE);
  BSA_REQUIRE(cu_q || (T == B && max_q == 1), BSA_ERR_SHAPE);
  BSA_REQUIRE(max_q <= std::max(T, 1), BSA_ERR_SHAPE);
  BSA_REQUIRE(group_ok(Hq, Hk) && head_dim_ok(d) && page_ok(page), BSA_ERR_UNSUPPORTED);
  // rows of the pool and of the packed queries, and a request's tokens, are 32-bit
  BSA_REQUIRE((long long)num_pages * Hk * page <= INT_MAX && (long long)T * Hq <= INT_MAX &&
                  (long long)T + B <= INT_MAX && prefix_len <= kMaxKeys &&
                  (long long)table_ld * page <= kMaxKeys, BSA_ERR_UNSUPPORTED);
  BSA_REQUIRE(T <= 1 || q_stride >= (long long)Hq * d, BSA_ERR_SHAPE);
  const int es = dt == BSA_BF16 ? 2 : 4;
  BSA_REQUIRE(all_aligned16(q, k_pages, v_pages, o) && (T <= 1 || q_stride * es % 16 == 0),
              BSA_ERR_ARG);
  if (T == 0 || B == 0) return BSA_OK;
  const PrefixPlan w = plan_of(dt, T, B, Hq, Hk, d, page, table_ld, prefix_len, max_q);
  const size_t need = w.bytes();
  BSA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), BSA_ERR_WORKSPACE);
  BSA_REQUIRE(aligned16(workspace), BSA_ERR_ARG);
  PrefixParams p;
  p.q = q; p.k = k_pages; p.v = v_pages;
  p.q_stride = T <= 1 ? (long long)Hq * d : q_stride;
  p.T = T; p.B = B; p.Hq = Hq; p.Hk = Hk; p.G = Hq / Hk;
  p.g_shift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3;
  p.page_shift = page_shift_of(page);
  p.num_pages = num_pages;
  p.table = table; p.table_ld = table_ld; p.lens = lens;
  p.ptable = prefix_table; p.prefix_len = prefix_len;
  p.cu_q = cu_q; p.max_q = max_q;
  p.slots = slots; p.num_slots = num_slots;
  p.give_up = t_give_up;
  p.o = o; p.lse = lse;
  BSA_REQUIRE(w.items <= INT_MAX - kRowsCtas, BSA_ERR_UNSUPPORTED);
  char* ws = static_cast<char*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(ws);
  p.part_o = reinterpret_cast<float*>(ws += w.ml_bytes);
  p.item_cta = reinterpret_cast<int2*>(ws += w.o_bytes);
  p.item_ml = reinterpret_cast<float2*>(ws += w.cta_bytes);
  p.item_o = reinterpret_cast<float*>(ws += w.item_ml_bytes);
  p.ns1 = w.ns1; p.ns2 = w.ns2;
  p.prefix_rows = w.prefix_rows;
  p.own_rows = w.own_rows;
  p.item_ctas = w.item_ctas;
  p.groups = w.groups;
  p.cluster = w.cluster;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dt == BSA_BF16)
    return d == 64 ? launch_parts<__nv_bfloat16, 64>(p, w, status, st)
                   : launch_parts<__nv_bfloat16, 128>(p, w, status, st);
  return d == 64 ? launch_parts<float, 64>(p, w, status, st)
                 : launch_parts<float, 128>(p, w, status, st);
}

extern "C" bsa_status bsa_prefix_attn(const void* q, long long q_stride, const void* k_pages,
                                      const void* v_pages, bsa_dtype dt, int T, int B, int Hq,
                                      int Hk, int d, int page, int num_pages, const int* table,
                                      int table_ld, const int* lens, const int* prefix_table,
                                      int prefix_len, const int* cu_q, int max_q, void* o,
                                      float* lse, int* status, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return bsa_prefix_attn_slots(q, q_stride, k_pages, v_pages, dt, T, B, Hq, Hk, d, page, num_pages,
                               table, table_ld, lens, prefix_table, prefix_len, cu_q, max_q, nullptr,
                               0, o, lse, status, workspace, workspace_bytes, stream);
}

extern "C" bsa_status bsa_selftest_prefix_timeout(int on) {
  t_give_up = on != 0;
  return BSA_OK;
}
