// Attention of a drafted tree of tokens over a paged cache, for sm_100a.
//
// Sequence b has len cache rows, the last n of them its drafted nodes; node i sees the
// context, rows [0, len - n), and of the drafted rows its own and its ancestors'.  The query
// rows of one KV head are all n nodes times the G query heads of its group, so one pass over
// the cached K and V serves n G rows.
//
// Bound: the cache bytes, 4 d a row and KV head, while n G stays under about 250 rows (measured
// tensor rate over measured bandwidth); above that the two products.  So the work is cut by
// cache rows and not by sequences: a unit is one 128-key tile of one (sequence, KV head, block
// of query rows) segment, and every CTA of a persistent grid takes an equal run of
// consecutive units, whatever the lengths are.  The lengths are read on the device: each CTA
// takes the prefix sums over the sequences itself, nothing is planned on the host and a
// captured graph follows the lengths of each replay.  A segment that lies in one CTA's run
// is finished there; of one that is cut, each CTA leaves a piece (sum, max, row sums; at most
// two pieces a CTA), and a second kernel joins them.
//
// Inside a CTA (tcgen05, 384 threads):
//   * warp 9 loads K and V tiles by TMA from the pages, 64 rows a copy, into a ring of
//     128-key tiles; warp 10 the query tile, (nodes x group) rows from [T, Hq, d];
//   * warp 8 issues S = Q K^T and O += P V, P read from tensor memory; before the product of
//     a sequence's last tile it zeroes the V rows past the end: what a page holds there may
//     be anything, and 0 * NaN would reach the sum.  For the same reason it looks through the
//     drafted rows of V, which not every node sees: infinities and NaN among them become zeros,
//     and the rows that do see them get them after the run (never, in a sound model);
//   * two softmax warpgroups, a thread a row.  With n G <= 128 rows there is one query tile;
//     each warpgroup takes one half of every key tile, with its own max, sum and O, and the
//     two O's are joined from tensor memory at the end of a piece.  A thread then has 64
//     scores of a tile and two tiles' scores are in tensor memory at a time, so that the way
//     from scores to product (half as long) does not hold up the loads.  With more rows each
//     warpgroup has a query tile of its own and every K/V tile feeds both.
// Measured: 16 sequences of 16384 to 32768 rows, 8 KV heads, 64 query rows each: 239 us, 6.3 TB/s
// of cache (266 us in long runs, clocked by the power limit); 256 rows: 990 TFLOP/s.
// Scores keep fp32; P is rounded to bf16 for the product (2^-8 relative, as in the prefill
// kernel), its row sum is taken before the rounding.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_serve.h"
#include "sm100_ptx.cuh"
#include "tmem_ldst.cuh"

namespace attn {

namespace {

constexpr int kTreeThreads = 384;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kTreeMma = 8, kTreeKv = 9, kTreeQ = 10;   // warp 11 is spare
// 2 * 128 * 192 + 128 * 112 = 63488 <= 384 * 168 launch registers
constexpr uint32_t kTreeRegsSoftmax = 192;
constexpr uint32_t kTreeRegsOther = 112;
constexpr int kKeys = 128;                    // keys of a tile
// What a segment costs beside its key tiles (the first and last tile's latencies, its output),
// in tiles: without it a CTA that gets many short segments ends long after the others.  With 0, 1,
// 2, 3 and 4 (us):
//   7 sequences of up to 5000 rows, one of them new, 16 KV heads    57   47   39   40   40
//   8 of up to 8192 rows, 8 KV heads, up to 256 query rows          80   72   63   63   63
//   8 of up to 8192 rows, 8 KV heads, up to 64 query rows           59   45   42   42   41
//   16 of up to 32768 rows, 8 KV heads, up to 64 query rows        279  268  259  258  258
//   64 of up to 1500 rows, 8 KV heads, up to 32 query rows          76   73   69   69   69
//   20 of up to 6000 rows, 8 KV heads, up to 64 query rows, d 64    73   66   55   53   53
constexpr int kPieceCost = 2;
constexpr float kTreeThreshold = 8.0f;        // O is rescaled when its max grows by 2^8
constexpr float kTreeLn2 = 0.69314718055994531f;
constexpr uint32_t kNegInf = 0xff800000u;

enum : uint32_t {
  kSiteTreeQ = 201, kSiteTreeEmpty, kSiteTreeFullK, kSiteTreeFullV, kSiteTreeP, kSiteTreeS,
  kSiteTreeO, kSiteTreeDrain, kSiteTreeQFree, kSiteTreeAlign,
  kSiteTreePv,
};

template <int D, bool kTwo>
struct TreeCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kKeys * 128;
  static constexpr int kTile = kKeys * D * 2;              // one Q, K or V tile
  static constexpr int kQTiles = kTwo ? 2 : 1;
  static constexpr int kStages = D == 128 ? (kTwo ? 4 : 6) : 8;
  static constexpr int kRing = kQTiles * kTile;
  static constexpr int kMl = kRing + kStages * kTile;      // float2 [2][128]: (m, l)
  static constexpr int kBar = kMl + 2 * 128 * 8;
  // barriers: q[2], q_free[2], full[S], empty[S], s[2], p[2][2], o[2], done, pv[2]
  static constexpr int kNumBars = 15 + 2 * kStages;
  static constexpr int kSlot = kBar + kNumBars * 8;        // tmem slot, abort flag, wait limit
  static constexpr int kStart = kSlot + 16;                // CTA's first sequence, prefixes
  static constexpr int kState = kStart + 32 + kTreeWarps * 8;   // Run [8]: softmax warps'
  static constexpr int kFound = kState + 8 * 16;           // int: a drafted row's V is no number
  static constexpr int kSmem = kFound + 16;
};

// ---------------------------------------------------------------------------- schedule

// Lengths, offsets, parents and table entries are read with ordinary loads throughout: the kernels
// are launched while the one before them, which may write those arrays, still runs, and a load
// through the read-only path is defined only for what no one writes while the kernel lives.

// Sequence b as its query rows, its rows in the cache and the units of its segments see it.
struct Seq {
  int first, n, nodes;   // first token, drafted rows, rows computed (n, at most max_nodes)
  int len;               // cache rows
  int ktiles, blocks;    // key tiles (one at least), blocks of query rows
  int span;              // units of one segment: its key tiles and kPieceCost more
  int units;             // Hkv * blocks * span (below 2^31: the host checks the largest)
};

__device__ __forceinline__ Seq load_seq(const TreeParams& p, int b, int block_nodes) {
  Seq s;
  s.first = min(max(p.offsets[b], 0), p.T);
  s.n = max(min(p.offsets[b + 1], p.T) - s.first, 0);
  s.nodes = min(s.n, p.max_nodes);
  s.len = min(max(p.seq_lens[b], 0), p.cap);
  s.ktiles = max((int)(((unsigned)s.len + kKeys - 1) / kKeys), 1);
  s.blocks = (s.nodes + block_nodes - 1) / block_nodes;
  s.span = s.ktiles + kPieceCost;
  s.units = p.Hkv * s.blocks * s.span;
  return s;
}

// One CTA's run within a segment: key tiles [tile0, tile0 + tiles) of a block of query rows
// (from node node0 on) and KV head hk of sequence b; `units` of the run (the segment's first
// kPieceCost units are no tiles, and a run may begin or end among them).
struct Piece {
  int b, hk, node0, tile0, tiles, units;
  Seq s;
};

// A run of units: `count` of them from unit `within` of sequence b0 on.
struct Run {
  int b0, within, count;
};

// The piece that a run begins with, from its first sequence's data.
__device__ __forceinline__ Piece first_piece(const Seq& s, const Run& r, int block_nodes) {
  Piece pc;
  pc.s = s;
  const int seg = r.within / s.span;
  const int at = r.within - seg * s.span;
  pc.b = r.b0;
  pc.units = min(s.span - at, r.count);
  pc.tile0 = max(at - kPieceCost, 0);
  pc.tiles = max(at + pc.units - kPieceCost, 0) - pc.tile0;
  pc.hk = seg / s.blocks;
  pc.node0 = (seg - pc.hk * s.blocks) * block_nodes;
  return pc;
}

template <typename F>
__device__ __forceinline__ void for_each_piece(const TreeParams& p, Run r, int block_nodes,
                                               F&& f) {
  while (r.count > 0) {
    const Seq s = load_seq(p, r.b0, block_nodes);
    if (r.within >= s.units) {
      r.within -= s.units;
      ++r.b0;
      continue;
    }
    const Piece pc = first_piece(s, r, block_nodes);
    if (pc.tiles > 0) f(pc);
    r.within += pc.units;
    r.count -= pc.units;
  }
}

// CTAs that get a run: no run is empty, so the pieces of a segment lie with consecutive CTAs.
__device__ __forceinline__ long long run_count(const TreeParams& p, long long total) {
  return min((long long)p.grid, total);
}

// Units of all sequences and this CTA's run of them; block 0 leaves the prefix sums for the
// join.  All threads call it; sums: kTreeWarps values, out: shared memory for the result.
__device__ __forceinline__ Run plan_run(const TreeParams& p, int block_nodes, long long* sums,
                                        Run* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += load_seq(p, b, block_nodes).units;
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  if (tid == 0) *out = Run{0, 0, 0};
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kTreeWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  before += x - mine;
  const long long parts = run_count(p, total);
  const long long begin = (long long)blockIdx.x * total / max(parts, 1LL);
  const long long end = ((long long)blockIdx.x + 1) * total / max(parts, 1LL);
  if ((long long)blockIdx.x < parts && begin >= before && begin < before + mine) {
    long long pre = before;
    for (int b = b0; b < b1; ++b) {
      const int u = load_seq(p, b, block_nodes).units;
      if (begin < pre + u) {
        *out = Run{b, (int)(begin - pre), (int)(end - begin)};
        break;
      }
      pre += u;
    }
  }
  if (blockIdx.x == 0) {
    long long pre = before;
    for (int b = b0; b < b1; ++b) {
      p.prefix[b] = pre;
      pre += load_seq(p, b, block_nodes).units;
    }
    if (tid == 0) p.prefix[p.B] = total;
  }
  __syncthreads();
  return *out;
}

// Places in the ring, counted from a piece's first, of its K and V tiles.  They are loaded in
// the order of their use: step j takes V_(j - lag), then K_j.  A V tile loaded beside its K
// would hold its place for `lag` steps before its product can be issued, and with six places
// the loads then run out of room (16 sequences of 32768 rows: 247 us instead of 239, and 277
// instead of 266 in long runs under the power limit).
template <int kLag>
struct KvOrder {
  static __device__ __forceinline__ int k(int j) { return j < kLag ? j : 2 * j - kLag + 1; }
  static __device__ __forceinline__ int v(int j, int n) {
    return j + kLag < n ? 2 * j + kLag : n + j;
  }
};

// ------------------------------------------------------------------------------- rows

__device__ __forceinline__ float fl(uint32_t u) { return __uint_as_float(u); }

template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&s)[N]) {
  float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int c = 0; c < N; c += 8) {
    m0 = max3f(m0, fl(s[c]), fl(s[c + 1]));
    m1 = max3f(m1, fl(s[c + 2]), fl(s[c + 3]));
    m2 = max3f(m2, fl(s[c + 4]), fl(s[c + 5]));
    m3 = max3f(m3, fl(s[c + 6]), fl(s[c + 7]));
  }
  return max3f(m0, m1, fmaxf(m2, m3));
}

// 2^(x ks - m) of 64 keys from s[base] on, packed in bf16 pairs; returns their fp32 sum.
template <int N>
__device__ __forceinline__ float row_exp_64(const uint32_t (&s)[N], int base, float ks, float m,
                                            uint32_t (&pk)[32]) {
  float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    float x0, x1, x2, x3;
    ffma2(x0, x1, fl(s[base + c]), fl(s[base + c + 1]), ks, ks, -m, -m);
    ffma2(x2, x3, fl(s[base + c + 2]), fl(s[base + c + 3]), ks, ks, -m, -m);
    const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
    const float e2 = ex2_approx(x2), e3 = ex2_approx(x3);
    add2(a0, a1, e0, e1);
    add2(b0, b1, e2, e3);
    pk[c >> 1] = pack_bf16x2(e0, e1);
    pk[(c >> 1) + 1] = pack_bf16x2(e2, e3);
  }
  return (a0 + a1) + (b0 + b1);
}

__device__ __forceinline__ void tmem_scores(uint32_t taddr, uint32_t (&s)[64]) {
  tmem_ld_x64(taddr, s);
}
__device__ __forceinline__ void tmem_scores(uint32_t taddr, uint32_t (&s)[128]) {
  tmem_ld_x128(taddr, s);
}

// Keys of the tile that starts at row k0 which a node sees, bit c for key k0 + c: all of the
// context (rows before ctx), and of the drafted rows those in `seen` (bit j: row ctx + j).
// A call of its own: inlined, its 128-bit shifts made the compiler spill registers that the
// scores need.
__device__ __noinline__ unsigned __int128 visible_keys(unsigned __int128 seen, int k0, int ctx) {
  const long long j0 = (long long)k0 - ctx;       // drafted row of key k0
  if (j0 >= 128) return 0;
  if (j0 >= 0) return seen >> (int)j0;
  if (j0 <= -128) return ~(unsigned __int128)0;
  return (seen << (int)-j0) | (((unsigned __int128)1 << (int)-j0) - 1);
}

// A sequence's parents into shared memory, a warp together; an entry that is no earlier node
// becomes -1.  All loads come before the first store, which they could not pass.
__device__ __noinline__ void load_parents(const int* parents, int nodes, int8_t* to) {
  const int lane = threadIdx.x & 31;
  int q[kTreeMaxNodes / 32];
#pragma unroll
  for (int k = 0; k < kTreeMaxNodes / 32; ++k)
    q[k] = lane + 32 * k < nodes ? parents[lane + 32 * k] : -1;
#pragma unroll
  for (int k = 0; k < kTreeMaxNodes / 32; ++k) {
    const int i = lane + 32 * k;
    if (i < nodes) to[i] = (int8_t)((q[k] >= 0 && q[k] < i) ? q[k] : -1);
  }
}

// Whether drafted rows [from, end) of a V tile hold an infinity or a NaN (the warp together).
// 0 * x is NaN for those and 0 for the rest: one instruction a pair of values.
template <int kChunks>
__device__ __forceinline__ bool rows_off(const uint8_t* v, int from, int end) {
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll 4
    for (int o = from * 128 + 16 * (int)(threadIdx.x & 31); o < end * 128; o += 512) {
      const uint4 x = *reinterpret_cast<const uint4*>(v + c * (kKeys * 128) + o);
      acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, acc[0]);
      acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, acc[1]);
      acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, acc[2]);
      acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, acc[3]);
    }
  const float2 a = __bfloat1622float2(__hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3])));
  return __any_sync(0xffffffffu, a.x != 0.f || a.y != 0.f);
}

// A bf16 pair with zeros in place of infinities and NaN.
__device__ __forceinline__ uint32_t pair_clean(uint32_t w) {
  return w & (((w & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
              ((w & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u));
}

// Puts zeros in their place, so that the product does not carry them to nodes that do not see
// them, and notes it in *found.  The look itself goes by while the softmax works on the tile's
// scores: 38.5 us with and without it at 7 sequences of 16 KV heads, 59.3 us instead of 57.8 with
// two query tiles at 64 segments of 8192 rows.  Inlined, or with the rows patched at the end of
// each piece, the tile loop lost 5 to 9 % there.
template <int kChunks>
__device__ __noinline__ void clean_rows(uint8_t* v, int from, int end, volatile int* found) {
  if (!rows_off<kChunks>(v, from, end)) return;
  *found = 1;
  for (int c = 0; c < kChunks; ++c)
    for (int o = from * 128 + 16 * (int)(threadIdx.x & 31); o < end * 128; o += 512) {
      uint4* at = reinterpret_cast<uint4*>(v + c * (kKeys * 128) + o);
      const uint4 x = *at;
      *at = make_uint4(pair_clean(x.x), pair_clean(x.y), pair_clean(x.z), pair_clean(x.w));
    }
  fence_proxy_async_smem();
  __syncwarp();
}

// After the run, adds what clean_rows took out to the rows that this thread has written: to
// finished ones, or to the pieces' sums.  Each gets it from the drafted rows that its node sees
// among the piece's.
template <int D, bool kTwo>
__device__ __noinline__ void patch_rows(const TreeParams p, const Run* run) {
  const int block_nodes = p.tile_nodes * (kTwo ? 2 : 1);
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  constexpr int kCols = kTwo ? D : D / 2;
  const int col0 = kTwo ? 0 : t * kCols, tile = kTwo ? t : 0;
  for_each_piece(p, *run, block_nodes, [&](const Piece& pc) {
    const int node = pc.node0 + tile * p.tile_nodes + r / p.G;
    if (r >= p.tile_nodes * p.G || node >= pc.s.nodes) return;
    const size_t orow = (size_t)(pc.s.first + node) * p.Hq + (size_t)(pc.hk * p.G + r % p.G);
    const bool whole = pc.tiles == pc.s.ktiles;
    const size_t ptile =
        (size_t)(2 * (int)blockIdx.x + (pc.tile0 == 0 ? 1 : 0)) * (kTwo ? 2 : 1) + tile;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.o) + orow * D;
    float* part = p.o_part + ptile * (D * kTreeRows) + 4 * r;
    const int k0 = pc.tile0 * kKeys, k1 = min(k0 + pc.tiles * kKeys, pc.s.len);
    for (int j = node; j >= 0;) {
      const int pos = pc.s.len - pc.s.n + j;
      if (pos >= k0 && pos < k1) {
        const int pg = pos / p.page_size;
        const int page = p.block_table[(size_t)pc.b * p.max_pages + pg];
        // a page outside the cache reads zeros
        if ((unsigned)page < (unsigned)p.num_pages) {
          const __nv_bfloat16* v =
              reinterpret_cast<const __nv_bfloat16*>(p.v_pages) +
              (((size_t)page * p.Hkv + pc.hk) * p.page_size + (pos - pg * p.page_size)) * D;
#pragma unroll 1
          for (int c = col0; c < col0 + kCols; ++c) {
            const float x = __bfloat162float(v[c]);
            if (isfinite(x)) continue;
            if (whole) out[c] = __float2bfloat16(__bfloat162float(out[c]) + x);
            else part[(c >> 2) * (4 * kTreeRows) + (c & 3)] += x;
          }
        }
      }
      const int q = p.parents == nullptr ? j - 1 : p.parents[pc.s.first + j];
      j = q < j ? q : -1;
    }
  });
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

template <int D, bool kTwo>
__global__ void __launch_bounds__(kTreeThreads, 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TreeCfg<D, kTwo>;
  constexpr int NS = C::kStages;
  constexpr int kLag = kTwo ? 1 : 2;      // steps from a tile's QK^T to its PV
  using Order = KvOrder<kLag>;
  // six 32 KB stages leave no room to round the base up: the declaration aligns it
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t base_u32 = smem_u32(base);
  if (base_u32 & 1023u) {
    if (threadIdx.x == 0) report_error(p.err, kErrBadArgument, kSiteTreeAlign);
    return;
  }
  const uint32_t sQ = base_u32, sRing = base_u32 + C::kRing, sBar = base_u32 + C::kBar;
  auto bar = [&](int i) -> uint32_t { return sBar + 8u * (uint32_t)i; };
  const int BAR_Q = 0, BAR_QF = 2, BAR_FULL = 4, BAR_EMPTY = 4 + NS, BAR_S = 4 + 2 * NS,
            BAR_P = 6 + 2 * NS, BAR_O = 10 + 2 * NS, BAR_DONE = 12 + 2 * NS,
            BAR_PV = 13 + 2 * NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* found = reinterpret_cast<volatile int*>(base + C::kFound);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_rows = p.tile_nodes * p.G;
  const int block_nodes = p.tile_nodes * C::kQTiles;

  if (threadIdx.x == kTreeKv * 32) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_Q + t), 1);
      mbar_init(bar(BAR_QF + t), 1);
      mbar_init(bar(BAR_S + t), 1);
      mbar_init(bar(BAR_P + 2 * t), 4);
      mbar_init(bar(BAR_P + 2 * t + 1), 4);
      mbar_init(bar(BAR_O + t), 1);
      mbar_init(bar(BAR_PV + t), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(BAR_FULL + s), 1);
      mbar_init(bar(BAR_EMPTY + s), 1);
    }
    mbar_init(bar(BAR_DONE), 1);
    *abort_flag = 0;
    *found = 0;
    init_wait_limit(abort_flag, p.err);
    fence_mbar_init();
  }
  if (warp == kTreeMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Query rows that no load fills are zeros: their products cost the tensor cores less power,
  // and a long run of calls is clocked by the power limit (43 -> 41 us at 7 sequences of 2500
  // to 5000 rows, 16 KV heads, 5 query rows each).
  for (int i = threadIdx.x; i < C::kQTiles * C::kChunks * (kTreeRows - tile_rows) * 8;
       i += kTreeThreads) {
    const int part = i / ((kTreeRows - tile_rows) * 8), at = i - part * (kTreeRows - tile_rows) * 8;
    *reinterpret_cast<uint4*>(base + part * C::kChunkBytes + tile_rows * 128 + at * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  // Launched while the kernel before it ends: of memory only the wait limit is read before this (its
  // setter synchronises the device), and nothing is written.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Run run = plan_run(p, block_nodes, reinterpret_cast<long long*>(base + C::kStart + 32),
                           reinterpret_cast<Run*>(base + C::kStart));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Whether query tile t of a piece has a row (t = 1 only with two tiles a CTA).
  auto tile_used = [&](const Piece& pc, int t) -> bool {
    return pc.node0 + t * p.tile_nodes < pc.s.nodes;
  };

  if (warp >= kTreeMma) {
    regs_decrease<kTreeRegsOther>();
    if (warp == kTreeKv) {
      // -------------------------------------------------------------- K/V loads
      if (lane == 0) {
        int issued = 0;
        bool ok = true;
        for_each_piece(p, run, block_nodes, [&](const Piece& pc) {
          const int* table = p.block_table + (size_t)pc.b * p.max_pages;
          // One 64-row half of a tile: its page (a half never crosses one), or a coordinate
          // past the map, which reads zeros, for rows past the sequence or a page outside the
          // cache
          struct Half {
            int z, row;
          };
          auto find = [&](int tile, int h) -> Half {
            const int k = tile * kKeys + 64 * h;
            Half x{p.num_pages * p.Hkv, 0};
            if (k < pc.s.len) {
              const int pg = k / p.page_size;
              const int page = table[pg];
              if ((unsigned)page < (unsigned)p.num_pages) x.z = page * p.Hkv + pc.hk;
              x.row = k - pg * p.page_size;
            }
            return x;
          };
          auto load = [&](const CUtensorMap* map, const Half (&x)[2]) {
            const int s = issued % NS, round = issued / NS;
            if (ok && round > 0)
              ok = mbar_wait(bar(BAR_EMPTY + s), (round - 1) & 1, abort_flag, p.err, kSiteTreeEmpty);
            if (!ok) return;
            mbar_arrive_expect_tx(bar(BAR_FULL + s), C::kTile);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(sRing + s * C::kTile + c * C::kChunkBytes + h * 64 * 128, map,
                            bar(BAR_FULL + s), c * 64, x[h].row, x[h].z);
            ++issued;
          };
          // in the order of use (KvOrder): V a step or two behind its K
          Half at[kLag + 1][2];
          for (int j = 0; ok && j < pc.tiles + kLag; ++j) {
#pragma unroll
            for (int i = kLag; i > 0; --i)
#pragma unroll
              for (int h = 0; h < 2; ++h) at[i][h] = at[i - 1][h];
            if (j < pc.tiles)
#pragma unroll
              for (int h = 0; h < 2; ++h) at[0][h] = find(pc.tile0 + j, h);
            if (j >= kLag) load(&tmV, at[kLag]);
            if (j < pc.tiles) load(&tmK, at[0]);
          }
        });
        // outstanding copies must land before the CTA may exit
        for (int s = 0; s < NS && s < issued; ++s) {
          const int last = s + ((issued - 1 - s) / NS) * NS;
          mbar_wait(bar(BAR_FULL + s), (last / NS) & 1, nullptr, p.err, kSiteTreeDrain);
        }
      }
      __syncwarp();
    } else if (warp == kTreeQ) {
      // -------------------------------------------------------------- query tiles
      if (lane == 0) {
        int loads[2] = {0, 0};
        bool ok = true;
        for_each_piece(p, run, block_nodes, [&](const Piece& pc) {
#pragma unroll
          for (int t = 0; t < C::kQTiles; ++t) {
            if (!ok || !tile_used(pc, t)) continue;
            if (loads[t] > 0 && !mbar_wait(bar(BAR_QF + t), (loads[t] - 1) & 1, abort_flag, p.err,
                                           kSiteTreeQFree)) {
              ok = false;
              continue;
            }
            mbar_arrive_expect_tx(bar(BAR_Q + t), C::kChunks * 128 * tile_rows);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_4d(sQ + t * C::kTile + c * C::kChunkBytes, &tmQ, bar(BAR_Q + t), c * 64, 0,
                          pc.hk, pc.s.first + pc.node0 + t * p.tile_nodes);
            ++loads[t];
          }
        });
        for (int t = 0; t < 2; ++t)
          if (loads[t] > 0)
            mbar_wait(bar(BAR_Q + t), (loads[t] - 1) & 1, nullptr, p.err, kSiteTreeDrain);
      }
      __syncwarp();
    } else if (warp == kTreeMma) {
      // -------------------------------------------------------------- tcgen05 issuer
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kKeys, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, true);
      const uint64_t dQ = smem_desc(sQ, 16, 1024);
      const uint64_t dK = smem_desc(sRing, 16, 1024);
      const uint64_t dV = smem_desc(sRing, C::kChunkBytes, 1024);
      // S_t = Q_q K^T (q: the query tile, 0 when the warpgroups share one)
      auto issue_qk = [&](int t, int sk) {
        const uint32_t q_off = kTwo ? (uint32_t)(t * C::kTile) >> 4 : 0u;
        const uint32_t k_off = (uint32_t)(sk * C::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
          umma_ss_warp(tmem + 128u * t, dQ + q_off + off, dK + k_off + off, idesc_qk,
                       kk > 0 ? 1u : 0u);
        }
      };
      // O_t += P V over 64 keys: half h of the tile in ring place sv, P from column `p_col` on
      auto issue_pv_half = [&](int t, uint32_t p_col, int sv, int h, bool first) {
        const uint32_t v_off = (uint32_t)(sv * C::kTile) >> 4;
#pragma unroll
        for (int k = 0; k < kKeys / 32; ++k)
          umma_ts_warp(tmem + 256u + 128u * t, tmem + p_col + 8u * k,
                       dV + v_off + (((h * (kKeys / 32) + k) * 16 * 128) >> 4), idesc_pv,
                       (!first || k > 0) ? 1u : 0u);
      };
      int kv = 0;
      int qloads[2] = {0, 0}, pcount[2] = {0, 0};
      bool ok = true;
      auto wait = [&](int b, uint32_t parity, uint32_t site) -> bool {
        if (ok) ok = mbar_wait_warp(bar(b), parity, abort_flag, p.err, site);
        return ok;
      };
      for_each_piece(p, run, block_nodes, [&](const Piece& pc) {
        if (!ok) return;
        const bool used1 = kTwo && tile_used(pc, 1);
#pragma unroll
        for (int t = 0; t < C::kQTiles; ++t) {
          if (t == 1 && !used1) continue;
          if (!wait(BAR_Q + t, qloads[t] & 1, kSiteTreeQ)) return;
          ++qloads[t];
        }
        const int n = pc.tiles;
        // keys of the piece's last tile (all 128 unless it is the sequence's last)
        const int tail = min(pc.s.len - (pc.tile0 + n - 1) * kKeys, kKeys);
        // PV of tile j once its P is there.  Two query tiles: for tile t, in two halves of the
        // keys as they come.  One: both warpgroups' halves, b the scores' buffer.
        auto pv = [&](int tb, int j, bool last) -> bool {
          const int sv = (int)((unsigned)(kv + Order::v(j, n)) % NS);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(BAR_P + 2 * tb + h, pcount[tb] & 1, kSiteTreeP)) return false;
            tc_fence_after();
            if constexpr (kTwo)
              issue_pv_half(tb, 128u * tb + 64u + 32u * h, sv, h, j == 0 && h == 0);
            else
              issue_pv_half(h, 128u * tb + 64u * h + 32u, sv, h, j == 0);
          }
          ++pcount[tb];
          if (!kTwo) umma_commit_warp(bar(BAR_PV + tb));
          if (last) umma_commit_warp(bar(BAR_O + (kTwo ? tb : 0)));
          return true;
        };
        auto v_ready = [&](int j) -> bool {
          const unsigned iv = (unsigned)(kv + Order::v(j, n));
          if (!wait(BAR_FULL + iv % NS, (iv / NS) & 1, kSiteTreeFullV)) return false;
          // drafted rows of the tile: while the softmax works on its scores
          const int from = max(pc.s.len - pc.s.n - (pc.tile0 + j) * kKeys, 0);
          if (from < kKeys) {
            uint8_t* v = base + C::kRing + (iv % NS) * C::kTile;
            const int end = j == n - 1 ? tail : kKeys;
            clean_rows<C::kChunks>(v, from, end, found);
          }
          if (tail < kKeys && j == n - 1) {
            // rows past the sequence's end become zeros (a half without any row already is)
            uint8_t* v = base + C::kRing + (iv % NS) * C::kTile;
            const int end = (tail <= 64 ? 64 : 128) * 128;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              for (int o = tail * 128 + 16 * lane; o < end; o += 512)
                *reinterpret_cast<uint4*>(v + c * C::kChunkBytes + o) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          return true;
        };
        auto k_ready = [&](int j) -> bool {
          const unsigned ik = (unsigned)(kv + Order::k(j));
          if (!wait(BAR_FULL + ik % NS, (ik / NS) & 1, kSiteTreeFullK)) return false;
          tc_fence_after();
          return true;
        };
        auto k_slot = [&](int j) -> int { return (int)((unsigned)(kv + Order::k(j)) % NS); };
        auto v_slot = [&](int j) -> int { return (int)((unsigned)(kv + Order::v(j, n)) % NS); };
        if constexpr (kTwo) {
          // step j: for each query tile PV of tile j - 1, then QK^T of tile j
          for (int j = 0; j <= n; ++j) {
            if (j < n && !k_ready(j)) return;
            if (j > 0 && !v_ready(j - 1)) return;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t == 1 && !used1) continue;
              if (j > 0 && !pv(t, j - 1, j == n)) return;
              if (j < n) {
                issue_qk(t, k_slot(j));
                umma_commit_warp(bar(BAR_S + t));
                if (j == n - 1) umma_commit_warp(bar(BAR_QF + t));
              }
            }
            if (j > 0) umma_commit_warp(bar(BAR_EMPTY + v_slot(j - 1)));
            if (j < n) umma_commit_warp(bar(BAR_EMPTY + k_slot(j)));
          }
        } else {
          // step j, scores' buffer t = j mod 2: PV of tile j - 2, then QK^T of tile j into the
          // same buffer (the tensor pipe runs in order, so P has been read by then)
          for (int j = 0; j < n + 2; ++j) {
            const int t = j & 1;
            if (j < n && !k_ready(j)) return;
            if (j >= 2 && j - 2 < n) {
              if (!v_ready(j - 2)) return;
              if (!pv(t, j - 2, j == n + 1)) return;
              umma_commit_warp(bar(BAR_EMPTY + v_slot(j - 2)));
            }
            if (j < n) {
              issue_qk(t, k_slot(j));
              umma_commit_warp(bar(BAR_S + t));
              umma_commit_warp(bar(BAR_EMPTY + k_slot(j)));
              if (j == n - 1) umma_commit_warp(bar(BAR_QF + 0));
            }
          }
        }
        kv += 2 * n;
      });
      // every product issued above must be complete before TMEM is released
      umma_commit_warp(bar(BAR_DONE));
      mbar_wait_warp(bar(BAR_DONE), 0, nullptr, p.err, kSiteTreeDrain);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    regs_increase<kTreeRegsSoftmax>();
    const int t = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;                         // row of the tile
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    constexpr int kN = kTwo ? 128 : 64;                   // scores of a tile that a thread takes
    // this warpgroup's scores (one query tile: of buffer 0, the other is 128 columns on)
    const uint32_t tS = tmem + lane_off + (kTwo ? 128u : 64u) * t;
    const uint32_t tO = tmem + lane_off + 256u;           // O_0; O_1 is 128 columns on
    float2* ml = reinterpret_cast<float2*>(base + C::kMl);
    // the sequence's parents, a copy a warp: in the 256 bytes that take this warp's own (m, l)
    // at the end of a piece, after its last look at them
    int8_t* par = reinterpret_cast<int8_t*>(ml + 32 * warp);
    // What is left of the run lies in shared memory, and the piece is derived from it anew
    // wherever it is needed: 128 scores a thread leave no registers for its fields.
    volatile int* left = reinterpret_cast<volatile int*>(base + C::kState) + 4 * warp;
    auto piece = [&]() -> Piece {
      const Run rest{left[0], left[1], left[2]};
      return first_piece(load_seq(p, rest.b0, block_nodes), rest, block_nodes);
    };
    // the node of this thread's row
    auto node_of = [&](const Piece& pc) -> int {
      return pc.node0 + (kTwo ? t : 0) * p.tile_nodes + r / p.G;
    };
    auto is_row = [&](const Piece& pc, int node) -> bool {
      return r < tile_rows && node < pc.s.nodes;
    };
    int scount = 0, ocount = 0;      // parities of the next waits for scores and for O
    bool ok = true;

    for (Run rest = run; rest.count > 0;) {
      int tiles, masked_from;      // key tiles; the first of them that ends past the context
      bool busy;
      {
        const Seq s = load_seq(p, rest.b0, block_nodes);
        if (rest.within >= s.units) {
          rest.within -= s.units;
          ++rest.b0;
          continue;
        }
        const Piece pc = first_piece(s, rest, block_nodes);
        tiles = pc.tiles;
        masked_from = max(s.len - s.n, 0) / kKeys - pc.tile0;
        // a warp without a row only keeps the barriers
        busy = __any_sync(0xffffffffu, is_row(pc, node_of(pc)));
        if (tiles == 0 || (kTwo && !tile_used(pc, t))) {
          rest.within += pc.units;
          rest.count -= pc.units;
          continue;
        }
        if (p.parents != nullptr && busy && masked_from < tiles) {
          // the parents of a piece that reaches the drafted rows, for its masked tiles
          load_parents(p.parents + s.first, s.nodes, par);
        }
        __syncwarp();
        if (lane == 0) {
          left[0] = rest.b0;
          left[1] = rest.within;
          left[2] = rest.count;
        }
        __syncwarp();
      }

      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j) {
        const int buf = kTwo ? t : j & 1;      // of the scores' barriers
        if (ok) {
          ok = mbar_wait(bar(BAR_S + buf), (kTwo ? scount : scount >> buf) & 1, abort_flag, p.err,
                         kSiteTreeS);
          ok = __all_sync(0xffffffffu, ok);
        }
        // waits so far: their parity, one bit for each buffer where both are waited for
        scount ^= kTwo ? 1 : 1 << buf;
        if (!ok) continue;
        tc_fence_after();
        if (busy) {
          const uint32_t tSb = kTwo ? tS : tS + 128u * buf;
          uint32_t w[kN / 32];  // the keys of a tile that this row's node sees, past the context
          if (j >= masked_from) {
            const Piece pc = piece();
            const int node = node_of(pc);
            unsigned __int128 seen = 0;
            if (p.parents == nullptr) {
              seen = node >= 127 ? ~(unsigned __int128)0 : ((unsigned __int128)1 << (node + 1)) - 1;
            } else {
              for (int i = is_row(pc, node) ? node : -1; i >= 0; i = par[i])
                seen |= (unsigned __int128)1 << i;
            }
            const unsigned __int128 vis =
                visible_keys(seen, (pc.tile0 + j) * kKeys, pc.s.len - pc.s.n);
#pragma unroll
            for (int i = 0; i < kN / 32; ++i)
              w[i] = (uint32_t)(vis >> (32 * i + (kTwo ? 0 : 64 * t)));
          }
          uint32_t s[kN];
          tmem_scores(tSb, s);
          if (j >= masked_from) {
#pragma unroll
            for (int c = 0; c < kN; ++c)
              if (!((w[c >> 5] >> (c & 31)) & 1u)) s[c] = kNegInf;
          }
          const float mx = row_max(s) * p.kscale;
          const float m_new = fmaxf(m_ref, mx);
          const bool need = m_new > m_ref + kTreeThreshold;
          float alpha = 1.f;
          if (need) {
            alpha = ex2_approx(m_ref - m_new);
            m_ref = m_new;
          }
          if (j > 0 && __any_sync(0xffffffffu, need)) {
            // The product of the tile before has to be in O.  Two query tiles: it was issued
            // before the one whose commit signalled these scores.  One: it comes after, so wait
            // for its own commit (no later one can follow before this warpgroup's next P).
            if (!kTwo) {
              ok = mbar_wait(bar(BAR_PV + (buf ^ 1)), ((scount >> (buf ^ 1)) & 1) ^ 1, abort_flag,
                             p.err, kSiteTreePv);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) continue;
              tc_fence_after();
            }
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {
              uint32_t o[16];
              tmem_ld_x16(tO + 128u * t + 16u * cc, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(fl(o[k]) * alpha);
              tmem_st_x16(tO + 128u * t + 16u * cc, o);
            }
          }
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          float sum = 0.f;
#pragma unroll
          for (int half = 0; half < kN / 64; ++half) {
            uint32_t pk[32];
            sum += row_exp_64(s, 64 * half, p.kscale, m_use, pk);
            tmem_st_x32(kTwo ? tSb + 64u + 32u * half : tSb + 32u, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_P + 2 * buf + (kTwo ? half : t)));
          }
          l = l * alpha + sum;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kTwo) {
              mbar_arrive(bar(BAR_P + 2 * buf));
              mbar_arrive(bar(BAR_P + 2 * buf + 1));
            } else {
              mbar_arrive(bar(BAR_P + 2 * buf + t));
            }
          }
        }
      }

      // ---- end of the piece: O of this row, its max and sum, from one or both warpgroups
      const Piece pc = piece();
      const int node = node_of(pc), tile = kTwo ? t : 0;
      const bool valid = is_row(pc, node);
      float f0, f1 = 0.f, m = m_ref, lsum = l;
      constexpr int kCols = kTwo ? D : D / 2;         // columns this thread writes
      const int col0 = kTwo ? 0 : t * (D / 2);
      if constexpr (kTwo) {
        f0 = 1.f;
      } else {
        // (m, l) cross through shared memory; both O's are in this row's TMEM lane
        ml[t * 128 + r] = make_float2(m_ref, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 a = ml[r], b = ml[128 + r];
        m = fmaxf(a.x, b.x);
        const float mu = m == -INFINITY ? 0.f : m;
        f0 = ex2_approx(a.x - mu);
        f1 = ex2_approx(b.x - mu);
        lsum = a.y * f0 + b.y * f1;
      }
      if (ok) {
        ok = mbar_wait(bar(BAR_O + (kTwo ? t : 0)), ocount & 1, abort_flag, p.err, kSiteTreeO);
        ok = __all_sync(0xffffffffu, ok);
      }
      ocount ^= 1;
      if (ok && busy) {
        tc_fence_after();
        // no key: l = 0, and O is 0, not 0 * (what V holds).  A NaN (of q, or of a K that the row
        // sees) stays one.
        const bool some = lsum != 0.f;
        const float inv = some ? 1.f / lsum : 0.f;
        // a whole segment is finished here; of a cut one, the piece that starts inside it is
        // this CTA's first, the one that starts with it this CTA's last
        const bool whole = pc.tiles == pc.s.ktiles;
        const int slot = 2 * (int)blockIdx.x + (pc.tile0 == 0 ? 1 : 0);
        const float g0 = whole ? f0 * inv : f0, g1 = whole ? f1 * inv : f1;
        const size_t token = (size_t)(pc.s.first + node);
        const size_t orow = token * p.Hq + (size_t)(pc.hk * p.G + r % p.G);
        const size_t ptile = (size_t)slot * C::kQTiles + tile;
        const uint32_t src = tO + (kTwo ? 128u * t : 0u) + (uint32_t)col0;
#pragma unroll 1
        for (int cc = 0; cc < kCols / 16; ++cc) {
          uint32_t a[16];
          float v[16];
          tmem_ld_x16(src + 16u * cc, a);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = fl(a[k]) * g0;
          if (!kTwo) {
            tmem_ld_x16(src + 128u + 16u * cc, a);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = fmaf(fl(a[k]), g1, v[k]);
          }
          if (valid && whole) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + orow * D +
                                                  col0 + 16 * cc);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              dst[k] = some ? make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]),
                                         pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                         pack_bf16x2(v[8 * k + 4], v[8 * k + 5]),
                                         pack_bf16x2(v[8 * k + 6], v[8 * k + 7]))
                            : make_uint4(0u, 0u, 0u, 0u);
          } else if (valid) {
            // 4 columns of 128 rows together: a warp's store is 512 bytes on end
            float4* dst = reinterpret_cast<float4*>(p.o_part) + ptile * (D / 4 * kTreeRows) +
                          (col0 / 4 + 4 * cc) * kTreeRows + r;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k * kTreeRows] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if (valid && (kTwo || t == 0)) {
          if (whole)
            p.lse[orow] = some ? (m + log2f(lsum)) * kTreeLn2 : -INFINITY;
          else
            p.ml_part[ptile * kTreeRows + r] = make_float2(m, lsum);
        }
        tc_fence_before();
      }
      // the next piece's products overwrite O, and its rows ml: both warpgroups are done
      if (!kTwo) asm volatile("bar.sync 1, 256;" ::: "memory");
      rest = Run{pc.b, left[1] + pc.units, left[2] - pc.units};
    }
  }

  if (threadIdx.x < 256 && *found)
    patch_rows<D, kTwo>(p, reinterpret_cast<const Run*>(base + C::kStart));
  tc_fence_before();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kTreeMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the segments that were cut: a thread takes 16 columns of one row (token,
// query head), a warp 32 neighbouring rows of one KV head, so that its loads are 512 bytes on
// end like the stores that left the pieces, and its own stores whole sectors.  The pieces of a
// segment lie with consecutive CTAs; rows of a segment in one piece are already written.
constexpr int kJoinCols = 16;
constexpr int kJoinPieces = 4;

template <int D>
__global__ void __launch_bounds__(256) attn_tree_join_kernel(const TreeParams p, int tiles) {
  // launched while the pieces' kernel ends: everything it leaves is read after the wait.  The
  // kernel after this one may be launched as soon as all blocks are here.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = (int)blockIdx.x * 32 + (threadIdx.x & 31);        // token * G + head of the group
  const int col = (int)(threadIdx.x >> 5) * kJoinCols;
  if (x >= p.T * p.G || col >= D) return;
  const int token = x / p.G, hk = blockIdx.y;
  // the last sequence that starts at or before the token and has nodes
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.offsets[mid] <= token) lo = mid; else hi = mid - 1;
  }
  const int block_nodes = p.tile_nodes * tiles;
  const Seq s = load_seq(p, lo, block_nodes);
  const int node = token - s.first;
  if (node < 0 || node >= s.nodes) return;
  const int block = node / block_nodes, in_block = node - block * block_nodes;
  const int tile = in_block / p.tile_nodes;
  const int r = (in_block - tile * p.tile_nodes) * p.G + (x - token * p.G);
  const long long total = p.prefix[p.B];
  const long long u1 = p.prefix[lo] + ((long long)hk * s.blocks + block + 1) * s.span;
  const long long u0 = u1 - s.ktiles;              // the segment's first tile
  // CTA c of N runs [c total / N, (c + 1) total / N): unit u is with ceil((u + 1) N / total) - 1
  const long long parts = run_count(p, total);
  const int c0 = (int)(((u0 + 1) * parts - 1) / total);
  const int c1 = (int)((u1 * parts - 1) / total);
  if (c0 == c1) return;
  auto part = [&](int c) -> size_t { return (size_t)(2 * c + (c == c0 ? 1 : 0)) * tiles + tile; };
  // kJoinPieces pieces at a time, their loads issued together: most rows have no more
  float m = -INFINITY, l = 0.f, acc[kJoinCols] = {};
  for (int c = c0; c <= c1; c += kJoinPieces) {
    float2 a[kJoinPieces];
    float4 v[kJoinPieces][kJoinCols / 4];
#pragma unroll
    for (int i = 0; i < kJoinPieces; ++i) {
      a[i] = make_float2(-INFINITY, 0.f);
      if (c + i > c1) continue;
      const size_t at = part(c + i);
      a[i] = p.ml_part[at * kTreeRows + r];
      const float4* src = reinterpret_cast<const float4*>(p.o_part) + at * (D / 4 * kTreeRows) +
                          col / 4 * kTreeRows + r;
#pragma unroll
      for (int k = 0; k < kJoinCols / 4; ++k) v[i][k] = src[k * kTreeRows];
    }
    // a piece without a key for this row (and none at all) has l = 0; one with a NaN has l = NaN
    // and may have no max
    float mn = m;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kJoinPieces; ++i) {
      mn = fmaxf(mn, a[i].x);
      some = some || a[i].y != 0.f;
    }
    if (!some) continue;
    const float old = m == -INFINITY ? 0.f : ex2_approx(m - mn);
    m = mn;
    l *= old;
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k) acc[k] *= old;
#pragma unroll
    for (int i = 0; i < kJoinPieces; ++i) {
      if (a[i].y == 0.f) continue;
      const float w = ex2_approx(a[i].x - m);
      l = fmaf(w, a[i].y, l);
#pragma unroll
      for (int k = 0; k < kJoinCols / 4; ++k) {
        acc[4 * k] = fmaf(w, v[i][k].x, acc[4 * k]);
        acc[4 * k + 1] = fmaf(w, v[i][k].y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(w, v[i][k].z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(w, v[i][k].w, acc[4 * k + 3]);
      }
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const size_t orow = (size_t)token * p.Hq + (size_t)(hk * p.G + (x - token * p.G));
  uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + orow * D + col);
#pragma unroll
  for (int k = 0; k < kJoinCols; k += 8)
    dst[k / 8] = make_uint4(pack_bf16x2(acc[k] * inv, acc[k + 1] * inv),
                            pack_bf16x2(acc[k + 2] * inv, acc[k + 3] * inv),
                            pack_bf16x2(acc[k + 4] * inv, acc[k + 5] * inv),
                            pack_bf16x2(acc[k + 6] * inv, acc[k + 7] * inv));
  if (col == 0) p.lse[orow] = l != 0.f ? (m + log2f(l)) * kTreeLn2 : -INFINITY;
}

template <int D, bool kTwo>
int launch_tree_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                  const TreeParams& p, cudaStream_t stream) {
  using C = TreeCfg<D, kTwo>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory budget");
  static std::atomic<bool> ready[64];
  if (!allow_smem(reinterpret_cast<const void*>(&attn_tree_kernel<D, kTwo>), C::kSmem, ready))
    return -4;
  // Both kernels are launched while the one before them ends (the join's blocks come in as the
  // pieces' leave) and wait for all of it: 2 to 3 us less for each.
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_tree_kernel<D, kTwo>, tq, tk, tv, p) != cudaSuccess) return -4;
  cfg.gridDim = dim3((unsigned)(((long long)p.T * p.G + 31) / 32), (unsigned)p.Hkv);
  cfg.blockDim = dim3(32 * D / kJoinCols);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_tree_join_kernel<D>, p, kTwo ? 2 : 1) == cudaSuccess ? 0
                                                                                            : -4;
}

}  // namespace

int launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                const TreeParams& p, int d, bool two_tiles, cudaStream_t stream) {
  if (d == 128)
    return two_tiles ? launch_tree_t<128, true>(tq, tk, tv, p, stream)
                     : launch_tree_t<128, false>(tq, tk, tv, p, stream);
  return two_tiles ? launch_tree_t<64, true>(tq, tk, tv, p, stream)
                   : launch_tree_t<64, false>(tq, tk, tv, p, stream);
}

}  // namespace attn
