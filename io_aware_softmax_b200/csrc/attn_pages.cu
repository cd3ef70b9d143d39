// Block tables and slot maps of a paged cache from request lengths, on the GPU.
//
// Sequence b holds c = ctx_lens[b] cache rows and adds n = new_lens[b] tokens.  With page size
// P it owns ceil(c / P) pages, or more where rows behind c were taken back (held_rows), and
// takes what ceil((c + n) / P) exceeds them by; these come off the free list in sequence order.
// Token i of the sequence lands in row c + i.  Everything follows from two prefix sums over
// the sequences, of tokens and of taken pages.
//
// The bytes (12 a token, 8 a new page) take microseconds at most, so the launch and the
// latencies on the way to the first store are the cost.  One launch does all: every block
// takes both sums over all sequences itself (8 bytes a sequence from L2) in one scan and keeps
// them in shared memory, which needs no block to wait for another, and then maps its share of
// the tokens by a binary search.  Divisions by the page size are products with its reciprocal.
// Depths in drafted trees come from doubling links in shared memory, a sequence to a warp or a
// block: their cost goes by the number of tokens, however deep the tree is.
// Measured (replayed back to back): 5.9 us for 64 sequences of one token, 10.0 us for 1.3 million
// tokens of 256 (16 MB), 6.5 us for 37 trees of up to 60 nodes; a chain of 8192 given by its
// parents beside 16 trees of 40: 35 us, where a walk through each token's ancestors took 1.4 ms.
// A page taken in this call is read from the free list, never from the table entry another
// block may be writing; entries of pages owned before are only read.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "attn_serve.h"

namespace attn {

namespace {

constexpr int kPagesThreads = 256;
constexpr int kPagesWarps = kPagesThreads / 32;
constexpr int kTokensPerThread = 4;   // one 16-byte store of positions, two of slots

// Sums over the block's threads before this one, and over all, of two 64-bit values each.
// 64 bits: lengths are caller data, and many of them can pass 2^31.
struct Sums {
  long long tokens, pages;
};

// A tree of up to kWarpNodes tokens is one warp's, a longer one goes through a block in chunks of
// kChunkNodes.  16 trees of 128 nodes: 7.6 us by warps, 15.2 by blocks; of 256 nodes 9.6 and
// 10.3; one tree of 256 alone 8.8 and 5.2.
constexpr int kWarpNodes = 256;
constexpr int kChunkNodes = kPagesWarps * kWarpNodes;

// A block's shared memory: what every call has, and the dynamic part, of sequences and of trees.
struct BlockShared {
  Sums warp_sums[2][kPagesWarps];
};
constexpr int kSmemOfSm = 228 * 1024;     // 1 KB a block is the system's
constexpr int kTreeBytes = kChunkNodes * 8;
constexpr int dynamic_bytes(int B, bool trees) { return (3 * B + 1) * 4 + (trees ? kTreeBytes : 0); }

__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.tokens, o);
    const long long g = __shfl_up_sync(0xffffffffu, x.pages, o);
    if (lane >= o) {
      x.tokens += t;
      x.pages += g;
    }
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  Sums before{0, 0};
  total = Sums{0, 0};
#pragma unroll
  for (int w = 0; w < kPagesWarps; ++w) {
    const Sums s = warp_sums[w];
    if (w < warp) {
      before.tokens += s.tokens;
      before.pages += s.pages;
    }
    total.tokens += s.tokens;
    total.pages += s.pages;
  }
  return Sums{before.tokens + x.tokens - v.tokens, before.pages + x.pages - v.pages};
}

// Doubles the links of n nodes until each names the topmost of its ancestors there (which names
// itself, 0 steps away).  In place: whichever of its values another thread's link is read at,
// it names an ancestor and the steps to it, and a link to a topmost node changes no more.
// kThreads threads call it, a warp or the block, thread `me` of them.
template <int kThreads>
__device__ __forceinline__ void double_links(volatile unsigned* links, int n, int me) {
  auto sync = [](bool more) -> bool {
    if (kThreads > 32) return __syncthreads_or(more);
    __syncwarp();
    return __any_sync(0xffffffffu, more);
  };
  sync(false);
  for (bool more = true; more;) {
    more = false;
    for (int i = me; i < n; i += kThreads) {
      const unsigned mine = links[i], up = links[mine >> 16];
      if ((up >> 16) != (mine >> 16)) {
        links[i] = up + (mine & 0xffffu);
        more = true;
      }
    }
    more = sync(more);
  }
}

template <bool kTrees>
__global__ void __launch_bounds__(kPagesThreads) attn_page_tables_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* off = smem;                  // [B + 1] first token of each sequence
  int* held = smem + p.B + 1;       // [B] cache rows before the step
  int* first = held + p.B;          // [B] free-list index of the first new page
  // with parents: ancestor << 16 | steps to it, nodes counted from the chunk's first, and the
  // depth of a node whose parent is none, or in an earlier chunk
  unsigned* links = reinterpret_cast<unsigned*>(first + p.B);   // [kChunkNodes]
  int* base = first + p.B + kChunkNodes;                        // [kChunkNodes]
  __shared__ BlockShared sh;
  const int tid = threadIdx.x;
  const int cap = p.max_pages * p.page_size;        // below 2^31 (host check)
  const int per = (p.B + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  // row / page_size for rows below 2^31 (see page_divisor)
  auto page_of = [&](int row) -> int {
    return (int)(((unsigned long long)(unsigned)row * p.div_mul) >> p.div_shift);
  };
  auto pages_of = [&](int rows) -> int { return rows > 0 ? page_of(rows - 1) + 1 : 0; };
  // pages that sequence b owns before the step, with c rows held
  auto owned = [&](int b, int c) -> int {
    return pages_of(p.held_rows != nullptr ? min(max(__ldg(p.held_rows + b), c), cap) : c);
  };
  auto grown = [&](int c, long long n) -> int {
    return (int)min((long long)c + n, (long long)cap);
  };

  Sums mine{0, 0}, total;
  for (int b = b0; b < b1; ++b) {
    const int c = min(max(__ldg(p.ctx_lens + b), 0), cap), n = max(__ldg(p.new_lens + b), 0);
    held[b] = c;
    mine.tokens += n;
    mine.pages += max(pages_of(grown(c, n)) - owned(b, c), 0);
  }
  const long long used0 = p.free_used != nullptr ? max(__ldg(p.free_used), 0) : 0;
  Sums run = block_scan(mine, sh.warp_sums[0], total);
  if (total.tokens > p.num_tokens) {
    // more tokens than there is room for: the lengths that count are cut, and the pages follow
    long long t = run.tokens;
    mine.pages = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = max(__ldg(p.new_lens + b), 0);
      const long long room = max((long long)p.num_tokens - t, 0LL);
      const int e = grown(held[b], min((long long)n, room));
      mine.pages += max(pages_of(e) - owned(b, held[b]), 0);
      t += n;
    }
    run = block_scan(mine, sh.warp_sums[1], total);
  }
  run.pages += used0;
  total.pages += used0;
  for (int b = b0; b < b1; ++b) {
    const int n = max(__ldg(p.new_lens + b), 0);
    const int o = (int)min(run.tokens, (long long)p.num_tokens);
    run.tokens += n;
    const int end = (int)min(run.tokens, (long long)p.num_tokens);
    const int e = grown(held[b], end - o);
    off[b] = o;
    first[b] = (int)min(run.pages, (long long)INT_MAX);
    run.pages += max(pages_of(e) - owned(b, held[b]), 0);
    if (blockIdx.x == 0) {
      p.seq_lens[b] = e;
      p.token_offsets[b] = o;
    }
  }
  if (tid == 0) {
    off[p.B] = (int)min(total.tokens, (long long)p.num_tokens);
    if (blockIdx.x == 0) {
      p.token_offsets[p.B] = off[p.B];
      p.pages_used[0] = (int)min(total.pages, (long long)INT_MAX);
    }
  }
  __syncthreads();
  const int tokens = off[p.B];

  auto free_page = [&](int b, int j) -> int {
    const long long x = (long long)first[b] + j;
    return x < p.num_free ? __ldg(p.free_pages + x) : -1;
  };

  // positions of drafted trees: c + depth, the depth being the number of steps to a node without
  // a parent (an entry that is no earlier node counts as none)
  if (kTrees) {
    const int lane = tid & 31, warp = tid >> 5;
    auto place = [&](int b, int i, long long depth) {
      p.positions[off[b] + i] = (int)min(held[b] + depth, (long long)INT_MAX);
    };
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      const int n = off[b + 1] - off[b];
      if (n <= kWarpNodes) continue;
      for (int c0 = 0; c0 < n; c0 += kChunkNodes) {
        const int m = min(n - c0, kChunkNodes);
        for (int i = tid; i < m; i += kPagesThreads) {
          const int q = __ldg(p.parents + off[b] + c0 + i);
          const bool up = q >= 0 && q < c0 + i;
          links[i] = up && q >= c0 ? ((unsigned)(q - c0) << 16) + 1u : (unsigned)i << 16;
          // this block has written the positions of earlier chunks
          if (!up) base[i] = 0;
          else if (q < c0) base[i] = p.positions[off[b] + q] - held[b] + 1;
        }
        double_links<kPagesThreads>(links, m, tid);
        for (int i = tid; i < m; i += kPagesThreads) {
          const unsigned w = links[i];
          place(b, c0 + i, (long long)base[w >> 16] + (w & 0xffffu));
        }
        __syncthreads();
      }
    }
    for (int b = blockIdx.x * kPagesWarps + warp; b < p.B; b += gridDim.x * kPagesWarps) {
      const int n = off[b + 1] - off[b];
      if (n > kWarpNodes) continue;
      unsigned* mine = links + warp * kWarpNodes;
      for (int i = lane; i < n; i += 32) {
        const int q = __ldg(p.parents + off[b] + i);
        mine[i] = q >= 0 && q < i ? ((unsigned)q << 16) + 1u : (unsigned)i << 16;
      }
      double_links<32>(mine, n, lane);
      for (int i = lane; i < n; i += 32) place(b, i, mine[i] & 0xffffu);
      __syncwarp();
    }
  }

  // slots, and the other positions
  const long long stride = (long long)gridDim.x * kPagesThreads * kTokensPerThread;
  for (long long t0 = ((long long)blockIdx.x * kPagesThreads + tid) * kTokensPerThread;
       t0 < p.num_tokens; t0 += stride) {
    long long slot[kTokensPerThread];
    int pos[kTokensPerThread];
    int b = 0;
    if (t0 < tokens) {
      int lo = 0, hi = p.B - 1;     // the last b with off[b] <= t0 (it owns t0: off[b + 1] > t0)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= t0) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    int known = -1, page = -1;      // the page of logical page `known` of sequence b
#pragma unroll
    for (int u = 0; u < kTokensPerThread; ++u) {
      const int t = (int)t0 + u;
      slot[u] = -1;
      pos[u] = 0;
      if (t >= tokens) continue;
      while (off[b + 1] <= t) {
        ++b;
        known = -1;
      }
      const int i = t - off[b];
      const int c = held[b];
      const long long row = (long long)c + i;
      if (row < cap) {
        const int pg = page_of((int)row);
        if (pg != known) {
          const int have = owned(b, c);
          known = pg;
          page = pg < have ? p.block_table[(size_t)b * p.max_pages + pg] : free_page(b, pg - have);
        }
        if (page >= 0) slot[u] = (long long)page * p.page_size + ((int)row - pg * p.page_size);
      }
      pos[u] = (int)min(row, (long long)INT_MAX);
    }
    const bool full = t0 + kTokensPerThread <= p.num_tokens;
    if (full) {
      if (!kTrees)
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<longlong2*>(p.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(p.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
    }
#pragma unroll
    for (int u = 0; u < kTokensPerThread; ++u) {
      if (t0 + u >= p.num_tokens) continue;
      if (!full) p.slots[t0 + u] = slot[u];
      // a tree's positions are written above
      if (kTrees ? t0 + u >= tokens : !full) p.positions[t0 + u] = pos[u];
    }
  }

  // new table entries: a warp for each sequence
  const int lane = tid & 31;
  for (int b = blockIdx.x * kPagesWarps + (tid >> 5); b < p.B; b += gridDim.x * kPagesWarps) {
    const int c = held[b], have = owned(b, c);
    const int need = pages_of(grown(c, off[b + 1] - off[b])) - have;
    int* row = p.block_table + (size_t)b * p.max_pages + have;
    for (int j = lane; j < need; j += 32) row[j] = free_page(b, j);
  }
}

// row mul >> shift = row / d for every row below 2^31.  With 2^s >= d, mul is 2^(31 + s) / d
// rounded up: (2^(31 + s) + e) / d with e < d.  The product exceeds the quotient by
// row e / (d 2^(31 + s)) < e / (d 2^s) < 1 / d, which changes no whole part; mul fits 32 bits.
void page_divisor(int d, unsigned& mul, int& shift) {
  int s = 0;
  while ((1LL << s) < d) ++s;
  shift = 31 + s;
  mul = (unsigned)(((1ULL << shift) + d - 1) / d);
}

}  // namespace

template <bool kTrees>
static int launch_t(const PagesParams& p, int num_sms, cudaStream_t stream) {
  const int smem = dynamic_bytes(p.B, kTrees);
  static std::atomic<bool> ready[64];
  // without the attribute a block has 48 KB, of which the fixed part comes first
  if (smem + (int)sizeof(BlockShared) > 48 * 1024 &&
      !allow_smem(reinterpret_cast<const void*>(attn_page_tables_kernel<kTrees>),
                  dynamic_bytes(kPagesMaxSeqs, kTrees), ready))
    return -4;
  const long long per_block = kPagesThreads * kTokensPerThread;
  long long blocks = std::max(((long long)p.num_tokens + per_block - 1) / per_block, 1LL);
  // A warp for each of a few trees; of many, the blocks for the tokens take several each (4000
  // trees of 100 nodes: 33 us with the tokens' 250 blocks, 37 with 444).
  if (kTrees)
    blocks = std::max(blocks, std::min(((long long)p.B + kPagesWarps - 1) / kPagesWarps,
                                       (long long)num_sms));
  // Four blocks an SM, or what fits there at a time: each takes the sums of all sequences anew,
  // and a second wave would do so one after the other.
  const int resident = std::min(4, kSmemOfSm / (smem + (int)sizeof(BlockShared) + 1024));
  blocks = std::min(blocks, (long long)std::max(resident, 1) * num_sms);
  attn_page_tables_kernel<kTrees><<<(unsigned)blocks, kPagesThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_page_tables(const PagesParams& args, int num_sms, cudaStream_t stream) {
  PagesParams p = args;
  page_divisor(p.page_size, p.div_mul, p.div_shift);
  return p.parents != nullptr ? launch_t<true>(p, num_sms, stream)
                              : launch_t<false>(p, num_sms, stream);
}

}  // namespace attn
