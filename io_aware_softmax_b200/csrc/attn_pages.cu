// Block tables and slot maps of a paged cache from request lengths, on the GPU.
//
// Sequence b holds c = ctx_lens[b] cache rows and adds n = new_lens[b] tokens.  With page size
// P it owns ceil(c / P) pages and takes ceil((c + n) / P) - ceil(c / P) more, which come off
// the free list in sequence order; token i of the sequence lands in row c + i.  Everything
// follows from two prefix sums over the sequences, of tokens and of taken pages.
//
// The bytes (12 a token, 8 a new page) take microseconds at most, so the launch and the two
// prefix sums are the cost.  One launch does all: every block takes both sums over all
// sequences itself (8 bytes a sequence from L2) and keeps them in shared memory, which needs
// no block to wait for another, and then maps its share of the tokens by a binary search.
// A page taken in this call is read from the free list, never from the table entry another
// block may be writing; entries of pages owned before are only read.
#include <cuda_runtime.h>

#include <climits>

#include "attn_serve.h"

namespace attn {

namespace {

constexpr int kPagesThreads = 256;
constexpr int kPagesWarps = kPagesThreads / 32;
constexpr int kTokensPerThread = 4;   // one 16-byte store of positions, two of slots

// Exclusive prefix sum of one 64-bit value a thread over the block; total: the whole sum.
// Sums are kept in 64 bits: lengths are caller data, and many of them can pass 2^31.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums,
                                                long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPagesWarps; ++w) {
    const long long s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kPagesThreads) attn_page_tables_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* off = smem;                 // [B + 1] first token of each sequence
  int* first = smem + p.B + 1;     // [B] free-list index of each sequence's first new page
  __shared__ long long warp_sums[kPagesWarps];
  const int tid = threadIdx.x;
  const long long cap = (long long)p.max_pages * p.page_size;   // <= 2^31 - 1 (host check)
  const int per = (p.B + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  auto held_rows = [&](int b) -> int {
    return (int)min((long long)max(__ldg(p.ctx_lens + b), 0), cap);
  };
  auto pages_of = [&](long long rows) -> int {
    return (int)((rows + p.page_size - 1) / p.page_size);
  };

  // tokens: off[b] = min(sum of the lengths before b, num_tokens)
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += max(__ldg(p.new_lens + b), 0);
  long long total;
  long long run = block_scan(sum, warp_sums, total);
  for (int b = b0; b < b1; ++b) {
    off[b] = (int)min(run, (long long)p.num_tokens);
    run += max(__ldg(p.new_lens + b), 0);
  }
  if (tid == 0) off[p.B] = (int)min(total, (long long)p.num_tokens);
  __syncthreads();

  // pages
  auto need_pages = [&](int b) -> int {
    const int c = held_rows(b);
    const long long e = min((long long)c + (off[b + 1] - off[b]), cap);
    return pages_of(e) - pages_of(c);
  };
  sum = 0;
  for (int b = b0; b < b1; ++b) sum += need_pages(b);
  run = block_scan(sum, warp_sums, total);
  const long long used0 = p.free_used != nullptr ? max(__ldg(p.free_used), 0) : 0;
  run += used0;
  total += used0;
  for (int b = b0; b < b1; ++b) {
    first[b] = (int)min(run, (long long)INT_MAX);
    run += need_pages(b);
  }
  __syncthreads();

  auto free_page = [&](int b, int j) -> int {
    const long long x = (long long)first[b] + j;
    return x < p.num_free ? __ldg(p.free_pages + x) : -1;
  };

  if (blockIdx.x == 0) {
    for (int b = tid; b < p.B; b += kPagesThreads)
      p.seq_lens[b] = (int)min((long long)held_rows(b) + (off[b + 1] - off[b]), cap);
    for (int b = tid; b <= p.B; b += kPagesThreads) p.token_offsets[b] = off[b];
    if (tid == 0) p.pages_used[0] = (int)min(total, (long long)INT_MAX);
  }

  // new table entries: a warp for each sequence
  const int lane = tid & 31;
  for (int b = blockIdx.x * kPagesWarps + (tid >> 5); b < p.B; b += gridDim.x * kPagesWarps) {
    const int need = need_pages(b);
    int* row = p.block_table + (size_t)b * p.max_pages + pages_of(held_rows(b));
    for (int j = lane; j < need; j += 32) row[j] = free_page(b, j);
  }

  // slots and positions
  const long long stride = (long long)gridDim.x * kPagesThreads * kTokensPerThread;
  for (long long t0 = ((long long)blockIdx.x * kPagesThreads + tid) * kTokensPerThread;
       t0 < p.num_tokens; t0 += stride) {
    long long slot[kTokensPerThread];
    int pos[kTokensPerThread];
    int b = 0;
    if (t0 < off[p.B]) {
      int lo = 0, hi = p.B - 1;     // the last b with off[b] <= t0 (it owns t0: off[b + 1] > t0)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= t0) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
#pragma unroll
    for (int u = 0; u < kTokensPerThread; ++u) {
      const long long t = t0 + u;
      slot[u] = -1;
      pos[u] = 0;
      if (t >= off[p.B]) continue;
      while (off[b + 1] <= t) ++b;
      const int i = (int)t - off[b];
      const int c = held_rows(b);
      const long long row = (long long)c + i;
      if (row < cap) {
        const int pg = (int)(row / p.page_size);
        const int have = pages_of(c);
        const int page = pg < have ? p.block_table[(size_t)b * p.max_pages + pg]
                                   : free_page(b, pg - have);
        if (page >= 0) slot[u] = (long long)page * p.page_size + (row - (long long)pg * p.page_size);
      }
      if (p.parents == nullptr) {
        pos[u] = (int)min(row, (long long)INT_MAX);
      } else {
        // depth in the tree: steps to a node without a parent.  A parent lies before its
        // node (any other entry counts as none), so the walk ends after at most i steps.
        int depth = 0;
        for (int j = i;;) {
          const int q = __ldg(p.parents + off[b] + j);
          if (q < 0 || q >= j) break;
          j = q;
          ++depth;
        }
        pos[u] = (int)min((long long)c + depth, (long long)INT_MAX);
      }
    }
    if (t0 + kTokensPerThread <= p.num_tokens) {
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<longlong2*>(p.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(p.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int u = 0; u < kTokensPerThread; ++u)
        if (t0 + u < p.num_tokens) {
          p.positions[t0 + u] = pos[u];
          p.slots[t0 + u] = slot[u];
        }
    }
  }
}

}  // namespace

int launch_page_tables(const PagesParams& p, int num_sms, cudaStream_t stream) {
  const int smem = (2 * p.B + 1) * 4;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(attn_page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (2 * kPagesMaxSeqs + 1) * 4) != cudaSuccess)
    return -4;
  const long long per_block = kPagesThreads * kTokensPerThread;
  long long blocks = ((long long)p.num_tokens + per_block - 1) / per_block;
  blocks = blocks < 1 ? 1 : blocks;
  if (blocks > 2 * num_sms) blocks = 2 * num_sms;
  attn_page_tables_kernel<<<(unsigned)blocks, kPagesThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace attn
