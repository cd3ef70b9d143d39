// Declarations of the operators around the attention kernels (page tables, query/key
// preparation, tree attention) shared by their launch wrappers and the C-ABI entry points.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

// Allows a kernel `bytes` of dynamic shared memory, once a device (ready: one flag a device,
// of this kernel alone): the attribute keeps, and setting it costs host time in every call.
inline bool allow_smem(const void* kernel, int bytes, std::atomic<bool> (&ready)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const bool known = dev >= 0 && dev < 64;
  if (known && ready[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  if (known) ready[dev].store(true, std::memory_order_release);
  return true;
}

// Sequences of one attn_page_tables call: 12 bytes each stay in shared memory (192 KB at this
// bound).
constexpr int kPagesMaxSeqs = 16384;

struct PagesParams {
  const int* ctx_lens;      // [B]
  const int* new_lens;      // [B]
  const int* free_pages;    // [num_free]
  const int* free_used;     // [1] or null
  const int* held_rows;     // [B] or null
  const int* parents;       // [num_tokens] or null
  int* block_table;         // [B, max_pages] (new entries written)
  long long* slots;         // [num_tokens] (written)
  int* positions;           // [num_tokens] (written)
  int* seq_lens;            // [B] (written)
  int* token_offsets;       // [B + 1] (written)
  int* pages_used;          // [1] (written)
  int B, max_pages, page_size, num_free, num_tokens;
  unsigned div_mul;         // row / page_size = row * div_mul >> div_shift (set by the launch)
  int div_shift;
};

struct PrepParams {
  const void* qkv;          // bf16 [tokens, H, d], H = Hq + 2 Hkv
  const void* wq;           // bf16 [d] or null (no norm)
  const void* wk;
  const float* table;       // fp32 [table_rows, rot]: cos | sin
  const int* positions;     // [tokens] or null (position n of row n)
  void* q;                  // forward: bf16 [B, Hq, N, d]; paged: [tokens, Hq, d]
  void* k;                  // forward: bf16 [B, Hkv, N, d]; paged: [pages, Hkv, page_size, d]
  void* v;
  const long long* slots;   // paged: [tokens]
  int num_slots;            // paged: num_pages * page_size
  int page_size;
  int tokens, N, Hq, Hkv, H;
  int rot, table_rows, interleaved;
  float eps;
};

struct PrepBwdParams {
  PrepParams f;             // q, k, v: dq, dk, dv (read)
  void* dqkv;               // bf16 [tokens, H, d] (written)
  float* partials;          // fp32 [blocks, 2, d]
  float* dwq;               // fp32 [d] (written)
  float* dwk;
};

// Heads of a token at most (query, key and value), and blocks of the backward: the workspace
// holds one partial gain gradient for each block.
constexpr int kPrepMaxHeads = 4096;
constexpr int kPrepBwdMaxBlocks = 592;

// Nodes of a sequence at most (a node's visible nodes are a 128-bit word), and rows of one
// query tile.
constexpr int kTreeMaxNodes = 128;
constexpr int kTreeRows = 128;

struct TreeParams {
  const int* block_table;   // [B, max_pages]
  const int* seq_lens;      // [B]
  const int* offsets;       // [B + 1]
  const int* parents;       // [T] or null (a chain)
  const void* v_pages;      // bf16 [num_pages, Hkv, page_size, d]: for values that are no numbers
  void* o;                  // bf16 [T, Hq, d]
  float* lse;               // fp32 [T, Hq]
  // workspace: prefix sums of the sequences' units, then the pieces' partial results
  long long* prefix;        // [B + 1]
  float* o_part;            // [2 grid, tiles a CTA, d / 4, 128, 4]: sums of exp(x - m) V
  float2* ml_part;          // [2 grid, tiles a CTA, 128]: (m in base 2, l)
  int B, T, Hq, Hkv, G;
  int page_size, max_pages, num_pages, max_nodes;
  int cap;                  // max_pages * page_size
  int tile_nodes;           // nodes of a query tile: tile_nodes * G <= 128 rows
  int grid;
  float kscale;             // scale * log2(e)
  uint32_t* err;
};

int launch_page_tables(const PagesParams& p, int num_sms, cudaStream_t stream);
int launch_qk_prep(const PrepParams& p, int d, bool paged, int num_sms, cudaStream_t stream);
int launch_qk_prep_bwd(const PrepBwdParams& p, int d, int num_sms, cudaStream_t stream);

// tq: q as (d, G, Hkv, T) in boxes of 64 x G x 1 x tile_nodes; tk, tv: pages as
// (d, page_size, num_pages * Hkv) in boxes of 64 x 64.
int launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                const TreeParams& p, int d, bool two_tiles, cudaStream_t stream);

}  // namespace attn
