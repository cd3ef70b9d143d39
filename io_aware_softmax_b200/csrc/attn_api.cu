// C-ABI entry points: argument validation, TMA descriptor construction and launches.
// Nothing here allocates device memory or synchronises (except attn_get_device_status).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "attn_serve.h"
#include "sm100_ptx.cuh"
#include "tanh_poly.cuh"

namespace attn {

// The library's device error word: [0] = error bits, [1] = first failing wait site,
// [2..3] = limit of the kernels' pipeline waits in ns (64-bit; 0: the built-in 0.5 s).
__device__ __align__(8) uint32_t g_error[4] = {0u, 0u, 0u, 0u};

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 3-D tensor map of bytes over [z, rows, inner] (inner = `extent` valid bytes of each
// `stride`-byte row) with a (128 x box_rows x 1) box and 128-byte swizzle; bytes past the
// extent read as zero.
bool make_map_3d_u8(CUtensorMap* map, const void* ptr, long long extent, long long stride,
                    long long rows, long long z, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)extent, (cuuint64_t)rows, (cuuint64_t)z};
  cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)stride * (cuuint64_t)rows};
  cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D bf16 tensor map over [z, rows, d] (d innermost) with a (64 x box_rows x 1) box and
// 128-byte swizzle: one box fills `box_rows` rows of 128 bytes in shared memory.
bool make_map_3d(CUtensorMap* map, const void* ptr, int d, long long rows, long long z,
                 int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)z};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * (cuuint64_t)rows};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Query rows of the tree attention: q [T, Hkv * G, d] as (d, G, Hkv, T) in boxes of
// 64 x G x 1 x nodes, so one box is the rows (node, head of the group) of one KV head.
bool make_map_tree_q(CUtensorMap* map, const void* ptr, int d, int G, int Hkv, int T, int nodes) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)T};
  cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * G, (cuuint64_t)d * 2 * G * Hkv};
  cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)nodes};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The soft-cap's polynomial tanh in the raw score s: cap_log2 tanh(s cap_scale) =
// s sum_i b_i s^(2i) with b_i = cap_log2 a_i cap_scale^(2i + 1), for |s cap_scale| <= 1/2
// (fast_max = 1 / (2 cap_scale) in raw units).  The kernels take it only when every b_i is a
// normal float (no term flushed to zero); otherwise fast_max = -1 turns it off.
void soft_cap_poly(float cap_scale, float cap_log2, float (&poly)[kTanhPolyTerms],
                   float& fast_max) {
  // The leading coefficient is positive, so a masked score (-inf) comes out of the
  // polynomial as -inf: the kernels need no other mask on the polynomial path.
  static_assert(kTanhPoly[kTanhPolyTerms - 1] > 0.f, "leading coefficient");
  fast_max = -1.f;
  for (int i = 0; i < kTanhPolyTerms; ++i) poly[i] = 0.f;
  if (!(cap_scale > 0.f)) return;
  bool normal = true;
  double cs_pow = (double)cap_scale;
  for (int i = 0; i < kTanhPolyTerms; ++i) {
    poly[i] = (float)((double)kTanhPoly[i] * (double)cap_log2 * cs_pow);
    normal = normal && std::isnormal(poly[i]);
    cs_pow *= (double)cap_scale * (double)cap_scale;
  }
  if (normal) fast_max = kTanhPolyMaxY / cap_scale;
}

int check_mask(int mask_kind, int window, const int* doc_offsets, int num_docs, int Nq, int Nk) {
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_SLIDING) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_NONE && Nq != Nk) return ATTN_ERR_UNSUPPORTED;
  if ((mask_kind == ATTN_MASK_SLIDING_CAUSAL || mask_kind == ATTN_MASK_SLIDING) && window < 0)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_DOCUMENT_CAUSAL) {
    if (doc_offsets == nullptr || num_docs < 1) return ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(doc_offsets) & 3u) return ATTN_ERR_MISALIGNED;
  }
  return ATTN_OK;
}

MaskParams mask_params(int mask_kind, int window, const int* doc_offsets, int num_docs, int Nq,
                       int Nk) {
  MaskParams m;
  m.kind = mask_kind;
  m.window = window;
  m.doc_offsets = doc_offsets;
  m.num_docs = num_docs;
  m.Nq = Nq;
  m.Nk = Nk;
  return m;
}

int sm_count(int device) {
  static int cached[64] = {0};
  if (device >= 0 && device < 64 && cached[device] > 0) return cached[device];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1)
    n = 148;
  if (device >= 0 && device < 64) cached[device] = n;
  return n;
}

// Device address of g_error on the current device (looked up once per device).
uint32_t* error_word_ptr(int device) {
  static std::mutex mu;
  static uint32_t* cache[64] = {};
  if (device < 0 || device >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[device] == nullptr) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_error) != cudaSuccess) return nullptr;
    cache[device] = reinterpret_cast<uint32_t*>(ptr);
  }
  return cache[device];
}

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return dev;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int attn_version(void) { return 100; }

extern "C" const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case ATTN_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case ATTN_ERR_CUDA: return "CUDA error";
    case ATTN_ERR_DEVICE_TIMEOUT: return "device wait timed out";
    case ATTN_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
  }
}

extern "C" int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int Hq, int Hkv, int Nq, int Nk, int d, float scale, int mask_kind,
                        int window, float softcap, const int* doc_offsets, int num_docs,
                        cudaStream_t stream) {
  return attn_fwd_alibi(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, mask_kind, window, softcap,
                        doc_offsets, num_docs, nullptr, stream);
}

extern "C" int attn_fwd_alibi(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                              int mask_kind, int window, float softcap, const int* doc_offsets,
                              int num_docs, const float* alibi_slopes, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || Nq < 0 || Nk < 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  int st = check_mask(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  if (st != ATTN_OK) return st;
  if (std::isnan(scale) || std::isnan(softcap)) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(alibi_slopes) & 3u) return ATTN_ERR_MISALIGNED;
  if (alibi_slopes != nullptr && softcap > 0.f) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || Hq == 0 || Nq == 0) return ATTN_OK;
  if (o == nullptr || lse == nullptr || q == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(o) || !aligned16(lse) || !aligned16(q)) return ATTN_ERR_MISALIGNED;
  const long long rows = (long long)B * Hq * Nq;
  if (Nk == 0) return launch_fill_empty(o, lse, (size_t)rows, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
  if (k == nullptr || v == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return ATTN_ERR_MISALIGNED;
  if ((long long)B * Hq > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;

  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);
  FwdParams p{};
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  // GQA with an even group: a CTA's two query tiles are two heads of one KV group at the
  // same rows (same keys, same mask, each K/V tile used by both); otherwise two adjacent
  // 128-row tiles of one head
  p.head_pairs = (p.G % 2 == 0) ? 1 : 0;
  p.num_pairs = p.head_pairs ? (Nq + 127) / 128 : (Nq + 255) / 256;
  p.num_sms = sm_count(current_device());
  // Packed documents: a unit's cost follows the document layout, so the units are dealt by
  // cost (sorted in every CTA) when they are few enough to sort in shared memory.
  p.sched = 0;
  if (mask_kind == ATTN_MASK_DOCUMENT_CAUSAL) {
    const long long U = (long long)p.num_pairs * B * (p.head_pairs ? Hq / 2 : Hq);
    const long long G = std::min<long long>(U, p.num_sms);
    if (U <= kSchedUnits && (U + G - 1) / G + 1 <= kSchedMax) p.sched = 1;
  }
  p.kscale = scale * kLog2e;
  p.softcap = softcap > 0.f ? softcap : 0.f;
  p.cap_scale = softcap > 0.f ? scale / softcap : 0.f;
  p.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
  soft_cap_poly(p.cap_scale, p.cap_log2, p.cap_poly, p.cap_fast_max);
  p.mask = mask_params(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  p.alibi = alibi_slopes;
  p.kv_reverse = alibi_slopes != nullptr ? 1 : 0;
  if ((long long)p.num_pairs * B * Hq > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  p.err = error_word_ptr(current_device());
  if (p.err == nullptr) return ATTN_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  if (!make_map_3d(&tq, q, d, Nq, (long long)B * Hq, 128) ||
      !make_map_3d(&tk, k, d, Nk, (long long)B * Hkv, 128) ||
      !make_map_3d(&tv, v, d, Nk, (long long)B * Hkv, 128))
    return ATTN_ERR_CUDA;
  return launch_attn_fwd(tq, tk, tv, p, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_blockmap(int B, int Nq, int Nk, int mask_kind, int window,
                             const int* doc_offsets, int num_docs, unsigned char* map,
                             cudaStream_t stream) {
  if (B < 0 || Nq < 0 || Nk < 0) return ATTN_ERR_INVALID_ARG;
  int st = check_mask(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  if (st != ATTN_OK) return st;
  if (B == 0 || Nq == 0 || Nk == 0) return ATTN_OK;
  if (map == nullptr) return ATTN_ERR_INVALID_ARG;
  MaskParams m = mask_params(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  return launch_blockmap(m, B, Nq, Nk, map, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" size_t attn_decode_workspace_bytes(int B, int Hq, int d, int num_splits) {
  if (B <= 0 || Hq <= 0 || d <= 0 || num_splits <= 0) return 0;
  const size_t rows = (size_t)B * Hq * num_splits;
  const size_t o_bytes = (rows * d * 4 + 255) & ~(size_t)255;
  return o_bytes + rows * 4;
}

extern "C" int attn_decode_default_splits(int B, int Hkv, int T, int device) {
  // Work items are (batch, kv head, split); a persistent grid of (SMs x resident CTAs)
  // slots walks them.  Take the smallest split count whose items fill the slots in whole
  // waves to within 1 %, keeping at least 128 keys per split.
  if (B <= 0 || Hkv <= 0 || T <= 0) return 1;
  const long long slots = (long long)sm_count(device) * 2;   // 2 resident CTAs at d=128, G<=8
  const long long heads = (long long)B * Hkv;
  const int max_splits = (int)std::max(1LL, std::min<long long>(256, (long long)T / 128));
  int best = 1;
  double best_eff = -1.0;
  for (int s = 1; s <= max_splits; ++s) {
    const long long items = heads * s;
    const long long waves = (items + slots - 1) / slots;
    const double eff = (double)items / (double)(waves * slots);
    if (eff > best_eff + 1e-9) {
      best_eff = eff;
      best = s;
    }
    if (eff >= 0.99) break;
  }
  return best;
}

extern "C" int attn_decode_merge(const float* o_part, const float* lse_part, void* o, float* lse,
                                 long long rows, int num_splits, int d, cudaStream_t stream) {
  if (rows < 0 || num_splits < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (rows == 0) return ATTN_OK;
  if (!o_part || !lse_part || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(o_part) || !aligned16(o) || ((uintptr_t)lse_part & 3u) || ((uintptr_t)lse & 3u))
    return ATTN_ERR_MISALIGNED;
  return launch_merge(o_part, lse_part, o, lse, rows, num_splits, d, stream) == 0 ? ATTN_OK
                                                                                  : ATTN_ERR_CUDA;
}

extern "C" int attn_decode_splitkv(const void* q, const void* k_cache, const void* v_cache,
                                   void* o, float* lse, int B, int Hq, int Hkv, int T, int d,
                                   float scale, int num_splits, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || T < 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  if (std::isnan(scale)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0) return ATTN_OK;
  const int G = Hq / Hkv;
  if (G > 16) return ATTN_ERR_UNSUPPORTED;
  if (!q || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse)) return ATTN_ERR_MISALIGNED;
  if (T == 0) return launch_fill_empty(o, lse, (size_t)B * Hq, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
  if (!k_cache || !v_cache) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return ATTN_ERR_MISALIGNED;
  const int dev = current_device();
  if (num_splits <= 0) num_splits = attn_decode_default_splits(B, Hkv, T, dev);
  if (num_splits > T) num_splits = T;
  const size_t need = attn_decode_workspace_bytes(B, Hq, d, num_splits);
  if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);

  DecParams p{};
  p.q = q;
  p.o_part = reinterpret_cast<float*>(workspace);
  const size_t rows = (size_t)B * Hq * num_splits;
  p.lse_part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                        ((rows * d * 4 + 255) & ~(size_t)255));
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.T = T;
  p.S = num_splits;
  p.num_items = B * Hkv * num_splits;
  p.kscale = scale * kLog2e;
  if ((long long)B * Hkv * num_splits > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  p.err = error_word_ptr(dev);
  if (p.err == nullptr) return ATTN_ERR_CUDA;

  CUtensorMap tk, tv;
  if (!make_map_3d(&tk, k_cache, d, T, (long long)B * Hkv, 64) ||
      !make_map_3d(&tv, v_cache, d, T, (long long)B * Hkv, 64))
    return ATTN_ERR_CUDA;
  const int slots = sm_count(dev) * decode_ctas_per_sm(d, G);
  const int grid = (int)std::min<long long>(p.num_items, slots);
  if (launch_decode_split(tk, tv, p, d, G, grid, stream) != 0) return ATTN_ERR_CUDA;
  return launch_merge(p.o_part, p.lse_part, o, lse, (long long)B * Hq, num_splits, d, stream) == 0
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

static int g_last_site = 0;

extern "C" int attn_get_device_status(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  uint32_t word[2] = {0u, 0u};
  const uint32_t zero[2] = {0u, 0u};
  if (cudaMemcpyFromSymbol(word, g_error, sizeof(word)) != cudaSuccess) return ATTN_ERR_CUDA;
  if (word[0] == 0) return ATTN_OK;
  if (cudaMemcpyToSymbol(g_error, zero, sizeof(zero)) != cudaSuccess) return ATTN_ERR_CUDA;
  g_last_site = (int)word[1];
  return (word[0] & kErrWaitTimeout) ? ATTN_ERR_DEVICE_TIMEOUT : ATTN_ERR_CUDA;
}

extern "C" int attn_last_error_site(void) { return g_last_site; }

extern "C" int attn_set_wait_limit_ns(unsigned long long ns) {
  const uint64_t v = ns;
  if (cudaDeviceSynchronize() != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaMemcpyToSymbol(g_error, &v, sizeof(v), 2 * sizeof(uint32_t)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

extern "C" int attn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                 const int* block_table, const int* seq_lens, void* o, float* lse,
                                 int B, int Hq, int Hkv, int num_pages, int page_size,
                                 int max_pages_per_seq, int d, float scale, int num_splits,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || num_pages < 0 || page_size <= 0 || max_pages_per_seq < 0)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size % 64 != 0) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  if (std::isnan(scale)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0) return ATTN_OK;
  const int G = Hq / Hkv;
  if (G > 16) return ATTN_ERR_UNSUPPORTED;
  if (!q || !o || !lse || !seq_lens || !block_table) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse)) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(seq_lens) & 3u) || (reinterpret_cast<uintptr_t>(block_table) & 3u))
    return ATTN_ERR_MISALIGNED;
  const long long t_cap = (long long)max_pages_per_seq * page_size;
  if (num_pages == 0 || t_cap == 0)
    return launch_fill_empty(o, lse, (size_t)B * Hq, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
  if (!k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return ATTN_ERR_MISALIGNED;
  if (t_cap > (1LL << 31) - 1 || (long long)num_pages * Hkv > (1LL << 31) - 1)
    return ATTN_ERR_UNSUPPORTED;
  const int dev = current_device();
  const int tiles = (int)((t_cap + 63) / 64);
  if (num_splits <= 0) num_splits = attn_decode_default_splits(B, Hkv, (int)t_cap, dev);
  if (num_splits > tiles) num_splits = tiles;
  const size_t need = attn_decode_workspace_bytes(B, Hq, d, num_splits);
  if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);

  DecParams p{};
  p.q = q;
  p.o_part = reinterpret_cast<float*>(workspace);
  const size_t rows = (size_t)B * Hq * num_splits;
  p.lse_part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                        ((rows * d * 4 + 255) & ~(size_t)255));
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.T = (int)t_cap;
  p.S = num_splits;
  if ((long long)B * Hkv * num_splits > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  p.num_items = B * Hkv * num_splits;
  p.kscale = scale * kLog2e;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.page_size = page_size;
  p.max_pages = max_pages_per_seq;
  p.err = error_word_ptr(dev);
  if (p.err == nullptr) return ATTN_ERR_CUDA;

  CUtensorMap tk, tv;
  if (!make_map_3d(&tk, k_pages, d, page_size, (long long)num_pages * Hkv, 64) ||
      !make_map_3d(&tv, v_pages, d, page_size, (long long)num_pages * Hkv, 64))
    return ATTN_ERR_CUDA;
  const int slots = sm_count(dev) * decode_ctas_per_sm(d, G);
  const int grid = (int)std::min<long long>(p.num_items, slots);
  if (launch_decode_split(tk, tv, p, d, G, grid, stream) != 0) return ATTN_ERR_CUDA;
  return launch_merge(p.o_part, p.lse_part, o, lse, (long long)B * Hq, num_splits, d, stream) == 0
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

extern "C" size_t attn_bwd_workspace_bytes(int B, int Hq, int Nq) {
  if (B <= 0 || Hq <= 0 || Nq <= 0) return 0;
  const size_t rows = (size_t)B * Hq * Nq;
  return 2 * ((rows * 4 + 255) & ~(size_t)255);
}

extern "C" int attn_bwd(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int Hq, int Hkv, int Nq, int Nk, int d, float scale, int mask_kind,
                        int window, float softcap, const int* doc_offsets, int num_docs,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attn_bwd_alibi(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale,
                        mask_kind, window, softcap, doc_offsets, num_docs, nullptr, workspace,
                        workspace_bytes, stream);
}

extern "C" int attn_bwd_alibi(const void* q, const void* k, const void* v, const void* o,
                              const void* dout, const float* lse, void* dq, void* dk, void* dv,
                              int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                              int mask_kind, int window, float softcap, const int* doc_offsets,
                              int num_docs, const float* alibi_slopes, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || Nq < 0 || Nk < 0) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(alibi_slopes) & 3u) return ATTN_ERR_MISALIGNED;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  int st = check_mask(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  if (st != ATTN_OK) return st;
  if (std::isnan(scale) || std::isnan(softcap)) return ATTN_ERR_INVALID_ARG;
  if (softcap > 0.f && alibi_slopes != nullptr) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || Hq == 0 || (Nq == 0 && Nk == 0)) return ATTN_OK;
  const void* ptrs[] = {q, k, v, o, dout, lse, dq, dk, dv};
  const int needed[] = {Nq > 0, Nk > 0, Nk > 0, Nq > 0, Nq > 0, Nq > 0, Nq > 0, Nk > 0, Nk > 0};
  for (int i = 0; i < 9; ++i) {
    if (!needed[i]) continue;
    if (ptrs[i] == nullptr) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(ptrs[i])) return ATTN_ERR_MISALIGNED;
  }
  const size_t rows = (size_t)B * Hq * Nq;
  const size_t need = attn_bwd_workspace_bytes(B, Hq, Nq);
  if (Nq > 0 && (workspace == nullptr || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (Nq > 0 && !aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  if ((long long)B * Hq > (1LL << 31) - 1 || (long long)B * Hkv * ((Nk + 127) / 128) > (1LL << 31) - 1 ||
      (long long)B * Hq * ((Nq + 127) / 128) > (1LL << 31) - 1)
    return ATTN_ERR_UNSUPPORTED;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);
  const int dev = current_device();

  BwdParams p{};
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dvec = reinterpret_cast<float*>(workspace);
  p.l2 = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + need / 2);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.kscale = scale * kLog2e;
  p.scale = scale;
  p.mask = mask_params(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  p.alibi = alibi_slopes;
  p.cap_scale = softcap > 0.f ? scale / softcap : 0.f;
  p.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
  soft_cap_poly(p.cap_scale, p.cap_log2, p.cap_poly, p.cap_fast_max);
  p.err = error_word_ptr(dev);
  if (p.err == nullptr) return ATTN_ERR_CUDA;
  if (Nq > 0 && launch_bwd_rowdot(o, dout, lse, const_cast<float*>(p.dvec),
                                  const_cast<float*>(p.l2), (long long)rows, d, stream) != 0)
    return ATTN_ERR_CUDA;

  // With no query rows dK = dV = 0; with no keys dQ = 0 (the kernels write these too, but
  // their maps need a non-empty tensor).
  CUtensorMap tq, tdo, tk, tv;
  if (Nq == 0 || Nk == 0) {
    if (Nk > 0) {
      if (cudaMemsetAsync(dk, 0, (size_t)B * Hkv * Nk * d * 2, stream) != cudaSuccess ||
          cudaMemsetAsync(dv, 0, (size_t)B * Hkv * Nk * d * 2, stream) != cudaSuccess)
        return ATTN_ERR_CUDA;
    }
    if (Nq > 0 && cudaMemsetAsync(dq, 0, rows * d * 2, stream) != cudaSuccess)
      return ATTN_ERR_CUDA;
    return ATTN_OK;
  }
  if (!make_map_3d(&tq, q, d, Nq, (long long)B * Hq, 128) ||
      !make_map_3d(&tdo, dout, d, Nq, (long long)B * Hq, 128) ||
      !make_map_3d(&tk, k, d, Nk, (long long)B * Hkv, 128) ||
      !make_map_3d(&tv, v, d, Nk, (long long)B * Hkv, 128))
    return ATTN_ERR_CUDA;
  return launch_attn_bwd(tq, tdo, tk, tv, p, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_quantize_fp8(const void* x, void* out, float* scales, int B, int H, int N,
                                 int d, int block_rows, int transpose, int n_pad,
                                 const float* signs, cudaStream_t stream) {
  if (B < 0 || H < 0 || N < 0 || block_rows <= 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (transpose && n_pad < N) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || N == 0) return ATTN_OK;
  if (!x || !out || !scales) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || (reinterpret_cast<uintptr_t>(scales) & 3u) ||
      (reinterpret_cast<uintptr_t>(signs) & 3u))
    return ATTN_ERR_MISALIGNED;
  if (!transpose && (reinterpret_cast<uintptr_t>(out) & 3u)) return ATTN_ERR_MISALIGNED;
  uint32_t* err = error_word_ptr(current_device());
  if (err == nullptr) return ATTN_ERR_CUDA;
  // row-major blocks of at most 128 rows take tiled copies (the other layouts plain loads)
  CUtensorMap tx;
  const bool tiled = !transpose && block_rows <= 128 &&
                     make_map_3d(&tx, x, d, N, (long long)B * H, block_rows);
  return launch_quantize_e4m3(tiled ? &tx : nullptr, x, out, scales, B, H, N, d, block_rows,
                              transpose, n_pad, signs, err, sm_count(current_device()),
                              stream) == 0
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

extern "C" int attn_fwd_fp8(const void* q8, const void* k8, const void* vt8,
                            const float* q_scales, const float* k_scales, const float* v_scales,
                            void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Nk,
                            int nk_pad, int d, float scale, int mask_kind, int window,
                            const int* doc_offsets, int num_docs, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || Nq < 0 || Nk < 0) return ATTN_ERR_INVALID_ARG;
  if (d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  int st = check_mask(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  if (st != ATTN_OK) return st;
  if (std::isnan(scale)) return ATTN_ERR_INVALID_ARG;
  if (nk_pad < Nk || (nk_pad & 15)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0 || Nq == 0) return ATTN_OK;
  if (!o || !lse || !q8 || !q_scales) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(o) || !aligned16(lse) || !aligned16(q8)) return ATTN_ERR_MISALIGNED;
  const long long rows = (long long)B * Hq * Nq;
  if (Nk == 0) return launch_fill_empty(o, lse, (size_t)rows, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
  if (!k8 || !vt8 || !k_scales || !v_scales) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k8) || !aligned16(vt8)) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(q_scales) | reinterpret_cast<uintptr_t>(k_scales) |
       reinterpret_cast<uintptr_t>(v_scales)) & 3u)
    return ATTN_ERR_MISALIGNED;
  if ((long long)B * Hq > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;

  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);
  FwdParams p{};
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  // GQA with an even group: a CTA's two query tiles are two heads of one KV group at the
  // same rows (same keys, same mask, each K/V tile used by both); otherwise two adjacent
  // 128-row tiles of one head
  p.head_pairs = (p.G % 2 == 0) ? 1 : 0;
  p.num_pairs = p.head_pairs ? (Nq + 127) / 128 : (Nq + 255) / 256;
  p.num_sms = sm_count(current_device());
  p.kscale = scale * kLog2e;
  p.mask = mask_params(mask_kind, window, doc_offsets, num_docs, Nq, Nk);
  p.q_scales = q_scales;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.nqt = (Nq + 127) / 128;
  p.nkt = (Nk + 127) / 128;
  if ((long long)p.num_pairs * B * Hq > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  p.err = error_word_ptr(current_device());
  if (p.err == nullptr) return ATTN_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  if (!make_map_3d_u8(&tq, q8, d, d, Nq, (long long)B * Hq, 128) ||
      !make_map_3d_u8(&tk, k8, d, d, Nk, (long long)B * Hkv, 128) ||
      !make_map_3d_u8(&tv, vt8, Nk, nk_pad, d, (long long)B * Hkv, d))
    return ATTN_ERR_CUDA;
  return launch_attn_fwd(tq, tk, tv, p, d, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

// ------------------------------------------------------------------ page tables and slots

namespace {

// Bytes that a call reads or writes (a null pointer: none).
struct Range {
  const void* ptr;
  size_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return a.ptr != nullptr && b.ptr != nullptr && a.bytes > 0 && b.bytes > 0 &&
         x < y + b.bytes && y < x + a.bytes;
}

// Whether an output lies on an input or on another output: blocks read while others write.
template <size_t I, size_t O>
bool overlaps(const Range (&ins)[I], const Range (&outs)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (size_t i = 0; i < I; ++i)
      if (overlap(ins[i], outs[o])) return true;
    for (size_t i = 0; i < o; ++i)
      if (overlap(outs[i], outs[o])) return true;
  }
  return false;
}

}  // namespace

extern "C" int attn_page_tables(const int* ctx_lens, const int* new_lens, const int* free_pages,
                                const int* free_used, const int* held_rows, const int* parents,
                                int* block_table, long long* slots, int* positions, int* seq_lens,
                                int* token_offsets, int* pages_used, int B, int max_pages_per_seq,
                                int page_size, int num_free, int num_tokens,
                                cudaStream_t stream) {
  if (B < 0 || max_pages_per_seq < 0 || page_size <= 0 || num_free < 0 || num_tokens < 0)
    return ATTN_ERR_INVALID_ARG;
  if (B > kPagesMaxSeqs || num_tokens > INT_MAX - 4 ||
      (long long)max_pages_per_seq * page_size > (1LL << 31) - 1)
    return ATTN_ERR_UNSUPPORTED;
  if (!token_offsets || !pages_used || (num_tokens > 0 && (!slots || !positions)) ||
      (B > 0 && (!ctx_lens || !new_lens || !seq_lens)) ||
      (B > 0 && max_pages_per_seq > 0 && !block_table) || (num_free > 0 && !free_pages))
    return ATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {slots, positions};
  for (const void* q : ptrs)
    if (!aligned16(q)) return ATTN_ERR_MISALIGNED;
  const void* ints[] = {ctx_lens,  new_lens,    free_pages, free_used,     held_rows,
                        parents,   block_table, seq_lens,   token_offsets, pages_used};
  for (const void* q : ints)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return ATTN_ERR_MISALIGNED;
  // every block reads the inputs while block 0 writes the outputs
  const size_t nb = (size_t)B * 4, nt = (size_t)num_tokens * 4;
  const Range ins[] = {{ctx_lens, nb}, {new_lens, nb}, {free_pages, (size_t)num_free * 4},
                       {free_used, 4}, {held_rows, nb}, {parents, nt}};
  const Range outs[] = {{block_table, nb * max_pages_per_seq}, {slots, 2 * nt}, {positions, nt},
                        {seq_lens, nb}, {token_offsets, nb + 4}, {pages_used, 4}};
  if (overlaps(ins, outs)) return ATTN_ERR_INVALID_ARG;
  PagesParams p{ctx_lens, new_lens, free_pages, free_used, held_rows, parents, block_table, slots, positions,
                seq_lens, token_offsets, pages_used, B, max_pages_per_seq, page_size, num_free,
                num_tokens};
  return launch_page_tables(p, sm_count(current_device()), stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

// ----------------------------------------------------------- query / key norm and rotation

// The checks that the three forms share; fills the common fields of p.
static int check_prep(PrepParams& p, const void* qkv, const void* q_weight, const void* k_weight,
                      const float* rope_table, const int* positions, long long tokens, int N,
                      int Hq, int Hkv, int d, int rot, int table_rows, float eps,
                      int interleaved) {
  if (tokens < 0 || N < 0 || Hq < 0 || Hkv < 0 || rot < 0 || table_rows < 0)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (rot > d || rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (q_weight != nullptr && !(eps >= FLT_MIN && eps <= FLT_MAX)) return ATTN_ERR_INVALID_ARG;
  const long long H = (long long)Hq + 2LL * Hkv;
  // rows of one call: a warp takes several, and their number is a 32-bit index
  if (tokens * H > (1LL << 31) - 1 || H > kPrepMaxHeads) return ATTN_ERR_UNSUPPORTED;
  if (tokens > 0 && H > 0) {
    if (qkv == nullptr || (rot > 0 && table_rows > 0 && rope_table == nullptr))
      return ATTN_ERR_INVALID_ARG;
    // without positions they are 0 to N - 1, and all of them have to be in the table
    if (rot > 0 && positions == nullptr && table_rows < N) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(rope_table) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u))
      return ATTN_ERR_MISALIGNED;
  }
  p.qkv = qkv;
  p.wq = q_weight;
  p.wk = k_weight;
  p.table = rope_table;
  p.positions = positions;
  p.tokens = (int)tokens;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.H = (int)H;
  p.rot = rot;
  p.table_rows = table_rows;
  p.interleaved = interleaved != 0;
  p.eps = eps;
  return ATTN_OK;
}

extern "C" int attn_qk_norm_rope(const void* qkv, const void* q_weight, const void* k_weight,
                                 const float* rope_table, const int* positions, void* q, void* k,
                                 void* v, int B, int N, int Hq, int Hkv, int d, int rot,
                                 int table_rows, float eps, int interleaved,
                                 cudaStream_t stream) {
  if (B < 0) return ATTN_ERR_INVALID_ARG;
  PrepParams p{};
  const int st = check_prep(p, qkv, q_weight, k_weight, rope_table, positions, (long long)B * N, N,
                            Hq, Hkv, d, rot, table_rows, eps, interleaved);
  if (st != ATTN_OK) return st;
  if (p.tokens == 0 || p.H == 0) return ATTN_OK;
  if ((Hq > 0 && !q) || (Hkv > 0 && (!k || !v))) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return ATTN_ERR_MISALIGNED;
  const size_t head = (size_t)p.tokens * d * 2;
  const Range ins[] = {{qkv, head * p.H}, {q_weight, (size_t)d * 2}, {k_weight, (size_t)d * 2},
                       {rope_table, (size_t)table_rows * rot * 4},
                       {positions, (size_t)p.tokens * 4}};
  const Range outs[] = {{q, head * Hq}, {k, head * Hkv}, {v, head * Hkv}};
  if (overlaps(ins, outs)) return ATTN_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.v = v;
  return launch_qk_prep(p, d, false, sm_count(current_device()), stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_qk_norm_rope_paged(const void* qkv, const void* q_weight,
                                       const void* k_weight, const float* rope_table,
                                       const int* positions, const long long* slots, void* q,
                                       void* k_pages, void* v_pages, int T, int Hq, int Hkv, int d,
                                       int num_pages, int page_size, int rot, int table_rows,
                                       float eps, int interleaved, cudaStream_t stream) {
  if (num_pages < 0 || page_size <= 0) return ATTN_ERR_INVALID_ARG;
  PrepParams p{};
  const int st = check_prep(p, qkv, q_weight, k_weight, rope_table, positions, T, 1, Hq, Hkv, d,
                            rot, table_rows, eps, interleaved);
  if (st != ATTN_OK) return st;
  if ((long long)num_pages * page_size > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  if (p.tokens == 0 || p.H == 0) return ATTN_OK;
  if ((Hq > 0 && !q) || !positions || !slots || (Hkv > 0 && num_pages > 0 && (!k_pages || !v_pages)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u))
    return ATTN_ERR_MISALIGNED;
  const size_t head = (size_t)T * d * 2, cache = (size_t)num_pages * page_size * Hkv * d * 2;
  const Range ins[] = {{qkv, head * p.H}, {q_weight, (size_t)d * 2}, {k_weight, (size_t)d * 2},
                       {rope_table, (size_t)table_rows * rot * 4}, {positions, (size_t)T * 4},
                       {slots, (size_t)T * 8}};
  const Range outs[] = {{q, head * Hq}, {k_pages, cache}, {v_pages, cache}};
  if (overlaps(ins, outs)) return ATTN_ERR_INVALID_ARG;
  p.q = q;
  p.k = k_pages;
  p.v = v_pages;
  p.slots = slots;
  p.page_size = page_size;
  p.num_slots = num_pages * page_size;
  return launch_qk_prep(p, d, true, sm_count(current_device()), stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" size_t attn_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d > 0 ? (size_t)kPrepBwdMaxBlocks * 2 * d * sizeof(float) : 0;
}

extern "C" int attn_qk_norm_rope_bwd(const void* qkv, const void* q_weight, const void* k_weight,
                                     const float* rope_table, const int* positions,
                                     const void* dq, const void* dk, const void* dv, void* dqkv,
                                     float* dq_weight, float* dk_weight, int B, int N, int Hq,
                                     int Hkv, int d, int rot, int table_rows, float eps,
                                     int interleaved, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  if (B < 0) return ATTN_ERR_INVALID_ARG;
  PrepBwdParams p{};
  const int st = check_prep(p.f, qkv, q_weight, k_weight, rope_table, positions, (long long)B * N,
                            N, Hq, Hkv, d, rot, table_rows, eps, interleaved);
  if (st != ATTN_OK) return st;
  const bool norm = q_weight != nullptr;
  if (norm) {
    if (!dq_weight || !dk_weight) return ATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u)
      return ATTN_ERR_MISALIGNED;
  }
  if (p.f.tokens == 0 || p.f.H == 0) {      // no rows: the gains' gradients are empty sums
    if (norm && (cudaMemsetAsync(dq_weight, 0, (size_t)d * 4, stream) != cudaSuccess ||
                 cudaMemsetAsync(dk_weight, 0, (size_t)d * 4, stream) != cudaSuccess))
      return ATTN_ERR_CUDA;
    return ATTN_OK;
  }
  if ((Hq > 0 && !dq) || (Hkv > 0 && (!dk || !dv)) || !dqkv) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dqkv))
    return ATTN_ERR_MISALIGNED;
  if (norm) {
    if (workspace == nullptr || workspace_bytes < attn_qk_norm_rope_bwd_workspace_bytes(d))
      return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  }
  const size_t head = (size_t)p.f.tokens * d * 2, gain = (size_t)d * 4;
  const Range ins[] = {{qkv, head * p.f.H}, {q_weight, gain / 2}, {k_weight, gain / 2},
                       {rope_table, (size_t)table_rows * rot * 4},
                       {positions, (size_t)p.f.tokens * 4}, {dq, head * Hq}, {dk, head * Hkv},
                       {dv, head * Hkv}};
  const Range outs[] = {{dqkv, head * p.f.H}, {norm ? dq_weight : nullptr, gain},
                        {norm ? dk_weight : nullptr, gain},
                        {norm ? workspace : nullptr, attn_qk_norm_rope_bwd_workspace_bytes(d)}};
  if (overlaps(ins, outs)) return ATTN_ERR_INVALID_ARG;
  p.f.q = const_cast<void*>(dq);
  p.f.k = const_cast<void*>(dk);
  p.f.v = const_cast<void*>(dv);
  p.dqkv = dqkv;
  p.partials = static_cast<float*>(workspace);
  p.dwq = dq_weight;
  p.dwk = dk_weight;
  return launch_qk_prep_bwd(p, d, sm_count(current_device()), stream) == 0 ? ATTN_OK
                                                                           : ATTN_ERR_CUDA;
}

// ---------------------------------------------------------------------- tree attention

namespace {

// How a tree call is cut: nodes of a query tile, whether a CTA takes two of them, and where
// the workspace's arrays begin.
struct TreePlan {
  int tile_nodes, tiles, grid;
  size_t ml, o, bytes;
};

TreePlan tree_plan(int B, int G, int max_nodes, int d, int device) {
  TreePlan t;
  t.tile_nodes = std::min(kTreeRows / G, std::max(max_nodes, 1));
  t.tiles = max_nodes > t.tile_nodes ? 2 : 1;
  t.grid = sm_count(device);
  const size_t rows = (size_t)2 * t.grid * t.tiles * kTreeRows;
  t.ml = (((size_t)B + 1) * 8 + 255) & ~(size_t)255;
  t.o = t.ml + ((rows * 8 + 255) & ~(size_t)255);
  t.bytes = t.o + rows * d * 4;
  return t;
}

}  // namespace

extern "C" size_t attn_decode_tree_workspace_bytes(int B, int Hq, int Hkv, int max_nodes, int d,
                                                   int device) {
  if (B <= 0 || Hkv <= 0 || Hq < Hkv || Hq / Hkv > 16 || max_nodes <= 0 || d <= 0) return 0;
  return tree_plan(B, Hq / Hkv, max_nodes, d, device).bytes;
}

extern "C" int attn_decode_tree(const void* q, const void* k_pages, const void* v_pages,
                                const int* block_table, const int* seq_lens,
                                const int* token_offsets, const int* parents, void* o, float* lse,
                                int B, int T, int Hq, int Hkv, int num_pages, int page_size,
                                int max_pages_per_seq, int max_nodes, int d, float scale,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || num_pages < 0 || page_size <= 0 ||
      max_pages_per_seq < 0 || max_nodes < 0)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size % 64 != 0 || max_nodes > kTreeMaxNodes) return ATTN_ERR_UNSUPPORTED;
  if (Hkv == 0 && Hq > 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && Hq % Hkv != 0) return ATTN_ERR_UNSUPPORTED;
  if (std::isnan(scale)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || Hq == 0 || max_nodes == 0) return ATTN_OK;
  const int G = Hq / Hkv;
  if (G > 16) return ATTN_ERR_UNSUPPORTED;
  const long long cap = (long long)max_pages_per_seq * page_size;
  if (!q || !o || !lse || !seq_lens || !token_offsets || (cap > 0 && !block_table) ||
      (num_pages > 0 && (!k_pages || !v_pages)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned16(k_pages) ||
      !aligned16(v_pages))
    return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(token_offsets) | reinterpret_cast<uintptr_t>(parents)) & 3u)
    return ATTN_ERR_MISALIGNED;
  const int dev = current_device();
  const TreePlan plan = tree_plan(B, G, max_nodes, d, dev);
  const long long blocks = (max_nodes + plan.tile_nodes * plan.tiles - 1) /
                           (plan.tile_nodes * plan.tiles);
  if (cap > (1LL << 31) - 1 - 256 || (long long)num_pages * Hkv > (1LL << 31) - 1 ||
      (long long)T * Hq > (1LL << 31) - 1 ||
      Hkv > 65535 || blocks * Hkv * ((cap + 127) / 128 + 8) > (1LL << 31) - 1)
    return ATTN_ERR_UNSUPPORTED;
  // a CTA counts its share of the units in 32 bits as well
  if (blocks * Hkv * ((cap + 127) / 128 + 8) * std::min(B, T) > plan.grid * ((1LL << 31) - 2))
    return ATTN_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < plan.bytes) return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  const size_t row = (size_t)T * Hq, cache = (size_t)num_pages * page_size * Hkv * d * 2;
  const Range ins[] = {{q, row * d * 2}, {k_pages, cache}, {v_pages, cache},
                       {block_table, (size_t)B * max_pages_per_seq * 4}, {seq_lens, (size_t)B * 4},
                       {token_offsets, (size_t)B * 4 + 4}, {parents, (size_t)T * 4}};
  const Range outs[] = {{o, row * d * 2}, {lse, row * 4}, {workspace, plan.bytes}};
  if (overlaps(ins, outs)) return ATTN_ERR_INVALID_ARG;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);

  TreeParams p{};
  p.v_pages = v_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.offsets = token_offsets;
  p.parents = parents;
  p.o = o;
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.prefix = reinterpret_cast<long long*>(ws);
  p.ml_part = reinterpret_cast<float2*>(ws + plan.ml);
  p.o_part = reinterpret_cast<float*>(ws + plan.o);
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.page_size = page_size;
  p.max_pages = max_pages_per_seq;
  // without a page there is no row: every length counts as 0
  p.num_pages = num_pages;
  p.cap = num_pages > 0 ? (int)cap : 0;
  p.max_nodes = max_nodes;
  p.tile_nodes = plan.tile_nodes;
  p.grid = plan.grid;
  p.kscale = scale * kLog2e;
  p.err = error_word_ptr(dev);
  if (p.err == nullptr) return ATTN_ERR_CUDA;
  if (num_pages == 0) {      // the maps need a tensor: nothing of it is read
    k_pages = v_pages = q;
    p.num_pages = 0;
  }
  CUtensorMap tq, tk, tv;
  const long long z = std::max((long long)num_pages * Hkv, 1LL);
  if (!make_map_tree_q(&tq, q, d, G, Hkv, T, plan.tile_nodes) ||
      !make_map_3d(&tk, k_pages, d, num_pages > 0 ? page_size : 1, z, 64) ||
      !make_map_3d(&tv, v_pages, d, num_pages > 0 ? page_size : 1, z, 64))
    return ATTN_ERR_CUDA;
  return launch_tree(tq, tk, tv, p, d, plan.tiles == 2, stream) == 0 ? ATTN_OK : ATTN_ERR_CUDA;
}
