// Per-head RMS norm of queries and keys and the rotary position rotation in one pass over the
// projection's output, forward and backward.
//
// A row is one head of one token, x of d values.  With gain w and the token's angles,
//   r = 1 / sqrt(mean(x^2) + eps),  z = r w x,  (y_a, y_b) = (z_a cos - z_b sin, z_b cos + z_a sin)
// over the pairs (a, b) of the first rot values: (i, i + rot/2), or (2i, 2i + 1) interleaved.
// V rows are copied.  The input is [token][head][d], as the projection leaves it; the output
// is the layout the attention kernels read ([B, H, N, d]), or q in token order with the K and V
// rows put into the pages of a paged cache.  Backward, with dy rotated back to dz (the
// rotation's transpose):
//   dx = r (w dz) - x r^3 / d sum(x w dz),   dw = sum over rows of dz x r.
//
// All of it is bound by the bytes: 2 to 3 passes over the rows and some ten operations a
// value.  16 (d = 128) or 8 (d = 64) lanes hold a row, 16 bytes each, so loads and stores are
// whole lines, the sums are shuffles, and a pair's other half is in the same lane
// (interleaved) or a fixed number of lanes away.  A warp takes kSteps * 32 / lanes rows of ONE
// token: it issues all their loads first, and reads the token's angles once for all of them.
// Sums, statistics and the rotation are in fp32; each output is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_serve.h"

namespace attn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kFwdSteps = 4;
constexpr int kBwdSteps = 2;

template <int D>
struct Row {
  static constexpr int kLanes = D / 8;           // lanes a row
  static constexpr int kRows = 32 / kLanes;      // rows a warp holds at a time
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

__device__ __forceinline__ uint4 load_once(const void* base, size_t elem) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<const __nv_bfloat16*>(base) + elem));
  return v;
}

__device__ __forceinline__ void store8(void* base, size_t elem, const uint4& v) {
  *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + elem) = v;
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This lane's coefficients: y[i] = z[i] c[i] + z_partner[i] s[i].  A position outside the
// table reads a row of zeros, as a page outside the cache does.
template <bool kInter>
struct Angles {
  float c[8], s[8];
  bool rotates;
  int partner;      // lane that holds the pairs' other halves (halves layout)

  __device__ __forceinline__ void load(const PrepParams& p, int pos, int e0, int lane) {
    const int half = p.rot >> 1;
    rotates = e0 < p.rot;
    partner = lane;
    if (!rotates) return;
    const bool valid = (unsigned)pos < (unsigned)p.table_rows;
    const float* row = p.table + (size_t)(valid ? pos : 0) * p.rot;
    if (kInter) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (valid) {
        a = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
        b = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
      }
      const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = cc[i];
        s[2 * i] = -ss[i];
        s[2 * i + 1] = ss[i];
      }
    } else {
      const bool low = e0 < half;
      const int j = low ? e0 : e0 - half;
      partner = low ? lane + (half >> 3) : lane - (half >> 3);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (valid) {
          a = __ldg(reinterpret_cast<const float4*>(row + j + i));
          b = __ldg(reinterpret_cast<const float4*>(row + half + j + i));
        }
        c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
        s[i] = low ? -b.x : b.x;
        s[i + 1] = low ? -b.y : b.y;
        s[i + 2] = low ? -b.z : b.z;
        s[i + 3] = low ? -b.w : b.w;
      }
    }
  }

  // z rotated (sign 1) or rotated back (sign -1), in place; every lane of the warp calls it.
  __device__ __forceinline__ void apply(float (&z)[8], float sign) const {
    float zp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      zp[i] = kInter ? z[i ^ 1] : __shfl_sync(0xffffffffu, z[i], partner);
    if (!rotates) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = fmaf(z[i], c[i], zp[i] * (sign * s[i]));
  }
};

template <int D, bool kNorm, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kPrepThreads, 3) attn_qk_prep_kernel(const PrepParams p) {
  using R = Row<D>;
  const int lane = threadIdx.x & 31;
  const int sub = lane / R::kLanes, e0 = (lane % R::kLanes) * 8;
  constexpr int kItemRows = kFwdSteps * R::kRows;
  const int bpt = (p.H + kItemRows - 1) / kItemRows;     // items a token
  const unsigned item = blockIdx.x * kPrepWarps + (threadIdx.x >> 5);
  const int t = (int)(item / (unsigned)bpt);
  if (t >= p.tokens) return;
  const int h0 = (int)(item % (unsigned)bpt) * kItemRows + sub;

  uint4 x[kFwdSteps];
  const size_t in0 = ((size_t)t * p.H + h0) * D + e0;
#pragma unroll
  for (int i = 0; i < kFwdSteps; ++i) {
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + i * R::kRows < p.H) x[i] = load_once(p.qkv, in0 + (size_t)i * R::kRows * D);
  }
  const int n = kPaged ? 0 : t % p.N, b = kPaged ? 0 : t / p.N;
  Angles<kInter> ang;
  ang.load(p, p.positions != nullptr ? __ldg(p.positions + t) : n, e0, lane);
  uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
  if (kNorm) {
    wq = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.wq) + e0));
    wk = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.wk) + e0));
  }
  int slot = -1;
  size_t kv0 = 0;            // first element of this token's row in KV head 0's pages
  if (kPaged) {
    const long long s = __ldg(p.slots + t);
    if (s >= 0 && s < p.num_slots) {
      slot = (int)s;
      const int page = slot / p.page_size;
      kv0 = ((size_t)page * p.Hkv * p.page_size + (size_t)(slot - page * p.page_size)) * D;
    }
  }

#pragma unroll
  for (int i = 0; i < kFwdSteps; ++i) {
    const int h = h0 + i * R::kRows;
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    uint4 out = x[i];
    if (h - sub < p.Hq + p.Hkv) {      // the warp's rows are not all V (warp-uniform)
      float z[8];
      unpack8(x[i], z);
      if (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(z[j], z[j], ss);
        const float r = rsqrtf(row_sum<R::kLanes>(ss) * (1.0f / D) + p.eps);
        float w[8];
        unpack8(is_q ? wq : wk, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] *= r * w[j];
      }
      ang.apply(z, 1.f);
      if (!is_v) out = pack8(z);
    }
    if (h >= p.H) continue;
    if (kPaged) {
      if (is_q) {
        store8(p.q, ((size_t)t * p.Hq + h) * D + e0, out);
      } else if (slot >= 0) {
        const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
        store8(is_v ? p.v : p.k, kv0 + (size_t)hk * p.page_size * D + e0, out);
      }
    } else {
      if (is_q) {
        store8(p.q, (((size_t)b * p.Hq + h) * p.N + n) * D + e0, out);
      } else {
        const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
        store8(is_v ? p.v : p.k, (((size_t)b * p.Hkv + hk) * p.N + n) * D + e0, out);
      }
    }
  }
}

// Backward.  The grid is persistent so that a warp keeps its share of the gains' gradients in
// registers over all its rows; a block adds its warps' shares in shared memory and leaves one
// partial, and a second kernel adds the partials in a fixed order (no atomics: the same
// inputs give the same bits).
template <int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kPrepThreads) attn_qk_prep_bwd_kernel(const PrepBwdParams pb) {
  using R = Row<D>;
  const PrepParams& p = pb.f;
  __shared__ float acc_s[kNorm ? kPrepWarps : 1][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / R::kLanes, e0 = (lane % R::kLanes) * 8;
  constexpr int kItemRows = kBwdSteps * R::kRows;
  const int bpt = (p.H + kItemRows - 1) / kItemRows;
  const unsigned items = (unsigned)p.tokens * (unsigned)bpt;
  uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
  if (kNorm) {
    wq = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.wq) + e0));
    wk = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.wk) + e0));
  }
  float aq[8], ak[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) aq[j] = ak[j] = 0.f;

  for (unsigned item = blockIdx.x * kPrepWarps + warp; item < items;
       item += gridDim.x * kPrepWarps) {
    const int t = (int)(item / (unsigned)bpt);
    const int h0 = (int)(item % (unsigned)bpt) * kItemRows + sub;
    const int n = t % p.N, b = t / p.N;
    uint4 x[kBwdSteps], dy[kBwdSteps];
    const size_t in0 = ((size_t)t * p.H + h0) * D + e0;
#pragma unroll
    for (int i = 0; i < kBwdSteps; ++i) {
      const int h = h0 + i * R::kRows;
      x[i] = dy[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < p.H) {
        if (kNorm && h < p.Hq + p.Hkv) x[i] = load_once(p.qkv, in0 + (size_t)i * R::kRows * D);
        if (h < p.Hq)
          dy[i] = load_once(p.q, (((size_t)b * p.Hq + h) * p.N + n) * D + e0);
        else if (h < p.Hq + p.Hkv)
          dy[i] = load_once(p.k, (((size_t)b * p.Hkv + h - p.Hq) * p.N + n) * D + e0);
        else
          dy[i] = load_once(p.v, (((size_t)b * p.Hkv + h - p.Hq - p.Hkv) * p.N + n) * D + e0);
      }
    }
    Angles<kInter> ang;
    ang.load(p, p.positions != nullptr ? __ldg(p.positions + t) : n, e0, lane);
#pragma unroll
    for (int i = 0; i < kBwdSteps; ++i) {
      const int h = h0 + i * R::kRows;
      uint4 out = dy[i];
      if (h - sub < p.Hq + p.Hkv) {
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        float dz[8];
        unpack8(dy[i], dz);
        ang.apply(dz, -1.f);
        if (kNorm) {
          float xv[8], w[8];
          unpack8(x[i], xv);
          unpack8(is_q ? wq : wk, w);
          float ss = 0.f, st = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            w[j] *= dz[j];
            ss = fmaf(xv[j], xv[j], ss);
            st = fmaf(xv[j], w[j], st);
          }
          const float r = rsqrtf(row_sum<R::kLanes>(ss) * (1.0f / D) + p.eps);
          const float m = row_sum<R::kLanes>(st) * (1.0f / D) * r * r;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float g = dz[j] * xv[j] * r;
            if (is_q) aq[j] += g;
            else if (!is_v) ak[j] += g;
            dz[j] = r * (w[j] - xv[j] * m);
          }
        }
        if (!is_v) out = pack8(dz);
      }
      if (h < p.H) store8(pb.dqkv, in0 + (size_t)i * R::kRows * D, out);
    }
  }

  if (kNorm) {
#pragma unroll
    for (int o = R::kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        aq[j] += __shfl_xor_sync(0xffffffffu, aq[j], o);
        ak[j] += __shfl_xor_sync(0xffffffffu, ak[j], o);
      }
    if (sub == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc_s[warp][0][e0 + j] = aq[j];
        acc_s[warp][1][e0 + j] = ak[j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kPrepThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kPrepWarps; ++w) s += acc_s[w][c / D][c % D];
      pb.partials[(size_t)blockIdx.x * 2 * D + c] = s;
    }
  }
}

// dw = sum of the blocks' partials: 32 columns a block, 32 threads a column, each adding
// every 32nd partial in order, then the 32 sums in order.
__global__ void __launch_bounds__(1024) attn_qk_prep_dw_kernel(const float* partials, int blocks,
                                                               int d, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float a = 0.f;
#pragma unroll 4
  for (int i = g; i < blocks; i += 32) a += partials[(size_t)i * 2 * d + col];
  s[g][c] = a;
  __syncthreads();
  if (g == 0) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][c];
    if (col < d) dwq[col] = v;
    else dwk[col - d] = v;
  }
}

template <int D, bool kNorm, bool kInter>
int launch_fwd_t(const PrepParams& p, bool paged, cudaStream_t stream) {
  constexpr int kItemRows = kFwdSteps * Row<D>::kRows;
  const long long items = (long long)p.tokens * ((p.H + kItemRows - 1) / kItemRows);
  const long long blocks = (items + kPrepWarps - 1) / kPrepWarps;   // items < 2^31 (host check)
  if (paged)
    attn_qk_prep_kernel<D, kNorm, kInter, true><<<(unsigned)blocks, kPrepThreads, 0, stream>>>(p);
  else
    attn_qk_prep_kernel<D, kNorm, kInter, false><<<(unsigned)blocks, kPrepThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int D, bool kNorm, bool kInter>
int launch_bwd_t(const PrepBwdParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kItemRows = kBwdSteps * Row<D>::kRows;
  const long long items = (long long)p.f.tokens * ((p.f.H + kItemRows - 1) / kItemRows);
  long long blocks = (items + kPrepWarps - 1) / kPrepWarps;
  if (blocks > 4LL * num_sms) blocks = 4LL * num_sms;
  if (blocks > kPrepBwdMaxBlocks) blocks = kPrepBwdMaxBlocks;
  attn_qk_prep_bwd_kernel<D, kNorm, kInter><<<(unsigned)blocks, kPrepThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -4;
  if (kNorm) {
    attn_qk_prep_dw_kernel<<<2 * D / 32, 1024, 0, stream>>>(p.partials, (int)blocks, D, p.dwq,
                                                            p.dwk);
    if (cudaGetLastError() != cudaSuccess) return -4;
  }
  return 0;
}

template <int D>
int launch_fwd_d(const PrepParams& p, bool paged, cudaStream_t s) {
  if (p.wq != nullptr)
    return p.interleaved ? launch_fwd_t<D, true, true>(p, paged, s)
                         : launch_fwd_t<D, true, false>(p, paged, s);
  return p.interleaved ? launch_fwd_t<D, false, true>(p, paged, s)
                       : launch_fwd_t<D, false, false>(p, paged, s);
}

template <int D>
int launch_bwd_d(const PrepBwdParams& p, int num_sms, cudaStream_t s) {
  if (p.f.wq != nullptr)
    return p.f.interleaved ? launch_bwd_t<D, true, true>(p, num_sms, s)
                           : launch_bwd_t<D, true, false>(p, num_sms, s);
  return p.f.interleaved ? launch_bwd_t<D, false, true>(p, num_sms, s)
                         : launch_bwd_t<D, false, false>(p, num_sms, s);
}

}  // namespace

int launch_qk_prep(const PrepParams& p, int d, bool paged, cudaStream_t stream) {
  if (p.tokens <= 0) return 0;
  return d == 128 ? launch_fwd_d<128>(p, paged, stream) : launch_fwd_d<64>(p, paged, stream);
}

int launch_qk_prep_bwd(const PrepBwdParams& p, int d, int num_sms, cudaStream_t stream) {
  return d == 128 ? launch_bwd_d<128>(p, num_sms, stream) : launch_bwd_d<64>(p, num_sms, stream);
}

}  // namespace attn
