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
// (interleaved) or a fixed number of lanes away.  A warp takes a chunk of a token's query
// heads or of its key and value heads: the angles and the gain are read and multiplied once,
//   y = r (x A + x_partner B),  A = w cos,  B = +-w_partner sin,
// and stay in registers for all rows of the chunk.  The rows come through shared memory, into
// places that every lane fills and reads for itself (cp.async, no barrier): what is in flight
// then costs no registers, and one row at a time is computed.  Sums, statistics and the
// rotation are in fp32; each output is rounded once.  Measured: forward, [8, 4096] tokens of 32 +
// 2 x 32 heads of 128, 240 us (6.7 TB/s, the copy rate); backward, [4, 4096] of 32 + 2 x 8, 101 us
// (5.7 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_serve.h"
#include "sm100_ptx.cuh"

namespace attn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
// Steps of a chunk at most, all in flight at once (a step is a row a lane: 2 or 4 rows a
// warp).  Measured on a B200: [8, 4096] tokens of 32 + 2 x 32 heads of 128, forward: 8 steps
// 240 us, 4 steps 267; [4, 4096] of 32 + 2 x 8, backward: 8 steps 101 us, 4 steps 111.
constexpr int kChunkSteps = 8;
// Blocks an SM: the forward at 64 registers a thread, the backward at 128 (with 80 it spills,
// 128 us instead of 101).
constexpr int kFwdBlocks = 4;
constexpr int kBwdBlocks = 2;

template <int D>
struct Row {
  static constexpr int kLanes = D / 8;           // lanes a row
  static constexpr int kRows = 32 / kLanes;      // rows a warp holds at a time
};

// Two values of a packed bf16 pair.
__device__ __forceinline__ void unpack2(uint32_t u, float& lo, float& hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  unpack2(u.x, x[0], x[1]);
  unpack2(u.y, x[2], x[3]);
  unpack2(u.z, x[4], x[5]);
  unpack2(u.w, x[6], x[7]);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 16 bytes to this lane's place in shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 read16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}

__device__ __forceinline__ uint4 load_gain(const void* w, int e0) {
  return __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(w) + e0));
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

// What this lane's values meet in the rotation: the lane of their partners, and the
// coefficients of y[i] = z[i] c[i] + z_partner[i] s[i].  A position outside the table reads a
// row of zeros, as a page outside the cache does.
template <bool kInter>
struct Angles {
  float c[8], s[8];
  bool rotates;
  int partner;

  __device__ __forceinline__ void place(const PrepParams& p, int e0, int lane) {
    const int half = p.rot >> 1;
    rotates = e0 < p.rot;
    partner = lane;
    if (!kInter && rotates) partner = e0 < half ? lane + (half >> 3) : lane - (half >> 3);
  }

  // back: the coefficients of the inverse rotation (its transpose has the sines' signs turned)
  template <bool kBack>
  __device__ __forceinline__ void load(const PrepParams& p, int pos, int e0) {
    const int half = p.rot >> 1;
    const bool valid = rotates && (unsigned)pos < (unsigned)p.table_rows;
    const float* row = p.table + (valid ? (size_t)pos * p.rot : 0);
    const float other = rotates ? 0.f : 1.f;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kInter) {
      float4 a = make_float4(other, other, other, other), b = zero;
      if (valid) {
        a = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
        b = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
      }
      c[0] = c[1] = a.x; c[2] = c[3] = a.y; c[4] = c[5] = a.z; c[6] = c[7] = a.w;
      const float ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[2 * i] = kBack ? ss[i] : -ss[i];
        s[2 * i + 1] = kBack ? -ss[i] : ss[i];
      }
    } else {
      const bool low = e0 < half;
      const int j = low ? e0 : e0 - half;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        float4 a = make_float4(other, other, other, other), b = zero;
        if (valid) {
          a = __ldg(reinterpret_cast<const float4*>(row + j + i));
          b = __ldg(reinterpret_cast<const float4*>(row + half + j + i));
        }
        c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
        const bool neg = low != kBack;
        s[i] = neg ? -b.x : b.x;
        s[i + 1] = neg ? -b.y : b.y;
        s[i + 2] = neg ? -b.z : b.z;
        s[i + 3] = neg ? -b.w : b.w;
      }
    }
  }

  // The partners of this lane's packed values, as floats, 0 where nothing rotates (what lies
  // there may be infinite, and a coefficient of 0 would make it NaN); every lane of the warp
  // calls it.  The mask costs nothing: it is part of the unpacking.
  __device__ __forceinline__ void partners(const uint4& x, float (&y)[8]) const {
    const uint32_t low = rotates ? 0x10000u : 0u, high = rotates ? 0xffff0000u : 0u;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kInter) {
        y[2 * i] = __uint_as_float(w[i] & high);
        y[2 * i + 1] = __uint_as_float(w[i] * low);
      } else {
        w[i] = __shfl_sync(0xffffffffu, w[i], partner);
        y[2 * i] = __uint_as_float(w[i] * low);
        y[2 * i + 1] = __uint_as_float(w[i] & high);
      }
    }
  }
};

// 1 / sqrt of a mean square plus eps (a normal number: the host refuses a smaller eps).
__device__ __forceinline__ float inv_sqrt(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Chunks of a token, `steps` times the rows of a warp each: of its query heads, and of its key
// and value heads, which follow each other (with few of them one chunk has both: 281 -> 261 us
// at 65536 tokens of 32 + 2 x 8 heads into a paged cache).
struct Chunks {
  int rows, q, kv;

  __host__ __device__ Chunks(int Hq, int Hkv, int warp_rows, int steps)
      : rows(warp_rows * steps), q((Hq + rows - 1) / rows), kv((2 * Hkv + rows - 1) / rows) {}
  __host__ __device__ int all() const { return q + kv; }
};

enum { kQuery = 0, kKey = 1, kValue = 2 };

template <int D, bool kNorm, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kPrepThreads, kFwdBlocks)
attn_qk_prep_kernel(const PrepParams p, int steps, int ahead) {
  using R = Row<D>;
  __shared__ __align__(16) uint4 rows[kChunkSteps][kPrepThreads];
  const int lane = threadIdx.x & 31;
  const int sub = lane / R::kLanes, e0 = (lane % R::kLanes) * 8;
  const Chunks ch(p.Hq, p.Hkv, R::kRows, steps);
  const unsigned item = blockIdx.x * kPrepWarps + (threadIdx.x >> 5);
  const int t = (int)(item / (unsigned)ch.all());
  if (t >= p.tokens) return;
  const int c = (int)(item - (unsigned)t * ch.all());
  const bool is_q = c < ch.q;
  // rows [h0, h1) of the query heads, or of the key heads and the value heads behind them
  const int h0 = (is_q ? c : c - ch.q) * ch.rows;
  const int h1 = min(h0 + ch.rows, is_q ? p.Hq : 2 * p.Hkv);
  const uint32_t mine = smem_u32(&rows[0][threadIdx.x]);
  constexpr uint32_t kSlot = kPrepThreads * 16;
  // the first of two loads, one after the other, on the way to the angles
  const int pos = kPaged || p.positions != nullptr ? __ldg(p.positions + t) : t % p.N;
  // the position of a token that warps launched a wave later will take
  int later = -1;
  if (c == 0 && (kPaged || p.positions != nullptr) && t + ahead < p.tokens)
    later = __ldg(p.positions + t + ahead);

  {
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.qkv) +
                               ((size_t)t * p.H + (is_q ? 0 : p.Hq)) * D + e0;
    if (h1 - h0 == kChunkSteps * R::kRows) {      // a full chunk, as most are
      const __nv_bfloat16* from = src + (h0 + sub) * D;
#pragma unroll
      for (int i = 0; i < kChunkSteps; ++i) {
        copy16(mine + i * kSlot, from + i * R::kRows * D);
        if (i == kChunkSteps / 2 - 1) copy_commit();
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunkSteps; ++i) {
        const int h = h0 + i * R::kRows + sub;
        if (i < steps) copy16(mine + i * kSlot, src + min(h, h1 - 1) * D, h < h1);
        if (i == kChunkSteps / 2 - 1) copy_commit();
      }
    }
    copy_commit();
  }

  // this lane's part of the token's row of head 0 (of the query, or the key and value heads),
  // and what a head adds
  size_t dst, head;
  bool keep = true;
  if (kPaged) {
    if (is_q) {
      dst = (size_t)t * p.Hq * D;
      head = D;
    } else {
      const long long s = __ldg(p.slots + t);
      keep = s >= 0 && s < p.num_slots;
      const int place = keep ? (int)s : 0;
      const int page = place / p.page_size;
      dst = ((size_t)page * p.Hkv * p.page_size + (size_t)(place - page * p.page_size)) * D;
      head = (size_t)p.page_size * D;
    }
  } else {
    const int b = t / p.N, n = t - b * p.N;
    dst = ((size_t)b * (is_q ? p.Hq : p.Hkv) * p.N + n) * D;
    head = (size_t)p.N * D;
  }
  dst += e0;
  __nv_bfloat16* const v_out = reinterpret_cast<__nv_bfloat16*>(p.v) + dst;
  const int first_v = is_q ? h1 : p.Hkv;      // rows from here on are values
  int h = h0 + sub;
  __nv_bfloat16* out = h < first_v || is_q
                           ? reinterpret_cast<__nv_bfloat16*>(is_q ? p.q : p.k) + dst + h * head
                           : v_out + (h - first_v) * head;
  const int n_steps = (h1 - h0 - 1) / R::kRows + 1;

  Angles<kInter> ang;
  if (h0 < first_v) {
    ang.place(p, e0, lane);
    ang.template load<false>(p, pos, e0);
    if (kNorm) {      // A = w c, B = w_partner s
      const uint4 w = load_gain(is_q ? p.wq : p.wk, e0);
      float g[8];
      unpack8(w, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) ang.c[j] *= g[j];
      ang.partners(w, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) ang.s[j] *= g[j];
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    half == 0 ? copy_wait<1>() : copy_wait<0>();
    const int end = half == 0 ? min(n_steps, kChunkSteps / 2) : n_steps;
#pragma unroll 1
    for (int i = half * (kChunkSteps / 2); i < end; ++i) {
      uint4 x = read16(mine + i * kSlot);
      if (h - sub < first_v) {      // not all of the warp's rows are values
        float v[8], vp[8];
        unpack8(x, v);
        ang.partners(x, vp);
        float r = 1.f;
        if (kNorm) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int j = 0; j < 8; j += 2) ffma2(s0, s1, v[j], v[j + 1], v[j], v[j + 1], s0, s1);
          r = inv_sqrt(row_sum<R::kLanes>(s0 + s1) * (1.0f / D) + p.eps);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          fmul2(v[j], v[j + 1], v[j], v[j + 1], ang.c[j], ang.c[j + 1]);
          ffma2(v[j], v[j + 1], vp[j], vp[j + 1], ang.s[j], ang.s[j + 1], v[j], v[j + 1]);
          if (kNorm) fmul2(v[j], v[j + 1], v[j], v[j + 1], r, r);
        }
        if (h < first_v) x = pack8(v);
      }
      if (h < h1 && keep) store8(out, 0, x);
      out += R::kRows * head;
      h += R::kRows;
      if (h >= first_v && h - R::kRows < first_v) out = v_out + (h - first_v) * head;
    }
  }
  // its angles on their way to L2 meanwhile: rows of a large table come from memory, and a
  // warp's start would wait for the position and then for them
  if ((unsigned)later < (unsigned)p.table_rows && lane * 32 < p.rot)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + (size_t)later * p.rot + lane * 32));
}

// Backward.  A block takes a run of tokens and goes through their query chunks, then their key
// chunks, then their value chunks, each kind spread evenly over its warps.  A warp so keeps
// its share of one gain's gradient in registers over all its rows of that kind; the block
// adds its warps' shares in shared memory and leaves one partial, and a second kernel adds the
// partials in a fixed order (no atomics: the same inputs give the same bits).  While a step
// is computed, the same step of the warp's next chunk is on its way.
template <int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kPrepThreads, kBwdBlocks)
attn_qk_prep_bwd_kernel(const PrepBwdParams pb, int steps) {
  using R = Row<D>;
  const PrepParams& p = pb.f;
  extern __shared__ __align__(16) uint4 bwd_rows[];      // [steps][x, dy][kPrepThreads]
  __shared__ float acc_s[kNorm ? kPrepWarps : 1][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / R::kLanes, e0 = (lane % R::kLanes) * 8;
  const uint32_t mine = smem_u32(bwd_rows + threadIdx.x);
  constexpr uint32_t kHalf = kPrepThreads * 16, kSlot = 2 * kHalf;
  const int t_begin = (int)((long long)blockIdx.x * p.tokens / gridDim.x);
  const int t_end = (int)(((long long)blockIdx.x + 1) * p.tokens / gridDim.x);

  Angles<kInter> ang;
  ang.place(p, e0, lane);

#pragma unroll 1
  for (int kind = kQuery; kind <= kValue; ++kind) {
    const int heads = kind == kQuery ? p.Hq : p.Hkv;
    const int head0 = kind == kQuery ? 0 : kind == kKey ? p.Hq : p.Hq + p.Hkv;
    const int n_steps = min(steps, (heads + R::kRows - 1) / R::kRows);
    const int chunk = n_steps * R::kRows;
    const int chunks = heads > 0 ? (heads + chunk - 1) / chunk : 0;
    const int items = (t_end - t_begin) * chunks;
    const bool x_too = kNorm && kind != kValue;
    const __nv_bfloat16* dy_of = reinterpret_cast<const __nv_bfloat16*>(kind == kQuery ? p.q
                                                                        : kind == kKey ? p.k : p.v);
    float w[8], acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = acc[j] = 0.f;
    if (x_too) unpack8(load_gain(kind == kQuery ? p.wq : p.wk, e0), w);

    // An item's token, and this lane's first row of it: offsets in the input and the gradient,
    // and how many of its steps have a row for this lane.
    int t, n_rows, pos;
    size_t in, dy_in;
    auto aim = [&](int item) {
      t = item / chunks;
      const int h = (item - t * chunks) * chunk + sub;
      t += t_begin;
      const int b = t / p.N;
      in = ((size_t)t * p.H + head0 + h) * D + e0;
      dy_in = (((size_t)b * heads + h) * p.N + (t - b * p.N)) * D + e0;
      n_rows = h < heads ? min((heads - h - 1) / R::kRows + 1, n_steps) : 0;
      // (read an item ahead: the angles wait for it)
      pos = p.positions != nullptr ? __ldg(p.positions + t) : t - b * p.N;
    };
    const __nv_bfloat16 *cx = nullptr, *cdy = nullptr;
    const __nv_bfloat16* any = reinterpret_cast<const __nv_bfloat16*>(p.qkv);   // for no row
    const size_t dy_step = (size_t)p.N * D * R::kRows;
    auto copy_step = [&](int i) {
      const bool valid = i < n_rows;
      copy16(mine + i * kSlot + kHalf, valid ? cdy : any, valid);
      if (x_too) copy16(mine + i * kSlot, valid ? cx : any, valid);
      cdy += dy_step;
      cx += R::kRows * D;
    };
    auto start = [&](int item) {
      aim(item);
      cx = any + in;
      cdy = dy_of + dy_in;
    };
    int item = warp;
    if (item < items) {
      start(item);
      for (int i = 0; i < n_steps; ++i) {
        copy_step(i);
        copy_commit();
      }
    }
    for (; item < items; item += kPrepWarps) {
      if (kind != kValue) ang.template load<true>(p, pos, e0);
      __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(pb.dqkv) + in;
      const int rows = n_rows;
      const bool more = item + kPrepWarps < items;
      if (more) start(item + kPrepWarps);
      for (int i = 0; i < n_steps; ++i) {
        // Copies in flight: this item's steps i .. n - 1 and, of the next, 0 .. i - 2 (a place
        // is filled again one step after it was read).
        if (n_steps >= 8) copy_wait<7>();
        else if (n_steps >= 4) copy_wait<3>();
        else if (n_steps >= 2) copy_wait<1>();
        else copy_wait<0>();
        const uint4 x = x_too ? read16(mine + i * kSlot) : make_uint4(0u, 0u, 0u, 0u);
        uint4 dy = read16(mine + i * kSlot + kHalf);
        if (more && i > 0) copy_step(i - 1);
        copy_commit();
        if (kind != kValue) {
          float dz[8], dp[8];
          unpack8(dy, dz);
          ang.partners(dy, dp);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            fmul2(dz[j], dz[j + 1], dz[j], dz[j + 1], ang.c[j], ang.c[j + 1]);
            ffma2(dz[j], dz[j + 1], dp[j], dp[j + 1], ang.s[j], ang.s[j + 1], dz[j], dz[j + 1]);
          }
          if (kNorm) {
            float xv[8], wd[8];
            unpack8(x, xv);
            float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              fmul2(wd[j], wd[j + 1], w[j], w[j + 1], dz[j], dz[j + 1]);
              ffma2(s0, s1, xv[j], xv[j + 1], xv[j], xv[j + 1], s0, s1);
              ffma2(t0, t1, xv[j], xv[j + 1], wd[j], wd[j + 1], t0, t1);
            }
            const float r = inv_sqrt(row_sum<R::kLanes>(s0 + s1) * (1.0f / D) + p.eps);
            const float m = row_sum<R::kLanes>(t0 + t1) * (-1.0f / D) * r * r;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              ffma2(wd[j], wd[j + 1], xv[j], xv[j + 1], m, m, wd[j], wd[j + 1]);
              fmul2(xv[j], xv[j + 1], xv[j], xv[j + 1], r, r);
              ffma2(acc[j], acc[j + 1], dz[j], dz[j + 1], xv[j], xv[j + 1], acc[j], acc[j + 1]);
              fmul2(dz[j], dz[j + 1], wd[j], wd[j + 1], r, r);
            }
          }
          dy = pack8(dz);
        }
        if (i < rows) store8(to, 0, dy);
        to += R::kRows * D;
      }
      if (more) copy_step(n_steps - 1);
      copy_commit();
    }
    copy_wait<0>();

    if (x_too) {
#pragma unroll
      for (int o = R::kLanes; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (sub == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_s[warp][kind][e0 + j] = acc[j];
      }
    }
  }
  if (kNorm) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kPrepThreads) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kPrepWarps; ++v) s += acc_s[v][c / D][c % D];
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

// Steps of a chunk: many for a large call, so that the angles are read and multiplied seldom,
// fewer while that leaves SMs with fewer than 16 warps.  With 4, 8, 16, 32 and 64 warps an SM for
// the 16 (us):
//   200 tokens of 32 + 2 x 8 heads of 128, paged     4.0   4.0   3.8   4.7   4.9
//   800 tokens                                       5.6   5.8   5.7   6.5   8.0
//   backward, 250 tokens                            11.0   9.9   9.2   9.7   9.4
//   backward, 1000 tokens                           14.2  14.1  14.1  14.6  15.8
//   500 tokens of 32 + 2 x 32 heads                  5.9   5.9   6.0   7.2   9.5
int chunk_steps(long long tokens, int Hq, int Hkv, int warp_rows, int num_sms) {
  int steps = kChunkSteps;
  while (steps > 1 &&
         tokens * Chunks(Hq, Hkv, warp_rows, steps).all() < (long long)num_sms * 16)
    steps /= 2;
  return steps;
}

template <int D, bool kNorm, bool kInter>
int launch_fwd_t(const PrepParams& p, bool paged, int num_sms, cudaStream_t stream) {
  const int steps = chunk_steps(p.tokens, p.Hq, p.Hkv, Row<D>::kRows, num_sms);
  const long long items = (long long)p.tokens * Chunks(p.Hq, p.Hkv, Row<D>::kRows, steps).all();
  const unsigned blocks = (unsigned)((items + kPrepWarps - 1) / kPrepWarps);   // items < 2^31
  const int ahead = kFwdBlocks * num_sms * kPrepWarps /
                    Chunks(p.Hq, p.Hkv, Row<D>::kRows, steps).all();
  if (paged)
    attn_qk_prep_kernel<D, kNorm, kInter, true>
        <<<blocks, kPrepThreads, 0, stream>>>(p, steps, ahead);
  else
    attn_qk_prep_kernel<D, kNorm, kInter, false>
        <<<blocks, kPrepThreads, 0, stream>>>(p, steps, ahead);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int D, bool kNorm, bool kInter>
int launch_bwd_t(const PrepBwdParams& p, int num_sms, cudaStream_t stream) {
  const int steps = chunk_steps(p.f.tokens, p.f.Hq, p.f.Hkv, Row<D>::kRows, num_sms);
  const long long blocks = std::min<long long>(
      p.f.tokens, std::min<long long>((long long)kBwdBlocks * num_sms, kPrepBwdMaxBlocks));
  const int smem = steps * 2 * kPrepThreads * 16;
  auto kernel = attn_qk_prep_bwd_kernel<D, kNorm, kInter>;
  static std::atomic<bool> ready[64];
  if (!allow_smem(reinterpret_cast<const void*>(kernel), kChunkSteps * 2 * kPrepThreads * 16,
                  ready))
    return -4;
  kernel<<<(unsigned)blocks, kPrepThreads, smem, stream>>>(p, steps);
  if (cudaGetLastError() != cudaSuccess) return -4;
  if (kNorm) {
    attn_qk_prep_dw_kernel<<<2 * D / 32, 1024, 0, stream>>>(p.partials, (int)blocks, D, p.dwq,
                                                            p.dwk);
    if (cudaGetLastError() != cudaSuccess) return -4;
  }
  return 0;
}

template <int D>
int launch_fwd_d(const PrepParams& p, bool paged, int num_sms, cudaStream_t s) {
  if (p.wq != nullptr)
    return p.interleaved ? launch_fwd_t<D, true, true>(p, paged, num_sms, s)
                         : launch_fwd_t<D, true, false>(p, paged, num_sms, s);
  return p.interleaved ? launch_fwd_t<D, false, true>(p, paged, num_sms, s)
                       : launch_fwd_t<D, false, false>(p, paged, num_sms, s);
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

int launch_qk_prep(const PrepParams& p, int d, bool paged, int num_sms, cudaStream_t stream) {
  if (p.tokens <= 0) return 0;
  return d == 128 ? launch_fwd_d<128>(p, paged, num_sms, stream)
                  : launch_fwd_d<64>(p, paged, num_sms, stream);
}

int launch_qk_prep_bwd(const PrepBwdParams& p, int d, int num_sms, cudaStream_t stream) {
  return d == 128 ? launch_bwd_d<128>(p, num_sms, stream) : launch_bwd_d<64>(p, num_sms, stream);
}

}  // namespace attn
