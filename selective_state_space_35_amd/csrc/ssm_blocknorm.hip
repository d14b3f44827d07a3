// ssm_blocknorm.hip -- what stands between two blocks: the RMS norm after one, its gate, the scale of each channel, the
// residual, and the RMS norm before the next, forward and backward, with the sums of the parameters' gradients.
//
// A row is one [W] slice of x [rows, H, W]; the parameters are [H, W] (H = 1: over the model's width; H > 1: each head's
// channels).  Every step can be left out.
//   p = x r1 w1,  r1 = 1 / sqrt(mean(x^2) + eps);  u = p silu(z);  h = residual + s u;  n = h r2 w2,  r2 as r1 of h
// Backward, with xh = x r1 and hh = h r2 (h is computed again, in float):
//   t = dn w2,  e = dh + r2 (t - hh mean(t hh))  (the gradient of h, and of the residual)
//   c = e s,  dz = c p silu'(z),  d = c silu(z) w1,  dx = r1 (d - xh mean(d xh))
//   dw1 = sum over rows of c silu(z) xh,  ds = sum of e u,  dw2 = sum of dn hh
// Both directions read every streamed value once, hold it for the two sums of its row, one after the other, and write
// once: bound by HBM (65536 rows of 2560 in bf16 with the residual: both norms, forward 254 us, 5.3 TB/s, backward with the
// parameters' sums 430 us, 4.7 TB/s; the norm before the next block alone 254 and 395 us).  A group of threads keeps one
// head's parameters, and in the backward its part of their gradients, in registers and walks rows, the next row's loads under
// way while one is summed (the parameters read again for every row, 16 registers a thread fewer: 742 us; rows of 640 threads
// and more do); the gate is a form of its own (with its values in registers that nobody used 510 us).  What does not fit in
// the registers goes through scratch: in the backward, rows of more than 512 threads that are gated or not whole pieces (6 to
// 514 registers) and nearly all of two or four vectors a thread (13 to 1321 registers; 2^27 bf16 elements in rows of 8192,
// one vector, 376 us, of 8200, two, 1515 us); in the forward, those of two or four vectors that are gated or not whole pieces
// (up to 280).  All sums are float.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ssm_blocknorm.h"
#include "ssm_device.h"
#include "ssm_kinds.h"

namespace ssm {
namespace {

// N consecutive elements of a row as they come from memory, 16 bytes at once from any address (unaligned access is on for
// global memory).  TAIL: the width is not whole pieces, and `left` elements from here on are inside the row.  A row's last
// piece of 8 is then read so that it ends with the row, and shifted into place, zeros behind it, when it is used.  65536 rows
// of 2561 in bf16, backward, 624 us; shifted when it is loaded, that is, waited for, 1089; 40000 gated rows of 4095 789 us
// and 1214, element by element 1210.  Pieces of 4 and rows shorter than a piece go element by element (65536 float rows of
// 1001, backward, 305 us; shifted 515).
__host__ __device__ constexpr bool shifted(int n, int W) { return n == 8 && W >= n; }
template <typename T, int N>
struct Raw {
  uint32_t w[N * int(sizeof(T)) / 4];
};
template <bool TAIL, typename T, int N>
__device__ __forceinline__ void load_raw(Raw<T, N>& r, const T* p, int left, int W) {
  constexpr int kPer = 16 / int(sizeof(T)), kPieces = N / kPer;
  if constexpr (!TAIL) {
    __builtin_memcpy(r.w, p, N * sizeof(T));
  } else if (shifted(N, W)) {
#pragma unroll
    for (int k = 0; k < kPieces; k++) {
      const int over = max((k + 1) * kPer - left, 0);
      __builtin_memcpy(r.w + 4 * k, p + k * kPer - over, 16);
    }
  } else if (left >= N) {
    __builtin_memcpy(r.w, p, N * sizeof(T));
  } else {
#pragma unroll
    for (int k = 0; k < N * int(sizeof(T)) / 4; k++) r.w[k] = 0;
#pragma unroll
    for (int j = 0; j < N - 1; j++) {
      if (j < left) {
        if constexpr (sizeof(T) == 4) r.w[j] = __float_as_uint(p[j]);
        else r.w[j / 2] |= uint32_t(p[j]) << (16 * (j % 2));
      }
    }
  }
}
template <bool TAIL, typename T, int N>
__device__ __forceinline__ void floats(Raw<T, N> r, float (&v)[N], int left, int W) {
  if constexpr (TAIL && N == 8) {
    constexpr int kPer = 16 / int(sizeof(T)), kPieces = N / kPer;
#pragma unroll
    for (int k = 0; k < kPieces; k++) {
      const int bits = !shifted(N, W) ? 0 : min(max((k + 1) * kPer - left, 0), kPer) * 8 * int(sizeof(T));
      unsigned __int128 x;
      __builtin_memcpy(&x, r.w + 4 * k, 16);
      x = kPieces == 1 ? x >> bits : x >> (bits / 2) >> (bits / 2);  // a piece behind the row shifts by all 128
      __builtin_memcpy(r.w + 4 * k, &x, 16);
    }
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < N; j++) v[j] = __uint_as_float(r.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N / 2; j++) {
      v[2 * j] = __uint_as_float(r.w[j] << 16);
      v[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
  }
}
template <bool TAIL, typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&v)[N], int left) {
  if (!TAIL || left >= N) {
    uint32_t w[N * int(sizeof(T)) / 4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < N; j++) w[j] = __float_as_uint(v[j]);
    } else {
      typedef __attribute__((ext_vector_type(2))) float f2;
      typedef __attribute__((ext_vector_type(2))) __bf16 b2;
#pragma unroll
      for (int j = 0; j < N / 2; j++) w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), b2));
    }
    __builtin_memcpy(p, w, N * sizeof(T));
  } else {
#pragma unroll
    for (int j = 0; j < N - 1; j++)
      if (j < left) store_elem(p + j, v[j]);
  }
}

// The sum over the TPR threads of a row, the same in every one of them: shuffles, and for wider rows LDS with one barrier
// a call (the whole workgroup comes to it).  That is enough only if no two calls in a row have the same buffer, over the rows
// too: a wave may be at the next call's write while another still reads this one's sums.  Callers alternate two of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float* buf) {
#pragma unroll
  for (int off = (TPR < kWave ? TPR : kWave) / 2; off > 0; off >>= 1) s += __shfl_xor(s, off);
  if constexpr (TPR > kWave) {
    constexpr int kWaves = TPR / kWave;
    if (threadIdx.x % kWave == 0) buf[threadIdx.x / kWave % kWaves] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) s += buf[w];
  }
  return s;
}

constexpr int block_threads(int tpr) { return tpr > 128 ? tpr : 256; }

// A parameter of a group's head, one where there is none: in registers, or for the rows of many threads, whose registers
// are few, read again for every row (from the caches).
template <bool TAIL, int NV, int VEC, int TPR>
struct Par {
  static constexpr bool kHeld = TPR < 640;
  const float* w;
  int lane, W;
  float v[kHeld ? NV : 1][VEC];
  __device__ __forceinline__ void init(const float* weight, int64_t at, int lane_, int W_) {
    w = weight ? weight + at : nullptr;
    lane = lane_;
    W = W_;
    if constexpr (kHeld)
#pragma unroll
      for (int j = 0; j < NV; j++) load(j, v[j]);
  }
  __device__ __forceinline__ void load(int j, float (&o)[VEC]) const {
#pragma unroll
    for (int e = 0; e < VEC; e++) o[e] = 1.f;
    const int c = (j * TPR + lane) * VEC;
    if (!w || c >= W) return;
    if (!TAIL || c + VEC <= W) {
      __builtin_memcpy(o, w + c, VEC * 4);
    } else {
#pragma unroll
      for (int e = 0; e < VEC - 1; e++)
        if (c + e < W) o[e] = w[c + e];
    }
  }
  __device__ __forceinline__ void get(int j, float (&o)[VEC]) const {
    if constexpr (kHeld) {
#pragma unroll
      for (int e = 0; e < VEC; e++) o[e] = v[j][e];
    } else {
      load(j, o);
    }
  }
};

// One group of TPR threads walks the rows slice, slice + n_slices, ... of head h; each thread has NV vectors of VEC
// elements of a row, at columns (j TPR + lane) VEC.  TAIL: the width is not whole vectors.  R: the residual stream's type.
template <typename T, typename R, bool GATE, bool TAIL, int VEC, int NV, int TPR>
__global__ __launch_bounds__(block_threads(TPR)) void bn_fwd_kernel(BlockNormArgs a, int64_t n_slices) {
  constexpr int kGroups = block_threads(TPR) / TPR;
  __shared__ float buf[2][kGroups][TPR > kWave ? TPR / kWave : 1];
  const int W = int(a.W), H = int(a.H);
  const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int64_t gid = int64_t(blockIdx.x) * kGroups + group;
  const bool live = gid < n_slices * H;  // the others keep the workgroup's barriers
  const int h = live ? int(gid % H) : 0;
  const int64_t slice = live ? gid / H : a.rows;
  const T* x = static_cast<const T*>(a.x);
  const T* z = static_cast<const T*>(a.z);
  const R* res = static_cast<const R*>(a.residual);
  Par<TAIL, NV, VEC, TPR> p1, ps, p2;
  p1.init(a.post ? a.post_weight : nullptr, int64_t(h) * W, lane, W);
  ps.init(a.scale, int64_t(h) * W, lane, W);
  p2.init(a.pre ? a.pre_weight : nullptr, int64_t(h) * W, lane, W);
  Raw<T, VEC> xn[NV], zn[GATE ? NV : 1];
  Raw<R, VEC> rn[NV];
  auto fetch = [&](int64_t i) {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int c = (j * TPR + lane) * VEC;
      const int64_t at = (i * H + h) * W + c;
      if (c < W) {
        load_raw<TAIL>(xn[j], x + at, W - c, W);
        if constexpr (GATE) load_raw<TAIL>(zn[j], z + at, W - c, W);
        if (res) load_raw<TAIL>(rn[j], res + at, W - c, W);
      }
    }
  };
  if (slice < a.rows) fetch(slice);
  const float inv_w = 1.f / float(W);
  const int64_t first = int64_t(blockIdx.x) * kGroups / H;  // the workgroup's first slice: it has the most rows
  int phase = 0;  // the buffer of the next row_sum, whichever norms there are
  for (int64_t k = first; k < a.rows; k += n_slices) {
    const int64_t i0 = slice + (k - first);
    const bool on = live && i0 < a.rows;
    float v[NV][VEC], g[NV][VEC], r[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const bool in = on && (j * TPR + lane) * VEC < W;
#pragma unroll
      for (int e = 0; e < VEC; e++) v[j][e] = g[j][e] = r[j][e] = 0.f;
      if (in) {
        floats<TAIL>(xn[j], v[j], W - (j * TPR + lane) * VEC, W);
        if constexpr (GATE) floats<TAIL>(zn[j], g[j], W - (j * TPR + lane) * VEC, W);
        if (res) floats<TAIL>(rn[j], r[j], W - (j * TPR + lane) * VEC, W);
      }
    }
    if (live && i0 + n_slices < a.rows) fetch(i0 + n_slices);
    float r1 = 1.f, r2 = 1.f;
    if (a.post) {
#pragma unroll
      for (int j = 0; j < NV; j++)
#pragma unroll
        for (int e = 0; e < VEC; e++) s = fmaf(v[j][e], v[j][e], s);
      s = row_sum<TPR>(s, buf[phase][group]);
      phase ^= 1;
      r1 = 1.f / sqrtf(fmaf(s, inv_w, a.eps));
    }
    s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float w1[VEC], sc[VEC];
      p1.get(j, w1);
      ps.get(j, sc);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        float u = v[j][e] * r1 * w1[e];
        if constexpr (GATE) u *= g[j][e] / (1.f + expf(-g[j][e]));
        v[j][e] = fmaf(u, sc[e], r[j][e]);
        s = fmaf(v[j][e], v[j][e], s);  // columns behind the width are zero: so is silu(0)
      }
    }
    const int64_t row = i0 * H + h;
    if (a.h && on) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int c = (j * TPR + lane) * VEC;
        if (c < W) store<TAIL>(static_cast<R*>(a.h) + row * W + c, v[j], W - c);
      }
    }
    if (a.pre) {
      s = row_sum<TPR>(s, buf[phase][group]);
      phase ^= 1;
      r2 = 1.f / sqrtf(fmaf(s, inv_w, a.eps));
      if (on) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
          const int c = (j * TPR + lane) * VEC;
          if (c < W) {
            float o[VEC], w2[VEC];
            p2.get(j, w2);
#pragma unroll
            for (int e = 0; e < VEC; e++) o[e] = v[j][e] * r2 * w2[e];
            store<TAIL>(static_cast<T*>(a.n) + row * W + c, o, W - c);
          }
        }
      }
    }
    if (on && lane == 0) {
      if (a.post && a.rstd_post) a.rstd_post[row] = r1;
      if (a.pre && a.rstd_pre) a.rstd_pre[row] = r2;
    }
  }
}

// As the forward; a group writes its own row of the partial sums [3][n_slices][H W] (of w1, the scale, w2), which
// bn_reduce_kernel adds in a fixed order.
template <typename T, typename R, bool GATE, bool TAIL, int VEC, int NV, int TPR>
__global__ __launch_bounds__(block_threads(TPR)) void bn_bwd_kernel(BlockNormArgs a, int64_t n_slices, float* part) {
  constexpr int kGroups = block_threads(TPR) / TPR;
  __shared__ float buf[2][kGroups][TPR > kWave ? TPR / kWave : 1];
  const int W = int(a.W), H = int(a.H);
  const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int64_t gid = int64_t(blockIdx.x) * kGroups + group;
  const bool live = gid < n_slices * H;
  const int h = live ? int(gid % H) : 0;
  const int64_t slice = live ? gid / H : a.rows;
  const T* x = static_cast<const T*>(a.x);
  const T* z = static_cast<const T*>(a.z);
  const T* dn = a.pre ? static_cast<const T*>(a.dn) : nullptr;
  // h is needed for the norm before the next block only
  const R* res = a.pre ? static_cast<const R*>(a.residual) : nullptr;
  const R* dh = static_cast<const R*>(a.dh);
  Par<TAIL, NV, VEC, TPR> p1, ps, p2;
  p1.init(a.post ? a.post_weight : nullptr, int64_t(h) * W, lane, W);
  ps.init(a.scale, int64_t(h) * W, lane, W);
  p2.init(a.pre ? a.pre_weight : nullptr, int64_t(h) * W, lane, W);
  float dw1[NV][VEC], ds[NV][VEC], dw2[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; j++)
#pragma unroll
    for (int e = 0; e < VEC; e++) dw1[j][e] = ds[j][e] = dw2[j][e] = 0.f;
  Raw<T, VEC> xn[NV], zn[GATE ? NV : 1], nn[NV];
  Raw<R, VEC> rn[NV], hn[NV];
  float r1n = 1.f, r2n = 1.f;
  auto fetch = [&](int64_t i) {
    const int64_t row = i * H + h;
    if (a.post) r1n = a.rstd_post[row];
    if (a.pre) r2n = a.rstd_pre[row];
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int c = (j * TPR + lane) * VEC;
      const int64_t at = row * W + c;
      if (c < W) {
        load_raw<TAIL>(xn[j], x + at, W - c, W);
        if constexpr (GATE) load_raw<TAIL>(zn[j], z + at, W - c, W);
        if (res) load_raw<TAIL>(rn[j], res + at, W - c, W);
        if (dh) load_raw<TAIL>(hn[j], dh + at, W - c, W);
        if (dn) load_raw<TAIL>(nn[j], dn + at, W - c, W);
      }
    }
  };
  if (slice < a.rows) fetch(slice);
  const float inv_w = 1.f / float(W);
  const int64_t first = int64_t(blockIdx.x) * kGroups / H;
  int phase = 0;
  for (int64_t k = first; k < a.rows; k += n_slices) {
    const int64_t i0 = slice + (k - first), row = i0 * H + h;
    const bool on = live && i0 < a.rows;
    const float r1 = r1n, r2 = r2n;
    float xh[NV][VEC], g[NV][VEC], hh[NV][VEC], d[NV][VEC], t[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const bool in = on && (j * TPR + lane) * VEC < W;
#pragma unroll
      for (int e = 0; e < VEC; e++) xh[j][e] = g[j][e] = hh[j][e] = d[j][e] = t[j][e] = 0.f;
      if (in) {
        floats<TAIL>(xn[j], xh[j], W - (j * TPR + lane) * VEC, W);
        if constexpr (GATE) floats<TAIL>(zn[j], g[j], W - (j * TPR + lane) * VEC, W);
        if (res) floats<TAIL>(rn[j], hh[j], W - (j * TPR + lane) * VEC, W);
        if (dh) floats<TAIL>(hn[j], d[j], W - (j * TPR + lane) * VEC, W);
        if (dn) floats<TAIL>(nn[j], t[j], W - (j * TPR + lane) * VEC, W);
#pragma unroll
        for (int e = 0; e < VEC; e++) xh[j][e] *= r1;
      }
    }
    if (live && i0 + n_slices < a.rows) fetch(i0 + n_slices);
    // silu(z), and its derivative over what it multiplies, from one exponential
    float sl[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        sl[j][e] = 1.f;
        if constexpr (GATE) {
          const float sg = 1.f / (1.f + expf(-g[j][e]));
          sl[j][e] = g[j][e] * sg;
          g[j][e] = sg * fmaf(g[j][e], 1.f - sg, 1.f);
        }
      }
    if (a.pre) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        float w1[VEC], sc[VEC], w2[VEC];
        p1.get(j, w1);
        ps.get(j, sc);
        p2.get(j, w2);
#pragma unroll
        for (int e = 0; e < VEC; e++) {
          hh[j][e] = fmaf(xh[j][e] * w1[e] * sl[j][e], sc[e], hh[j][e]) * r2;
          dw2[j][e] = fmaf(t[j][e], hh[j][e], dw2[j][e]);
          t[j][e] *= w2[e];
          s = fmaf(t[j][e], hh[j][e], s);
        }
      }
      const float m = row_sum<TPR>(s, buf[phase][group]) * inv_w;
      phase ^= 1;
#pragma unroll
      for (int j = 0; j < NV; j++)
#pragma unroll
        for (int e = 0; e < VEC; e++) d[j][e] = fmaf(r2, fmaf(-hh[j][e], m, t[j][e]), d[j][e]);
    }
    if (a.dresidual && on) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int c = (j * TPR + lane) * VEC;
        if (c < W) store<TAIL>(static_cast<R*>(a.dresidual) + row * W + c, d[j], W - c);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float w1[VEC], sc[VEC];
      p1.get(j, w1);
      ps.get(j, sc);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const float p = xh[j][e] * w1[e], c = d[j][e] * sc[e];
        ds[j][e] = fmaf(d[j][e], p * sl[j][e], ds[j][e]);
        g[j][e] *= c * p;
        const float o = c * sl[j][e];
        dw1[j][e] = fmaf(o, xh[j][e], dw1[j][e]);
        d[j][e] = o * w1[e];
        s = fmaf(d[j][e], xh[j][e], s);
      }
    }
    if (GATE && on) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int c = (j * TPR + lane) * VEC;
        if (c < W) store<TAIL>(static_cast<T*>(a.dz) + row * W + c, g[j], W - c);
      }
    }
    if (a.post) {
      const float m = row_sum<TPR>(s, buf[phase][group]) * inv_w;
      phase ^= 1;
#pragma unroll
      for (int j = 0; j < NV; j++)
#pragma unroll
        for (int e = 0; e < VEC; e++) d[j][e] = r1 * fmaf(-xh[j][e], m, d[j][e]);
    }
    if (on) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int c = (j * TPR + lane) * VEC;
        if (c < W) store<TAIL>(static_cast<T*>(a.dx) + row * W + c, d[j], W - c);
      }
    }
  }
  if (!part || !live) return;
  const int64_t at = (slice * H + h) * int64_t(W), all = n_slices * H * W;
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const int c = (j * TPR + lane) * VEC;
    {
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        if (c + e >= W) continue;
        if (a.dpost_weight) part[at + c + e] = dw1[j][e];
        if (a.dscale) part[all + at + c + e] = ds[j][e];
        if (a.dpre_weight) part[2 * all + at + c + e] = dw2[j][e];
      }
    }
  }
}

struct Sums {
  const float* in[3];
  float* out[3];  // null: not asked for
};
// out[k][c] = sum of in[k per .. k per + per - 1][c] over its rows below n, in order: 64 columns and 4 row strides a
// workgroup; blockIdx.z chooses the parameter
__global__ __launch_bounds__(256) void bn_reduce_kernel(Sums a, int64_t n, int64_t per, int64_t cols) {
  __shared__ float sh[4][64];
  const float* in = a.in[blockIdx.z];
  float* out = a.out[blockIdx.z];
  if (!out) return;
  const int l = threadIdx.x % 64, g = threadIdx.x / 64;
  const int64_t c = int64_t(blockIdx.x) * 64 + l;
  const int64_t r0 = int64_t(blockIdx.y) * per, r1 = r0 + per < n ? r0 + per : n;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < cols) {
    int64_t r = r0 + g;
    for (; r + 12 < r1; r += 16) {
#pragma unroll
      for (int u = 0; u < 4; u++) s[u] += in[(r + 4 * u) * cols + c];
    }
    for (; r < r1; r += 4) s[0] += in[r * cols + c];
  }
  sh[g][l] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (g == 0 && c < cols) out[blockIdx.y * cols + c] = (sh[0][l] + sh[1][l]) + (sh[2][l] + sh[3][l]);
}

// Workgroups of a launch.  Forward, 65536 rows of 2560 in bf16 with both norms and the residual: 2048, 4096, 8192 of them 320,
// 275, 259 us.  The backward's partial sums grow with them: 512 or 768 of rows of many threads 464 or 472 us (with the sums),
// of rows of at most a wave (16384 rows of 24 heads of 64, gated) 91 or 74 us.
constexpr int64_t kFwdBlocks = 8192;
constexpr int64_t bwd_blocks(int tpr) { return tpr > kWave ? 512 : 768; }

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T, typename R, bool GATE, bool TAIL, int VEC, int NV, int TPR>
struct Form {
  static hipError_t fwd(const BlockNormArgs& a, int64_t n_slices) {
    constexpr int threads = block_threads(TPR), groups = threads / TPR;
    return launch_kind(kKindBlockNormFwd, bn_fwd_kernel<T, R, GATE, TAIL, VEC, NV, TPR>, ceil_div(n_slices * a.H, groups), threads, a.stream, a, n_slices);
  }
  static hipError_t bwd(const BlockNormArgs& a, int64_t n_slices, float* part) {
    constexpr int threads = block_threads(TPR), groups = threads / TPR;
    return launch_kind(kKindBlockNormBwd, bn_bwd_kernel<T, R, GATE, TAIL, VEC, NV, TPR>, ceil_div(n_slices * a.H, groups), threads, a.stream, a, n_slices, part);
  }
  static constexpr int tpr = TPR;
};

// The form of rows of W elements: one vector a thread, two only above 1024 threads.  The steps leave up to half of the
// threads of a row idle: 2^27 bf16 elements in rows of 2560 on 320 of 320 threads 205 us forward and 347 backward, of 2568 on
// 321 of 512 217 and 352, of 4096 on 512 of 512 197 and 315, of 4104 on 513 of 640 249 and 474, of 6400 on 800 of 1024
// 218 and 419.  768 threads may have 168 registers, 1024 of them 128: 16384 float rows of 5120, backward, 425 us with 768 and
// 535 with 1024, gated 857 and 1259; 8192 gated bf16 rows of 12288 1480 and 3046.
template <typename T, typename R, bool GATE, bool TAIL, typename Go>
auto with_size(int64_t W, Go go) {
  constexpr int V = 16 / sizeof(T);
  const int64_t n = ceil_div(W, V);
  if (n <= 8) return go(Form<T, R, GATE, TAIL, V, 1, 8>{});
  if (n <= 16) return go(Form<T, R, GATE, TAIL, V, 1, 16>{});
  if (n <= 32) return go(Form<T, R, GATE, TAIL, V, 1, 32>{});
  if (n <= 64) return go(Form<T, R, GATE, TAIL, V, 1, 64>{});
  if (n <= 128) return go(Form<T, R, GATE, TAIL, V, 1, 128>{});
  if (n <= 192) return go(Form<T, R, GATE, TAIL, V, 1, 192>{});
  if (n <= 256) return go(Form<T, R, GATE, TAIL, V, 1, 256>{});
  if (n <= 320) return go(Form<T, R, GATE, TAIL, V, 1, 320>{});
  if (n <= 512) return go(Form<T, R, GATE, TAIL, V, 1, 512>{});
  if (n <= 640) return go(Form<T, R, GATE, TAIL, V, 1, 640>{});
  if (n <= 1024) return go(Form<T, R, GATE, TAIL, V, 1, 1024>{});
  if (n <= 1536) return go(Form<T, R, GATE, TAIL, V, 2, 768>{});
  if (V == 4 && n <= 2048) return go(Form<T, R, GATE, TAIL, V, 8 / V, 1024>{});
  return go(Form<T, R, GATE, TAIL, V, 16 / V, 1024>{});
}
template <typename T, typename R, bool GATE, typename Go>
auto with_form(int64_t W, Go go) {
  return W % (16 / sizeof(T)) ? with_size<T, R, GATE, true>(W, go) : with_size<T, R, GATE, false>(W, go);
}

template <typename Go>
auto with_types(const BlockNormArgs& a, Go go) {
  auto types = [&](auto gate) {
    if (a.dtype == 0) return go(float{}, float{}, gate);
    return a.rdtype == 0 ? go(bf16_bits{}, float{}, gate) : go(bf16_bits{}, bf16_bits{}, gate);
  };
  return a.z ? types(std::true_type{}) : types(std::false_type{});
}

// Rows in flight: the groups of `blocks` workgroups, shared out over the heads.
int64_t slices_of(const BlockNormArgs& a, int tpr, int64_t blocks) {
  return std::max<int64_t>(1, std::min<int64_t>(a.rows, ceil_div(blocks * (block_threads(tpr) / tpr), a.H)));
}

// How the backward's parameter sums are cut: n_slices partial rows [H W], added in n_parts parts of `per` rows and then
// together.
struct NormPlan {
  int64_t n_slices, n_parts, per;
};
NormPlan plan_bwd(const BlockNormArgs& a) {
  NormPlan p;
  const int tpr = with_types(a, [&](auto t, auto r, auto gate) {
    return with_form<decltype(t), decltype(r), decltype(gate)::value>(a.W, [](auto f) { return int(f.tpr); });
  });
  p.n_slices = slices_of(a, tpr, bwd_blocks(tpr));
  const int64_t blocks = 3 * ceil_div(a.H * a.W, 64);
  p.n_parts = std::max<int64_t>(1, std::min<int64_t>(ceil_div(512, blocks), p.n_slices / 32));
  p.per = ceil_div(p.n_slices, p.n_parts);
  p.n_parts = ceil_div(p.n_slices, p.per);
  return p;
}
int64_t plan_floats(const BlockNormArgs& a, const NormPlan& p) {
  return 3 * (p.n_slices + (p.n_parts > 1 ? p.n_parts : 0)) * a.H * a.W;
}

}  // namespace

int64_t blocknorm_max_width() { return 16384; }

size_t blocknorm_workspace_bytes(const BlockNormArgs& a) {
  if (a.rows == 0 || a.H == 0 || a.W == 0) return 0;
  return size_t(plan_floats(a, plan_bwd(a))) * sizeof(float);
}

hipError_t launch_blocknorm_fwd(const BlockNormArgs& a) {
  return with_types(a, [&](auto t, auto r, auto gate) {
    typedef decltype(t) T;
    typedef decltype(r) R;
    return with_form<T, R, decltype(gate)::value>(a.W, [&](auto f) { return f.fwd(a, slices_of(a, f.tpr, kFwdBlocks)); });
  });
}

hipError_t launch_blocknorm_bwd(const BlockNormArgs& a, void* workspace) {
  const int64_t cols = a.H * a.W, blocks = ceil_div(cols, 64);
  const bool params = a.dpost_weight || a.dscale || a.dpre_weight;
  auto reduce = [&](const float* in, int64_t in_stride, float* o0, float* o1, float* o2, int64_t n, int64_t per, int64_t parts) {
    const Sums s{{in, in + in_stride, in + 2 * in_stride}, {o0, o1, o2}};
    return launch_kind_3d(kKindBlockNormReduce, bn_reduce_kernel, dim3(unsigned(blocks), unsigned(parts), 3), 256, a.stream, s, n, per, cols);
  };
  float* part = params ? static_cast<float*>(workspace) : nullptr;
  if (a.rows == 0)  // sums over no rows
    return params ? reduce(part, 0, a.dpost_weight, a.dscale, a.dpre_weight, 0, 0, 1) : hipSuccess;
  NormPlan p{};
  const hipError_t err = with_types(a, [&](auto t, auto r, auto gate) {
    typedef decltype(t) T;
    typedef decltype(r) R;
    p = plan_bwd(a);
    return with_form<T, R, decltype(gate)::value>(a.W, [&](auto f) { return f.bwd(a, p.n_slices, part); });
  });
  if (err != hipSuccess || !params) return err;
  const int64_t all = p.n_slices * cols, some = p.n_parts * cols;
  if (p.n_parts == 1) return reduce(part, all, a.dpost_weight, a.dscale, a.dpre_weight, p.n_slices, p.n_slices, 1);
  float* q = part + 3 * all;
  const hipError_t e = reduce(part, all, a.dpost_weight ? q : nullptr, a.dscale ? q + some : nullptr, a.dpre_weight ? q + 2 * some : nullptr,
                              p.n_slices, p.per, p.n_parts);
  if (e != hipSuccess) return e;
  return reduce(q, some, a.dpost_weight, a.dscale, a.dpre_weight, p.n_parts, p.n_parts, 1);
}

}  // namespace ssm
