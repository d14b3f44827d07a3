// ssm_layernorm.hip -- layer norm over the last axis, forward and backward, with the
// reduction of the parameters' gradients.
//
// A row is one [W] slice of x [rows, H, W]; the parameters are [H, W] (H = 1: the norm over
// the model's width; H > 1: each head's channels, with the head's own weight).
//   m = mean(x),  v = mean((x - m)^2),  r = 1 / sqrt(v + eps),  xh = (x - m) r
//   y = xh w + b
//   t = dy w,  dx = r (t - mean(t) - xh mean(t xh)),  dw = sum over rows of dy xh,  db = sum of dy
// Both directions read every streamed value once, hold it for the two sums of its row (the variance is taken around
// the mean, in a second pass over the registers), and write once; rows of whole 16-byte vectors are bound by HBM up to a
// width of 8192 (bf16; float 4096 backward, 16384 forward).  Wider rows take 1024 threads of 128 registers each,
// too few for their backward, which keeps three values a column more: 289 (bf16), 125 (float) and, of odd widths
// above 2048, 89 registers go through scratch.  TB/s of what has to be moved, at 2^27 elements, forward / backward: 5.1 / 5.4 at
// 2560 and 5.6 / 2.9 at 8192 in float; 3.7 / 4.6 at 8192 and 2.2 / 0.6 at 16384 in bf16; of odd widths, whose lanes read one
// element each, 3.8 / 5.1 at 1001 and 3.4 / 1.4 at 5001 in float, 2.5 / 2.4 and 1.7 / 0.7 in bf16.  A group of threads keeps one head's parameters in registers and
// walks rows, the next row's loads under way while one is summed; without them, a row a group and
// 1024 workgroups, the backward of 65536 rows of 2560 in bf16 took 338 us, with them 191 us (5.3 TB/s).
// All sums are float.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssm_device.h"
#include "ssm_layernorm.h"
#include "ssm_profile.h"

namespace ssm {
namespace {

// VEC consecutive elements, as floats
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
    static_assert(VEC == 1, "");
    v[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const bf16_bits* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    static_assert(VEC == 1, "");
    v[0] = load_elem(p);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void store_vec(bf16_bits* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const bf16_bits lo = __builtin_bit_cast(bf16_bits, static_cast<__bf16>(v[2 * j]));
      const bf16_bits hi = __builtin_bit_cast(bf16_bits, static_cast<__bf16>(v[2 * j + 1]));
      w[j] = uint32_t(lo) | (uint32_t(hi) << 16);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    store_elem(p, v[0]);
  }
}
// VEC elements as they come from memory, and as floats
template <typename T, int VEC>
struct RawVec {
  uint4 u;
};
template <typename T>
struct RawVec<T, 1> {
  T u;
};
template <typename T, int VEC>
__device__ __forceinline__ RawVec<T, VEC> load_raw(const T* p) {
  RawVec<T, VEC> r;
  if constexpr (VEC == 1) r.u = *p;
  else r.u = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void raw_floats(const RawVec<T, VEC>& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = load_elem(&r.u);
  else load_vec<VEC>(reinterpret_cast<const T*>(&r.u), v);
}
// VEC floats of a parameter row (only 4-byte aligned: W need not be a multiple of 4)
template <int VEC>
__device__ __forceinline__ void load_par(const float* p, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; j++) v[j] = p[j];
}

// Sums of N values over the TPR threads of a row, the same in every one of them.  Rows of at
// most a wave's lanes are summed with shuffles; wider ones through LDS, two calls in turn with a
// buffer each, so that one barrier a call is enough (the whole workgroup comes to it).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* buf) {
#pragma unroll
  for (int off = (TPR < kWave ? TPR : kWave) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; i++) s[i] += __shfl_xor(s[i], off);
  if constexpr (TPR > kWave) {
    constexpr int kWaves = TPR / kWave;
    if (threadIdx.x % kWave == 0)
#pragma unroll
      for (int i = 0; i < N; i++) buf[i * kWaves + threadIdx.x / kWave % kWaves] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; w++) t += buf[i * kWaves + w];
      s[i] = t;
    }
  }
}

constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256; }

// One group of TPR threads walks the rows slice, slice + n_slices, ... of head h; each thread has NV
// vectors of VEC elements of a row, at columns (j TPR + lane) VEC.
template <typename T, int VEC, int NV, int TPR>
__global__ __launch_bounds__(block_threads(TPR)) void ln_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias, float eps,
    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int64_t n_slices, int H, int W) {
  constexpr int kGroups = block_threads(TPR) / TPR;
  __shared__ float buf[2][kGroups][TPR > kWave ? TPR / kWave : 1];
  const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int64_t gid = int64_t(blockIdx.x) * kGroups + group;
  const bool live = gid < n_slices * H;  // the others keep the workgroup's barriers
  const int h = live ? int(gid % H) : 0;
  const int64_t slice = live ? gid / H : rows;
  float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const int c = (j * TPR + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      wv[j][i] = 1.f;
      bv[j][i] = 0.f;
    }
    if (weight && c < W) load_par<VEC>(weight + int64_t(h) * W + c, wv[j]);
    if (bias && c < W) load_par<VEC>(bias + int64_t(h) * W + c, bv[j]);
  }
  RawVec<T, VEC> xn[NV];
  auto fetch = [&](int64_t i) {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int c = (j * TPR + lane) * VEC;
      if (c < W) xn[j] = load_raw<T, VEC>(x + (i * H + h) * W + c);
    }
  };
  if (slice < rows) fetch(slice);
  const int64_t first = int64_t(blockIdx.x) * kGroups / H;  // the workgroup's first slice: it has the most rows
  for (int64_t k = first; k < rows; k += n_slices) {
    const int64_t i0 = slice + (k - first);
    const bool on = live && i0 < rows;
    float v[NV][VEC], s[1] = {0.f}, q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (on && (j * TPR + lane) * VEC < W) {
        raw_floats<T, VEC>(xn[j], v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) v[j][i] = 0.f;
      }
    }
    if (live && i0 + n_slices < rows) fetch(i0 + n_slices);
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int i = 0; i < VEC; i++) s[0] += v[j][i];
    row_sum<TPR>(s, buf[0][group]);
    const float m = s[0] / float(W);
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if ((j * TPR + lane) * VEC < W) {
#pragma unroll
        for (int i = 0; i < VEC; i++) {
          v[j][i] -= m;
          q[0] = fmaf(v[j][i], v[j][i], q[0]);
        }
      }
    }
    row_sum<TPR>(q, buf[1][group]);
    const float r = 1.f / sqrtf(q[0] / float(W) + eps);
    if (on) {
      const int64_t row = i0 * H + h;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int c = (j * TPR + lane) * VEC;
        if (c < W) {
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; i++) o[i] = fmaf(v[j][i] * r, wv[j][i], bv[j][i]);
          store_vec<VEC>(y + row * W + c, o);
        }
      }
      if (lane == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
      }
    }
  }
}

// As the forward; a group keeps its head's parameter gradients in registers and writes its own row of the
// partial sums [n_slices][H W], which ln_reduce_kernel adds in a fixed order.
template <typename T, int VEC, int NV, int TPR>
__global__ __launch_bounds__(block_threads(TPR)) void ln_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx, float* __restrict__ part_w,
    float* __restrict__ part_b, int64_t rows, int64_t n_slices, int H, int W) {
  constexpr int kGroups = block_threads(TPR) / TPR;
  __shared__ float buf[2][kGroups][TPR > kWave ? 2 * (TPR / kWave) : 1];
  const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int64_t gid = int64_t(blockIdx.x) * kGroups + group;
  const bool live = gid < n_slices * H;
  const int h = live ? int(gid % H) : 0;
  const int64_t slice = live ? gid / H : rows;
  float wv[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const int c = (j * TPR + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      wv[j][i] = 1.f;
      dw[j][i] = 0.f;
      db[j][i] = 0.f;
    }
    if (weight && c < W) load_par<VEC>(weight + int64_t(h) * W + c, wv[j]);
  }
  const float inv_w = 1.f / float(W);
  // the next row is on its way while one is worked on
  RawVec<T, VEC> xn[NV], gn[NV];
  float mn = 0.f, rn = 0.f;
  auto fetch = [&](int64_t i) {
    const int64_t row = i * H + h;
    mn = mean[row];
    rn = rstd[row];
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int c = (j * TPR + lane) * VEC;
      if (c < W) {
        xn[j] = load_raw<T, VEC>(x + row * W + c);
        gn[j] = load_raw<T, VEC>(dy + row * W + c);
      }
    }
  };
  if (slice < rows) fetch(slice);
  int phase = 0;
  const int64_t first = int64_t(blockIdx.x) * kGroups / H;
  for (int64_t k = first; k < rows; k += n_slices) {
    const int64_t i0 = slice + (k - first), row = i0 * H + h;
    const bool on = live && i0 < rows;
    const float m = on ? mn : 0.f, r = on ? rn : 0.f;
    float xh[NV][VEC], g[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (on && (j * TPR + lane) * VEC < W) {
        raw_floats<T, VEC>(xn[j], xh[j]);
        raw_floats<T, VEC>(gn[j], g[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) {
          xh[j][i] = m;
          g[j][i] = 0.f;
        }
      }
    }
    if (live && i0 + n_slices < rows) fetch(i0 + n_slices);
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        xh[j][i] = (xh[j][i] - m) * r;
        dw[j][i] = fmaf(g[j][i], xh[j][i], dw[j][i]);
        db[j][i] += g[j][i];
        g[j][i] *= wv[j][i];
        s[0] += g[j][i];
        s[1] = fmaf(g[j][i], xh[j][i], s[1]);
      }
    row_sum<TPR>(s, buf[phase][group]);
    phase ^= 1;  // a row's sums are read before the barrier of the next one, which frees this half
    const float c1 = s[0] * inv_w, c2 = s[1] * inv_w;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int c = (j * TPR + lane) * VEC;
      if (on && c < W) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i++) o[i] = r * (g[j][i] - fmaf(xh[j][i], c2, c1));
        store_vec<VEC>(dx + row * W + c, o);
      }
    }
  }
  if (!part_w || !live) return;
  const int64_t at = (slice * H + h) * int64_t(W);
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const int c = (j * TPR + lane) * VEC;
    if (c < W) {
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        part_w[at + c + i] = dw[j][i];
        part_b[at + c + i] = db[j][i];
      }
    }
  }
}

// out[k][c] = sum of in[k per .. k per + per - 1][c] over its rows below n, in order: 64 columns
// and 4 row strides a workgroup; blockIdx.z chooses the weight's or the bias's sums.
__global__ __launch_bounds__(256) void ln_reduce_kernel(const float* __restrict__ in_w, const float* __restrict__ in_b,
                                                        float* __restrict__ out_w, float* __restrict__ out_b,
                                                        int64_t n, int64_t per, int64_t cols) {
  __shared__ float sh[4][64];
  const float* in = blockIdx.z ? in_b : in_w;
  float* out = blockIdx.z ? out_b : out_w;
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

// Workgroups of a launch.  Forward, 65536 rows in bf16: 512, 1024, 2048 of them 316, 311, 255 us at a width of 4096 and
// 223, 154, 155 us at 2560; backward: two a CU (four times as many 233, 191 us, with four times the partial sums).
constexpr int64_t kFwdBlocks = 2048, kBwdBlocks = 512;

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T, int VEC, int NV, int TPR>
struct Form {
  static hipError_t fwd(const LayerNormArgs& a, int64_t n_slices) {
    constexpr int threads = block_threads(TPR), groups = threads / TPR;
    return launch_kind(kKindNormFwd, ln_fwd_kernel<T, VEC, NV, TPR>, ceil_div(n_slices * a.H, groups), threads, a.stream,
                       static_cast<const T*>(a.x), a.weight, a.bias, a.eps, static_cast<T*>(a.y), a.mean, a.rstd, a.rows,
                       n_slices, int(a.H), int(a.W));
  }
  static hipError_t bwd(const LayerNormArgs& a, int64_t n_slices, float* pw, float* pb) {
    constexpr int threads = block_threads(TPR), groups = threads / TPR;
    return launch_kind(kKindNormBwd, ln_bwd_kernel<T, VEC, NV, TPR>, ceil_div(n_slices * a.H, groups), threads, a.stream,
                       static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
                       static_cast<T*>(a.dx), pw, pb, a.rows, n_slices, int(a.H), int(a.W));
  }
  static constexpr int tpr = TPR;
};

// rows read and written in 16-byte vectors: whole vectors a row, aligned tensors
template <typename T>
bool whole_vectors(const LayerNormArgs& a) {
  constexpr int VEC = 16 / sizeof(T);
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                      reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dx);
  return a.W % VEC == 0 && p % 16 == 0;
}

// The form of rows of W elements: as few threads as hold a row in at most 4 vectors each (one element at a time, 8 or
// 16), in whole waves above one.  Measured, 65536 rows of 2560 in bf16, forward / backward: 3 vectors of 128 threads
// 157 / 212 us where 2 of 256 took 191 / 253 us and 1 of 512 242 / 254 us.  Between 129 and 256 vectors the forward has
// one wave a row (1536: 77 us, 94 us with two) and the backward, which keeps twice as much, two (114 us, 126 us with one).
template <typename T, bool FWD, typename Go>
auto with_form(bool vec, int64_t W, Go go) {
  constexpr int V = 16 / sizeof(T);
  if (!vec) {
    if (W <= 64) return go(Form<T, 1, 8, 8>{});
    if (W <= 512) return go(Form<T, 1, 8, 64>{});
    if (W <= 2048) return go(Form<T, 1, 8, 256>{});
    return go(Form<T, 1, 16, 1024>{});
  }
  const int64_t n = W / V;
  if (n <= 8) return go(Form<T, V, 1, 8>{});
  if (n <= 16) return go(Form<T, V, 1, 16>{});
  if (n <= 32) return go(Form<T, V, 1, 32>{});
  if (n <= 64) return go(Form<T, V, 1, 64>{});
  if (n <= 128) return go(Form<T, V, 2, 64>{});
  if (FWD && n <= 192) return go(Form<T, V, 3, 64>{});
  if (FWD && n <= 256) return go(Form<T, V, 4, 64>{});
  if (n <= 256) return go(Form<T, V, 2, 128>{});
  if (n <= 384) return go(Form<T, V, 3, 128>{});
  if (n <= 512) return go(Form<T, V, 4, 128>{});
  if (n <= 768) return go(Form<T, V, 3, 256>{});
  if (n <= 1024) return go(Form<T, V, 4, 256>{});
  return go(Form<T, V, 4, 1024>{});
}

// Rows in flight: the groups of `blocks` workgroups, shared out over the heads.
int64_t slices_of(const LayerNormArgs& a, int tpr, int64_t blocks) {
  return std::max<int64_t>(1, std::min<int64_t>(a.rows, ceil_div(blocks * (block_threads(tpr) / tpr), a.H)));
}

template <typename T>
hipError_t launch_fwd(const LayerNormArgs& a) {
  return with_form<T, true>(whole_vectors<T>(a), a.W, [&](auto f) { return f.fwd(a, slices_of(a, f.tpr, kFwdBlocks)); });
}
template <typename T>
hipError_t launch_bwd(const LayerNormArgs& a, int64_t n_slices, float* pw, float* pb) {
  return with_form<T, false>(whole_vectors<T>(a), a.W, [&](auto f) { return f.bwd(a, n_slices, pw, pb); });
}

// How the backward's parameter sums are cut: n_slices partial rows [H W], added in n_parts parts of
// `per` rows and then together.
struct NormPlan {
  int64_t n_slices, n_parts, per;
};
NormPlan plan_bwd(const LayerNormArgs& a, bool vec) {
  NormPlan p;
  auto tpr_of = [](auto f) { return int(f.tpr); };
  const int tpr = a.dtype == 0 ? with_form<float, false>(vec, a.W, tpr_of) : with_form<bf16_bits, false>(vec, a.W, tpr_of);
  p.n_slices = slices_of(a, tpr, kBwdBlocks);
  const int64_t blocks = 2 * ceil_div(a.H * a.W, 64);
  p.n_parts = std::max<int64_t>(1, std::min<int64_t>(ceil_div(512, blocks), p.n_slices / 32));
  p.per = ceil_div(p.n_slices, p.n_parts);
  p.n_parts = ceil_div(p.n_slices, p.per);
  return p;
}
int64_t plan_floats(const LayerNormArgs& a, const NormPlan& p) {
  return 2 * (p.n_slices + (p.n_parts > 1 ? p.n_parts : 0)) * a.H * a.W;
}

}  // namespace

int64_t layernorm_max_width() { return 16384; }

size_t layernorm_workspace_bytes(const LayerNormArgs& a) {
  if (a.rows == 0 || a.H == 0 || a.W == 0) return 0;
  // tensors of any alignment: the larger of the two forms
  const int64_t n = std::max(plan_floats(a, plan_bwd(a, true)), plan_floats(a, plan_bwd(a, false)));
  return size_t(n) * sizeof(float);
}

hipError_t launch_layernorm_fwd(const LayerNormArgs& a) {
  return a.dtype == 0 ? launch_fwd<float>(a) : launch_fwd<bf16_bits>(a);
}

hipError_t launch_layernorm_bwd(const LayerNormArgs& a, void* workspace) {
  const int64_t cols = a.H * a.W, blocks = ceil_div(cols, 64);
  const bool params = a.dweight != nullptr;
  auto reduce = [&](const float* iw, const float* ib, float* ow, float* ob, int64_t n, int64_t per, int64_t parts) {
    return launch_kind_3d(kKindNormReduce, ln_reduce_kernel, dim3(unsigned(blocks), unsigned(parts), 2), 256, a.stream,
                          iw, ib, ow, ob, n, per, cols);
  };
  if (a.rows == 0)  // sums over no rows
    return params ? reduce(nullptr, nullptr, a.dweight, a.dbias, 0, 0, 1) : hipSuccess;
  const bool vec = a.dtype == 0 ? whole_vectors<float>(a) : whole_vectors<bf16_bits>(a);
  const NormPlan p = plan_bwd(a, vec);
  float* pw = params ? static_cast<float*>(workspace) : nullptr;
  float* pb = params ? pw + p.n_slices * cols : nullptr;
  hipError_t err = a.dtype == 0 ? launch_bwd<float>(a, p.n_slices, pw, pb) : launch_bwd<bf16_bits>(a, p.n_slices, pw, pb);
  if (err != hipSuccess || !params) return err;
  if (p.n_parts == 1) return reduce(pw, pb, a.dweight, a.dbias, p.n_slices, p.n_slices, 1);
  float* qw = pb + p.n_slices * cols;
  float* qb = qw + p.n_parts * cols;
  err = reduce(pw, pb, qw, qb, p.n_slices, p.per, p.n_parts);
  if (err != hipSuccess) return err;
  return reduce(qw, qb, a.dweight, a.dbias, p.n_parts, p.n_parts, 1);
}

}  // namespace ssm
