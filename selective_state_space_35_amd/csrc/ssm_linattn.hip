// ssm_linattn.hip -- linear attention with a decay for each head: whole sequences, the
// gradients, and the step for one token.
//
// Definition, for each batch row and head (q and k belong to the head's group):
//   r_t = exp(A_h + g_t),  S_t = r_t S_{t-1} + k_t v_t^T  [Dk, Dv],  y_t = scale S_t^T q_t
//
// The gradients are the same operator with the roles changed.  With D_t the gradient of S_t,
//   D_t = scale q_t dy_t^T + r_{t+1} D_{t+1},  D of the last token also + d_last
//   dq_t = scale S_t dy_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  d_initial = r_0 D_0
// so dq sweeps the tokens forwards with (dy, v, k) in the places of (q, k, v) and the state S^T,
// dk sweeps them backwards with (v, dy, q) and the state D^T, and dv backwards with (k, q, dy)
// and the state D; in reversed time a state is decayed by the gate of the token after.
// The gate's gradient is <D_t, r_t S_{t-1}>.  Token i adds q_i . dq_i to <D, S> as it is read
// and k_i . dk_i leaves it as it is written (counting backwards), so
//   dg_t = <d_last, S_last> + sum over i >= t of (q_i . dq_i - k_i . dk_i),
// where the product of token i with itself, in both terms, is left out of both: a difference of
// rounded values would not cancel it, and with strong decays it is much larger than dg.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssm_device.h"
#include "ssm_internal.h"
#include "ssm_profile.h"

namespace ssm {
namespace {

constexpr int kMaxDim = 128;

// One sweep over the sequence, in the roles of the forward: queries xq and keys xk of KD
// elements, values xv and outputs of VD elements.
struct Sweep {
  const void* xq;
  const void* xk;
  const void* xv;
  int gq, gk, gv;          // heads that share a row of xq, xk, xv (H / their heads)
  const void* g;
  const float* A;
  const int32_t* lengths;
  float wscale, rscale;    // factors of the products written into the state, and of the readout
  const float* init;       // state before the first token of the sweep, or null
  bool init_t;             // it is stored [VD][KD]
  void* out;               // [b, L, H, VD], of the streamed type or (out_f32) float; null: not written
  bool out_f32;
  float* last;             // [b, H, KD, VD], or null
  bool final_decay;        // `last` takes the first token's decay too (gradient of the initial state)
  // with dots: dots[b, L, H] = (output without the token's own product) . xd
  const void* xd;
  int gd;
  float* dots;
  const float* dstate;     // [b, H, VD, KD] (transposed); dstate_dot[b, H] = its product with the last state
  float* dstate_dot;
  int64_t b, L;
  int H, KD, VD;
  hipStream_t stream;
};

// A log decay below -10^4 counts as -10^4 (its factor is zero in float either way), so that
// minus infinity is a reset and differences of running sums stay numbers.
__device__ __forceinline__ float clamp_log(float x) { return x < -1e4f ? -1e4f : x; }

template <typename T>
__device__ __forceinline__ float log_decay(const Sweep& p, int64_t bi, int64_t t, int h) {
  float x = p.A ? p.A[h] : 0.f;
  if (p.g) x += load_elem(static_cast<const T*>(p.g) + (bi * p.L + t) * p.H + h);
  return clamp_log(x);
}

__device__ __forceinline__ int64_t live_length(const int32_t* lengths, int64_t bi, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[bi];
  return n < 0 ? 0 : n > L ? L : n;
}

// sum of v over the 128 threads of the workgroup, in every thread
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if (threadIdx.x % kWave == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  return sh[0] + sh[1];
}

// The recurrence token by token: a workgroup holds a head's state, thread j its column j.
template <typename T, bool REVERSE>
__global__ __launch_bounds__(128) void lin_sweep_kernel(Sweep p) {
  __shared__ float ks[kMaxDim], qs[kMaxDim], sh[2];
  const int h = blockIdx.x % p.H;
  const int64_t bi = blockIdx.x / p.H;
  const int j = threadIdx.x;
  const bool live = j < p.VD;
  const int Hq = p.H / p.gq, Hk = p.H / p.gk, Hv = p.H / p.gv;
  const int64_t n = live_length(p.lengths, bi, p.L);
  float S[kMaxDim];
#pragma unroll
  for (int i = 0; i < kMaxDim; i++) {
    S[i] = 0.f;
    if (p.init && live && i < p.KD) {
      const int64_t at = (bi * p.H + h) * p.KD * p.VD;
      S[i] = p.init_t ? p.init[at + int64_t(j) * p.KD + i] : p.init[at + int64_t(i) * p.VD + j];
    }
  }
  for (int64_t i = 0; i < p.L; i++) {
    const int64_t t = REVERSE ? p.L - 1 - i : i, row = bi * p.L + t;
    const int64_t oat = (row * p.H + h) * p.VD + j;
    if (t >= n) {
      if (p.out && live) {
        if (p.out_f32) static_cast<float*>(p.out)[oat] = 0.f;
        else store_elem(static_cast<T*>(p.out) + oat, 0.f);
      }
      if (p.dots && j == 0) p.dots[row * p.H + h] = 0.f;
      continue;
    }
    __syncthreads();
    if (j < p.KD) {
      ks[j] = load_elem(static_cast<const T*>(p.xk) + (row * Hk + h / p.gk) * p.KD + j);
      qs[j] = load_elem(static_cast<const T*>(p.xq) + (row * Hq + h / p.gq) * p.KD + j);
    } else {
      ks[j] = 0.f;
      qs[j] = 0.f;
    }
    __syncthreads();
    const float v = live ? load_elem(static_cast<const T*>(p.xv) + (row * Hv + h / p.gv) * p.VD + j) * p.wscale : 0.f;
    float dec;
    if (REVERSE) dec = t + 1 < n ? expf(log_decay<T>(p, bi, t + 1, h)) : 1.f;
    else dec = expf(log_decay<T>(p, bi, t, h));
    float o = 0.f, qk = 0.f;
#pragma unroll
    for (int i2 = 0; i2 < kMaxDim; i2++) {
      S[i2] *= dec;
      o = fmaf(qs[i2], S[i2], o);
      qk = fmaf(qs[i2], ks[i2], qk);
      S[i2] = fmaf(ks[i2], v, S[i2]);
    }
    o *= p.rscale;
    if (p.dots) {
      const int Hd = p.H / p.gd;
      const float x = live ? load_elem(static_cast<const T*>(p.xd) + (row * Hd + h / p.gd) * p.VD + j) : 0.f;
      const float d = block_sum(o * x, sh);
      if (j == 0) p.dots[row * p.H + h] = d;
    }
    o = fmaf(qk * p.rscale, v, o);
    if (p.out && live) {
      if (p.out_f32) static_cast<float*>(p.out)[oat] = o;
      else store_elem(static_cast<T*>(p.out) + oat, o);
    }
  }
  if (p.dstate_dot) {
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxDim; i++)
      if (p.dstate && live && i < p.KD) d += S[i] * p.dstate[((bi * p.H + h) * p.VD + j) * p.KD + i];
    d = block_sum(d, sh);
    if (j == 0) p.dstate_dot[bi * p.H + h] = d;
  }
  if (p.last && live) {
    const float f = p.final_decay && n > 0 ? expf(log_decay<T>(p, bi, 0, h)) : 1.f;
#pragma unroll
    for (int i = 0; i < kMaxDim; i++)
      if (i < p.KD) p.last[((bi * p.H + h) * p.KD + i) * p.VD + j] = S[i] * f;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the gates: dg_t = end + sum over i >= t of (a_i - c_i), per batch row and head, where
// end = <d_last, S_last>.  a and c are [b, L, H].  Tiles of kGateTile tokens: first each tile's
// sum, then each tile adds the sums of the later ones to its own running sum (double: the terms
// cancel over the sequence).
constexpr int kGateTile = 256;
constexpr int kGateHeads = 16;  // heads of a workgroup: 16 consecutive floats of a row, times 16 tokens

__global__ __launch_bounds__(256) void lin_gate_tiles_kernel(const float* __restrict__ a, const float* __restrict__ c,
                                                             double* __restrict__ sums, int64_t L, int H, int n_tiles,
                                                             int h_blocks) {
  __shared__ double sh[16][kGateHeads];
  const int h = (blockIdx.x % h_blocks) * kGateHeads + threadIdx.x % kGateHeads;
  const int64_t rest = blockIdx.x / h_blocks;
  const int tile = int(rest % n_tiles);
  const int64_t bi = rest / n_tiles;
  const int s = threadIdx.x / kGateHeads;
  double d = 0.0;
  for (int i = 0; i < kGateTile / 16; i++) {
    const int64_t t = int64_t(tile) * kGateTile + i * 16 + s;
    if (t < L && h < H) {
      const int64_t at = (bi * L + t) * H + h;
      d += double(a[at]) - double(c[at]);
    }
  }
  sh[s][threadIdx.x % kGateHeads] = d;
  __syncthreads();
  if (s == 0 && h < H) {
    double tot = 0.0;
    for (int i = 0; i < 16; i++) tot += sh[i][threadIdx.x];
    sums[(bi * n_tiles + tile) * H + h] = tot;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void lin_gate_kernel(const float* __restrict__ a, const float* __restrict__ c,
                                                       const double* __restrict__ sums, const float* __restrict__ end,
                                                       const int32_t* __restrict__ lengths, T* __restrict__ dg,
                                                       int64_t L, int H, int n_tiles, int h_blocks) {
  __shared__ double sh[16][kGateHeads];
  __shared__ double after[16][kGateHeads];
  const int hl = threadIdx.x % kGateHeads;
  const int h = (blockIdx.x % h_blocks) * kGateHeads + hl;
  const int64_t rest = blockIdx.x / h_blocks;
  const int tile = int(rest % n_tiles);
  const int64_t bi = rest / n_tiles;
  const int s = threadIdx.x / kGateHeads;  // 16 consecutive tokens of the tile
  const bool ok = h < H;
  const int64_t t0 = int64_t(tile) * kGateTile + s * 16;
  double d[16], own = 0.0, later = 0.0;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int64_t at = (bi * L + t0 + i) * H + h;
    d[i] = ok && t0 + i < L ? double(a[at]) - double(c[at]) : 0.0;
    own += d[i];
  }
  for (int k = tile + 1 + s; k < n_tiles; k += 16)
    if (ok) later += sums[(bi * n_tiles + k) * H + h];
  sh[s][hl] = own;
  after[s][hl] = later;
  __syncthreads();
  double run = ok && end ? double(end[bi * H + h]) : 0.0;
  for (int i = 0; i < 16; i++) run += after[i][hl];
  for (int i = s + 1; i < 16; i++) run += sh[i][hl];
  const int64_t n = live_length(lengths, bi, L);
#pragma unroll
  for (int i = 15; i >= 0; i--) {
    run += d[i];
    const int64_t t = t0 + i;
    if (ok && t < L) store_elem(dg + (bi * L + t) * H + h, t < n ? float(run) : 0.f);
  }
}

// out[row, g, :] = sum over the group's heads of in[row, h, :] (float), rounded once
template <typename T>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float* __restrict__ in, T* __restrict__ out,
                                                            int64_t n, int share, int D) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t rg = i / D;
  const int d = int(i % D);
  float s = 0.f;
  for (int k = 0; k < share; k++) s += in[(rg * share + k) * D + d];
  store_elem(out + i, s);
}

// ---------------------------------------------------------------------------
// One token: a workgroup holds one head of one batch row.  Lanes run along the columns of the
// state, the workgroup's row groups along its rows; the readout is summed over the row groups in LDS.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void lin_update_kernel(float* __restrict__ state, const T* __restrict__ q,
                                                         const T* __restrict__ k, const T* __restrict__ v,
                                                         const T* __restrict__ g, const float* __restrict__ A,
                                                         const int32_t* __restrict__ lengths, float scale,
                                                         T* __restrict__ y, int H, int share, int Dk, int Dv,
                                                         int lanes) {
  __shared__ float qs[kMaxDim], ks[kMaxDim];
  __shared__ float part[256 * VEC];
  const int h = blockIdx.x % H;
  const int64_t bi = blockIdx.x / H;
  const int64_t bh = bi * H + h, qrow = bi * (H / share) + h / share;
  if (lengths && lengths[bi] <= 0) {
    for (int j = threadIdx.x; j < Dv; j += 256) store_elem(y + bh * Dv + j, 0.f);
    return;
  }
  for (int j = threadIdx.x; j < Dk; j += 256) {
    qs[j] = load_elem(q + qrow * Dk + j);
    ks[j] = load_elem(k + qrow * Dk + j);
  }
  __syncthreads();
  const float dec = expf(clamp_log((A ? A[h] : 0.f) + (g ? load_elem(g + bh) : 0.f)));
  const int l = threadIdx.x % lanes, r0 = threadIdx.x / lanes, rows = 256 / lanes;
  const int c = l * VEC;
  float acc[VEC], vv[VEC];
#pragma unroll
  for (int i = 0; i < VEC; i++) {
    acc[i] = 0.f;
    vv[i] = c + i < Dv ? load_elem(v + bh * Dv + c + i) : 0.f;
  }
  if (c < Dv) {
    float* S = state + bh * Dk * Dv + c;
#pragma unroll 8
    for (int r = r0; r < Dk; r += rows) {
      float s[VEC];
      if constexpr (VEC == 4) {
        const float4 u = *reinterpret_cast<const float4*>(S + r * Dv);
        s[0] = u.x; s[1] = u.y; s[2] = u.z; s[3] = u.w;
      } else {
        s[0] = S[r * Dv];
      }
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        s[i] = fmaf(s[i], dec, ks[r] * vv[i]);
        acc[i] = fmaf(qs[r], s[i], acc[i]);
      }
      if constexpr (VEC == 4) *reinterpret_cast<float4*>(S + r * Dv) = make_float4(s[0], s[1], s[2], s[3]);
      else S[r * Dv] = s[0];
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; i++) part[(r0 * lanes + l) * VEC + i] = acc[i];
  __syncthreads();
  for (int j = threadIdx.x; j < Dv; j += 256) {
    float s = 0.f;
    for (int r = 0; r < rows; r++) s += part[r * lanes * VEC + j];
    store_elem(y + bh * Dv + j, s * scale);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <typename T>
hipError_t run_sweep(const Sweep& p, bool reverse) {
  if (reverse) return launch_kind(kKindLinSweep, lin_sweep_kernel<T, true>, p.b * p.H, 128, p.stream, p);
  return launch_kind(kKindLinSweep, lin_sweep_kernel<T, false>, p.b * p.H, 128, p.stream, p);
}

Sweep common(const LinAttnArgs& a) {
  Sweep p{};
  p.g = a.g; p.A = a.A; p.lengths = a.lengths;
  p.wscale = p.rscale = 1.f;
  p.gq = p.gk = p.gv = p.gd = 1;
  p.b = a.b; p.L = a.L; p.H = int(a.H);
  p.stream = a.stream;
  return p;
}

// The backward's workspace, in bytes from its start.
struct BwdWork {
  size_t dot_q, dot_k, end, sums, dq, dk, total;
  int n_tiles;
};
BwdWork plan_bwd(const LinAttnArgs& a) {
  BwdWork w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += up256(bytes);
    return r;
  };
  const size_t rows = size_t(a.b) * a.L * a.H;
  w.n_tiles = int(ceil_div(a.L, kGateTile));
  w.dot_q = take(rows * 4);
  w.dot_k = take(rows * 4);
  w.end = take(size_t(a.b) * a.H * 4);
  w.sums = take(size_t(a.b) * w.n_tiles * a.H * 8);
  if (a.G != a.H) {
    w.dq = take(rows * a.Dk * 4);
    w.dk = take(rows * a.Dk * 4);
  }
  w.total = at;
  return w;
}

template <typename T>
hipError_t bwd_impl(const LinAttnArgs& a, char* ws) {
  const BwdWork w = plan_bwd(a);
  const int share = int(a.H / a.G);
  const bool gate = a.dg != nullptr;
  float* end = gate && a.dlast ? reinterpret_cast<float*>(ws + w.end) : nullptr;
  Sweep p = common(a);  // dq: forwards, the state is S^T [Dv, Dk]
  p.xq = a.dy; p.xk = a.v; p.xv = a.k; p.gv = share;
  p.KD = int(a.Dv); p.VD = int(a.Dk);
  p.rscale = a.scale;
  p.init = a.h0; p.init_t = true;
  p.out = share > 1 ? static_cast<void*>(ws + w.dq) : a.dq; p.out_f32 = share > 1;
  if (gate) {
    p.xd = a.q; p.gd = share;
    p.dots = reinterpret_cast<float*>(ws + w.dot_q);
    p.dstate = a.dlast;
    p.dstate_dot = end;
  }
  hipError_t err = run_sweep<T>(p, false);
  if (err != hipSuccess) return err;
  p = common(a);  // dk: backwards, the state is D^T [Dv, Dk]
  p.xq = a.v; p.xk = a.dy; p.xv = a.q; p.gv = share;
  p.KD = int(a.Dv); p.VD = int(a.Dk);
  p.wscale = a.scale;
  p.init = a.dlast; p.init_t = true;
  p.out = share > 1 ? static_cast<void*>(ws + w.dk) : a.dk; p.out_f32 = share > 1;
  if (gate) {
    p.xd = a.k; p.gd = share;
    p.dots = reinterpret_cast<float*>(ws + w.dot_k);
  }
  err = run_sweep<T>(p, true);
  if (err != hipSuccess) return err;
  p = common(a);  // dv: backwards, the state is D [Dk, Dv]
  p.xq = a.k; p.gq = share; p.xk = a.q; p.gk = share; p.xv = a.dy;
  p.KD = int(a.Dk); p.VD = int(a.Dv);
  p.wscale = a.scale;
  p.init = a.dlast;
  p.out = a.dv;
  p.last = a.dh0; p.final_decay = true;
  err = run_sweep<T>(p, true);
  if (err != hipSuccess || a.L == 0) return err;
  if (share > 1) {
    const int64_t n = a.b * a.L * a.G * a.Dk;
    for (int k = 0; k < 2; k++) {
      err = launch_kind(kKindLinReduce, lin_group_sum_kernel<T>, ceil_div(n, 256), 256, a.stream,
                        reinterpret_cast<const float*>(ws + (k ? w.dk : w.dq)), static_cast<T*>(k ? a.dk : a.dq), n,
                        share, int(a.Dk));
      if (err != hipSuccess) return err;
    }
  }
  if (gate) {
    const int h_blocks = int(ceil_div(a.H, kGateHeads));
    const float* dq = reinterpret_cast<const float*>(ws + w.dot_q);
    const float* dk = reinterpret_cast<const float*>(ws + w.dot_k);
    double* sums = reinterpret_cast<double*>(ws + w.sums);
    const int64_t blocks = a.b * w.n_tiles * h_blocks;
    err = launch_kind(kKindLinGate, lin_gate_tiles_kernel, blocks, 256, a.stream, dq, dk, sums, a.L, int(a.H),
                      w.n_tiles, h_blocks);
    if (err != hipSuccess) return err;
    err = launch_kind(kKindLinGate, lin_gate_kernel<T>, blocks, 256, a.stream, dq, dk, sums, end, a.lengths,
                      static_cast<T*>(a.dg), a.L, int(a.H), w.n_tiles, h_blocks);
  }
  return err;
}

template <typename T>
hipError_t update_impl(const LinAttnArgs& a) {
  const bool vec = a.Dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.last) % 16 == 0;
  int lanes = 1;
  while (lanes * (vec ? 4 : 1) < a.Dv) lanes *= 2;
  const int share = int(a.H / a.G);
  auto go = [&](auto kern) {
    return launch_kind(kKindLinUpdate, kern, a.b * a.H, 256, a.stream, a.last, static_cast<const T*>(a.q),
                       static_cast<const T*>(a.k), static_cast<const T*>(a.v), static_cast<const T*>(a.g), a.A,
                       a.lengths, a.scale, static_cast<T*>(a.y), int(a.H), share, int(a.Dk), int(a.Dv), lanes);
  };
  return vec ? go(lin_update_kernel<T, 4>) : go(lin_update_kernel<T, 1>);
}

}  // namespace

int64_t linattn_max_dim() { return kMaxDim; }
int64_t linattn_max_heads() { return 65535; }

size_t linattn_workspace_bytes(const LinAttnArgs& a, bool backward) {
  if (a.b == 0 || a.H == 0 || !backward) return 0;
  return plan_bwd(a).total;
}

hipError_t launch_linattn_fwd(const LinAttnArgs& a, void*) {
  const int share = int(a.H / a.G);
  Sweep p = common(a);
  p.xq = a.q; p.xk = a.k; p.xv = a.v; p.gq = p.gk = share;
  p.KD = int(a.Dk); p.VD = int(a.Dv);
  p.rscale = a.scale;
  p.init = a.h0;
  p.out = a.y;
  p.last = a.last;
  return a.dtype == 0 ? run_sweep<float>(p, false) : run_sweep<bf16_bits>(p, false);
}

hipError_t launch_linattn_bwd(const LinAttnArgs& a, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  return a.dtype == 0 ? bwd_impl<float>(a, ws) : bwd_impl<bf16_bits>(a, ws);
}

hipError_t launch_linattn_update(const LinAttnArgs& a) {
  return a.dtype == 0 ? update_impl<float>(a) : update_impl<bf16_bits>(a);
}

}  // namespace ssm
