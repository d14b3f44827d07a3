// ssm_deltarule.hip -- the gated delta rule: whole sequences, the gradients, and the step for one token.
//
// Definition, for each batch row and head (q and k belong to the head's group):
//   r_t = exp(A_h + g_t),  u_t = beta_t (v_t - r_t S_{t-1}^T k_t),  S_t = r_t S_{t-1} + k_t u_t^T  [Dk, Dv],
//   y_t = scale S_t^T q_t
// What a token writes is what its value differs by from what the state answers for its key.
//
// In chunks of C tokens, with G the running sum of the log decays inside the chunk, S the state entering it, products by
// exp(G) taken row by row, and X_ts = exp(G_t - G_s) k_t . k_s for s < t (zero else):
//   R = V - exp(G) K S,  (I + X diag(beta)) N = R,  U = beta N
//   Y = scale (exp(G) Q S + P U),  P_ts = exp(G_t - G_s) q_t . k_s for s <= t
//   S' = exp(G_C) S + K^T (exp(G_C - G) U)
// The inverse Z = (I + X diag(beta))^-1 needs the keys only, so it is taken for all chunks at once (delta_tri_kernel); what runs
// from chunk to chunk are products with the state (sweep).
//
// Backward, D the gradient of the state leaving the chunk:
//   dU = scale P^T dY + exp(G_C - G) K D,  dR = Z^T beta dU,  dV = dR
//   D' = exp(G_C) D + scale (exp(G) Q)^T dY - (exp(G) K)^T dR
// is the same sweep from the last chunk to the first.  With S, D, N and dR of every chunk the rest is each chunk's own
// (delta_grad_kernel), W = scale exp(G_t - G_s) dY U^T (s <= t), B = -exp(G_t - G_s) dR U^T (s < t):
//   dQ = scale exp(G) dY S^T + W K,  dK = W^T Q + (B + B^T) K + exp(G_C - G) U D^T - exp(G) dR S^T
//   dbeta_t = dR_t . N_t / beta_t
// and dg_t sums, over the terms above that hold a factor exp(G) with token t's gate in it, the term: the entries of
// W o QK^T + B o KK^T with row >= t > column, and the rows' products of q and k with the state parts.  It is computed as the
// sum from t on of row sums less column sums, of the same rounded entries, so that what cancels cancels to float's
// rounding of one chunk; at a reset (a factor that is zero in float) it is zero and the sum starts again.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ssm_chunks.h"
#include "ssm_deltarule.h"
#include "ssm_device.h"
#include "ssm_kinds.h"

namespace ssm {
namespace {

constexpr int kMaxDim = 128;
// exp of a log decay below this is zero in float, denormal numbers included (2^-150)
constexpr float kZeroLog = -104.f;
// The backward's dR is beta E, and dbeta needs E: where beta is nearer to zero than this, dR is computed with this in its
// place, and its own part taken where dR itself is meant
constexpr float kLeastBeta = 8.673617379884035e-19f;  // 2^-60

constexpr int kTile = 64;  // columns of the values a workgroup of the sweep or of the token step has

struct Rule {
  const void* q;
  const void* k;
  const void* v;           // the sweep's values: v, or (backwards) dy
  const void* beta;
  const void* g;
  const float* A;
  const int32_t* lengths;
  float scale;
  bool backward;           // a small beta is moved away from zero (delta_tri_kernel)
  const float* init;       // the state before the sweep's first chunk, or (backwards) the gradient behind its last
  void* y;
  float* last;             // the state after the sweep's last chunk
  const float* tri;        // [b H n_chunks] inverses as operand fragments
  // what the backward keeps of a chunk, 16 rows by 16 rows and in those by columns, as a lane of the sweep has them
  float* states;           // [b H n_chunks][KP / 16][VP][16]: states entering the chunks, or gradients of those leaving them
  float* left;             // [b H n_chunks][C / 16][VP][16]: N, or dR of the moved beta
  // the cut, in the sweep's order of the chunks: n_segs segments of `parts` parts of part_chunks chunks.  With more than one
  // segment, what the n_parts parts of all but the last do to a state is S -> map S + own
  float* part_own;         // [b H n_parts][KP / 16][VP][16]; after the chain the states leaving the parts
  float* part_map;         // [b H n_parts][KP / 16][KP][16]
  int n_segs, parts, part_chunks, n_parts;
  int64_t b, L;
  int H, share, Dk, Dv, KP, VP, n_chunks, n_tiles;
  hipStream_t stream;
};

template <typename T>
struct Shape {
  static constexpr int kC = kChunk<T>;
  static constexpr int TB = kC / 16;           // blocks of 16 tokens
  static constexpr int kSteps = kC / 32;       // operand fragments along the tokens
  static constexpr int kTri = TB == 4 ? 6 : 2; // fragments of a triangular matrix
  static constexpr bool kTwo = sizeof(T) == 2; // operands that are not given in bf16 are taken in parts
};
// Which of the kTri fragments holds rows 16 tb.. and columns 32 ks.. of a lower triangular matrix, or of an upper one
template <int TB>
__device__ __forceinline__ constexpr int lower_frag(int tb, int ks) { return tb < 2 ? tb : 2 * tb - 2 + ks; }
template <int TB>
__device__ __forceinline__ constexpr int upper_frag(int tb, int ks) { return TB == 2 ? tb : tb < 2 ? 2 * tb + ks : tb + 2; }

template <typename T>
__device__ __forceinline__ float beta_of(const Rule& p, int64_t bi, int64_t t, int h, int n) {
  if (t >= n) return 0.f;
  return p.beta ? load_elem(static_cast<const T*>(p.beta) + (bi * p.L + t) * p.H + h) : 1.f;
}
__device__ __forceinline__ float moved_beta(float x) { return fabsf(x) < kLeastBeta ? copysignf(kLeastBeta, x) : x; }
template <typename T>
__device__ __forceinline__ float gate_of(const Rule& p, int64_t bi, int64_t t, int h, int n) {
  if (t >= n) return 0.f;
  return clamp_log((p.g ? load_elem(static_cast<const T*>(p.g) + (bi * p.L + t) * p.H + h) : 0.f) + (p.A ? p.A[h] : 0.f));
}

// A 16 x 16 product in float: rows of a, a lane's four contraction indices 4 (l / 16) .. + 3, with b, which has the layout
// of a result
__device__ __forceinline__ f32x4 mma16(const float4& a, const f32x4& b, f32x4 c) {
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b[2], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b[3], c, 0, 0, 0);
}

// Rows r .. r + 3 (of a lane's group of 16) of column c0 + lane % 16 of an LDS tile
__device__ __forceinline__ uint2 quad_bits(const bf16_bits* t, int ld, int r, int c0) {
  const int m = threadIdx.x % 16;
  const bf16_bits* p = t + (r + m / 4) * ld + c0 + 4 * (m % 4);
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)p));
}
__device__ __forceinline__ f32x4 quad_rows(const bf16_bits* t, int ld, int r, int c0) {
  const uint2 v = quad_bits(t, ld, r, c0);
  return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
               __uint_as_float(v.y & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 quad_rows(const float* t, int ld, int r, int c0) {
  const float* p = t + r * ld + c0 + threadIdx.x % 16;
  return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]};
}
// the fragment of rows r .. r + 3 and r + 16 .. r + 19 of that column: the contraction in the order of two results
__device__ __forceinline__ bf16x8 col_pair(const bf16_bits* t, int ld, int r, int c0) {
  const uint2 a = quad_bits(t, ld, r, c0), b = quad_bits(t, ld, r + 16, c0);
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
__device__ __forceinline__ f32x8 col_pair(const float* t, int ld, int r, int c0) {
  const f32x4 a = quad_rows(t, ld, r, c0), b = quad_rows(t, ld, r + 16, c0);
  return f32x8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}

// One value a token of [b, L, H], as it comes from memory, lane l with the chunk's token l: nothing but the load, and no
// branch around it, so that what waits for one chunk's does not wait for the next one's.
template <typename T, int kC>
struct Scalars {
  const T* base;
  int voff, chunk;
  __device__ __forceinline__ void init(const void* x, int64_t row, int H, int h) {
    const int l = threadIdx.x % kWave;
    base = static_cast<const T*>(x) + row * H + h;
    chunk = kC * H;
    voff = x && l < kC ? l * H * int(sizeof(T)) : 0x7fffffff;
  }
  __device__ __forceinline__ uint32_t load(int nv) {
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(base);
    base += chunk;
    const int at = int(threadIdx.x % kWave) < nv ? voff : 0x7fffffff;
    if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
  }
  // those of the chunk whose first token's value is x[at]
  static __device__ __forceinline__ uint32_t load_at(const void* x, int64_t at, int H, int nv) {
    const int l = threadIdx.x % kWave;
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(static_cast<const T*>(x) + at);
    const int o = x && l < nv ? l * H * int(sizeof(T)) : 0x7fffffff;
    if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0);
  }
  static __device__ __forceinline__ float value(uint32_t raw) { return __uint_as_float(sizeof(T) == 4 ? raw : raw << 16); }
};

// Two floats rounded to bf16, in one instruction
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) float f2;
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
}

// Floats as operand fragments: bf16 in N parts of 8 bits each (2^-9, 2^-17, 2^-25 of them is lost), float as they are
template <typename T, int N>
struct Parts {
  static constexpr int kN = sizeof(T) == 2 ? N : 1;
  Frag<T> f[kN];
  __device__ __forceinline__ void set(const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
      make_frag(x, f[0]);
    } else {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] = x[j];
#pragma unroll
      for (int k = 0; k < kN; k++) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          w[j] = pack_pair(y[2 * j], y[2 * j + 1]);
          if (k + 1 < kN) {
            y[2 * j] -= __uint_as_float(w[j] << 16);
            y[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
          }
        }
        f[k] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
  __device__ __forceinline__ void set(const f32x4& a, const f32x4& b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    set(x);
  }
};
// c + a b, of parts whose numbers add up to less than `least` (the products beyond are below the last part's rounding)
template <typename T, int NA, int NB>
__device__ __forceinline__ f32x4 mma_parts(const Parts<T, NA>& a, const Parts<T, NB>& b, f32x4 c) {
  constexpr int na = Parts<T, NA>::kN, nb = Parts<T, NB>::kN, least = na > nb ? na : nb;
#pragma unroll
  for (int i = 0; i < na; i++)
#pragma unroll
    for (int j = 0; j < nb; j++)
      if (i + j < least) c = mma(a.f[i], b.f[j], c);
  return c;
}

// ---------------------------------------------------------------------------
// Z = (I + X diag(beta))^-1 of every chunk, written as operand fragments in float: lane l of fragment (tb, ks) has row
// 16 tb + l % 16 and columns 32 ks + 4 (l / 16) .. + 3 and 16 more; for the backward also those of Z^T beta.
// The 16 x 16 blocks on the diagonal are inverted by forward substitution, a column a lane, and joined block by block,
// Z_ij = -Z_ii (sum over j <= k < i of X_ik Z_kj), a column of blocks a wave, in float products.  An entry of X that is not
// finite is taken as zero: where a key, a beta or a gate is not finite the sweep makes NaN of everything from its token on by
// itself.
// Bound by the latency of its phases (scores, blocks, joining, a barrier between): b8 L2048 H24 D64 bf16 36 us, of the backward,
// with both forms, 49; b1 L32768 H40 D128 bf16 128 us, 3 TB/s of keys and inverses.  Four workgroups a CU hide some of it.
// ---------------------------------------------------------------------------
template <typename T, int KDP, bool VEC>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4))) void delta_tri_kernel(Rule p, float* lower, float* upper) {
  typedef Shape<T> Z;
  constexpr int kC = Z::kC, TB = Z::TB, KS = KDP / 32, ldk = Tile<T, KDP, kKey>::ld, ld = kC + 4;
  __shared__ __attribute__((aligned(16))) T Ks[Tile<T, KDP, kKey>::kElems];
  __shared__ __attribute__((aligned(16))) float X[kC * ld];  // X diag(beta); block by block its inverse takes its place
  __shared__ Decays<kC> d;
  __shared__ __attribute__((aligned(16))) float beta[kC];
  const int64_t id = blockIdx.x, bh = id / p.n_chunks, bi = bh / p.H;
  const int c = int(id % p.n_chunks), h = int(bh % p.H), n = live_length(p.lengths, bi, p.L);
  if (c * kC >= n) return;  // behind the sequence: not read
  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid / kWave), l = tid % kWave;
  const int lr = l % 16, g4 = 4 * (l / 16), g8 = 8 * (l / 16);
  Stage<T, KDP, kKey, VEC> sk;
  uint4 rk[Tile<T, KDP, kKey>::kPieces];
  const int G = p.H / p.share;
  sk.init(static_cast<const T*>(p.k) + ((bi * p.L + int64_t(c) * kC) * G + h / p.share) * p.Dk, G * p.Dk, p.Dk, false, tid);
  sk.load(rk, n - c * kC, tid);
  if (wv == 0) {
    const float g = l < kC ? gate_of<T>(p, bi, int64_t(c) * kC + l, h, n) : 0.f;
    fill_decays(d, g, 1.f);
  } else if (wv == 1 && l < kC) {
    const float x = beta_of<T>(p, bi, int64_t(c) * kC + l, h, n);
    beta[l] = p.backward ? moved_beta(x) : x;
  }
  sk.store(Ks, rk, tid);
  __syncthreads();
  for (int j = wv; j < TB * (TB + 1) / 2; j += 4) {  // X diag(beta), its blocks on and below the diagonal
    int tb = 0, sb = j;
    while (sb > tb) sb -= ++tb;
    f32x4 a{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KS; kk++)
      a = mma(row_frag(Ks + (16 * sb + lr) * ldk + 32 * kk + g8), row_frag(Ks + (16 * tb + lr) * ldk + 32 * kk + g8), a);
    const int t = 16 * tb + lr, s0 = 16 * sb + g4;
    const float th = d.hi[t], tl = d.lo[t];
    const float4 h4 = lds4(d.hi + s0), l4 = lds4(d.lo + s0), b4 = lds4(beta + s0);
    const float sh[4] = {h4.x, h4.y, h4.z, h4.w}, sl[4] = {l4.x, l4.y, l4.z, l4.w}, be[4] = {b4.x, b4.y, b4.z, b4.w};
    float x[4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const float e = a[r] * exp2_fast((th - sh[r]) + (tl - sl[r])) * be[r];
      x[r] = s0 + r < t && e * 0.f == 0.f ? e : 0.f;
    }
    *reinterpret_cast<float4*>(X + t * ld + s0) = make_float4(x[0], x[1], x[2], x[3]);
  }
  __syncthreads();
  if (tid < kC) {  // lane l has column l % 16 of block l / 16
    const int b0 = 16 * (l / 16);
    float4 a4[4][4];  // four rows at a time, read two rows ahead
    auto read = [&](int i) {
#pragma unroll
      for (int k4 = 0; k4 < (i + 3) / 4; k4++) a4[i % 4][k4] = lds4(X + (b0 + i) * ld + b0 + 4 * k4);
    };
    read(1);
    read(2);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
      if (i > 0 && i + 2 < 16) read(i + 2);
      float s[2] = {i == lr ? 1.f : 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < i; k++) {
        const float4& r = a4[i % 4][k / 4];
        s[k % 2] = fmaf(-(k % 4 == 0 ? r.x : k % 4 == 1 ? r.y : k % 4 == 2 ? r.z : r.w), x[k], s[k % 2]);
      }
      x[i] = s[0] + s[1];
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_sched_barrier(0);  // one wave reads and writes the blocks, in this order
#pragma unroll
    for (int i = 0; i < 16; i++) X[(b0 + i) * ld + b0 + lr] = x[i];
  }
  __syncthreads();
  f32x4 col[TB];
  if (wv < TB - 1) {
#pragma unroll
    for (int r = 0; r < 4; r++) col[0][r] = X[(16 * wv + g4 + r) * ld + 16 * wv + lr];
#pragma unroll
    for (int o = 1; o < TB; o++) {  // block row wv + o
      const int i = wv + o;
      if (i < TB) {
        f32x4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < o; k++) t = mma16(lds4(X + (16 * i + lr) * ld + 16 * (wv + k) + g4), col[k], t);
        f32x4 z{0.f, 0.f, 0.f, 0.f};
        z = mma16(lds4(X + (16 * i + lr) * ld + 16 * i + g4), t, z);
#pragma unroll
        for (int r = 0; r < 4; r++) col[o][r] = -z[r];
      }
    }
  }
  __syncthreads();  // the blocks below the diagonal have been read by all
  if (wv < TB - 1) {
    float* here = X + (16 * wv + g4) * ld + 16 * wv + lr;
#pragma unroll
    for (int o = 1; o < TB; o++)
      if (wv + o < TB)
#pragma unroll
        for (int r = 0; r < 4; r++) here[(16 * o + r) * ld] = col[o][r];
  }
  __syncthreads();
  float4* out = reinterpret_cast<float4*>(lower + id * (Z::kTri * 512));
  float4* out_t = upper ? reinterpret_cast<float4*>(upper + id * (Z::kTri * 512)) : nullptr;
  for (int j = tid; j < Z::kTri * 64; j += kThreads) {
    const int f = j / 64, ll = j % 64, r16 = ll % 16, q4 = 4 * (ll / 16);
    int tb = 0, ks = 0;
#pragma unroll
    for (int a = 0; a < TB; a++)
      for (int b = 0; b <= a / 2; b++)
        if (lower_frag<TB>(a, b) == f) tb = a, ks = b;
    const float* row = X + (16 * tb + r16) * ld + 32 * ks + q4;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    out[2 * j] = lds4(row);
    out[2 * j + 1] = 2 * ks + 1 <= tb ? lds4(row + 16) : zero;
    if (out_t) {
      int sb = 0;
      ks = 0;
#pragma unroll
      for (int a = 0; a < TB; a++)
        for (int b = a / 2; b < Z::kSteps; b++)
          if (upper_frag<TB>(a, b) == f) sb = a, ks = b;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int t = 32 * ks + q4 + e % 4 + 16 * (e / 4);
        x[e] = t / 16 >= sb ? X[t * ld + 16 * sb + r16] * beta[t] : 0.f;
      }
      out_t[2 * j] = make_float4(x[0], x[1], x[2], x[3]);
      out_t[2 * j + 1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

// In the block of code around it: FIRST vector instructions, then N matrix instructions with EACH vector ones after each (a
// wave's matrix instructions run beside its vector ones, if they are issued in turn)
template <int FIRST, int N, int EACH>
__device__ __forceinline__ void interleave() {
  if constexpr (FIRST > 0) __builtin_amdgcn_sched_group_barrier(0x2, FIRST, 0);
#pragma unroll
  for (int i = 0; i < N; i++) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, EACH, 0);
  }
}

// ---------------------------------------------------------------------------
// The sweep over a head's chunks, for VT columns of the values: columns of the state do not meet, so each of the state
// waves has 16 NT of them to itself, with the state, R, N and U in registers.  A result of 16 x 16 has, in lane l, rows
// 4 (l / 16) .. + 3 of column l % 16, so two results side by side are the next product's operand as they are, as long as the
// other operand is read in that order of the contraction.
// Four other waves stage the chunk after and compute its P; two barriers a chunk.
// bf16: a product's operands that are not given in bf16 are taken in parts.  What a state or N is made of keeps all 24 bits
// (three parts, six products where both sides are floats); what an output alone is made of two (2^-17).
// ---------------------------------------------------------------------------
enum Mode { kForward, kStates, kBackwards };

constexpr int state_waves(int vt) { return vt >= 64 ? 4 : vt / 16; }

template <typename T, int KDP, int VT>
struct SweepLds {
  typedef Shape<T> Z;
  static constexpr int kC = Z::kC;
  __attribute__((aligned(16))) T q[2][Tile<T, KDP, kQuery>::kElems];
  __attribute__((aligned(16))) T k[2][Tile<T, KDP, kKey>::kElems];
  __attribute__((aligned(16))) T v[2][Tile<T, VT, kValue>::kElems];
  __attribute__((aligned(16))) T z[2][Z::kTwo ? 3 : 1][Z::kTri * 512];
  __attribute__((aligned(16))) T P[2][Z::kTwo ? 2 : 1][Z::kTri * 512];
  Decays<kC> d[4];  // written two chunks ahead
  __attribute__((aligned(16))) float beta[4][kC];  // backwards the part of dR that is beta's own
};

// A wave's step of a chunk is a chain: K S and Q S, R, Z R, U, the state; 64 columns a workgroup give each SIMD one wave of state
// and one that stages, and the chain bounds the sweep: at D64 in bf16 a wave takes 6400 cycles a chunk, in which a SIMD's matrix
// units are busy for 1970, its vector instructions issue for 2850 and the CU's LDS is busy for 2900 (840 of them bank conflicts);
// at D128 8800, 3070, 3240 and 5190 (2220).  Keeping S and N it takes 7200 and 8900, backwards 8000 and 10800.
// b8 L2048 H24 D64 bf16 101 us, keeping S and N 106, backwards 131; b4 L4096 H32 D128 bf16 keeping S and N 263, backwards 321
// (0.8 GB of states and values written by each, beside what it reads).
//
// PART: the pass that a cut needs before.  A workgroup takes one part of a head's chunks, from a state of zero for VT columns
// of the values, or from the unit matrix and without values for VT columns of the part's map; nothing is kept but where the
// state arrives.
template <typename T, int KDP, int VT, Mode MODE, bool PART, bool VEC>
__global__ __launch_bounds__(kThreads + kWave * state_waves(VT)) __attribute__((amdgpu_waves_per_eu(2, 2)))
void delta_sweep_kernel(Rule p) {
  typedef Shape<T> Z;
  constexpr int kC = Z::kC, TB = Z::TB, kSteps = Z::kSteps, kTri = Z::kTri, KS = KDP / 32, MT = KDP / 16;
  constexpr bool kTwo = Z::kTwo, kBack = MODE == kBackwards, kOut = MODE == kForward;
  constexpr int SW = state_waves(VT), NT = VT / (16 * SW);
  constexpr int ldq = Tile<T, KDP, kQuery>::ld, ldk = Tile<T, KDP, kKey>::ld, ldv = Tile<T, VT, kValue>::ld;
  __shared__ SweepLds<T, KDP, VT> sh;
  // Workgroups are dealt to the 8 XCDs in turn: those of a head, and of neighbouring ones that share rows, go to one
  const int tiles = PART ? p.n_tiles + (p.KP + VT - 1) / VT : p.n_tiles, pieces = PART ? p.n_parts : p.n_segs;
  const int64_t units = p.b * p.H * tiles * pieces, wg = blockIdx.x;
  const int64_t id = units % 8 == 0 ? (wg % 8) * (units / 8) + wg / 8 : wg;
  const bool unit = PART && int(id % tiles) >= p.n_tiles;  // columns of the map
  const int v0 = (int(id % tiles) - (unit ? p.n_tiles : 0)) * VT;
  const int piece = int(id / tiles % pieces);
  const int64_t bh = id / tiles / pieces, bi = bh / p.H;
  const int h = int(bh % p.H), n = live_length(p.lengths, bi, p.L), G = p.H / p.share;
  // its chunks first .. first + chunks - 1
  const int per = PART ? p.part_chunks : p.parts * p.part_chunks;
  const int from = kBack ? p.n_chunks - (piece + 1) * per : piece * per;
  const int lo = std::max(from, 0), chunks = std::max(0, std::min(from + per, (n + kC - 1) / kC) - lo);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = threadIdx.x % kWave;
  const int lr = l % 16, g4 = 4 * (l / 16), g8 = 8 * (l / 16);
  auto chunk_of = [&](int i) { return lo + (kBack ? chunks - 1 - i : i); };

  if (wv >= SW) {
    // ------------------------------------------------------------------ staging and scores
    const int pw = wv - SW, tid = threadIdx.x - kWave * SW;
    if constexpr (MODE != kStates) {  // the halves of P's fragments beyond the diagonal stay zero
      for (int i = tid; i < kSteps * 256; i += kThreads) {
        const int f = kBack ? upper_frag<TB>(2 * (i / 256) + 1, i / 256) : lower_frag<TB>(2 * (i / 256), i / 256);
        const int at = f * 512 + (i % 256) / 4 * 8 + i % 4 + (kBack ? 0 : 4);
#pragma unroll
        for (int b = 0; b < 2; b++) {
          sh.P[b][0][at] = T(0);
          if constexpr (kTwo) sh.P[b][1][at] = T(0);
        }
      }
    }
    Stage<T, KDP, kQuery, VEC> sq;
    Stage<T, KDP, kKey, VEC> sk;
    Stage<T, VT, kValue, VEC> sv;
    const int64_t t0 = bi * p.L + int64_t(chunk_of(0)) * kC;
    sq.init(static_cast<const T*>(p.q) + (t0 * G + h / p.share) * p.Dk, G * p.Dk, p.Dk, false, tid);
    sk.init(static_cast<const T*>(p.k) + (t0 * G + h / p.share) * p.Dk, G * p.Dk, p.Dk, false, tid);
    sv.init(static_cast<const T*>(p.v) + (t0 * p.H + h) * p.Dv + v0, p.H * p.Dv, p.Dv - v0, false, tid);
    if (kBack) {
      sq.chunk = -sq.chunk;
      sk.chunk = -sk.chunk;
      sv.chunk = -sv.chunk;
    }
    constexpr int kZ = (kTri * 64 + kThreads - 1) / kThreads;
    struct Regs {
      uint4 q[Tile<T, KDP, kQuery>::kPieces], k[Tile<T, KDP, kKey>::kPieces], v[Tile<T, VT, kValue>::kPieces];
      float4 z[kZ][2];
      uint32_t gate, beta;
    };
    Regs r0, r1;
    auto live = [&](int i) { return i < chunks ? n - chunk_of(i) * kC : 0; };
    const float fixed = p.A ? p.A[h] : 0.f;
    Scalars<T, kC> sg, sb;
    sg.init(p.g, t0, p.H, h);
    sb.init(p.beta, t0, p.H, h);
    if (kBack) {
      sg.chunk = -sg.chunk;
      sb.chunk = -sb.chunk;
    }
    const int last = std::max(chunks - 1, 0);
    const float* tri = p.tri + bh * p.n_chunks * (kTri * 512);
    auto fetch = [&](Regs& r, int i) {  // the i-th chunk of the sweep; behind its end nothing is read and the rows are zero
      const int nv = live(i);
      if constexpr (MODE != kStates) sq.load(r.q, nv, tid);
      sk.load(r.k, nv, tid);
      sv.load(r.v, unit ? 0 : nv, tid);
      const float4* from = reinterpret_cast<const float4*>(tri + int64_t(chunk_of(std::min(i, last))) * (kTri * 512));
#pragma unroll
      for (int j = 0; j < kZ; j++) {
        const int at = std::min(tid + j * kThreads, kTri * 64 - 1);
        r.z[j][0] = from[2 * at];
        r.z[j][1] = from[2 * at + 1];
      }
      r.gate = sg.load(nv);
      r.beta = sb.load(nv);
    };
    auto place = [&](const Regs& r, int i) {
      if (i >= chunks) return;
      const int b = i & 1;
      if constexpr (MODE != kStates) sq.store(sh.q[b], r.q, tid);
      sk.store(sh.k[b], r.k, tid);
      sv.store(sh.v[b], r.v, tid);
#pragma unroll
      for (int j = 0; j < kZ; j++) {
        const int at = tid + j * kThreads;
        if (at < kTri * 64) {
          const float x[8] = {r.z[j][0].x, r.z[j][0].y, r.z[j][0].z, r.z[j][0].w, r.z[j][1].x, r.z[j][1].y, r.z[j][1].z, r.z[j][1].w};
          Parts<T, 3> f;
          f.set(x);
#pragma unroll
          for (int k = 0; k < Parts<T, 3>::kN; k++) *reinterpret_cast<Frag<T>*>(sh.z[b][k] + at * 8) = f.f[k];
        }
      }
    };
    auto decays = [&](const Regs& r, int i) {  // by the wave with the fewest blocks of P
      if (pw != 3 || i >= chunks) return;
      const bool on = l < std::min(kC, live(i));
      fill_decays(sh.d[i & 3], on ? clamp_log(sg.value(r.gate) + fixed) : 0.f, 1.f);
      const float beta = on ? p.beta ? sb.value(r.beta) : 1.f : 0.f;
      const bool finite = beta * 0.f == 0.f;
      if (l < kC) sh.beta[i & 3][l] = kBack ? beta / moved_beta(beta) : finite ? beta : 0.f;
      // a beta that is no number makes its token's R, and so all from it on, NaN
      if (!kBack && l < kC && !finite) sh.d[i & 3].in[l] = beta * 0.f;
    };
    // N blocks of P, rows t of q with columns s of k, to their halves of fragments: forwards of P, backwards of its
    // transpose.  All reads come first, all products next.
    auto score_blocks = [&](int i, auto count, int t0, int s0, int t1, int s1, int t2, int s2) {
      constexpr int N = decltype(count)::value;
      const int tbs[3] = {t0, t1, t2}, sbs[3] = {s0, s1, s2};
      const T* Qs = sh.q[i & 1];
      const T* Ks = sh.k[i & 1];
      const Decays<kC>& d = sh.d[i & 3];
      Frag<T> qf[N][KS], kf[N][KS];
      float ch[N], cl[N];
      float4 h4[N], l4[N];
#pragma unroll
      for (int j = 0; j < N; j++)
#pragma unroll
        for (int kk = 0; kk < KS; kk++) {
          qf[j][kk] = row_frag(Qs + (16 * tbs[j] + lr) * ldq + 32 * kk + g8);
          kf[j][kk] = row_frag(Ks + (16 * sbs[j] + lr) * ldk + 32 * kk + g8);
        }
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int cb = kBack ? sbs[j] : tbs[j], rb = kBack ? tbs[j] : sbs[j];  // the blocks along lanes, and along a lane's four
        ch[j] = d.hi[16 * cb + lr];
        cl[j] = d.lo[16 * cb + lr];
        h4[j] = lds4(d.hi + 16 * rb + g4);
        l4[j] = lds4(d.lo + 16 * rb + g4);
      }
      __builtin_amdgcn_sched_barrier(0);
      f32x4 a[N];
#pragma unroll
      for (int j = 0; j < N; j++) a[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KS; kk++)
#pragma unroll
        for (int j = 0; j < N; j++) a[j] = kBack ? mma(qf[j][kk], kf[j][kk], a[j]) : mma(kf[j][kk], qf[j][kk], a[j]);
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int tb = tbs[j], sb = sbs[j], rb = kBack ? tb : sb;
        const float rh[4] = {h4[j].x, h4[j].y, h4[j].z, h4[j].w}, rl[4] = {l4[j].x, l4[j].y, l4[j].z, l4[j].w};
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const float diff = (ch[j] - rh[r]) + (cl[j] - rl[r]);
          const bool in = tb > sb || (kBack ? lr <= g4 + r : g4 + r <= lr);
          x[r] = in ? a[j][r] * exp2_fast(kBack ? -diff : diff) * p.scale : 0.f;
        }
        const int f = kBack ? upper_frag<TB>(sb, tb / 2) : lower_frag<TB>(tb, sb / 2);
        const int at = f * 512 + l * 8 + 4 * (rb % 2);
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(sh.P[i & 1][0] + at) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
          const uint2 hi = make_uint2(pack_pair(x[0], x[1]), pack_pair(x[2], x[3]));
          *reinterpret_cast<uint2*>(sh.P[i & 1][0] + at) = hi;
          *reinterpret_cast<uint2*>(sh.P[i & 1][kTwo ? 1 : 0] + at) =
              make_uint2(pack_pair(x[0] - __uint_as_float(hi.x << 16), x[1] - __uint_as_float(hi.x & 0xffff0000u)),
                         pack_pair(x[2] - __uint_as_float(hi.y << 16), x[3] - __uint_as_float(hi.y & 0xffff0000u)));
        }
      }
    };
    auto score = [&](int i) {
      if (MODE == kStates || i >= chunks) return;
      using std::integral_constant;
      if constexpr (TB == 4) {
        if (pw < 3) {
          if constexpr (KDP == 64) {
            score_blocks(i, integral_constant<int, 3>{}, 3 - pw, 0, 3 - pw, 1, pw == 2 ? 0 : 3 - pw, pw == 2 ? 0 : 2);
          } else {
            score_blocks(i, integral_constant<int, 2>{}, 3 - pw, 0, 3 - pw, 1, 0, 0);
            score_blocks(i, integral_constant<int, 1>{}, pw == 2 ? 0 : 3 - pw, pw == 2 ? 0 : 2, 0, 0, 0, 0);
          }
        } else score_blocks(i, integral_constant<int, 1>{}, 3, 3, 0, 0, 0, 0);
      } else {
        if (pw < 3) score_blocks(i, integral_constant<int, 1>{}, pw > 0, pw > 1, 0, 0, 0, 0);
      }
    };
    if (chunks > 0) {
      fetch(r0, 0);
      fetch(r1, 1);
      place(r0, 0);
      decays(r0, 0);
      fetch(r0, 2);
      decays(r1, 1);
      __syncthreads();
      score(0);
      __syncthreads();
      // at the top of step i: chunk i is in the tiles and in P; chunks i + 1 (in r) and i + 2 (in the other set) are in
      // registers or under way
      constexpr bool kLate = MODE != kForward;
      auto step = [&](Regs& r, const Regs& other, int i) {
        place(r, i + 1);
        if (!kLate) fetch(r, i + 3);
        __syncthreads();
        if (kLate) fetch(r, i + 3);
        score(i + 1);
        decays(other, i + 2);
        __syncthreads();
      };
      for (int i = 0; i < chunks; i += 2) {
        step(r1, r0, i);
        step(r0, r1, i + 1);
      }
    } else {  // no chunk to bring (and maybe no inverses to read): the state waves' two barriers
      __syncthreads();
      __syncthreads();
    }
    if (kOut && piece == p.n_segs - 1) {  // rows behind the length are zero
      const int cols = std::min(VT, p.Dv - v0);
      for (int64_t t = n + pw; t < p.L; t += 4) {
        T* y = static_cast<T*>(p.y) + ((bi * p.L + t) * p.H + h) * p.Dv + v0;
        for (int j = l; j < cols; j += kWave) store_elem(y + j, 0.f);
      }
    }
    return;
  }

  // -------------------------------------------------------------------- the state
  const int vw = 16 * NT * wv;  // the wave's first column of the tile
  f32x4 S[MT][NT];
  if (!PART && piece > 0) {
    const float* init = p.part_own + (bh * p.n_parts + piece * p.parts - 1) * p.KP * p.VP;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int v = v0 + vw + 16 * j + lr;
        const float4 x = 16 * m < p.KP && v < p.VP ? lds4(init + (m * p.VP + v) * 16 + g4) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[m][j] = f32x4{x.x, x.y, x.z, x.w};
      }
  } else {
    const float* init = !PART && p.init ? p.init + bh * p.Dk * p.Dv : nullptr;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int i = 16 * m + g4 + r, v = v0 + vw + 16 * j + lr;
          S[m][j][r] = unit ? (i == v ? 1.f : 0.f) : init && i < p.Dk && v < p.Dv ? init[i * p.Dv + v] : 0.f;
        }
  }
  constexpr int kN3 = Parts<T, 3>::kN, kN2 = Parts<T, 2>::kN;
  Frag<T> kf[2][TB], qf[2][TB];
  auto read_rows = [&](int i, int kk) {  // 32 elements of the i-th chunk's keys (and queries)
#pragma unroll
    for (int tt = 0; tt < TB; tt++) {
      const T* kt = sh.k[i & 1] + (16 * tt + lr) * ldk + 32 * kk + g4;
      kf[kk % 2][tt] = pair_frag(kt, kt + 16);
      if constexpr (kOut) {
        const T* qt = sh.q[i & 1] + (16 * tt + lr) * ldq + 32 * kk + g4;
        qf[kk % 2][tt] = pair_frag(qt, qt + 16);
      }
    }
  };
  // outputs: a lane has 4 columns of the tokens 16 tt + lane % 16
  const int yrow = p.H * p.Dv, yoff = (lr * yrow + vw + g4) * int(sizeof(T));
  T* ybase = kOut ? static_cast<T*>(p.y) + (bi * p.L * p.H + h) * p.Dv + v0 : nullptr;
  __builtin_amdgcn_s_setprio(2);  // before the wave beside it, whose work is not waited for step by step
  __syncthreads();
  __syncthreads();
  read_rows(0, 0);
  for (int i = 0; i < chunks; i++) {
    const int c = chunk_of(i), nv = std::min(kC, n - c * kC);
    const Decays<kC>& d = sh.d[i & 3];
    const float* beta = sh.beta[i & 3];
    const T* Qs = sh.q[i & 1];
    const T* Ks = sh.k[i & 1];
    const T* Vs = sh.v[i & 1];
    // ---- the state's answers for the keys (and, transposed, for the queries): reads a step ahead of their products ----
    f32x4 x[TB][NT], o[TB][NT];
#pragma unroll
    for (int tt = 0; tt < TB; tt++)
#pragma unroll
      for (int j = 0; j < NT; j++) x[tt][j] = o[tt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto times_state = [&](int kk) {
      Parts<T, 3> s[NT];
#pragma unroll
      for (int j = 0; j < NT; j++) s[j].set(S[2 * kk][j], S[2 * kk + 1][j]);
#pragma unroll
      for (int e = 0; e < kN3; e++)
#pragma unroll
        for (int tt = 0; tt < TB; tt++)
#pragma unroll
          for (int j = 0; j < NT; j++) {
            x[tt][j] = mma(kf[kk % 2][tt], s[j].f[e], x[tt][j]);
            if constexpr (kOut)
              if (e < kN2) o[tt][j] = mma(s[j].f[e], qf[kk % 2][tt], o[tt][j]);
          }
    };
#pragma unroll
    for (int kk = 0; kk + 1 < KS; kk++) {
      read_rows(i, kk + 1);
      __builtin_amdgcn_sched_barrier(0);
      times_state(kk);
      if constexpr (kTwo) interleave<14, kOut ? 20 : 12, kOut ? 2 : 3>();
      __builtin_amdgcn_sched_barrier(0);
    }
    Frag<T> zf[2][kTri], pf[kTri][kN2], yf[kBack ? kSteps : 1][NT];
    f32x4 vq[kBack ? 1 : TB][NT];
    float w4[TB][4], b4[TB][4];
    auto read_z = [&](int e) {
#pragma unroll
      for (int f = 0; f < kTri; f++) zf[e % 2][f] = row_frag(sh.z[i & 1][e] + f * 512 + l * 8);
    };
    auto read_p = [&]() {
#pragma unroll
      for (int f = 0; f < kTri; f++)
#pragma unroll
        for (int e = 0; e < kN2; e++) pf[f][e] = row_frag(sh.P[i & 1][e] + f * 512 + l * 8);
    };
#pragma unroll
    for (int tt = 0; tt < TB; tt++) {
      const float4 a = lds4((kBack ? d.out : d.in) + 16 * tt + g4), be = lds4(beta + 16 * tt + g4);
      w4[tt][0] = a.x; w4[tt][1] = a.y; w4[tt][2] = a.z; w4[tt][3] = a.w;
      b4[tt][0] = be.x; b4[tt][1] = be.y; b4[tt][2] = be.z; b4[tt][3] = be.w;
    }
    if constexpr (kBack) {
#pragma unroll
      for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
        for (int j = 0; j < NT; j++) yf[ks][j] = col_pair(Vs, ldv, 32 * ks + g4, vw + 16 * j);
      read_p();
    } else {
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++) vq[tt][j] = quad_rows(Vs, ldv, 16 * tt + g4, vw + 16 * j);
      read_z(0);
    }
    times_state(KS - 1);
    if constexpr (MODE != kForward && !PART) {  // what delta_grad_kernel reads: the state entering the chunk, or the gradient leaving it
      float* to = p.states + (bh * p.n_chunks + c) * int64_t(p.KP) * p.VP;
#pragma unroll
      for (int m = 0; m < MT; m++)
#pragma unroll
        for (int j = 0; j < NT; j++) {
          const int v = v0 + vw + 16 * j + lr;
          if (16 * m < p.KP && v < p.VP)
            *reinterpret_cast<float4*>(to + (m * p.VP + v) * 16 + g4) = make_float4(S[m][j][0], S[m][j][1], S[m][j][2], S[m][j][3]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    // ---- R, or dU ----
    if constexpr (kBack) {
      read_z(0);
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) x[tt][j][r] *= w4[tt][r];
#pragma unroll
      for (int e = 0; e < kN2; e++)
#pragma unroll
        for (int ks = kSteps - 1; ks >= 0; ks--)
#pragma unroll
          for (int sb = 0; sb < TB; sb++)
            if (sb / 2 <= ks)
#pragma unroll
              for (int j = 0; j < NT; j++) x[sb][j] = mma(pf[upper_frag<TB>(sb, ks)][e], yf[ks][j], x[sb][j]);
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) x[tt][j][r] = fmaf(-w4[tt][r], x[tt][j][r], vq[tt][j][r]);
    }
    // A row that is not finite must not meet Z's zeros: the rows before it would be no numbers.  From it on N is NaN, and so
    // are the outputs and the state's column.
    int first[NT] = {};
    bool bad = false;
    if constexpr (!kBack) {
      float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) z[r] = fmaf(x[tt][j][r], 0.f, z[r]);
      bad = __ballot(!((z[0] + z[1]) + (z[2] + z[3]) == 0.f)) != 0;
#pragma unroll
      for (int j = 0; j < NT; j++) first[j] = kC;
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
#pragma unroll
          for (int tt = TB - 1; tt >= 0; tt--)
#pragma unroll
            for (int r = 3; r >= 0; r--)
              if (!(x[tt][j][r] * 0.f == 0.f)) {
                first[j] = 16 * tt + g4 + r;
                x[tt][j][r] = 0.f;
              }
          first[j] = std::min(first[j], __shfl_xor(first[j], 16));
          first[j] = std::min(first[j], __shfl_xor(first[j], 32));
        }
      }
    }
    // ---- N = Z R, or dR = Z^T beta dU ----
    f32x4 nn[TB][NT];
#pragma unroll
    for (int tt = 0; tt < TB; tt++)
#pragma unroll
      for (int j = 0; j < NT; j++) nn[tt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    {
      Parts<T, 3> xf[kSteps][NT];
#pragma unroll
      for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
        for (int j = 0; j < NT; j++) xf[ks][j].set(x[2 * ks][j], x[2 * ks + 1][j]);
      auto times = [&](int ea, int eb) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
          for (int tt = 0; tt < TB; tt++)
            if (kBack ? tt / 2 <= ks : ks <= tt / 2)
#pragma unroll
              for (int j = 0; j < NT; j++)
                nn[tt][j] = mma(zf[ea % 2][kBack ? upper_frag<TB>(tt, ks) : lower_frag<TB>(tt, ks)], xf[ks][j].f[eb], nn[tt][j]);
      };
      if constexpr (kTwo) {  // Z's parts in the order 0, 1, 2 and each read while the one before is multiplied
        read_z(1);
        __builtin_amdgcn_sched_barrier(0);
        times(0, 0);
        times(0, 1);
        times(0, 2);
        interleave<28, 18, 4>();
        __builtin_amdgcn_sched_barrier(0);
        read_z(2);
        times(1, 0);
        times(1, 1);
        __builtin_amdgcn_sched_barrier(0);
        times(2, 0);
      } else {
        times(0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // the keys (and queries) as the state's update reads them, for 32 of its rows, a step ahead
    Frag<T> kc[2][2][kSteps], qc[2][2][kSteps];
    auto read_cols = [&](int step) {
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int ks = 0; ks < kSteps; ks++) {
          kc[step % 2][m][ks] = col_pair(Ks, ldk, 32 * ks + g4, 16 * (2 * step + m));
          if constexpr (kBack) qc[step % 2][m][ks] = col_pair(Qs, ldq, 32 * ks + g4, 16 * (2 * step + m));
        }
    };
    if constexpr (kOut) read_p();
    read_cols(0);
    float in[kOut ? TB : 1];
    if constexpr (kOut) {
#pragma unroll
      for (int tt = 0; tt < TB; tt++) in[tt] = d.in[16 * tt + lr] * p.scale;
    }
#pragma unroll
    for (int tt = 0; tt < TB; tt++) {
      const float4 a = lds4((kBack ? d.in : d.out) + 16 * tt + g4);
      w4[tt][0] = a.x; w4[tt][1] = a.y; w4[tt][2] = a.z; w4[tt][3] = a.w;
    }
    const float all = d.all;
    __syncthreads();  // the middle of a step: the other waves have the next chunk in its tiles
    if constexpr (MODE != kForward && !PART) {
      float* to = p.left + (bh * p.n_chunks + c) * int64_t(kC) * p.VP;
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++) {
          const int v = v0 + vw + 16 * j + lr;
          float u[4];
#pragma unroll
          for (int r = 0; r < 4; r++) u[r] = bad && 16 * tt + g4 + r >= first[j] ? __builtin_nanf("") : nn[tt][j][r];
          if (v < p.VP) *reinterpret_cast<float4*>(to + (tt * p.VP + v) * 16 + g4) = make_float4(u[0], u[1], u[2], u[3]);
        }
    }
    // U, in the products' parts: as it is for the outputs, with its decay for the state; backwards the two rows that the
    // state's gradient takes, of dR and of dY
    Parts<T, 3> wf[kSteps][NT], wy[kBack ? kSteps : 1][NT];
    Parts<T, 2> uf[kOut ? kSteps : 1][NT];
#pragma unroll
    for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        float u[8];
        if constexpr (kBack) {
          float yv[8];
          frag_floats(yf[ks][j], yv);
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int tt = 2 * ks + e / 4;
            u[e] = -nn[tt][j][e % 4] * (w4[tt][e % 4] * b4[tt][e % 4]);
            yv[e] *= w4[tt][e % 4] * p.scale;
          }
          wy[ks][j].set(yv);
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int tt = 2 * ks + e / 4;
            u[e] = nn[tt][j][e % 4] * b4[tt][e % 4];
          }
          if constexpr (kOut) uf[ks][j].set(u);
#pragma unroll
          for (int e = 0; e < 8; e++) u[e] *= w4[2 * ks + e / 4][e % 4];
        }
        wf[ks][j].set(u);
      }
    if constexpr (kOut) {
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) o[tt][j][r] *= in[tt];
#pragma unroll
      for (int ea = 0; ea < kN2; ea++)
#pragma unroll
        for (int eb = 0; ea + eb < kN2; eb++)
#pragma unroll
          for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
            for (int tt = 0; tt < TB; tt++)
              if (ks <= tt / 2)
#pragma unroll
                for (int j = 0; j < NT; j++) o[tt][j] = mma(uf[ks][j].f[ea], pf[lower_frag<TB>(tt, ks)][eb], o[tt][j]);
      if constexpr (kTwo) interleave<60, 18, 6>();
    }
    __builtin_amdgcn_sched_barrier(0);
    // ---- the state after the chunk, 32 of its rows at a time ----
    auto update = [&](int step) {
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) S[2 * step + m][j][r] *= all;
#pragma unroll
      for (int e = 0; e < kN3; e++)
#pragma unroll
        for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
          for (int m = 0; m < 2; m++)
#pragma unroll
            for (int j = 0; j < NT; j++) {
              f32x4& to = S[2 * step + m][j];
              to = mma(kc[step % 2][m][ks], wf[ks][j].f[e], to);
              if constexpr (kBack) to = mma(qc[step % 2][m][ks], wy[ks][j].f[e], to);
            }
    };
#pragma unroll
    for (int step = 0; step + 1 < KS; step++) {
      read_cols(step + 1);
      __builtin_amdgcn_sched_barrier(0);
      update(step);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (i + 1 < chunks) read_rows(i + 1, 0);
    update(KS - 1);
    if constexpr (kOut) {
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) {
            const int at = __shfl(first[j], g4 + r);
#pragma unroll
            for (int tt = 0; tt < TB; tt++) o[tt][j][r] = 16 * tt + lr >= at ? __builtin_nanf("") : o[tt][j][r];
          }
      }
      const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(ybase + int64_t(c) * kC * yrow);
#pragma unroll
      for (int tt = 0; tt < TB; tt++) {
        const bool row = 16 * tt + lr < nv;
#pragma unroll
        for (int j = 0; j < NT; j++) {
          const int so = (16 * tt * yrow + 16 * j) * int(sizeof(T)), left = p.Dv - v0 - vw - 16 * j - g4;
          if constexpr (VEC) {
            const int at = row && left > 0 ? yoff : 0x7fffffff;
            if constexpr (kTwo) {
              typedef uint32_t u2 __attribute__((ext_vector_type(2)));
              __builtin_amdgcn_raw_buffer_store_b64(u2{pack_pair(o[tt][j][0], o[tt][j][1]), pack_pair(o[tt][j][2], o[tt][j][3])}, rs, at, so, 0);
            } else {
              typedef uint32_t u4 __attribute__((ext_vector_type(4)));
              __builtin_amdgcn_raw_buffer_store_b128(u4{__float_as_uint(o[tt][j][0]), __float_as_uint(o[tt][j][1]), __float_as_uint(o[tt][j][2]),
                                                        __float_as_uint(o[tt][j][3])}, rs, at, so, 0);
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; r++) buf_store(rs, row && r < left ? yoff + r * int(sizeof(T)) : 0x7fffffff, so, o[tt][j][r], static_cast<T*>(nullptr));
          }
        }
      }
    }
    if constexpr (!kBack) {
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int r = 0; r < 4; r++) S[m][j][r] = first[j] < kC ? __builtin_nanf("") : S[m][j][r];
      }
    }
    __syncthreads();
  }
  if (chunks % 2) {  // the staging waves' steps go by twos
    __syncthreads();
    __syncthreads();
  }
  if constexpr (PART) {
    const int VP = unit ? p.KP : p.VP;
    float* to = (unit ? p.part_map : p.part_own) + (bh * p.n_parts + piece) * p.KP * int64_t(VP);
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int v = v0 + vw + 16 * j + lr;
        if (16 * m < p.KP && v < VP)
          *reinterpret_cast<float4*>(to + (m * VP + v) * 16 + g4) = make_float4(S[m][j][0], S[m][j][1], S[m][j][2], S[m][j][3]);
      }
  } else if (p.last && piece == p.n_segs - 1) {
    float* last = p.last + bh * p.Dk * p.Dv;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int i = 16 * m + g4 + r, v = v0 + vw + 16 * j + lr;
          if (i < p.Dk && v < p.Dv) last[i * p.Dv + v] = S[m][j][r];
        }
  }
}

// ---------------------------------------------------------------------------
// The states leaving the parts of a cut sequence, one after the other: S = map S + own, 16 columns a workgroup, a quarter of
// the rows a wave, in float products.  The state goes through LDS, the next part's map is under way meanwhile.  Bound by the
// length of the chain: b1 L32768 H40 D128 42 us.
// ---------------------------------------------------------------------------
template <int KDP>
__global__ __launch_bounds__(kThreads) void delta_chain_kernel(Rule p) {
  constexpr int MT = KDP / 16, MW = MT / 4;
  __shared__ f32x4 S[2][MT][kWave];
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = threadIdx.x % kWave, lr = l % 16, g4 = 4 * (l / 16);
  const int blocks = p.KP / 16;
  const int64_t bh = blockIdx.x / (p.VP / 16);
  const int v = int(blockIdx.x % (p.VP / 16)) * 16 + lr;
  const float* init = p.init ? p.init + bh * p.Dk * p.Dv : nullptr;
#pragma unroll
  for (int k = 0; k < MW; k++) {
    f32x4 x;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int i = 16 * (wv * MW + k) + g4 + r;
      x[r] = init && i < p.Dk && v < p.Dv ? init[i * p.Dv + v] : 0.f;
    }
    S[0][wv * MW + k][l] = x;
  }
  float4 a[MW][MT], own[MW];
  auto fetch = [&](int part) {
    const float* from = p.part_own + (bh * p.n_parts + part) * p.KP * p.VP + v * 16 + g4;
    const float* map = p.part_map + (bh * p.n_parts + part) * p.KP * p.KP + lr;
#pragma unroll
    for (int k = 0; k < MW; k++) {
      const int m = std::min(wv * MW + k, blocks - 1);  // rows behind the state's: read again, not written
      own[k] = lds4(from + m * p.VP * 16);
#pragma unroll
      for (int kb = 0; kb < MT; kb++) {
        const float* at = map + (m * p.KP + 16 * std::min(kb, blocks - 1) + g4) * 16;
        a[k][kb] = make_float4(at[0], at[16], at[32], at[48]);
      }
    }
  };
  fetch(0);
  for (int part = 0; part < p.n_parts; part++) {
    __syncthreads();
    f32x4 x[MT], y[MW][2];
#pragma unroll
    for (int kb = 0; kb < MT; kb++) x[kb] = kb < blocks ? S[part % 2][kb][l] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < MW; k++) {
      y[k][0] = f32x4{own[k].x, own[k].y, own[k].z, own[k].w};
      y[k][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int kb = 0; kb < MT; kb++)
      if (kb < blocks)  // not a product with zero of what may be no number
#pragma unroll
        for (int k = 0; k < MW; k++) y[k][kb % 2] = mma16(a[k][kb], x[kb], y[k][kb % 2]);
    if (part + 1 < p.n_parts) fetch(part + 1);
    float* to = p.part_own + (bh * p.n_parts + part) * p.KP * p.VP + v * 16 + g4;
#pragma unroll
    for (int k = 0; k < MW; k++) {
      const int m = wv * MW + k;
      const f32x4 z = y[k][0] + y[k][1];
      S[(part + 1) % 2][m][l] = z;
      if (m < blocks) *reinterpret_cast<float4*>(to + m * p.VP * 16) = make_float4(z[0], z[1], z[2], z[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// What is a chunk's own of the backward: dq, dk, dv, dbeta and dg from S, D, N and dR.  A workgroup has one chunk of
// `heads` heads that share their q and k, one after the other (so that their dq and dk are summed in registers), eight waves.
// First the products along the values, 32 columns at a time: with the states (a wave has 16 of the keys' elements), and
// dY U^T and dR U^T (a wave has a block or two of them); then, with W and B in LDS, those along the tokens.  Results are
// transposed, so that a lane has consecutive elements of its own token.  S, D, U and dR lie in LDS by columns, as the
// sweeps wrote them, and are read transposed.  Bound by the latency of its loads with few workgroups a CU (one at D128, two at
// D64, by their LDS): b8 L2048 H24 D64 bf16 197 us; b4 L4096 H32 G8 D128 bf16 594, four heads a workgroup.
// ---------------------------------------------------------------------------
struct Grad {
  Rule p;                // v is v, y is dv
  const void* dy;
  const float* S;        // as Rule's states
  const float* D;
  const float* N;        // as Rule's left
  const float* dR;
  void* dq;              // [b, L, H / heads, Dk]: of the streamed type, or (where a group's heads are not one workgroup's) float
  void* dk;
  bool dqk_f32;
  int heads;
  void* dbeta;           // nullable
  void* dg;              // nullable
};

constexpr int kGradWaves = 8;
template <typename T, int KDP>
struct GradLds {
  typedef Shape<T> Z;
  static constexpr int kC = Z::kC, kN = Z::kTwo ? 2 : 1;
  static constexpr int ldw = kC + 16 / int(sizeof(T));
  static constexpr int ldv = 32 + 16 / int(sizeof(T));        // rows of 32 values
  static constexpr int ldt = kC + 32 / int(sizeof(T));        // columns: rows of kC tokens
  static constexpr int lds = KDP + 32 / int(sizeof(T));       // rows of KDP elements of the keys
  __attribute__((aligned(16))) T q[Tile<T, KDP, kQuery>::kElems];
  __attribute__((aligned(16))) T k[Tile<T, KDP, kKey>::kElems];
  union {
    struct {
      __attribute__((aligned(16))) T dy[kC * ldv], u[kN][32 * ldt], r[kN][32 * ldt], S[kN][32 * lds], D[kN][32 * lds];
    } a;
    struct {
      __attribute__((aligned(16))) T W[kN][kC * ldw], B[kN][kC * ldw];
    } b;
  };
  Decays<kC> d;
  __attribute__((aligned(16))) float beta[kC], own[kC];  // own: the part of dR that is beta's own
  __attribute__((aligned(16))) float rows[Z::TB][kC], cols[Z::TB][kC];      // sums of a block's rows and columns
  float dots[KDP / 16][kC], kept[KDP / 16][kC];  // of a token, over 16 of the keys' elements
  __attribute__((aligned(16))) float db[8][kC];  // a token's parts of dbeta
  float gate[kC];
  double sd[kGradWaves];
};

// four floats to a row of an LDS tile, in its parts
__device__ __forceinline__ void put4(const float (&x)[4], float* a, float*) { *reinterpret_cast<float4*>(a) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void put4(const float (&x)[4], bf16_bits* a, bf16_bits* b) {
  const uint2 hi = make_uint2(pack_pair(x[0], x[1]), pack_pair(x[2], x[3]));
  *reinterpret_cast<uint2*>(a) = hi;
  *reinterpret_cast<uint2*>(b) = make_uint2(pack_pair(x[0] - __uint_as_float(hi.x << 16), x[1] - __uint_as_float(hi.x & 0xffff0000u)),
                                            pack_pair(x[2] - __uint_as_float(hi.y << 16), x[3] - __uint_as_float(hi.y & 0xffff0000u)));
}
__device__ __forceinline__ void put1(float x, float* a, float*) { *a = x; }
__device__ __forceinline__ void put1(float x, bf16_bits* a, bf16_bits* b) {
  store_elem(a, x);
  store_elem(b, x - load_elem(a));
}
// four consecutive elements of a row in memory, of which `left` are inside
template <typename T>
__device__ __forceinline__ void store4(T* to, const float (&x)[4], int left, bool vec) {
  if (vec) {
    if (left <= 0) return;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<uint2*>(to) = make_uint2(pack_pair(x[0], x[1]), pack_pair(x[2], x[3]));
  } else {
#pragma unroll
    for (int r = 0; r < 4; r++)
      if (r < left) store_elem(to + r, x[r]);
  }
}
__device__ __forceinline__ void store8(bf16_bits* to, const bf16x8& x) { *reinterpret_cast<bf16x8*>(to) = x; }
__device__ __forceinline__ void store8(float* to, const f32x8& x) {
  reinterpret_cast<float4*>(to)[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}

// x and that of the lane 16 or 32 away, added
__device__ __forceinline__ float add_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// x and that of the lane N places on in its row of 16, added
template <int N>
__device__ __forceinline__ float add_ror(float x) {
  return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(x)), 0x120 + N, 0xF, 0xF, false));
}
// One step of a running sum over the lanes that starts again where `cut` is
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(double& x, int& cut) {
  const double before = dpp_or_zero<CTRL, ROWS>(x);
  const int c = __builtin_amdgcn_update_dpp(0, cut, CTRL, ROWS, 0xF, false);
  x += cut ? 0.0 : before;
  cut |= c;
}
__device__ __forceinline__ void running_sum(double& x, int cut) {
  scan_step<0x111, 0xF>(x, cut);
  scan_step<0x112, 0xF>(x, cut);
  scan_step<0x114, 0xF>(x, cut);
  scan_step<0x118, 0xF>(x, cut);
  scan_step<0x142, 0xA>(x, cut);
  scan_step<0x143, 0xC>(x, cut);
}
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u)), kWave - 1));
  const uint64_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u >> 32)), kWave - 1));
  return __builtin_bit_cast(double, (hi << 32) | lo);
}

template <typename T, int KDP, bool MULTI, bool VEC>
__global__ __launch_bounds__(kGradWaves * kWave) __attribute__((amdgpu_waves_per_eu(KDP == 64 ? 4 : 2)))
void delta_grad_kernel(Grad a) {
  typedef Shape<T> Z;
  typedef GradLds<T, KDP> Lds;
  constexpr int kC = Z::kC, TB = Z::TB, kSteps = Z::kSteps, KS = KDP / 32, MT = KDP / 16, kAll = kGradWaves * kWave;
  constexpr int TT = TB * MT / kGradWaves;  // blocks of tokens a wave has
  constexpr int ldq = Tile<T, KDP, kQuery>::ld, ldk = Tile<T, KDP, kKey>::ld, ldv = Lds::ldv, ldt = Lds::ldt, lds = Lds::lds, ldw = Lds::ldw;
  constexpr int kN = Lds::kN, NB = TB == 4 ? 2 : 1;  // blocks of W and B a wave has, at most
  const Rule& p = a.p;
  __shared__ Lds sh;
  const int sets = p.H / a.heads;  // sets of heads of one workgroup
  const int64_t units = p.b * sets * p.n_chunks, wg = blockIdx.x;
  const int64_t id = units % 8 == 0 ? (wg % 8) * (units / 8) + wg / 8 : wg;
  const int64_t bset = id / p.n_chunks, bi = bset / sets;
  const int c = int(id % p.n_chunks), set = int(bset % sets), n = live_length(p.lengths, bi, p.L), G = p.H / p.share;
  const int h0 = set * a.heads, gr = h0 / p.share;
  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid / kWave), l = tid % kWave;
  const int lr = l % 16, g4 = 4 * (l / 16);
  const int64_t t0 = int64_t(c) * kC, row0 = bi * p.L + t0;
  const int nv = std::max(0, std::min(kC, int(n - t0))), rows = int(std::min<int64_t>(kC, p.L - t0));
  auto zero_rows = [&](void* x, bool f32, int heads, int hh, int D, int from) {
    for (int j = tid; j < (rows - from) * D; j += kAll) {
      const int64_t at = ((row0 + from + j / D) * heads + hh) * D + j % D;
      if (f32) static_cast<float*>(x)[at] = 0.f;
      else store_elem(static_cast<T*>(x) + at, 0.f);
    }
  };
  if (nv < rows) {  // behind the length
    zero_rows(a.dq, a.dqk_f32, sets, set, p.Dk, nv);
    zero_rows(a.dk, a.dqk_f32, sets, set, p.Dk, nv);
    for (int h = h0; h < h0 + a.heads; h++) {
      zero_rows(p.y, false, p.H, h, p.Dv, nv);
      if (a.dbeta) zero_rows(a.dbeta, false, p.H, h, 1, nv);
      if (a.dg) zero_rows(a.dg, false, p.H, h, 1, nv);
    }
  }
  if (nv == 0) return;
  // waves 0..3 bring q, the others k
  const bool brings_q = wv < 4;
  constexpr int kRowsPieces = Tile<T, KDP, kQuery>::kPieces;
  static_assert(kRowsPieces == Tile<T, KDP, kKey>::kPieces, "q and k come alike");
  uint4 rqk[kRowsPieces];
  {
    Stage<T, KDP, kQuery, VEC> st;
    st.init(static_cast<const T*>(brings_q ? p.q : p.k) + (row0 * G + gr) * p.Dk, G * p.Dk, p.Dk, false, tid % kThreads);
    st.load(rqk, nv, tid % kThreads);
  }
  const int ib = wv % MT, tb0 = wv / MT * TT;  // the wave's 16 elements of the keys, and its first block of tokens
  const int n_blocks = TB * (TB + 1) / 2;
  int tbs[NB], sbs[NB];
#pragma unroll
  for (int j = 0; j < NB; j++) {
    int tb = 0, sb = std::min(wv + j * kGradWaves, n_blocks - 1);
    while (sb > tb) sb -= ++tb;
    tbs[j] = tb;
    sbs[j] = sb;
  }
  f32x4 sum_q[MULTI ? TT : 1], sum_k[MULTI ? TT : 1];
  if constexpr (MULTI)
#pragma unroll
    for (int j = 0; j < TT; j++) sum_q[j] = sum_k[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto store_qk = [&](int tt, const f32x4& dq, const f32x4& dk) {
    const int t = 16 * (tb0 + tt) + lr, i = 16 * ib + g4;
    if (t >= nv) return;
    const int64_t at = ((row0 + t) * sets + set) * p.Dk + i;
    const float x[4] = {dq[0], dq[1], dq[2], dq[3]}, y[4] = {dk[0], dk[1], dk[2], dk[3]};
    if (a.dqk_f32) {
      store4(static_cast<float*>(a.dq) + at, x, p.Dk - i, VEC);
      store4(static_cast<float*>(a.dk) + at, y, p.Dk - i, VEC);
    } else {
      store4(static_cast<T*>(a.dq) + at, x, p.Dk - i, VEC);
      store4(static_cast<T*>(a.dk) + at, y, p.Dk - i, VEC);
    }
  };

  // what a thread brings of 32 columns: a piece of dY's rows, four tokens of one column of N and dR, four of the keys'
  // elements of one column of S and D
  constexpr int kVec = 16 / int(sizeof(T)), kRowPieces = 32 / kVec;           // pieces of a row of dY
  constexpr int kDy = (kC * kRowPieces + kAll - 1) / kAll;
  constexpr int kLeft = kC * 8;                                                // float4 pieces of N, of dR
  constexpr int kStates = KDP * 8 / kAll;                                      // of S, of D, a thread
  struct Regs {
    uint4 dy[kDy];
    float4 n, r, S[kStates], D[kStates];
    uint32_t gate, beta;
  };
  Regs r;

#pragma unroll 1
  for (int h = h0; h < h0 + (MULTI ? a.heads : 1); h++) {
    // Over the heads neither what is read of q and k nor the lane's places in the tiles are kept: there are no registers
    int tid_here = threadIdx.x;
    if constexpr (MULTI) asm volatile("" : "+v"(tid_here) : : "memory");
    const int tid = tid_here, l = tid % kWave, lr = l % 16, g4 = 4 * (l / 16), g8 = 8 * (l / 16);
    const bool has_left = tid < kLeft;
    const int lt = tid % 4 * 4 + tid / 128 * 16, lv = tid / 4 % 32;  // a thread's tokens and column of N and dR
    // 32 columns of head hh from v0 on, through descriptors: what lies outside is zero, and no branch is around a load
    auto fetch = [&](int hh, int v0) {
      const int64_t at_chunk = (bi * p.H + hh) * p.n_chunks + c;
      const T* gY = static_cast<const T*>(a.dy) + (row0 * p.H + hh) * p.Dv;
      const __amdgpu_buffer_rsrc_t ry = uniform_rsrc(gY), rn = uniform_rsrc(a.N + at_chunk * kC * p.VP), rr = uniform_rsrc(a.dR + at_chunk * kC * p.VP);
      const __amdgpu_buffer_rsrc_t rS = uniform_rsrc(a.S + at_chunk * p.KP * p.VP), rD = uniform_rsrc(a.D + at_chunk * p.KP * p.VP);
      auto load = [](const __amdgpu_buffer_rsrc_t& rs, int at) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
        return make_uint4(v[0], v[1], v[2], v[3]);
      };
      auto quad = [&](const __amdgpu_buffer_rsrc_t& rs, int at) { return __builtin_bit_cast(float4, load(rs, at)); };
#pragma unroll
      for (int j = 0; j < kDy; j++) {
        const int i = tid + j * kAll, t = i / kRowPieces, v = v0 + kVec * (i % kRowPieces);
        if constexpr (VEC) {
          r.dy[j] = load(ry, t < nv && v < p.Dv ? (t * p.H * p.Dv + v) * int(sizeof(T)) : 0x7fffffff);
        } else {
          r.dy[j] = make_uint4(0, 0, 0, 0);
          if (t < nv && v < p.Dv) {
            const T* from = gY + int64_t(t) * p.H * p.Dv + v;
            T x[kVec];
#pragma unroll
            for (int e = 0; e < kVec; e++) x[e] = v + e < p.Dv ? from[e] : T(0);
            __builtin_memcpy(&r.dy[j], x, 16);
          }
        }
      }
      const int at = has_left && v0 + lv < p.VP ? 4 * ((lt / 16 * p.VP + v0 + lv) * 16 + lt % 16) : 0x7fffffff;
      r.n = quad(rn, at);
      r.r = quad(rr, at);
#pragma unroll
      for (int j = 0; j < kStates; j++) {
        const int i = tid + j * kAll, e = i % 4 * 4 + i / 128 * 16, v = v0 + i / 4 % 32;
        const int so = e < p.KP && v < p.VP ? 4 * ((e / 16 * p.VP + v) * 16 + e % 16) : 0x7fffffff;
        r.S[j] = quad(rS, so);
        r.D[j] = quad(rD, so);
      }
      if (v0 == 0) {  // a head's first
        r.gate = Scalars<T, kC>::load_at(p.g, (row0 * p.H + hh), p.H, nv);
        r.beta = Scalars<T, kC>::load_at(p.beta, (row0 * p.H + hh), p.H, nv);
      }
    };
    if (h == h0) fetch(h, 0);
    const float gate = l < nv ? clamp_log(Scalars<T, kC>::value(r.gate) + (p.A ? p.A[h] : 0.f)) : 0.f;
    const float beta = l < nv ? p.beta ? Scalars<T, kC>::value(r.beta) : 1.f : 0.f;
    if (wv == 0) {
      fill_decays(sh.d, gate, 1.f);
      if (l < kC) sh.gate[l] = gate;
    } else if (wv == 1 && l < kC) {
      sh.beta[l] = beta;
      sh.own[l] = beta / moved_beta(beta);
    }
    if (h == h0) {
      if (brings_q) Stage<T, KDP, kQuery, VEC>::store(sh.q, rqk, tid);
      else Stage<T, KDP, kKey, VEC>::store(sh.k, rqk, tid - kThreads);
    }
    f32x4 fq[TT], fk[TT], tk[TT], wu[NB], bu[NB];
#pragma unroll
    for (int j = 0; j < TT; j++) fq[j] = fk[j] = tk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NB; j++) wu[j] = bu[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    double sd = 0.0;
    float db[4] = {0.f, 0.f, 0.f, 0.f};  // the part of dbeta that this thread's columns give
    __syncthreads();
#pragma unroll 1
    for (int v0 = 0; v0 < p.Dv; v0 += 32) {
      if (v0) __syncthreads();
#pragma unroll
      for (int j = 0; j < kDy; j++) {
        const int i = tid + j * kAll;
        if (i < kC * kRowPieces) *reinterpret_cast<uint4*>(sh.a.dy + i / kRowPieces * ldv + kVec * (i % kRowPieces)) = r.dy[j];
      }
      if (has_left) {
        const float4 be4 = lds4(sh.beta + lt), ow4 = lds4(sh.own + lt);
        const float be[4] = {be4.x, be4.y, be4.z, be4.w}, own[4] = {ow4.x, ow4.y, ow4.z, ow4.w};
        const float x[4] = {r.n.x, r.n.y, r.n.z, r.n.w}, y[4] = {r.r.x, r.r.y, r.r.z, r.r.w};
        float u[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          db[e] = fmaf(x[e], y[e], db[e]);
          u[e] = x[e] * be[e];
          w[e] = y[e] * own[e];
        }
        put4(u, sh.a.u[0] + lv * ldt + lt, sh.a.u[kN - 1] + lv * ldt + lt);
        put4(w, sh.a.r[0] + lv * ldt + lt, sh.a.r[kN - 1] + lv * ldt + lt);
      }
#pragma unroll
      for (int j = 0; j < kStates; j++) {
        const int i = tid + j * kAll, at = i / 4 % 32 * lds + i % 4 * 4 + i / 128 * 16;
        const float x[4] = {r.S[j].x, r.S[j].y, r.S[j].z, r.S[j].w}, y[4] = {r.D[j].x, r.D[j].y, r.D[j].z, r.D[j].w};
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          if constexpr (sizeof(T) == 4) sd = fma(double(x[e]), double(y[e]), sd);
          else s = fmaf(x[e], y[e], s);
        }
        if constexpr (sizeof(T) == 2) sd += double(s);
        put4(x, sh.a.S[0] + at, sh.a.S[kN - 1] + at);
        put4(y, sh.a.D[0] + at, sh.a.D[kN - 1] + at);
      }
      __syncthreads();
      if (v0 + 32 < p.Dv) fetch(h, v0 + 32);
      if (wv < TB) {  // dv: the first part of dR is what rounding leaves of it
        const int t = 16 * wv + lr, v = v0 + g8;
        const Frag<T> f = col_frag(sh.a.r[0], ldt, g8, 16 * wv, 4);
        if (t < nv && v < p.Dv) {
          T* to = static_cast<T*>(p.y) + ((row0 + t) * p.H + h) * p.Dv + v;
          if constexpr (VEC) {
            if (v + 8 <= p.Dv) {
              store8(to, f);
            } else {  // (float) rows of whole 16-byte pieces may end inside the eight
              float x[8];
              frag_floats(f, x);
              const float x4[4] = {x[0], x[1], x[2], x[3]};
              store4(to, x4, p.Dv - v, true);
            }
          } else {
            float x[8];
            frag_floats(f, x);
#pragma unroll
            for (int e = 0; e < 8; e++)
              if (v + e < p.Dv) store_elem(to + e, x[e]);
          }
        }
      }
      {
        Parts<T, 2> sf, df;
#pragma unroll
        for (int e = 0; e < kN; e++) {
          sf.f[e] = col_frag(sh.a.S[e], lds, g8, 16 * ib, 4);
          df.f[e] = col_frag(sh.a.D[e], lds, g8, 16 * ib, 4);
        }
#pragma unroll
        for (int tt = 0; tt < TT; tt++) {
          const Frag<T> yf = row_frag(sh.a.dy + (16 * (tb0 + tt) + lr) * ldv + g8);
          Parts<T, 2> uf, rf;
#pragma unroll
          for (int e = 0; e < kN; e++) {
            uf.f[e] = col_frag(sh.a.u[e], ldt, g8, 16 * (tb0 + tt), 4);
            rf.f[e] = col_frag(sh.a.r[e], ldt, g8, 16 * (tb0 + tt), 4);
            fq[tt] = mma(sf.f[e], yf, fq[tt]);
          }
          fk[tt] = mma_parts(sf, rf, fk[tt]);
          tk[tt] = mma_parts(df, uf, tk[tt]);
          if (tt % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int j = 0; j < NB; j++) {
        if (wv + j * kGradWaves < n_blocks) {
          Parts<T, 2> uf, rf;
          const Frag<T> yf = row_frag(sh.a.dy + (16 * tbs[j] + lr) * ldv + g8);
#pragma unroll
          for (int e = 0; e < kN; e++) {
            uf.f[e] = col_frag(sh.a.u[e], ldt, g8, 16 * sbs[j], 4);
            rf.f[e] = col_frag(sh.a.r[e], ldt, g8, 16 * tbs[j], 4);
            wu[j] = mma(uf.f[e], yf, wu[j]);
          }
          bu[j] = mma_parts(uf, rf, bu[j]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (MULTI && h + 1 < h0 + a.heads) fetch(h + 1, 0);
    // dbeta: a row of 16 lanes has four columns of 16 tokens, four a lane
#pragma unroll
    for (int e = 0; e < 4; e++) db[e] = add_ror<4>(add_ror<8>(db[e]));
    if (has_left && lr < 4) *reinterpret_cast<float4*>(&sh.db[wv % 2 * 4 + l / 16][lt]) = make_float4(db[0], db[1], db[2], db[3]);
    __syncthreads();
    if (a.dbeta && tid < nv) {
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) x += sh.db[j][tid];
      store_elem(static_cast<T*>(a.dbeta) + (row0 + tid) * p.H + h, x / moved_beta(sh.beta[tid]));
    }
    // ---- W and B + B^T, and what they give the gate ----
#pragma unroll
    for (int j = 0; j < NB; j++) {
      if (wv + j * kGradWaves >= n_blocks) continue;
      const int tb = tbs[j], sb = sbs[j], t = 16 * tb + lr, s0 = 16 * sb + g4;
      const float th = sh.d.hi[t], tl = sh.d.lo[t];
      float w[4], b[4];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const float m = exp2_fast((th - sh.d.hi[s0 + r]) + (tl - sh.d.lo[s0 + r]));
        w[r] = s0 + r <= t ? wu[j][r] * m * p.scale : 0.f;
        b[r] = s0 + r < t ? -bu[j][r] * m : 0.f;
      }
      if (a.dg) {
        f32x4 qk{0.f, 0.f, 0.f, 0.f}, kk4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KS; kk++) {
          const Frag<T> kf = row_frag(sh.k + (16 * sb + lr) * ldk + 32 * kk + g8);
          qk = mma(kf, row_frag(sh.q + t * ldq + 32 * kk + g8), qk);
          kk4 = mma(kf, row_frag(sh.k + t * ldk + 32 * kk + g8), kk4);
        }
        float x[4], row = 0.f;
#pragma unroll
        for (int r = 0; r < 4; r++) {
          x[r] = s0 + r < t ? fmaf(w[r], qk[r], b[r] * kk4[r]) : 0.f;
          row += x[r];
        }
        row = add_xor32(add_xor16(row));
        if (l < 16) sh.rows[sb][t] = row;
#pragma unroll
        for (int r = 0; r < 4; r++) x[r] = add_ror<1>(add_ror<2>(add_ror<4>(add_ror<8>(x[r]))));
        if (lr == 0) *reinterpret_cast<float4*>(&sh.cols[tb][s0]) = make_float4(x[0], x[1], x[2], x[3]);
      }
      put4(w, sh.b.W[0] + t * ldw + s0, sh.b.W[kN - 1] + t * ldw + s0);
      __builtin_amdgcn_sched_barrier(0);
      if (tb > sb) {
        put4(b, sh.b.B[0] + t * ldw + s0, sh.b.B[kN - 1] + t * ldw + s0);
#pragma unroll
        for (int r = 0; r < 4; r++) put1(b[r], sh.b.B[0] + (s0 + r) * ldw + t, sh.b.B[kN - 1] + (s0 + r) * ldw + t);
      } else {
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int s = s0 + r;
          if (s <= t) put1(b[r], sh.b.B[0] + t * ldw + s, sh.b.B[kN - 1] + t * ldw + s);
          if (s < t) put1(b[r], sh.b.B[0] + s * ldw + t, sh.b.B[kN - 1] + s * ldw + t);
        }
        if (tb % 2 == 0 && tb + 1 < TB) {  // the block beside the diagonal that the products read
          const float z[4] = {0.f, 0.f, 0.f, 0.f};
          put4(z, sh.b.W[0] + t * ldw + s0 + 16, sh.b.W[kN - 1] + t * ldw + s0 + 16);
        }
      }
    }
    __syncthreads();
    // ---- dq, dk ----
#pragma unroll
    for (int tt = 0; tt < TT; tt++) {
      const int tb = tb0 + tt, t = 16 * tb + lr, i = 16 * ib + g4;
      const float in = sh.d.in[t], out = sh.d.out[t];
      f32x4 dq, dk;
#pragma unroll
      for (int r = 0; r < 4; r++) {
        fq[tt][r] *= in * p.scale;
        fk[tt][r] *= -in;
        tk[tt][r] *= out;
        dq[r] = fq[tt][r];
        dk[r] = fk[tt][r] + tk[tt][r];
      }
      if constexpr (MULTI) {
        dq += sum_q[tt];
        dk += sum_k[tt];
      }
      if (a.dg) {
        const float4 q4 = lds4(sh.q + t * ldq + i), k4 = lds4(sh.k + t * ldk + i);
        const float qv[4] = {q4.x, q4.y, q4.z, q4.w}, kv[4] = {k4.x, k4.y, k4.z, k4.w};
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int r = 0; r < 4; r++) {
          x = fmaf(qv[r], fq[tt][r], fmaf(kv[r], fk[tt][r], x));
          y = fmaf(kv[r], tk[tt][r], y);
        }
        x = add_xor32(add_xor16(x));
        y = add_xor32(add_xor16(y));
        if (l < 16) {
          sh.dots[ib][t] = x;
          sh.kept[ib][t] = y;
        }
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ks++) {
        const Frag<T> kf = col_frag(sh.k, ldk, 32 * ks + g8, 16 * ib, 4);
        if (ks <= tb / 2) {
#pragma unroll
          for (int e = 0; e < kN; e++) dq = mma(kf, row_frag(sh.b.W[e] + t * ldw + 32 * ks + g8), dq);
        }
        if (ks >= tb / 2) {
          const Frag<T> qf = col_frag(sh.q, ldq, 32 * ks + g8, 16 * ib, 4);
#pragma unroll
          for (int e = 0; e < kN; e++) dk = mma(qf, col_frag(sh.b.W[e], ldw, 32 * ks + g8, 16 * tb, 4), dk);
        }
#pragma unroll
        for (int e = 0; e < kN; e++) dk = mma(kf, row_frag(sh.b.B[e] + t * ldw + 32 * ks + g8), dk);
      }
      if constexpr (MULTI) {
        sum_q[tt] = dq;
        sum_k[tt] = dk;
      } else {
        store_qk(tt, dq, dk);
      }
      __builtin_amdgcn_sched_barrier(0);  // the next block's reads would not fit in the registers
    }
    if (a.dg) {
      running_sum(sd, 0);
      if (l == kWave - 1) sh.sd[wv] = sd;
    }
    __syncthreads();  // dots and sums are there; W and B have been read
    // dg: sums from a token on, that start again at a reset; lane l has the l-th token from the last
    if (a.dg && wv == 0) {
      const int t = kWave - 1 - l;
      double x = 0.0, kept = 0.0;
      int reset = 0;
      if (t < nv) {
#pragma unroll
        for (int j = 0; j < MT; j++) {
          x += double(sh.dots[j][t]);
          kept += double(sh.kept[j][t]);
        }
#pragma unroll
        for (int j = 0; j < TB; j++) {
          if (j <= t / 16) x += double(sh.rows[j][t]);
          if (j >= t / 16) x -= double(sh.cols[j][t]);
        }
        x -= kept;
        reset = sh.gate[t] < kZeroLog;
      }
      double all_kept = kept;
      running_sum(all_kept, 0);
      double end = 0.0;
#pragma unroll
      for (int j = 0; j < kGradWaves; j++) end += sh.sd[j];
      end = end * double(sh.d.all) + last_lane(all_kept);
      if (l == 0) x += end;
      if (reset) x = 0.0;
      running_sum(x, reset);
      if (t < nv) store_elem(static_cast<T*>(a.dg) + (row0 + t) * p.H + h, float(x));
    }
    if (MULTI && h + 1 < h0 + a.heads) __syncthreads();  // the small arrays have been read
  }
  if constexpr (MULTI)
#pragma unroll
    for (int tt = 0; tt < TT; tt++) store_qk(tt, sum_q[tt], sum_k[tt]);
}

// ---------------------------------------------------------------------------
// One token: a workgroup holds up to kTile columns of one head's state in registers (NR rows of VEC columns a thread): lanes
// run along its columns, groups of them along its rows.  What the state answers for k and for q is summed over
// the groups at once, in LDS: y = scale (r S^T q + (q . k) u).  The state is read and written once: bound by HBM (b256 H40
// D128 bf16 268 us, 5 TB/s).
// ---------------------------------------------------------------------------
template <typename T, int VEC, int NR>
__global__ __launch_bounds__(256) void delta_update_kernel(Rule p, float* __restrict__ state, int lanes) {
  __shared__ float qs[kMaxDim], ks[kMaxDim], pk[256 * VEC], pq[256 * VEC], kq_part[4];
  const int G = p.H / p.share;
  const int64_t bh = blockIdx.x / p.n_tiles, bi = bh / p.H;
  const int h = int(bh % p.H), c0 = int(blockIdx.x % p.n_tiles) * kTile;
  const int64_t qrow = bi * G + h / p.share;
  const int Dk = p.Dk, Dv = p.Dv;
  T* y = static_cast<T*>(p.y) + bh * Dv;
  if (p.lengths && p.lengths[bi] <= 0) {
    for (int j = c0 + threadIdx.x; j < Dv && j < c0 + kTile; j += 256) store_elem(y + j, 0.f);
    return;
  }
  const int l = threadIdx.x % lanes, r0 = threadIdx.x / lanes, groups = 256 / lanes, c = c0 + l * VEC;
  // the state through a descriptor: one lane offset, rows `groups` apart in steps of a scalar one
  const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(state + bh * Dk * Dv);
  const int at = 4 * (r0 * Dv + c), step = 4 * groups * Dv;
  auto place = [&](int i) { return r0 + i * groups < Dk && c < Dv ? at : 0x7fffffff; };
  float S[NR][VEC];
#pragma unroll
  for (int i = 0; i < NR; i++) {
    if constexpr (VEC == 4) {
      const auto u = __builtin_amdgcn_raw_buffer_load_b128(rs, place(i), i * step, 0);
#pragma unroll
      for (int j = 0; j < 4; j++) S[i][j] = __uint_as_float(u[j]);
    } else {
      S[i][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, place(i), i * step, 0));
    }
  }
  float kq = 0.f;
  if (int(threadIdx.x) < kMaxDim) {
    const int j = threadIdx.x;
    const float q = j < Dk ? load_elem(static_cast<const T*>(p.q) + qrow * Dk + j) : 0.f;
    const float k = j < Dk ? load_elem(static_cast<const T*>(p.k) + qrow * Dk + j) : 0.f;
    qs[j] = q;
    ks[j] = k;
    kq = q * k;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) kq += __shfl_xor(kq, off);
  if (threadIdx.x % kWave == 0) kq_part[threadIdx.x / kWave] = kq;
  const float beta = p.beta ? load_elem(static_cast<const T*>(p.beta) + bh) : 1.f;
  const float dec = expf(clamp_log((p.A ? p.A[h] : 0.f) + (p.g ? load_elem(static_cast<const T*>(p.g) + bh) : 0.f)));
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) v[j] = c + j < Dv ? load_elem(static_cast<const T*>(p.v) + bh * Dv + c + j) : 0.f;
  __syncthreads();
  float ak[VEC], aq[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) ak[j] = aq[j] = 0.f;
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const int r = std::min(r0 + i * groups, kMaxDim - 1);  // rows behind the state's are zero
    if (r0 + i * groups < Dk) {
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        S[i][j] *= dec;
        ak[j] = fmaf(ks[r], S[i][j], ak[j]);
        aq[j] = fmaf(qs[r], S[i][j], aq[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; j++) {
    pk[(r0 * lanes + l) * VEC + j] = ak[j];
    pq[(r0 * lanes + l) * VEC + j] = aq[j];
  }
  __syncthreads();
  float u[VEC], o[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) u[j] = o[j] = 0.f;
  for (int r = 0; r < groups; r++) {
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      u[j] += pk[(r * lanes + l) * VEC + j];
      o[j] += pq[(r * lanes + l) * VEC + j];
    }
  }
  kq = kq_part[0] + kq_part[1];
#pragma unroll
  for (int j = 0; j < VEC; j++) {
    u[j] = beta * (v[j] - u[j]);
    o[j] = fmaf(kq, u[j], o[j]) * p.scale;
  }
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const float k = ks[std::min(r0 + i * groups, kMaxDim - 1)];
    if constexpr (VEC == 4) {
      typedef uint32_t u4 __attribute__((ext_vector_type(4)));
      u4 w;
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = __float_as_uint(fmaf(k, u[j], S[i][j]));
      __builtin_amdgcn_raw_buffer_store_b128(w, rs, place(i), i * step, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(fmaf(k, u[0], S[i][0])), rs, place(i), i * step, 0);
    }
  }
  if (r0 == 0)
#pragma unroll
    for (int j = 0; j < VEC; j++)
      if (c + j < Dv) store_elem(y + c + j, o[j]);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kSumBlocks = int64_t(1) << 22;  // a grid holds less than 2^32 threads: beyond, a thread has several sums
constexpr size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// rows of whole 16-byte pieces, 16-byte aligned
template <typename T>
bool pieces(const void* x, int64_t D) {
  return D % (16 / int(sizeof(T))) == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

// The cut of a sequence.  A CU holds one workgroup of the sweep, so with fewer heads (times tiles of columns) than CUs the
// sequence is cut into segments, whose entering states a pass before gives: the part's own state and its map, Dk columns more.
// Of the cuts into up to 64 segments and 1, 2, 3 or 4 parts each the one whose generations of workgroups take the fewest chunks
// one after the other: a chunk of the pass before counts 3/4 of one of the sweep (measured: bf16, D128, 2.9 and 3.7 us), a step
// of the chain 1/3 or, above 64 elements of the keys, one (it is shorter, but with 1/5 and 2/5 b1 L2048 H32 D128 took 128 us, so 107),
// the launches 3.  Float takes the same counts.  Forward / backward in us, cut and uncut: float b1 L8192 H4 D64 90 / 206 and
// 673 / 1260, b1 L2048 H32 D128 200 / 601 and 288 / 706, b1 L32768 H40 D128 2914 / 9669 and 4534 / 11971, but b4 L1024 H24
// D64, where the counts are nearly even, 103 / 298 and 102 / 270; bf16 b1 L8192 H8 D128 140 / 383 and 480 / 1016.
constexpr int64_t kAtOnce = 256;
struct Cut {
  int n_segs = 1, parts = 1, part_chunks = 1, n_parts = 0;
};
Cut cut_of(const DeltaRuleArgs& a) {
  const int64_t chunks = ceil_div(a.L, a.dtype == 0 ? kChunk<float> : kChunk<bf16_bits>), heads = a.b * a.H;
  const int64_t tiles = ceil_div(a.Dv, kTile), more = tiles + ceil_div(ceil_div(a.Dk, 16) * 16, kTile);
  Cut best;
  best.part_chunks = int(std::max<int64_t>(1, chunks));
  double least = double(ceil_div(heads * tiles, kAtOnce) * chunks);
  if (heads * tiles >= kAtOnce) return best;
  for (int64_t segs = 2; segs <= std::min<int64_t>(64, chunks / 2); segs++)
    for (int64_t parts = 1; parts <= 4; parts++) {
      const int64_t pc = ceil_div(chunks, segs * parts), n = ceil_div(chunks, pc * parts), n_parts = (n - 1) * parts;
      if (n < 2) continue;
      const double cost = double(ceil_div(heads * tiles * n, kAtOnce) * pc * parts) + 0.75 * double(ceil_div(heads * more * n_parts, kAtOnce) * pc) +
                          (a.Dk <= 64 ? 0.35 : 1.0) * double(n_parts) + 3.0;
      if (cost < least) {
        least = cost;
        best.n_segs = int(n); best.parts = int(parts); best.part_chunks = int(pc); best.n_parts = int(n_parts);
      }
    }
  return best;
}

Rule rule_of(const DeltaRuleArgs& a) {
  Rule p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.beta = a.beta; p.g = a.g; p.A = a.A; p.lengths = a.lengths; p.scale = a.scale;
  p.stream = a.stream;
  p.b = a.b; p.L = a.L; p.H = int(a.H); p.share = int(a.H / a.G); p.Dk = int(a.Dk); p.Dv = int(a.Dv);
  p.KP = int(ceil_div(a.Dk, 16) * 16);
  p.VP = int(ceil_div(a.Dv, 16) * 16);
  p.n_chunks = int(ceil_div(a.L, a.dtype == 0 ? kChunk<float> : kChunk<bf16_bits>));
  p.n_tiles = int(ceil_div(a.Dv, kTile));
  const Cut c = cut_of(a);
  p.n_segs = c.n_segs; p.parts = c.parts; p.part_chunks = c.part_chunks; p.n_parts = c.n_parts;
  return p;
}

// Heads of a group that delta_grad_kernel takes one after the other, their dq and dk summed in registers: as many as leave
// the chip two generations of workgroups (a CU holds one or two), so that the others' partial sums, in float, are few.
int heads_together(const DeltaRuleArgs& a, int64_t chunks) {
  const int64_t share = a.H / a.G;
  int64_t heads = share;
  while (heads > 1 && (share % heads || a.b * (a.H / heads) * chunks < 1024)) heads--;
  return int(heads);
}

// Bytes from the workspace's start of its parts.
struct Work {
  size_t lower, upper, own, map, S, D, N, dR, dq, dk, total;
};
Work plan_work(const DeltaRuleArgs& a, bool backward) {
  Work w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += up256(bytes);
    return r;
  };
  const Rule p = rule_of(a);
  const size_t chunks = size_t(a.b) * a.H * p.n_chunks;
  const size_t tri = chunks * (a.dtype == 0 ? Shape<float>::kTri : Shape<bf16_bits>::kTri) * 512 * 4;
  w.lower = take(tri);
  w.own = take(size_t(a.b) * a.H * p.n_parts * p.KP * p.VP * 4);  // one direction after the other
  w.map = take(size_t(a.b) * a.H * p.n_parts * p.KP * p.KP * 4);
  if (backward) {
    const size_t state = chunks * p.KP * p.VP * 4;
    const size_t rows = chunks * (a.dtype == 0 ? kChunk<float> : kChunk<bf16_bits>) * p.VP * 4;
    w.upper = take(tri);
    w.S = take(state);
    w.D = take(state);
    w.N = take(rows);
    w.dR = take(rows);
    const int64_t sets = a.H / heads_together(a, p.n_chunks);
    if (sets != a.G) {
      w.dq = take(size_t(a.b) * a.L * sets * a.Dk * 4);
      w.dk = take(size_t(a.b) * a.L * sets * a.Dk * 4);
    }
  }
  w.total = at;
  return w;
}

template <typename T>
hipError_t run_tri(const Rule& p, float* lower, float* upper) {
  const int64_t blocks = p.b * p.H * p.n_chunks;
  const bool vec = pieces<T>(p.k, p.Dk);
  auto go = [&](auto kern) { return launch_kind(kKindDeltaTri, kern, blocks, kThreads, p.stream, p, lower, upper); };
  if (p.Dk <= 64) return vec ? go(delta_tri_kernel<T, 64, true>) : go(delta_tri_kernel<T, 64, false>);
  return vec ? go(delta_tri_kernel<T, 128, true>) : go(delta_tri_kernel<T, 128, false>);
}

template <typename T, Mode MODE>
hipError_t run_sweep(const Rule& p) {
  const int64_t heads = p.b * p.H;
  const bool vec = pieces<T>(p.q, p.Dk) && pieces<T>(p.k, p.Dk) && pieces<T>(p.v, p.Dv) && (MODE != kForward || pieces<T>(p.y, p.Dv));
  auto go = [&](auto kern, int64_t blocks) { return launch_kind(kKindDeltaSweep, kern, blocks, kThreads + kWave * state_waves(kTile), p.stream, p); };
  if (p.n_segs > 1) {
    constexpr Mode PM = MODE == kForward ? kStates : MODE;
    const int64_t blocks = heads * (p.n_tiles + ceil_div(p.KP, kTile)) * p.n_parts;
    hipError_t err = p.Dk <= 64 ? (vec ? go(delta_sweep_kernel<T, 64, kTile, PM, true, true>, blocks) : go(delta_sweep_kernel<T, 64, kTile, PM, true, false>, blocks))
                                : (vec ? go(delta_sweep_kernel<T, 128, kTile, PM, true, true>, blocks) : go(delta_sweep_kernel<T, 128, kTile, PM, true, false>, blocks));
    if (err != hipSuccess) return err;
    const int64_t tiles = heads * (p.VP / 16);
    err = p.Dk <= 64 ? launch_kind(kKindDeltaChain, delta_chain_kernel<64>, tiles, kThreads, p.stream, p)
                     : launch_kind(kKindDeltaChain, delta_chain_kernel<128>, tiles, kThreads, p.stream, p);
    if (err != hipSuccess) return err;
  }
  const int64_t blocks = heads * p.n_tiles * p.n_segs;
  if (p.Dk <= 64) return vec ? go(delta_sweep_kernel<T, 64, kTile, MODE, false, true>, blocks) : go(delta_sweep_kernel<T, 64, kTile, MODE, false, false>, blocks);
  return vec ? go(delta_sweep_kernel<T, 128, kTile, MODE, false, true>, blocks) : go(delta_sweep_kernel<T, 128, kTile, MODE, false, false>, blocks);
}

template <typename T>
hipError_t run_grad(const Grad& a) {
  const Rule& p = a.p;
  const int64_t blocks = p.b * (p.H / a.heads) * p.n_chunks;
  const bool vec = pieces<T>(p.q, p.Dk) && pieces<T>(p.k, p.Dk) && pieces<T>(a.dy, p.Dv) && pieces<T>(p.y, p.Dv) &&
                   pieces<T>(a.dq, p.Dk) && pieces<T>(a.dk, p.Dk);
  auto go = [&](auto kern) { return launch_kind(kKindDeltaGrad, kern, blocks, kGradWaves * kWave, p.stream, a); };
  auto width = [&](auto multi) {
    constexpr bool M = decltype(multi)::value;
    if (p.Dk <= 64) return vec ? go(delta_grad_kernel<T, 64, M, true>) : go(delta_grad_kernel<T, 64, M, false>);
    return vec ? go(delta_grad_kernel<T, 128, M, true>) : go(delta_grad_kernel<T, 128, M, false>);
  };
  return a.heads > 1 ? width(std::true_type{}) : width(std::false_type{});
}

template <typename T>
hipError_t fwd_impl(const DeltaRuleArgs& a, char* ws) {
  const Work w = plan_work(a, false);
  Rule p = rule_of(a);
  float* lower = reinterpret_cast<float*>(ws + w.lower);
  const hipError_t err = run_tri<T>(p, lower, nullptr);
  if (err != hipSuccess) return err;
  p.tri = lower;
  p.part_own = reinterpret_cast<float*>(ws + w.own);
  p.part_map = reinterpret_cast<float*>(ws + w.map);
  p.init = a.h0;
  p.y = a.y;
  p.last = a.last;
  return run_sweep<T, kForward>(p);
}

template <typename T>
hipError_t bwd_impl(const DeltaRuleArgs& a, char* ws) {
  const Work w = plan_work(a, true);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  Rule p = rule_of(a);
  p.backward = true;
  p.part_own = at(w.own);
  p.part_map = at(w.map);
  hipError_t err = run_tri<T>(p, at(w.lower), at(w.upper));
  if (err != hipSuccess) return err;
  Rule f = p, r = p;
  f.tri = at(w.lower);
  f.init = a.h0;
  f.states = at(w.S);
  f.left = at(w.N);
  err = run_sweep<T, kStates>(f);
  if (err != hipSuccess) return err;
  r.v = a.dy;
  r.tri = at(w.upper);
  r.init = a.dlast;
  r.states = at(w.D);
  r.left = at(w.dR);
  r.last = a.dh0;
  err = run_sweep<T, kBackwards>(r);
  if (err != hipSuccess || a.L == 0) return err;
  Grad g{};
  g.heads = heads_together(a, p.n_chunks);
  const int rest = p.share / g.heads;  // partial sums of a group
  const bool shared = rest > 1;
  g.p = p;
  g.p.y = a.dv;
  g.dy = a.dy;
  g.S = at(w.S); g.D = at(w.D); g.N = at(w.N); g.dR = at(w.dR);
  g.dq = shared ? static_cast<void*>(at(w.dq)) : a.dq;
  g.dk = shared ? static_cast<void*>(at(w.dk)) : a.dk;
  g.dqk_f32 = shared;
  g.dbeta = a.dbeta;
  g.dg = a.dg;
  err = run_grad<T>(g);
  if (err != hipSuccess || !shared) return err;
  const int64_t n = a.b * a.L * a.G * a.Dk;
  for (int k = 0; k < 2; k++) {
    const float* in = k ? at(w.dk) : at(w.dq);
    T* out = static_cast<T*>(k ? a.dk : a.dq);
    const bool vec = a.Dk % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0;
    err = vec ? launch_kind(kKindDeltaReduce, lin_group_sum_kernel<T, 4>, std::min(ceil_div(n, 1024), kSumBlocks), 256, a.stream, in, out, n, rest, int(a.Dk))
              : launch_kind(kKindDeltaReduce, lin_group_sum_kernel<T, 1>, std::min(ceil_div(n, 256), kSumBlocks), 256, a.stream, in, out, n, rest, int(a.Dk));
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <typename T>
hipError_t update_impl(const DeltaRuleArgs& a) {
  Rule p = rule_of(a);
  p.y = a.y;
  const bool vec = a.Dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.last) % 16 == 0;
  int lanes = 1;
  while (lanes * (vec ? 4 : 1) < std::min<int64_t>(a.Dv, kTile)) lanes *= 2;
  const int64_t rows = ceil_div(a.Dk, 256 / lanes);  // of the state a thread has: at most 8 in vectors, 32 else
  auto go = [&](auto kern) { return launch_kind(kKindDeltaUpdate, kern, a.b * a.H * p.n_tiles, 256, a.stream, p, a.last, lanes); };
  if (vec) return rows <= 4 ? go(delta_update_kernel<T, 4, 4>) : go(delta_update_kernel<T, 4, 8>);
  return rows <= 16 ? go(delta_update_kernel<T, 1, 16>) : go(delta_update_kernel<T, 1, 32>);
}

}  // namespace

int64_t deltarule_max_dim() { return kMaxDim; }
int64_t deltarule_max_heads() { return 65535; }

size_t deltarule_workspace_bytes(const DeltaRuleArgs& a, bool backward) {
  if (a.b == 0 || a.H == 0) return 0;
  return plan_work(a, backward).total;
}

hipError_t launch_deltarule_fwd(const DeltaRuleArgs& a, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  return a.dtype == 0 ? fwd_impl<float>(a, ws) : fwd_impl<bf16_bits>(a, ws);
}

hipError_t launch_deltarule_bwd(const DeltaRuleArgs& a, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  return a.dtype == 0 ? bwd_impl<float>(a, ws) : bwd_impl<bf16_bits>(a, ws);
}

hipError_t launch_deltarule_update(const DeltaRuleArgs& a) {
  return a.dtype == 0 ? update_impl<float>(a) : update_impl<bf16_bits>(a);
}

}  // namespace ssm
