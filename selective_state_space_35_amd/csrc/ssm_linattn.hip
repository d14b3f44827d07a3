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
// rounded values would not cancel it, and with strong decays it is much larger than dg.  Where r_t is
// zero (a reset) dg_t is zero, and the sums of the tokens before end there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ssm_chain.h"
#include "ssm_device.h"
#include "ssm_linattn.h"
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
  void* out;               // [b, L, H, VD], of the streamed type or (out_f32) float
  bool out_f32;
  float* last;             // [b, H, KD, VD], or null
  bool final_decay;        // `last` takes the first token's decay too (gradient of the initial state)
  // with dots: dots[b, L, H] = (output without the token's own product) . xd
  const void* xd;
  int gd;
  void* dots;              // Dot<T>
  const float* dstate;     // [b, H, VD, KD] (transposed); dstate_dot[b, H] = its product with the last state
  void* dstate_dot;        // Dot<T>
  bool exact;              // a sweep whose last state can be asked for: its products keep all bits of a float, asked for or not
  bool reverse;            // from the last token to the first
  int64_t b, L;
  int H, KD, VD;
  // the cut: n_segs segments of `parts` parts of part_chunks chunks.  With more than one segment, the states leaving the
  // n_parts parts of all but the last are in seg_state[b][n_parts][H], stored as `init` is, and the sums of the parts' log
  // decays in seg_decay
  int n_chunks, n_segs, parts, part_chunks, n_parts;
  float* seg_state;
  float* seg_decay;
  hipStream_t stream;
};

// The dots of one token, float or (float tensors, whose gate gradient has to be right to their last bits) double
template <typename T>
using Dot = typename std::conditional<sizeof(T) == 4, double, float>::type;

// A log decay below -10^4 counts as -10^4 (its factor is zero in float either way), so that
// minus infinity is a reset and differences of running sums stay numbers.
__device__ __forceinline__ float clamp_log(float x) { return x < -1e4f ? -1e4f : x; }

template <typename T>
__device__ __forceinline__ float log_decay(const Sweep& p, int64_t bi, int64_t t, int h) {
  float x = p.A ? p.A[h] : 0.f;
  if (p.g) x += load_elem(static_cast<const T*>(p.g) + (bi * p.L + t) * p.H + h);
  return clamp_log(x);
}

__device__ __forceinline__ int live_length(const int32_t* lengths, int64_t bi, int64_t L) {
  const int n = lengths ? lengths[bi] : int(L);
  return __builtin_amdgcn_readfirstlane(n < 0 ? 0 : n > L ? int(L) : n);
}

// ---------------------------------------------------------------------------
// Matrix products.  A fragment is one lane's 8 elements of an operand of 16 rows (or columns) by
// 32: lane l holds row l % 16 and the contraction indices 8 (l / 16) .. + 7.  bf16 takes one
// v_mfma_f32_16x16x32_bf16; float takes eight v_mfma_f32_16x16x4_f32, the j-th with every lane's
// j-th element (the order of the contraction index is free, as long as both operands share it).
// The result of 16 x 16 has, in lane l, rows 4 (l / 16) .. + 3 of column l % 16.
// ---------------------------------------------------------------------------
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
struct f32x8 {
  float v[8];
};
template <typename T>
struct FragOf;
template <>
struct FragOf<bf16_bits> {
  typedef bf16x8 type;
};
template <>
struct FragOf<float> {
  typedef f32x8 type;
};
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; j++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ bf16x8 row_frag(const bf16_bits* p) { return *reinterpret_cast<const bf16x8*>(p); }
__device__ __forceinline__ f32x8 row_frag(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return f32x8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// the same of two separate groups of four
__device__ __forceinline__ bf16x8 pair_frag(const bf16_bits* a, const bf16_bits* b) {
  const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(b);
  return __builtin_bit_cast(bf16x8, make_uint4(x.x, x.y, y.x, y.y));
}
__device__ __forceinline__ f32x8 pair_frag(const float* a, const float* b) {
  const float4 x = *reinterpret_cast<const float4*>(a), y = *reinterpret_cast<const float4*>(b);
  return f32x8{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
}

// Column c0 + step (i / 4) + i % 4 (i = lane % 16) of rows r .. r + 7 of a row-major LDS tile; r may
// differ between the groups of 16 lanes.  bf16 goes through the transposing LDS read of gfx950: in a group of 16
// lanes, lane m names 8 bytes and lane i receives element i % 4 of the bytes named by lanes
// i / 4 + 4 j, j = 0..3.
typedef short v4i16 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 col_frag(const bf16_bits* t, int ld, int r, int c0, int step) {
  const int m = threadIdx.x % 16;
  const bf16_bits* p = t + (r + m / 4) * ld + c0 + step * (m % 4);
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)p);
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(p + 4 * ld));
  const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
__device__ __forceinline__ f32x8 col_frag(const float* t, int ld, int r, int c0, int step) {
  const int i = threadIdx.x % 16;
  const float* p = t + r * ld + c0 + step * (i / 4) + i % 4;
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 8; j++) f.v[j] = p[j * ld];
  return f;
}

// x as one rounded fragment, and (bf16) what the rounding left, rounded again
__device__ __forceinline__ void make_frag(const float (&x)[8], bf16x8& hi) {
#pragma unroll
  for (int j = 0; j < 8; j++) hi[j] = static_cast<__bf16>(x[j]);
}
__device__ __forceinline__ void make_frag(const float (&x)[8], f32x8& hi) {
#pragma unroll
  for (int j = 0; j < 8; j++) hi.v[j] = x[j];
}
__device__ __forceinline__ bf16x8 rest_frag(const float (&x)[8], const bf16x8& hi) {
  bf16x8 lo;
#pragma unroll
  for (int j = 0; j < 8; j++) lo[j] = static_cast<__bf16>(x[j] - static_cast<float>(hi[j]));
  return lo;
}
__device__ __forceinline__ void frag_floats(const bf16x8& f, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) x[j] = static_cast<float>(f[j]);
}
__device__ __forceinline__ void frag_floats(const f32x8& f, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) x[j] = f.v[j];
}

// ---------------------------------------------------------------------------
// Waves of a SIMD that the registers are held to.  A sweep's workgroup alone is two.  The bound is also an upper one: it
// keeps a second workgroup off the CU where registers and LDS would allow it (float, widths of up to 64: 91 to 127
// registers, at most 72 KB).  What a second one gives there is not measured.
#define SSM_LIN_WAVES(n) __attribute__((amdgpu_waves_per_eu(n, n)))
constexpr int kSweepWaves = 2;
template <typename T>
constexpr int state_waves(int kd, int vd) {
  return sizeof(T) == 4 ? 2 : kd + vd > 128 ? 2 : 4;
}

// Chunks of kChunk tokens.  A sweep counts positions from its own start: position i is token i, or in
// reversed time token n - 1 - i of the row's n.  Rows of an LDS tile are positions.
// ---------------------------------------------------------------------------
template <typename T>
constexpr int kChunk = sizeof(T) == 4 ? 32 : 64;  // float tiles are twice as wide, and two chunks of them have to fit in the LDS
constexpr int kThreads = 256;  // four waves that hold a quarter of the state's columns each, or that stage and score

// Tiles in LDS: their rows are padded so that the reads of their kind fall on different banks (64 of 4 bytes).
// Row fragments (16 bytes a lane, 8 rows at once) and pairs of 8 bytes (16 rows at once) want rows 4 banks apart,
// transposing reads (4 rows by 32 or, of every other 8 bytes, 64 bytes) want 8 or 16.  At 64 elements a row of
// bf16 with one piece of padding is 36 banks on, which serves all of them.
enum Role { kQuery, kKey, kValue };
template <typename T, int DP, Role ROLE>
struct Tile {
  static constexpr int kVec = 16 / sizeof(T);                  // elements of a 16-byte piece
  static constexpr int kRow = DP / kVec;                       // pieces a row
  static constexpr int kC = kChunk<T>;
  static constexpr int kPieces = kC * kRow / kThreads;         // pieces a thread
  static constexpr int ld = DP + (sizeof(T) == 4 || DP == 64 ? 1 : ROLE == kQuery ? 1 : ROLE == kKey ? 2 : 4) * kVec;  // elements a row
  static constexpr int kElems = kC * ld;
};

// Where a workgroup is: its head, batch row, segment and the chunks of it.
struct Place {
  int h, seg, c0, c1, n;
  int64_t bi, bh;
};
// workgroup `id` of n pieces of `chunks` chunks a head
__device__ __forceinline__ Place place_of(const Sweep& p, int n, int chunks, int id) {
  Place w;
  // Workgroups are dealt to the 8 XCDs in turn: with H a multiple of 8, each XCD takes H / 8 neighbouring
  // heads, so that the heads of a group read their shared rows through one L2.
  w.h = p.H % 8 == 0 ? (id % 8) * (p.H / 8) + (id / 8) % (p.H / 8) : id % p.H;
  const int rest = id / p.H;
  w.seg = rest % n;
  w.bi = rest / n;
  w.bh = w.bi * p.H + w.h;
  w.n = live_length(p.lengths, w.bi, p.L);
  w.c0 = w.seg * chunks;
  w.c1 = min(w.c0 + chunks, p.n_chunks);
  return w;
}

// Descriptor at an address that is the same in every lane (said so: the compiler would loop over the lanes' values)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(int(uint32_t(u))), hi = __builtin_amdgcn_readfirstlane(int(uint32_t(u >> 32)));
  return make_rsrc(reinterpret_cast<const void*>((uint64_t(hi) << 32) | lo));
}

// Any bytes at any address: the compiler reads and writes them at once (unaligned access is on for global memory)
__device__ __forceinline__ uint4 load_16(const char* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// v moved down by n bytes, 0 < n < 16, zeros above
__device__ __forceinline__ uint4 down_bytes(const uint4& v, int n) {
  const uint64_t lo = uint64_t(v.x) | (uint64_t(v.y) << 32), hi = uint64_t(v.z) | (uint64_t(v.w) << 32);
  const int b = 8 * n;
  const uint64_t a = b >= 64 ? hi >> (b - 64) : (lo >> b) | (hi << (64 - b)), c = b >= 64 ? 0 : hi >> b;
  return make_uint4(uint32_t(a), uint32_t(a >> 32), uint32_t(c), uint32_t(c >> 32));
}

// A chunk's rows of one tensor, on their way from memory to LDS: rows of D <= DP elements, `stride`
// elements apart, the rest zero.  VEC: rows are whole 16-byte pieces, 16-byte aligned.  A thread's
// pieces are kStep rows apart, so one lane offset serves them all, the steps and the chunks being
// wave-uniform.  In reversed time the descriptor starts at the chunk's last position: position i is
// row kC - 1 - i of it, and rows below a short last chunk's, which are not read, may lie before the tensor.
template <typename T, int DP, Role ROLE, bool VEC>
struct Stage {
  typedef Tile<T, DP, ROLE> L;
  static constexpr int kStep = kThreads / L::kRow;  // rows between a thread's pieces
  const T* base;     // row of the chunk's first position, or (reversed) of its last
  int voff, soff, sstep, chunk, live_cols;
  bool wide;
  // first: row of position p0 of the sweep (reversed: of position p0 + kC - 1, maybe before the tensor); tid: of 256
  __device__ __forceinline__ void init(const T* first, int stride, int D, bool reverse, int tid) {
    const int i = tid / L::kRow, c = (tid % L::kRow) * L::kVec;
    base = first;
    chunk = reverse ? -L::kC * stride : L::kC * stride;
    sstep = kStep * stride * int(sizeof(T));
    soff = 0;
    if (reverse) {
      voff = ((kStep - 1 - i) * stride + c) * int(sizeof(T));
      soff = (L::kPieces - 1) * sstep;
      sstep = -sstep;
    } else {
      voff = (i * stride + c) * int(sizeof(T));
    }
    live_cols = D - c;
    wide = D >= L::kVec;
    if (VEC && live_cols <= 0) voff = 0x7fffffff;
  }
  // the next chunk, of nv live positions
  __device__ __forceinline__ void load(uint4 (&r)[L::kPieces], int nv, int tid) {
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(base);
    const int i = tid / L::kRow;
#pragma unroll
    for (int j = 0; j < L::kPieces; j++) {
      const int o = i + j * kStep < nv ? voff : 0x7fffffff;
      if constexpr (VEC) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, o, soff + j * sstep, 0);
        r[j] = make_uint4(v[0], v[1], v[2], v[3]);
      } else if (sizeof(T) == 2 && wide) {  // 16 bytes from any address; a row's last piece is moved to its place from a
                                            // read that ends with the row (b4 L2048 H24 D100: 322 us by elements, 205 so)
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i + j * kStep < nv && live_cols > 0) {
          const int over = live_cols < L::kVec ? (L::kVec - live_cols) * int(sizeof(T)) : 0;
          v = load_16(reinterpret_cast<const char*>(base) + (int64_t(voff) + soff + j * sstep - over));
          if (over) v = down_bytes(v, over);
        }
        r[j] = v;
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < L::kVec; e++) {
          const int oe = i + j * kStep < nv && e < live_cols ? voff + e * int(sizeof(T)) : 0x7fffffff;
          if constexpr (sizeof(T) == 4) w[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, oe, soff + j * sstep, 0);
          else w[e / 2] |= uint32_t(__builtin_amdgcn_raw_buffer_load_b16(rs, oe, soff + j * sstep, 0)) << (16 * (e % 2));
        }
        r[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    base += chunk;
  }
  static __device__ __forceinline__ void store(T* tile, const uint4 (&r)[L::kPieces], int tid) {
    T* to = tile + (tid / L::kRow) * L::ld + (tid % L::kRow) * L::kVec;
#pragma unroll
    for (int j = 0; j < L::kPieces; j++) *reinterpret_cast<uint4*>(to + j * kStep * L::ld) = r[j];
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return uint32_t(__builtin_bit_cast(bf16_bits, static_cast<__bf16>(lo))) |
         (uint32_t(__builtin_bit_cast(bf16_bits, static_cast<__bf16>(hi))) << 16);
}
// four consecutive elements of an LDS row, as floats
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 lds4(const bf16_bits* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

// A lane's part of a chunk's rows of one tensor in memory, of elements of `es` bytes: N consecutive elements at
// column c of position 16 tt + lane % 16.  As in Stage, one lane offset and wave-uniform steps; what is not live is
// read as zero and not written.
template <int N, bool VEC, int kC>
struct Rows {
  const char* base;
  int voff, soff, sstep, chunk, cols;
  __device__ __forceinline__ void init(const Sweep& p, const Place& w, const void* x, int es, int share, int c) {
    const int i = threadIdx.x % 16, D = p.VD, stride = p.H / share * D * es;
    const int64_t t = p.reverse ? int64_t(w.n) - int64_t(w.c0) * kC - kC : int64_t(w.c0) * kC;
    base = static_cast<const char*>(x) + ((w.bi * p.L + t) * (p.H / share) + w.h / share) * D * es;
    chunk = p.reverse ? -kC * stride : kC * stride;
    sstep = p.reverse ? -16 * stride : 16 * stride;
    soff = p.reverse ? (kC - 16) * stride : 0;
    voff = (p.reverse ? 15 - i : i) * stride + c * es;
    cols = D - c;
  }
  __device__ __forceinline__ void next() { base += chunk; }
  template <typename T>
  struct Raw {
    uint32_t w[N * int(sizeof(T)) / 4];
  };
  template <typename T>
  __device__ __forceinline__ Raw<T> load(int tt, int nv) const {
    constexpr int kBytes = int(sizeof(T));
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(base);
    const bool row = 16 * tt + int(threadIdx.x % 16) < nv;
    const int so = soff + tt * sstep;
    Raw<T> x;
    if constexpr (VEC) {
      if constexpr (N * kBytes == 8) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, row && cols > 0 ? voff : 0x7fffffff, so, 0);
        x.w[0] = v[0]; x.w[1] = v[1];
      } else {
#pragma unroll
        for (int k = 0; k < N * kBytes / 16; k++) {
          const int at = row && cols > k * 16 / kBytes ? voff + 16 * k : 0x7fffffff;
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, at, so, 0);
#pragma unroll
          for (int j = 0; j < 4; j++) x.w[4 * k + j] = v[j];
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < N * kBytes / 4; k++) x.w[k] = 0;
      if (kBytes == 2 && row && cols >= N) {
        __builtin_memcpy(x.w, base + (int64_t(voff) + so), N * kBytes);
        return x;
      }
#pragma unroll
      for (int e = 0; e < N; e++) {
        const int at = row && e < cols ? voff + e * kBytes : 0x7fffffff;
        if constexpr (kBytes == 4) x.w[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, so, 0);
        else x.w[e / 2] |= uint32_t(__builtin_amdgcn_raw_buffer_load_b16(rs, at, so, 0)) << (16 * (e % 2));
      }
    }
    return x;
  }
  template <typename T>
  static __device__ __forceinline__ float element(const Raw<T>& x, int j) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(x.w[j]);
    else return __uint_as_float(j % 2 ? x.w[j / 2] & 0xffff0000u : x.w[j / 2] << 16);
  }
  template <typename T>
  __device__ __forceinline__ void store(int tt, int nv, const float (&y)[N]) const {
    constexpr int kBytes = int(sizeof(T));
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(base);
    const bool row = 16 * tt + int(threadIdx.x % 16) < nv;
    const int so = soff + tt * sstep;
    uint32_t w[N * kBytes / 4];
    if constexpr (kBytes == 4) {
#pragma unroll
      for (int j = 0; j < N; j++) w[j] = __float_as_uint(y[j]);
    } else {
#pragma unroll
      for (int j = 0; j < N / 2; j++) w[j] = pack_bf16(y[2 * j], y[2 * j + 1]);
    }
    if constexpr (VEC) {
      if constexpr (N * kBytes == 8) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(u2{w[0], w[1]}, rs, row && cols > 0 ? voff : 0x7fffffff, so, 0);
      } else {
        typedef uint32_t u4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int k = 0; k < N * kBytes / 16; k++)
          __builtin_amdgcn_raw_buffer_store_b128(u4{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]}, rs,
                                                 row && cols > k * 16 / kBytes ? voff + 16 * k : 0x7fffffff, so, 0);
      }
    } else if (kBytes == 2 && row && cols >= N) {
      __builtin_memcpy(const_cast<char*>(base) + (int64_t(voff) + so), w, N * kBytes);
    } else {
#pragma unroll
      for (int e = 0; e < N; e++) {
        const int at = row && e < cols ? voff + e * kBytes : 0x7fffffff;
        if constexpr (kBytes == 4) __builtin_amdgcn_raw_buffer_store_b32(w[e], rs, at, so, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(w[e / 2] >> (16 * (e % 2))), rs, at, so, 0);
      }
    }
  }
};

// Decays of a chunk, for its kC positions, in LDS.  The running sum is kept in double, in units of
// log 2, and handed on in two floats: differences of it are exact to fp32 even where a reset
// put it at -10^4.
template <int kC>
struct __attribute__((aligned(16))) Decays {
  float hi[kC], lo[kC];  // running sum up to and with the position
  float in[kC];          // exp of it: what the state entering the chunk has kept
  float out[kC];         // exp(last - own) wscale: what a product written here keeps to the chunk's end
  float all;             // exp of the last
};
// Log decays of a chunk's positions, lane i of a wave with position i's: a token's own, or in reversed time
// the one of the token after it (the first position has none).
template <typename T, int kC>
struct Gates {
  const T* base;
  int voff, chunk;
  float fixed;
  bool given, reverse;
  __device__ __forceinline__ void init(const Sweep& p, const Place& w, int c0) {
    const int l = threadIdx.x % kWave;
    given = p.g != nullptr;
    reverse = p.reverse;
    fixed = p.A ? p.A[w.h] : 0.f;
    const int64_t t = reverse ? int64_t(w.n) - int64_t(c0) * kC - kC : int64_t(c0) * kC;
    base = static_cast<const T*>(p.g) + ((w.bi * p.L + t) * p.H + w.h);
    chunk = reverse ? -kC * p.H : kC * p.H;
    voff = (reverse ? kC - l : l) * p.H * int(sizeof(T));
  }
  // the next chunk, from position p0, nv live; the raw value, to be turned into a log decay later
  __device__ __forceinline__ float load(int p0, int nv) {
    const int l = threadIdx.x % kWave;
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(base);
    base += chunk;
    const int at = given && l < kC && l < nv && !(reverse && p0 + l == 0) ? voff : 0x7fffffff;
    if constexpr (sizeof(T) == 4) return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0));
    else return __uint_as_float(uint32_t(__builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0)) << 16);
  }
  __device__ __forceinline__ float log_of(float raw, int p0, int nv) const {
    const int l = threadIdx.x % kWave;
    return l < kC && l < nv && !(reverse && p0 + l == 0) ? clamp_log(raw + fixed) : 0.f;
  }
};
// x of the lane N below in the row of 16 (or, N = 16 and 32, of the last lane of the row or half below), else 0
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(u)), CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(u >> 32)), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}
// by one wave, lane i with position i's gate; returns the chunk's sum in natural units
template <int kC>
__device__ __forceinline__ double fill_decays(Decays<kC>& d, float gate, float wscale) {
  const int l = threadIdx.x % kWave;
  double run = double(gate) * 1.4426950408889634;
  run += dpp_or_zero<0x111, 0xF>(run);  // row_shr:1
  run += dpp_or_zero<0x112, 0xF>(run);  // row_shr:2
  run += dpp_or_zero<0x114, 0xF>(run);  // row_shr:4
  run += dpp_or_zero<0x118, 0xF>(run);  // row_shr:8
  run += dpp_or_zero<0x142, 0xA>(run);  // row_bcast:15 into rows 1 and 3
  run += dpp_or_zero<0x143, 0xC>(run);  // row_bcast:31 into rows 2 and 3
  const uint64_t u = __builtin_bit_cast(uint64_t, run);
  const uint64_t ul = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u)), kC - 1));
  const uint64_t uh = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u >> 32)), kC - 1));
  const double last = __builtin_bit_cast(double, (uh << 32) | ul);
  if (l < kC) {
    const float hi = float(run);
    d.hi[l] = hi;
    d.lo[l] = float(run - double(hi));
    d.in[l] = exp2_fast(hi);
    d.out[l] = exp2_fast(float(last - run)) * wscale;
    if (l == 0) d.all = exp2_fast(float(last));
  }
  return last * 0.6931471805599453;
}

// Whether a lane's fragments (or, bf16, those of lanes that share a row of 16 with it) hold what is not finite: its
// products with zero are no numbers.  bf16: one matrix product a fragment (b8 L2048 H24 D64 forward 63 us with and without
// it, b4 L4096 H32 G8 D128 backward 647 and 638 us).
template <int KS, int N>
__device__ __forceinline__ bool not_finite(const bf16x8 (&f)[KS][N]) {
  const bf16x8 zero = __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
  f32x4 z{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < KS; k++)
#pragma unroll
    for (int n = 0; n < N; n++) z = mma(f[k][n], zero, z);
  return !((z[0] + z[1]) + (z[2] + z[3]) == 0.f);
}
template <int KS, int N>
__device__ __forceinline__ bool not_finite(const f32x8 (&f)[KS][N]) {
  float z = 0.f;
#pragma unroll
  for (int k = 0; k < KS; k++)
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int j = 0; j < 8; j++) z = fmaf(f[k][n].v[j], 0.f, z);
  return !(z == 0.f);
}
// Zero in the place of what is not finite; the first such element, 8 if there is none
__device__ __forceinline__ int drop_not_finite(bf16x8& f) {
  uint4 u = __builtin_bit_cast(uint4, f);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
  int first = 8;
#pragma unroll
  for (int j = 7; j >= 0; j--) {
    const uint32_t exponent = 0x7f80u << (16 * (j % 2));
    if ((w[j / 2] & exponent) == exponent) {
      first = j;
      w[j / 2] &= j % 2 ? 0x0000ffffu : 0xffff0000u;
    }
  }
  f = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
  return first;
}
__device__ __forceinline__ int drop_not_finite(f32x8& f) {
  int first = 8;
#pragma unroll
  for (int j = 7; j >= 0; j--)
    if ((__float_as_uint(f.v[j]) & 0x7f800000u) == 0x7f800000u) {
      first = j;
      f.v[j] = 0.f;
    }
  return first;
}

// The state in registers: wave w holds its VDP / 4 columns, as 16 x 16 results whose rows run along
// the KDP index.  Two neighbouring results are an operand fragment as they are: a lane then has indices
// 32 kk + 4 (l / 16) .. + 3 and 16 more, and the other operand is read in that order (pair_frag).  Where a wave has two
// results side by side, their columns interleave by fours, so that a lane has 8 consecutive outputs.
template <int KDP, int VDP>
struct Layout {
  static constexpr int MT = KDP / 16, NT = VDP / 64, KS = KDP / 32;
  static constexpr int vstep = NT == 2 ? 8 : 4;
  static __device__ __forceinline__ int v0(int nt) { return int(threadIdx.x / kWave) * (VDP / 4) + 4 * nt; }  // waves 0..3
  // column of lane index i of result nt
  static __device__ __forceinline__ int col(int nt) {
    const int i = threadIdx.x % 16;
    return v0(nt) + vstep * (i / 4) + i % 4;
  }
  // first of the 4 rows that this lane holds of result m
  static __device__ __forceinline__ int row(int m) { return 16 * m + 4 * int((threadIdx.x % kWave) / 16); }
  typedef f32x4 State[MT][NT];
  static __device__ __forceinline__ void zero(State& S) {
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int n = 0; n < NT; n++) S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // a state in memory, [KD][VD] or transposed, through a descriptor: what lies outside is read as zero and not written
  static __device__ __forceinline__ void load(State& S, const float* src, bool transposed, int KD, int VD) {
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(src);
    const int dk = transposed ? 4 : 4 * VD;  // bytes from row to row
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int v = col(n);
      int at = row(0) * dk + (transposed ? 4 * v * KD : 4 * v);
#pragma unroll
      for (int m = 0; m < MT; m++) {
#pragma unroll
        for (int r = 0; r < 4; r++) {
          S[m][n][r] = __uint_as_float(
              __builtin_amdgcn_raw_buffer_load_b32(rs, row(m) + r < KD && v < VD ? at : 0x7fffffff, 0, 0));
          at += dk;
        }
        at += 12 * dk;
      }
    }
  }
  static __device__ __forceinline__ void store(const State& S, float* dst, int KD, int VD, float f) {
    const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(dst);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int v = col(n);
      int at = 4 * (row(0) * VD + v);
#pragma unroll
      for (int m = 0; m < MT; m++) {
#pragma unroll
        for (int r = 0; r < 4; r++) {
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[m][n][r] * f), rs,
                                                row(m) + r < KD && v < VD ? at : 0x7fffffff, 0, 0);
          at += 4 * VD;
        }
        at += 48 * VD;
      }
    }
  }
};

// S = all S + K^T (out o V) over a chunk.  The weighted values are split into two bf16 parts (half a step of 2^-8
// twice: 2^-16 of a product at most, 2 10^-6 of the state measured), and in the sweeps whose state can be an output
// (exact) into three, which hold all 24 bits of a float: whether it is asked for does not change the other outputs' bits
// (b1 L65536 H40 D128 forward 1030 us, with two parts 920 us).
template <typename T, int KDP, int VDP>
__device__ __forceinline__ void write_state(typename Layout<KDP, VDP>::State& S, const T* Ks,
                                            const Frag<T> (&vf)[kChunk<T> / 32][VDP / 64],
                                            const Decays<kChunk<T>>& d, bool exact) {
  typedef Layout<KDP, VDP> Y;
  constexpr int kSteps = kChunk<T> / 32;
  const int g8 = 8 * int((threadIdx.x % kWave) / 16);
  Frag<T> hi[kSteps][Y::NT], lo[kSteps][Y::NT], rest[kSteps][Y::NT];
#pragma unroll
  for (int ks = 0; ks < kSteps; ks++) {
    const float4 w0 = lds4(d.out + 32 * ks + g8), w1 = lds4(d.out + 32 * ks + g8 + 4);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int n = 0; n < Y::NT; n++) {
      float x[8];
      frag_floats(vf[ks][n], x);
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] *= w[j];
      make_frag(x, hi[ks][n]);
      if constexpr (sizeof(T) == 2) {
        lo[ks][n] = rest_frag(x, hi[ks][n]);
        if (exact) {
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] -= static_cast<float>(hi[ks][n][j]);
          rest[ks][n] = rest_frag(x, lo[ks][n]);
        }
      }
    }
  }
  const float all = d.all;
  constexpr int kHalf = Y::MT / 2;  // the keys' fragments are read half a round ahead of their products
  Frag<T> kf[2][kHalf][kSteps];
  auto read = [&](int half) {
#pragma unroll
    for (int m = 0; m < kHalf; m++)
#pragma unroll
      for (int ks = 0; ks < kSteps; ks++)
        kf[half][m][ks] = col_frag(Ks, Tile<T, KDP, kKey>::ld, 32 * ks + g8, 16 * (half * kHalf + m), 4);
  };
  auto multiply = [&](int half) {
#pragma unroll
    for (int i = 0; i < kHalf; i++) {
      const int m = half * kHalf + i;
#pragma unroll
      for (int n = 0; n < Y::NT; n++)
#pragma unroll
        for (int r = 0; r < 4; r++) S[m][n][r] *= all;
#pragma unroll
      for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
        for (int n = 0; n < Y::NT; n++) {
          S[m][n] = mma(kf[half][i][ks], hi[ks][n], S[m][n]);
          if constexpr (sizeof(T) == 2) S[m][n] = mma(kf[half][i][ks], lo[ks][n], S[m][n]);
        }
    }
    if constexpr (sizeof(T) == 2) {
      if (exact) {
#pragma unroll
        for (int i = 0; i < kHalf; i++)
#pragma unroll
          for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
            for (int n = 0; n < Y::NT; n++)
              S[half * kHalf + i][n] = mma(kf[half][i][ks], rest[ks][n], S[half * kHalf + i][n]);
      }
    }
  };
  read(0);
  __builtin_amdgcn_sched_barrier(0);
  read(1);
  multiply(0);
  __builtin_amdgcn_sched_barrier(0);
  multiply(1);
}

// The row of a tensor of `heads` heads of D elements that token t of a batch row has for head h
template <typename T>
__device__ __forceinline__ const T* row_of(const void* x, const Sweep& p, const Place& w, int share, int64_t t, int D) {
  return static_cast<const T*>(x) + ((w.bi * p.L + t) * (p.H / share) + w.h / share) * int64_t(D);
}

// Where the chunks of a tensor start: the row of the first chunk's first position, or in reversed time of its last
template <typename T, int kC>
__device__ __forceinline__ const T* start_of(const void* x, const Sweep& p, const Place& w, int share, int D) {
  const int64_t t = p.reverse ? int64_t(w.n) - int64_t(w.c0) * kC - kC : int64_t(w.c0) * kC;
  return row_of<T>(x, p, w, share, t, D);
}

// ---------------------------------------------------------------------------
// States of the parts of a cut sequence, each from zero, and the sums of their log decays; the workgroups from n on
// take the second sweep's.  The parts are shorter than the segments, so that a few heads fill the chip here too
// (b1 L65536 H40 D128: 300 us, 3.7 TB/s; with a part a segment 345 us).  Bound by HBM.
// ---------------------------------------------------------------------------
template <typename T, int KDP, int VDP, bool VEC>
__global__ __launch_bounds__(kThreads) SSM_LIN_WAVES(state_waves<T>(KDP, VDP)) void lin_state_kernel(Sweep p0, Sweep p1, int n) {
  const bool second = int(blockIdx.x) >= n;
  const Sweep& p = second ? p1 : p0;
  typedef Layout<KDP, VDP> Y;
  constexpr int kC = kChunk<T>;
  __shared__ __attribute__((aligned(16))) T Ks[Tile<T, KDP, kKey>::kElems];
  __shared__ __attribute__((aligned(16))) T Vs[Tile<T, VDP, kValue>::kElems];
  __shared__ Decays<kC> ds[2];
  const Place w = place_of(p, p.n_parts, p.part_chunks, int(blockIdx.x) - (second ? n : 0));
  const int tid = threadIdx.x, g8 = 8 * ((tid % kWave) / 16);
  Stage<T, KDP, kKey, VEC> sk;
  Stage<T, VDP, kValue, VEC> sv;
  uint4 rk[Tile<T, KDP, kKey>::kPieces], rv[Tile<T, VDP, kValue>::kPieces];
  sk.init(start_of<T, kC>(p.xk, p, w, p.gk, p.KD), p.H / p.gk * p.KD, p.KD, p.reverse, tid);
  sv.init(start_of<T, kC>(p.xv, p, w, p.gv, p.VD), p.H / p.gv * p.VD, p.VD, p.reverse, tid);
  Gates<T, kC> gates;
  gates.init(p, w, w.c0);
  float gate = 0.f;
  auto fetch = [&](int c) {
    const int nv = c < w.c1 ? w.n - c * kC : 0;  // behind the segment nothing is read
    sk.load(rk, nv, tid);
    sv.load(rv, nv, tid);
    gate = gates.load(c * kC, nv);
  };
  typename Y::State S;
  Y::zero(S);
  double total = 0.0;
  fetch(w.c0);
  if (tid < kWave) total += fill_decays(ds[0], gates.log_of(gate, w.c0 * kC, w.n - w.c0 * kC), p.wscale);
  for (int c = w.c0; c < w.c1; c++) {
    const Decays<kC>& d = ds[(c - w.c0) & 1];
    sk.store(Ks, rk, tid);
    sv.store(Vs, rv, tid);
    __syncthreads();
    fetch(c + 1);
    Frag<T> vf[kC / 32][Y::NT];
#pragma unroll
    for (int ks = 0; ks < kC / 32; ks++)
#pragma unroll
      for (int n = 0; n < Y::NT; n++) vf[ks][n] = col_frag(Vs, Tile<T, VDP, kValue>::ld, 32 * ks + g8, Y::v0(n), Y::vstep);
    write_state<T, KDP, VDP>(S, Ks, vf, d, p.exact);
    if (c + 1 < w.c1 && tid < kWave)
      total += fill_decays(ds[(c + 1 - w.c0) & 1], gates.log_of(gate, (c + 1) * kC, w.n - (c + 1) * kC), p.wscale);
    __syncthreads();
  }
  const int64_t at = (w.bi * p.n_parts + w.seg) * p.H + w.h;
  Y::store(S, p.seg_state + at * p.KD * p.VD, p.KD, p.VD, 1.f);
  if (tid == 0) p.seg_decay[at] = float(total);
}

// ---------------------------------------------------------------------------
// The sweep.  Per chunk:
//   P[t][s] = (q_t . k_s) exp(G_t - G_s) for s <= t, computed as K Q^T (a lane then has four
//             consecutive s of its t), to LDS
//   out     = exp(G_t) S^T q_t + P V, as its transpose: a lane has consecutive columns of its own t
//   S       = exp(G) S + K^T (out o V)
// bf16: P and S go into the products as two bf16 parts (2^-16 of a product at most), so that an output's error is its
// own rounding: against float64 1.7 10^-3 of y in the norm, with one part 2.3 10^-3; b8 L2048 H24 D64 forward 62 us, with
// one part 59 us.  With DOTS the output without the token's own product is multiplied with the rows of xd, for sums over
// the whole sequence that one part would not be right enough for at all.
//
// Only the state runs from chunk to chunk, so it has waves of its own: waves 0..3 take the outputs and
// the state's update, while waves 4..7 bring the next chunk's rows to the other half of the LDS tiles
// and then compute its P, in the other half of P; two barriers a chunk.  One SIMD has a wave of each kind.  The rows of the
// two chunks after are on their way into registers meanwhile.
//
// Measured (bf16): b8 L2048 H24 D64 forward 63 to 66 us (HBM floor 38 us; before the operands were split 59 us, and then
// all eight waves doing all the work in turn 84 us in segments, 105 us uncut); a chunk is 4700 cycles, of which the
// LDS is busy 2100 and each SIMD issues vector instructions in 2200, partly one after the other.  b1 L65536 H40 D128: 1030 us
// (floor 498 us) of which 300 us are the pass over k and v that the cut needs.  Backward, three sweeps: b8 L2048 H24
// D64 240 us, b4 L4096 H32 G8 D128 654 us (floors 66, 100 us), bound by the issue of VALU and MFMA instructions (a workgroup's
// eight waves have 4500 a chunk at D128, 700 of them MFMA; 2400 at D64).
// ---------------------------------------------------------------------------
template <typename T, int KDP, int VDP, bool DOTS>
struct SweepLds {
  static constexpr int kC = kChunk<T>;
  static constexpr bool kTwo = sizeof(T) == 2;  // operands that are not given in bf16 are taken in two parts
  static constexpr int ldp = kC + 16 / int(sizeof(T));
  __attribute__((aligned(16))) T q[2][Tile<T, KDP, kQuery>::kElems];
  __attribute__((aligned(16))) T k[2][Tile<T, KDP, kKey>::kElems];
  __attribute__((aligned(16))) T v[2][Tile<T, VDP, kValue>::kElems];
  __attribute__((aligned(16))) T P[2][kTwo ? 2 : 1][kC * ldp];
  Decays<kC> d[4];  // written two chunks ahead
  Dot<T> dot_part[2][DOTS ? 16 : 1][kC];
  float diag[2][DOTS ? kC : 1];
  Dot<T> red[4];
};

template <typename T, int KDP, int VDP, bool DOTS, bool VEC>
__device__ __forceinline__ void sweep(const Sweep& p, SweepLds<T, KDP, VDP, DOTS>& sh, int id) {
  typedef Layout<KDP, VDP> Y;
  typedef SweepLds<T, KDP, VDP, DOTS> Lds;
  constexpr int kC = Lds::kC, ldp = Lds::ldp, kN = 4 * Y::NT, TB = kC / 16, kSteps = kC / 32;
  constexpr bool kTwo = Lds::kTwo;
  constexpr int ldq = Tile<T, KDP, kQuery>::ld, ldk = Tile<T, KDP, kKey>::ld, ldv = Tile<T, VDP, kValue>::ld;
  const Place w = place_of(p, p.n_segs, p.parts * p.part_chunks, id);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = threadIdx.x % kWave;
  const int lr = l % 16, g4 = 4 * (l / 16), g8 = 8 * (l / 16);
  const int chunks = w.c1 - w.c0;
  // the blocks above the diagonal that the products read stay zero
  for (int i = threadIdx.x; i < (TB / 2) * 256; i += 2 * kThreads) {
    const int b = i / 256, t = 32 * b + (i / 16) % 16, s = 32 * b + 16 + i % 16;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      sh.P[k][0][t * ldp + s] = T(0);
      if constexpr (kTwo) sh.P[k][1][t * ldp + s] = T(0);
    }
  }

  if (wv >= 4) {
    // ------------------------------------------------------------------ staging and scores
    const int pw = wv - 4, tid = threadIdx.x - kThreads;
    const float sscale = p.wscale * p.rscale;
    Stage<T, KDP, kQuery, VEC> sq;
    Stage<T, KDP, kKey, VEC> sk;
    Stage<T, VDP, kValue, VEC> sv;
    sq.init(start_of<T, kC>(p.xq, p, w, p.gq, p.KD), p.H / p.gq * p.KD, p.KD, p.reverse, tid);
    sk.init(start_of<T, kC>(p.xk, p, w, p.gk, p.KD), p.H / p.gk * p.KD, p.KD, p.reverse, tid);
    sv.init(start_of<T, kC>(p.xv, p, w, p.gv, p.VD), p.H / p.gv * p.VD, p.VD, p.reverse, tid);
    struct Regs {
      uint4 q[Tile<T, KDP, kQuery>::kPieces], k[Tile<T, KDP, kKey>::kPieces], v[Tile<T, VDP, kValue>::kPieces];
      float gate;
    };
    Regs r0, r1;
    Gates<T, kC> gates;
    gates.init(p, w, w.c0);
    // behind the segment (i >= chunks) nothing is read and the rows are zero
    auto live = [&](int i) { return i < chunks ? w.n - (w.c0 + i) * kC : 0; };
    auto fetch = [&](Regs& r, int i) {  // the i-th chunk of the segment
      const int nv = live(i);
      sq.load(r.q, nv, tid);
      sk.load(r.k, nv, tid);
      sv.load(r.v, nv, tid);
      r.gate = gates.load((w.c0 + i) * kC, nv);
    };
    auto place = [&](const Regs& r, int i) {
      const int b = i & 1;
      sq.store(sh.q[b], r.q, tid);
      sk.store(sh.k[b], r.k, tid);
      sv.store(sh.v[b], r.v, tid);
    };
    auto decays = [&](const Regs& r, int i) {  // by the wave with the fewest blocks of P
      const float g = gates.log_of(r.gate, (w.c0 + i) * kC, live(i));
      if (pw == 3) fill_decays(sh.d[i & 3], g, p.wscale);
    };
    // P of the i-th chunk: its blocks (t block, s block) with s <= t, mostly of one t block a wave, so that the rows of Q
    // are read once; the wave that takes the decays has the fewest.  All reads come first, all products next.
    auto score_blocks = [&](int i, auto count, int t0, int s0, int t1, int s1, int t2, int s2) {
      constexpr int N = decltype(count)::value;
      const int tbs[3] = {t0, t1, t2}, sbs[3] = {s0, s1, s2};
      const T* Qs = sh.q[i & 1];
      const T* Ks = sh.k[i & 1];
      const Decays<kC>& d = sh.d[i & 3];
      const int pb = i & 1;
      Frag<T> qf[N][Y::KS], kf[N][Y::KS];
      float th[N], tl[N];
      float4 h4[N], l4[N];
#pragma unroll
      for (int j = 0; j < N; j++) {
#pragma unroll
        for (int kk = 0; kk < Y::KS; kk++) {
          qf[j][kk] = row_frag(Qs + (16 * tbs[j] + lr) * ldq + 32 * kk + g8);
          kf[j][kk] = row_frag(Ks + (16 * sbs[j] + lr) * ldk + 32 * kk + g8);
        }
      }
#pragma unroll
      for (int j = 0; j < N; j++) {
        th[j] = d.hi[16 * tbs[j] + lr];
        tl[j] = d.lo[16 * tbs[j] + lr];
        h4[j] = lds4(d.hi + 16 * sbs[j] + g4);
        l4[j] = lds4(d.lo + 16 * sbs[j] + g4);
      }
      __builtin_amdgcn_sched_barrier(0);
      f32x4 acc[N];
#pragma unroll
      for (int j = 0; j < N; j++) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < Y::KS; kk++)
#pragma unroll
        for (int j = 0; j < N; j++) acc[j] = mma(kf[j][kk], qf[j][kk], acc[j]);
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int tb = tbs[j], sb = sbs[j], t = 16 * tb + lr;
        const float shi[4] = {h4[j].x, h4[j].y, h4[j].z, h4[j].w}, slo[4] = {l4[j].x, l4[j].y, l4[j].z, l4[j].w};
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int s = 16 * sb + g4 + r;
          const float e = acc[j][r] * exp2_fast((th[j] - shi[r]) + (tl[j] - slo[r])) * sscale;
          x[r] = (DOTS ? s < t : s <= t) ? e : 0.f;
        }
        if (DOTS && tb == sb && lr / 4 == l / 16) {  // the lane with s == t among its four
          const float a01 = lr % 2 ? acc[j][1] : acc[j][0], a23 = lr % 2 ? acc[j][3] : acc[j][2];
          sh.diag[pb][t] = (lr % 4 < 2 ? a01 : a23) * sscale;
        }
        T* pr = sh.P[pb][0] + t * ldp + 16 * sb + g4;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(pr) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
          const uint2 hi = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
          *reinterpret_cast<uint2*>(pr) = hi;
          if constexpr (kTwo) {
            const float y[4] = {x[0] - __uint_as_float(hi.x << 16), x[1] - __uint_as_float(hi.x & 0xffff0000u),
                                x[2] - __uint_as_float(hi.y << 16), x[3] - __uint_as_float(hi.y & 0xffff0000u)};
            *reinterpret_cast<uint2*>(sh.P[pb][1] + t * ldp + 16 * sb + g4) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
          }
        }
      }
    };
    auto score = [&](int i) {
      using std::integral_constant;
      if constexpr (TB == 4) {
        if (pw < 3) {
          if constexpr (KDP == 64) {
            score_blocks(i, integral_constant<int, 3>{}, 3 - pw, 0, 3 - pw, 1, pw == 2 ? 0 : 3 - pw, pw == 2 ? 0 : 2);
          } else {  // three at once would not fit in the registers
            score_blocks(i, integral_constant<int, 1>{}, 3 - pw, 0, 0, 0, 0, 0);
            score_blocks(i, integral_constant<int, 1>{}, 3 - pw, 1, 0, 0, 0, 0);
            score_blocks(i, integral_constant<int, 1>{}, pw == 2 ? 0 : 3 - pw, pw == 2 ? 0 : 2, 0, 0, 0, 0);
          }
        } else score_blocks(i, integral_constant<int, 1>{}, 3, 3, 0, 0, 0, 0);
      } else {
        if (pw < 3) score_blocks(i, integral_constant<int, 1>{}, pw > 0, pw > 1, 0, 0, 0, 0);
      }
    };
    // what follows the outputs of the i-th chunk: the dots' sums (by one wave), and zero rows behind the length
    auto finish = [&](int i) {
      if (i < 0 || i >= chunks) return;
      const int p0 = (w.c0 + i) * kC, nv = max(0, min(kC, w.n - p0)), rows = min(kC, int(p.L) - p0);
      if (DOTS && pw == 3 && l < rows) {
        const int64_t t = l >= nv ? p0 + l : p.reverse ? w.n - 1 - p0 - l : p0 + l;
        Dot<T> s = 0;
#pragma unroll
        for (int k = 0; k < 16; k++) s += sh.dot_part[i & 1][DOTS ? k : 0][l];
        static_cast<Dot<T>*>(p.dots)[(w.bi * p.L + t) * p.H + w.h] = l < nv ? s : Dot<T>(0);
      }
      for (int r = nv + pw; r < rows; r += 4) {
        const int64_t at = ((w.bi * p.L + p0 + r) * p.H + w.h) * p.VD;
        for (int j = l; j < p.VD; j += kWave) {
          if (p.out_f32) static_cast<float*>(p.out)[at + j] = 0.f;
          else store_elem(static_cast<T*>(p.out) + at + j, 0.f);
        }
      }
    };
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
    // registers or under way.  Steps go by twos, each with its set, so that a wait is for the older loads only.
    auto step = [&](Regs& r, const Regs& other, int i) {
      place(r, i + 1);
      fetch(r, i + 3);
      __syncthreads();
      score(i + 1);
      decays(other, i + 2);
      finish(i - 1);
      __syncthreads();
    };
    for (int i = 0; i < chunks; i += 2) {
      step(r1, r0, i);
      step(r0, r1, i + 1);
    }
    if (chunks % 2 == 0) finish(chunks - 1);
    if (DOTS && p.dstate_dot && w.seg == p.n_segs - 1) __syncthreads();  // the state waves' sum
    return;
  }

  // -------------------------------------------------------------------- outputs and state
  const int vc = wv * (VDP / 4) + (l / 16) * kN;  // first of the kN columns that this lane has of an output row
  typedef Rows<kN, VEC, kC> R;
  R xr, yr;
  if constexpr (DOTS) xr.init(p, w, p.xd, int(sizeof(T)), p.gd, vc);
  yr.init(p, w, p.out, p.out_f32 ? 4 : int(sizeof(T)), 1, vc);
  typename R::template Raw<T> xd[DOTS ? TB : 1];  // the rows of xd for the lane's outputs
  auto fetch_xd = [&](int i) {
    if constexpr (DOTS) {
      const int nv = i < chunks ? w.n - (w.c0 + i) * kC : 0;
#pragma unroll
      for (int tt = 0; tt < TB; tt++) xd[tt] = xr.template load<T>(tt, nv);
      xr.next();
    }
  };
  typename Y::State S;
  const float* from = w.seg > 0 ? p.seg_state + ((w.bi * p.n_parts + w.seg * p.parts - 1) * p.H + w.h) * p.KD * p.VD
                                : p.init ? p.init + w.bh * p.KD * p.VD : nullptr;
  if (from) Y::load(S, from, p.init_t, p.KD, p.VD);
  else Y::zero(S);
  fetch_xd(0);
  __syncthreads();
  __syncthreads();
  for (int c = 0; c < chunks; c++) {
    const int nv = max(0, min(kC, w.n - (w.c0 + c) * kC));
    const Decays<kC>& d = sh.d[c & 3];
    const T* Qs = sh.q[c & 1];
    const T* Ks = sh.k[c & 1];
    const T* Vs = sh.v[c & 1];
    // ---- the entering state's part of the outputs, and the chunk's own: reads a step ahead of their products ----
    f32x4 o[TB][Y::NT];
#pragma unroll
    for (int tt = 0; tt < TB; tt++)
#pragma unroll
      for (int n = 0; n < Y::NT; n++) o[tt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kHalf = Y::KS / 2;
    Frag<T> qf[2][kHalf][TB];
    auto read_q = [&](int half) {
#pragma unroll
      for (int k = 0; k < kHalf; k++)
#pragma unroll
        for (int tt = 0; tt < TB; tt++) {
          const T* q = Qs + (16 * tt + lr) * ldq + 32 * (half * kHalf + k) + g4;
          qf[half][k][tt] = pair_frag(q, q + 16);
        }
    };
    auto times_state = [&](int half) {
#pragma unroll
      for (int k = 0; k < kHalf; k++) {
        const int kk = half * kHalf + k;
        Frag<T> shi[Y::NT], slo[Y::NT];
#pragma unroll
        for (int n = 0; n < Y::NT; n++) {
          float x[8];
#pragma unroll
          for (int r = 0; r < 8; r++) x[r] = S[2 * kk + r / 4][n][r % 4];
          make_frag(x, shi[n]);
          if constexpr (kTwo) slo[n] = rest_frag(x, shi[n]);
        }
#pragma unroll
        for (int tt = 0; tt < TB; tt++)
#pragma unroll
          for (int n = 0; n < Y::NT; n++) {
            o[tt][n] = mma(shi[n], qf[half][k][tt], o[tt][n]);
            if constexpr (kTwo) o[tt][n] = mma(slo[n], qf[half][k][tt], o[tt][n]);
          }
      }
    };
    Frag<T> vf[kSteps][Y::NT], pf[kTwo ? 2 : 1][TB][kSteps];
    read_q(0);
    __builtin_amdgcn_sched_barrier(0);
    read_q(1);
    times_state(0);
    __builtin_amdgcn_sched_barrier(0);
    float in[TB];
#pragma unroll
    for (int tt = 0; tt < TB; tt++) in[tt] = d.in[16 * tt + lr] * p.rscale;
#pragma unroll
    for (int ks = 0; ks < kSteps; ks++)
#pragma unroll
      for (int n = 0; n < Y::NT; n++) vf[ks][n] = col_frag(Vs, ldv, 32 * ks + g8, Y::v0(n), Y::vstep);
#pragma unroll
    for (int k = 0; k < (kTwo ? 2 : 1); k++)
#pragma unroll
      for (int tt = 0; tt < TB; tt++)
#pragma unroll
        for (int ks = 0; ks <= tt / 2; ks++) pf[k][tt][ks] = row_frag(sh.P[c & 1][k] + (16 * tt + lr) * ldp + 32 * ks + g8);
    times_state(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int tt = 0; tt < TB; tt++)
#pragma unroll
      for (int n = 0; n < Y::NT; n++)
#pragma unroll
        for (int r = 0; r < 4; r++) o[tt][n][r] *= in[tt];
    // A value that is not finite must not meet P's zeros: the outputs before it would be no numbers.  It is taken out, and
    // its column of the outputs from its own position on, and of the state, is set to NaN.  (With DOTS the own product is
    // added below, from the tile.)
    if (__builtin_expect(__ballot(not_finite(vf)) != 0, 0)) {
      const float nan = __builtin_nanf("");
#pragma unroll
      for (int n = 0; n < Y::NT; n++) {
        int first = kC;
#pragma unroll
        for (int ks = kSteps - 1; ks >= 0; ks--) {
          const int j = drop_not_finite(vf[ks][n]);
          if (j < 8) first = 32 * ks + g8 + j;
        }
        first = min(first, __shfl_xor(first, 16));
        first = min(first, __shfl_xor(first, 32));
#pragma unroll
        for (int m = 0; m < Y::MT; m++)
#pragma unroll
          for (int r = 0; r < 4; r++) S[m][n][r] = first < kC ? nan : S[m][n][r];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int at = __shfl(first, g4 + r);
#pragma unroll
          for (int tt = 0; tt < TB; tt++) o[tt][n][r] = 16 * tt + lr >= at + (DOTS ? 1 : 0) ? nan : o[tt][n][r];
        }
      }
    }
#pragma unroll
    for (int tt = 0; tt < TB; tt++)
#pragma unroll
      for (int ks = 0; ks <= tt / 2; ks++)
#pragma unroll
        for (int k = 0; k < (kTwo ? 2 : 1); k++)
#pragma unroll
          for (int n = 0; n < Y::NT; n++) o[tt][n] = mma(vf[ks][n], pf[k][tt][ks], o[tt][n]);
    // The middle of a step, after the products with P, so that neither half waits long (before them: float, b32 L512 H8
    // D128, backward, 340 us and here 330; bf16, b8 L2048 H24 D64, forward, 65 and 62 us)
    __syncthreads();
    // ---- outputs ----
#pragma unroll
    for (int tt = 0; tt < TB; tt++) {
      const int i = 16 * tt + lr;
      float y[kN];
#pragma unroll
      for (int j = 0; j < kN; j++) y[j] = o[tt][j / 4][j % 4];
      if constexpr (DOTS) {
        Dot<T> s = 0;
#pragma unroll
        for (int j = 0; j < kN; j++) s = fma(Dot<T>(y[j]), Dot<T>(R::template element<T>(xd[tt], j)), s);
        sh.dot_part[c & 1][4 * wv + l / 16][i] = s;
        const float dg = sh.diag[c & 1][i];
#pragma unroll
        for (int j = 0; j < kN; j += 4) {
          const float4 v = lds4(Vs + i * ldv + vc + j);
          y[j] = fmaf(dg, v.x, y[j]); y[j + 1] = fmaf(dg, v.y, y[j + 1]);
          y[j + 2] = fmaf(dg, v.z, y[j + 2]); y[j + 3] = fmaf(dg, v.w, y[j + 3]);
        }
      }
      if (sizeof(T) == 2 && p.out_f32) yr.template store<float>(tt, nv, y);
      else yr.template store<T>(tt, nv, y);
    }
    yr.next();
    fetch_xd(c + 1);
    write_state<T, KDP, VDP>(S, Ks, vf, d, !DOTS && p.exact);
    __syncthreads();
  }
  if (chunks % 2) {  // the staging waves' steps go by twos
    __syncthreads();
    __syncthreads();
  }
  if (w.seg != p.n_segs - 1) return;
  if (DOTS && p.dstate_dot) {
    typename Y::State D;
    Y::load(D, p.dstate + w.bh * p.KD * p.VD, true, p.KD, p.VD);
    Dot<T> s = 0;
#pragma unroll
    for (int m = 0; m < Y::MT; m++)
#pragma unroll
      for (int n = 0; n < Y::NT; n++)
#pragma unroll
        for (int r = 0; r < 4; r++) s = fma(Dot<T>(S[m][n][r]), Dot<T>(D[m][n][r]), s);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    if (l == 0) sh.red[wv] = s;
    __syncthreads();
    if (threadIdx.x == 0) static_cast<Dot<T>*>(p.dstate_dot)[w.bh] = (sh.red[0] + sh.red[1]) + (sh.red[2] + sh.red[3]);
  }
  if (p.last) {
    const float f = p.final_decay && w.n > 0 ? exp2_fast(log_decay<T>(p, w.bi, 0, w.h) * kLog2e) : 1.f;
    Y::store(S, p.last + w.bh * p.KD * p.VD, p.KD, p.VD, f);
  }
}

template <typename T, int KDP, int VDP, bool VEC>
__global__ __launch_bounds__(2 * kThreads) SSM_LIN_WAVES(kSweepWaves) void lin_fwd_kernel(Sweep p) {
  __shared__ SweepLds<T, KDP, VDP, false> sh;
  sweep<T, KDP, VDP, false, VEC>(p, sh, blockIdx.x);
}

// The three sweeps of the backward in one launch, n workgroups each: dq first, then dk and dv of the same heads on the
// same XCD side by side (both run backwards over the same rows, which the second to come finds in the L2).
template <typename T, int DKP, int DVP, bool GATE, bool VEC>
__global__ __launch_bounds__(2 * kThreads) SSM_LIN_WAVES(kSweepWaves) void lin_bwd_kernel(Sweep dq, Sweep dk, Sweep dv, int n) {
  typedef SweepLds<T, DVP, DKP, GATE> LdsK;
  typedef SweepLds<T, DKP, DVP, false> LdsV;
  __shared__ __attribute__((aligned(16))) char pool[sizeof(LdsK) > sizeof(LdsV) ? sizeof(LdsK) : sizeof(LdsV)];
  const int id = blockIdx.x, j = id - n, even = n / 8 * 16;  // pairs of 8 workgroups, and what is left over
  bool values;
  int at;
  if (id < n) {
    at = id;
    values = false;
  } else if (j < even) {
    at = j / 16 * 8 + j % 8;
    values = j % 16 >= 8;
  } else {
    at = n / 8 * 8 + (j - even) % (n % 8);
    values = j - even >= n % 8;
  }
  if (values) sweep<T, DKP, DVP, false, VEC>(dv, *reinterpret_cast<LdsV*>(pool), at);
  else sweep<T, DVP, DKP, GATE, VEC>(id < n ? dq : dk, *reinterpret_cast<LdsK*>(pool), at);
}

// ---------------------------------------------------------------------------
// Gradient of the gates: dg_t = end + sum over i >= t of (a_i - c_i), per batch row and head, where
// end = <d_last, S_last>.  a and c are [b, L, H].  At a reset, a token whose factor r_t is zero in float, dg_t = <D_t, 0> is
// zero, and so is the sum up to it: the sum starts again there, so that nothing of a document comes into the one before
// it.  Tiles of kGateTile tokens: first each tile's sum up to its first reset (and whether it has one), then each tile adds
// the later ones' up to the first reset to its own running sum (double: the terms cancel over the sequence).
// b8 L2048 H24: 10 and 9 us, by the latency of a row's 64-byte pieces.
constexpr int kGateTile = 256;
constexpr int kGateHeads = 16;  // heads of a workgroup: 16 consecutive floats of a row, times 16 tokens
// exp of a log decay below this is zero in float, denormal numbers included (2^-150)
constexpr float kZeroLog = -104.f;

template <typename T>
struct GateArgs {
  const Dot<T>* a;
  const Dot<T>* c;
  double* sums;      // [b, n_tiles, H]
  uint8_t* resets;   // [b, n_tiles, H]: whether the tile has a reset
  const Dot<T>* end; // [b, H], nullable
  const T* g;
  const float* A;    // nullable
  const int32_t* lengths;
  T* dg;
  int64_t L;
  int H, n_tiles, h_blocks;
};
template <typename T>
__device__ __forceinline__ bool is_reset(const T* g, float fixed) { return load_elem(g) + fixed < kZeroLog; }

template <typename T>
__global__ __launch_bounds__(256) void lin_gate_tiles_kernel(GateArgs<T> p) {
  __shared__ double sh[16][kGateHeads];
  __shared__ int first[kGateHeads];  // the tile's first reset of each head
  const int hl = threadIdx.x % kGateHeads;
  const int h = (blockIdx.x % p.h_blocks) * kGateHeads + hl;
  const int64_t rest = blockIdx.x / p.h_blocks;
  const int tile = int(rest % p.n_tiles);
  const int64_t bi = rest / p.n_tiles;
  const int s = threadIdx.x / kGateHeads;
  const int64_t n = live_length(p.lengths, bi, p.L);
  const float fixed = p.A && h < p.H ? p.A[h] : 0.f;
  if (s == 0) first[hl] = kGateTile;
  __syncthreads();
  double d[kGateTile / 16];
#pragma unroll
  for (int i = 0; i < kGateTile / 16; i++) {
    const int64_t t = int64_t(tile) * kGateTile + i * 16 + s;
    d[i] = 0.0;
    if (t < n && h < p.H) {  // the dots behind the length are zero
      const int64_t at = (bi * p.L + t) * p.H + h;
      d[i] = double(p.a[at]) - double(p.c[at]);
      if (is_reset(p.g + at, fixed)) atomicMin(&first[hl], i * 16 + s);
    }
  }
  __syncthreads();
  const int stop = first[hl];
  double own = 0.0;
#pragma unroll
  for (int i = 0; i < kGateTile / 16; i++)
    if (i * 16 + s < stop) own += d[i];
  sh[s][hl] = own;
  __syncthreads();
  if (s == 0 && h < p.H) {
    double tot = 0.0;
    for (int i = 0; i < 16; i++) tot += sh[i][hl];
    const int64_t at = (bi * p.n_tiles + tile) * p.H + h;
    p.sums[at] = tot;
    p.resets[at] = stop < kGateTile;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void lin_gate_kernel(GateArgs<T> p) {
  __shared__ double sh[16][kGateHeads];     // sums of 16 tokens up to their first reset
  __shared__ double after[16][kGateHeads];
  __shared__ int cut[16][kGateHeads];       // whether the 16 tokens have a reset
  __shared__ int last[kGateHeads];          // the first later tile with a reset: its sum is the last to count
  const int hl = threadIdx.x % kGateHeads;
  const int h = (blockIdx.x % p.h_blocks) * kGateHeads + hl;
  const int64_t rest = blockIdx.x / p.h_blocks;
  const int tile = int(rest % p.n_tiles);
  const int64_t bi = rest / p.n_tiles;
  const int s = threadIdx.x / kGateHeads;  // 16 consecutive tokens of the tile
  const bool ok = h < p.H;
  const int64_t t0 = int64_t(tile) * kGateTile + s * 16;
  const int64_t n = live_length(p.lengths, bi, p.L);
  const float fixed = p.A && ok ? p.A[h] : 0.f;
  if (s == 0) last[hl] = p.n_tiles;
  double d[16], own = 0.0, later = 0.0;
  uint32_t reset = 0;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    d[i] = 0.0;
    if (ok && t0 + i < n) {
      const int64_t at = (bi * p.L + t0 + i) * p.H + h;
      d[i] = double(p.a[at]) - double(p.c[at]);
      reset |= uint32_t(is_reset(p.g + at, fixed)) << i;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; i++)
    if (!(reset & ((2u << i) - 1))) own += d[i];
  sh[s][hl] = own;
  cut[s][hl] = reset != 0;
  __syncthreads();
  const int64_t col = bi * p.n_tiles * p.H + h;  // of sums and resets, H apart
  if (ok)
    for (int k = tile + 1 + s; k < p.n_tiles; k += 16)
      if (p.resets[col + int64_t(k) * p.H]) {
        atomicMin(&last[hl], k);
        break;
      }
  __syncthreads();
  const int stop = last[hl];
  for (int k = tile + 1 + s; k < p.n_tiles && k <= stop; k += 16)
    if (ok) later += p.sums[col + int64_t(k) * p.H];
  after[s][hl] = later;
  __syncthreads();
  // what comes after this thread's tokens, up to the first reset
  double run = 0.0;
  bool open = true;
  for (int i = s + 1; i < 16; i++) {
    if (open) run += sh[i][hl];
    open = open && !cut[i][hl];
  }
  if (open) {
    for (int i = 0; i < 16; i++) run += after[i][hl];
    if (ok && p.end && stop == p.n_tiles) run += double(p.end[bi * p.H + h]);
  }
#pragma unroll
  for (int i = 15; i >= 0; i--) {
    const int64_t t = t0 + i;
    run = reset >> i & 1 ? 0.0 : run + d[i];
    if (ok && t < p.L) store_elem(p.dg + (bi * p.L + t) * p.H + h, t < n ? float(run) : 0.f);
  }
}

// out[row, g, :] = sum over the group's heads of in[row, h, :] (float), rounded once; VEC elements a thread.  Bound by HBM
// (b4 L4096, 32 heads in 8 groups, D128: 57 us, 5.3 TB/s; one element a thread 91 us).
template <typename T, int VEC>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float* __restrict__ in, T* __restrict__ out,
                                                            int64_t n, int share, int D) {
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * VEC; i < n; i += int64_t(gridDim.x) * 256 * VEC) {
    const int64_t rg = i / D;
    const float* p = in + rg * share * D + i % D;
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) s[j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < share; k++) {
      if constexpr (VEC == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + int64_t(k) * D);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      } else {
        s[0] += p[int64_t(k) * D];
      }
    }
    if constexpr (VEC == 4 && sizeof(T) == 4) {
      *reinterpret_cast<float4*>(out + i) = make_float4(s[0], s[1], s[2], s[3]);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
    } else {
      store_elem(out + i, s[0]);
    }
  }
}

// ---------------------------------------------------------------------------
// One token: a workgroup holds one head of one batch row.  Lanes run along the columns of the
// state, the workgroup's row groups along its rows; the readout is summed over the row groups in LDS.  Bound by HBM, the
// state read and written once: b256 H40 D128 260 us, 5.2 TB/s.
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
constexpr int64_t kSumBlocks = int64_t(1) << 22;  // a grid holds less than 2^32 threads: beyond, a thread has several sums
constexpr size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// rows of whole 16-byte pieces, 16-byte aligned
template <typename T>
bool pieces(const void* x, int D) {
  return D % (16 / int(sizeof(T))) == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

template <typename T>
bool sweep_pieces(const Sweep& p) {
  return pieces<T>(p.xq, p.KD) && pieces<T>(p.xk, p.KD) && pieces<T>(p.xv, p.VD) && pieces<T>(p.out, p.VD) &&
         (!p.xd || pieces<T>(p.xd, p.VD));
}

template <typename T, int KDP, int VDP>
hipError_t fwd_kernel(const Sweep& p) {
  const int64_t blocks = p.b * p.H * p.n_segs;
  return sweep_pieces<T>(p) ? launch_kind(kKindLinSweep, lin_fwd_kernel<T, KDP, VDP, true>, blocks, 2 * kThreads, p.stream, p)
                            : launch_kind(kKindLinSweep, lin_fwd_kernel<T, KDP, VDP, false>, blocks, 2 * kThreads, p.stream, p);
}
template <typename T>
hipError_t run_fwd(const Sweep& p) {
  if (p.KD <= 64) return p.VD <= 64 ? fwd_kernel<T, 64, 64>(p) : fwd_kernel<T, 64, 128>(p);
  return p.VD <= 64 ? fwd_kernel<T, 128, 64>(p) : fwd_kernel<T, 128, 128>(p);
}

template <typename T, int DKP, int DVP, bool GATE>
hipError_t bwd_kernel(const Sweep& dq, const Sweep& dk, const Sweep& dv) {
  const int64_t n = dq.b * dq.H * dq.n_segs;
  const bool vec = sweep_pieces<T>(dq) && sweep_pieces<T>(dk) && sweep_pieces<T>(dv);
  return vec ? launch_kind(kKindLinSweep, lin_bwd_kernel<T, DKP, DVP, GATE, true>, 3 * n, 2 * kThreads, dq.stream, dq, dk, dv, int(n))
             : launch_kind(kKindLinSweep, lin_bwd_kernel<T, DKP, DVP, GATE, false>, 3 * n, 2 * kThreads, dq.stream, dq, dk, dv, int(n));
}
template <typename T, bool GATE>
hipError_t bwd_sizes(const Sweep& dq, const Sweep& dk, const Sweep& dv) {
  if (dv.KD <= 64) return dv.VD <= 64 ? bwd_kernel<T, 64, 64, GATE>(dq, dk, dv) : bwd_kernel<T, 64, 128, GATE>(dq, dk, dv);
  return dv.VD <= 64 ? bwd_kernel<T, 128, 64, GATE>(dq, dk, dv) : bwd_kernel<T, 128, 128, GATE>(dq, dk, dv);
}

template <typename T, int KDP, int VDP>
hipError_t state_kernel(const Sweep& p, const Sweep& q, int sweeps, bool vec) {
  const int64_t n = p.b * p.H * p.n_parts;
  return vec ? launch_kind(kKindLinState, lin_state_kernel<T, KDP, VDP, true>, sweeps * n, kThreads, p.stream, p, q, int(n))
             : launch_kind(kKindLinState, lin_state_kernel<T, KDP, VDP, false>, sweeps * n, kThreads, p.stream, p, q, int(n));
}
// States leaving the parts of a cut sequence, for one sweep or two of the same sizes: every part's own, then the chain
// over them.
template <typename T>
hipError_t run_states(const Sweep& p, const Sweep& q, int sweeps) {
  if (p.n_segs <= 1) return hipSuccess;
  const bool vec = pieces<T>(p.xk, p.KD) && pieces<T>(p.xv, p.VD) && pieces<T>(q.xk, q.KD) && pieces<T>(q.xv, q.VD);
  hipError_t err = p.KD <= 64 ? (p.VD <= 64 ? state_kernel<T, 64, 64>(p, q, sweeps, vec) : state_kernel<T, 64, 128>(p, q, sweeps, vec))
                              : (p.VD <= 64 ? state_kernel<T, 128, 64>(p, q, sweeps, vec) : state_kernel<T, 128, 128>(p, q, sweeps, vec));
  for (int k = 0; k < sweeps && err == hipSuccess; k++) {
    const Sweep& s = k ? q : p;
    if (s.n_parts == 1 && !s.init) continue;  // the one part's own state is the one that leaves it
    ChainArgs c{};
    c.agg = s.seg_state; c.sums = s.seg_decay;
    c.init = s.init;
    c.outer = s.b; c.mid = s.H; c.inner = s.KD * s.VD; c.N = c.inner;
    c.n_chunks = c.K = s.n_parts;
    err = launch_chain<false, false, false>(kKindLinChain, c, s.stream);
  }
  return err;
}

// The cut of a sequence: as many segments as give every CU a workgroup, and no second generation of them
// (a cut costs another reading of keys and values), so from 129 heads of batch rows on (43 in the backward) none; of at
// least kMinSeg chunks.  Measured, bf16, b8 L2048 H24 D64:
// 66 us in one piece, 96 us in two; b2 L8192 H32 D128: 422, 345, 246, 208 and 257 us in 1 to 5.
constexpr int kMinSeg = 4;
constexpr int64_t kAtOnce = 256;
struct Cut {
  int n_chunks, n_segs, parts, part_chunks, n_parts;
};
Cut cut_of(const LinAttnArgs& a, bool backward) {
  Cut c;
  c.n_chunks = int(ceil_div(a.L, a.dtype == 0 ? kChunk<float> : kChunk<bf16_bits>));
  const int64_t heads = a.b * a.H, sweeps = backward ? 3 : 1;
  const int64_t want = std::max<int64_t>(1, kAtOnce / std::max<int64_t>(heads * sweeps, 1));
  const int64_t segs = std::min(want, std::max<int64_t>(1, c.n_chunks / kMinSeg));
  int64_t seg = std::max<int64_t>(1, ceil_div(c.n_chunks, segs));
  c.parts = 1;
  if (segs > 1) {  // parts for two generations of the smaller workgroups of the states' pass
    const int64_t more = 2 * kAtOnce / std::max<int64_t>(heads * (segs - 1) * (backward ? 2 : 1), 1);
    c.parts = int(std::max<int64_t>(1, std::min(more, seg / kMinSeg)));
  }
  c.part_chunks = int(ceil_div(seg, c.parts));
  seg = int64_t(c.part_chunks) * c.parts;
  c.n_segs = int(std::max<int64_t>(1, ceil_div(c.n_chunks, seg)));
  c.n_parts = (c.n_segs - 1) * c.parts;
  return c;
}

Sweep common(const LinAttnArgs& a, bool backward) {
  Sweep p{};
  p.g = a.g; p.A = a.A; p.lengths = a.lengths;
  p.wscale = p.rscale = 1.f;
  p.gq = p.gk = p.gv = p.gd = 1;
  p.b = a.b; p.L = a.L; p.H = int(a.H);
  const Cut c = cut_of(a, backward);
  p.n_chunks = c.n_chunks; p.n_segs = c.n_segs; p.parts = c.parts; p.part_chunks = c.part_chunks; p.n_parts = c.n_parts;
  p.stream = a.stream;
  return p;
}

// Bytes from the workspace's start of its parts.
struct Work {
  size_t seg_f, dec_f, seg_r, dec_r;  // segment states and decays, forwards and (backward) in reversed time
  size_t dot_q, dot_k, end, sums, resets, dq, dk, total;
  int n_tiles;
};
Work plan_work(const LinAttnArgs& a, bool backward) {
  Work w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += up256(bytes);
    return r;
  };
  const size_t heads = size_t(a.b) * a.H, segs = heads * cut_of(a, backward).n_parts;
  w.seg_f = take(segs * a.Dk * a.Dv * 4);
  w.dec_f = take(segs * 4);
  if (backward) {
    const size_t rows = heads * a.L;
    w.n_tiles = int(ceil_div(a.L, kGateTile));
    w.seg_r = take(segs * a.Dk * a.Dv * 4);
    w.dec_r = take(segs * 4);
    w.dot_q = take(rows * (a.dtype == 0 ? sizeof(Dot<float>) : sizeof(Dot<bf16_bits>)));
    w.dot_k = take(rows * (a.dtype == 0 ? sizeof(Dot<float>) : sizeof(Dot<bf16_bits>)));
    w.end = take(heads * sizeof(double));
    w.sums = take(heads * w.n_tiles * 8);
    w.resets = take(heads * w.n_tiles);
    if (a.G != a.H) {
      w.dq = take(rows * a.Dk * 4);
      w.dk = take(rows * a.Dk * 4);
    }
  }
  w.total = at;
  return w;
}

template <typename T>
hipError_t fwd_impl(const LinAttnArgs& a, char* ws) {
  const Work w = plan_work(a, false);
  const int share = int(a.H / a.G);
  Sweep p = common(a, false);
  p.xq = a.q; p.xk = a.k; p.xv = a.v; p.gq = p.gk = share;
  p.KD = int(a.Dk); p.VD = int(a.Dv);
  p.rscale = a.scale;
  p.init = a.h0;
  p.seg_state = reinterpret_cast<float*>(ws + w.seg_f); p.seg_decay = reinterpret_cast<float*>(ws + w.dec_f);
  p.exact = true;
  const hipError_t err = run_states<T>(p, p, 1);
  if (err != hipSuccess) return err;
  p.out = a.y;
  p.last = a.last;
  return run_fwd<T>(p);
}

template <typename T>
hipError_t bwd_impl(const LinAttnArgs& a, char* ws) {
  const Work w = plan_work(a, true);
  const int share = int(a.H / a.G);
  const bool gate = a.dg != nullptr;
  Dot<T>* end = gate && a.dlast ? reinterpret_cast<Dot<T>*>(ws + w.end) : nullptr;
  float* seg_f = reinterpret_cast<float*>(ws + w.seg_f);
  float* dec_f = reinterpret_cast<float*>(ws + w.dec_f);
  float* seg_r = reinterpret_cast<float*>(ws + w.seg_r);
  float* dec_r = reinterpret_cast<float*>(ws + w.dec_r);
  hipError_t err = hipSuccess;
  if (common(a, true).n_segs > 1) {  // the segments' S and D, [Dk, Dv]; dq and dk read them transposed
    Sweep f = common(a, true), r = common(a, true);
    f.xk = a.k; f.gk = share; f.xv = a.v;
    f.init = a.h0; f.seg_state = seg_f; f.seg_decay = dec_f;
    r.xk = a.q; r.gk = share; r.xv = a.dy;
    r.wscale = a.scale; r.reverse = true;
    r.init = a.dlast; r.seg_state = seg_r; r.seg_decay = dec_r;
    r.exact = true;
    f.KD = r.KD = int(a.Dk); f.VD = r.VD = int(a.Dv);
    err = run_states<T>(f, r, 2);
    if (err != hipSuccess) return err;
  }
  Sweep dq = common(a, true);  // forwards, the state is S^T [Dv, Dk]
  dq.xq = a.dy; dq.xk = a.v; dq.xv = a.k; dq.gv = share;
  dq.KD = int(a.Dv); dq.VD = int(a.Dk);
  dq.rscale = a.scale;
  dq.init = a.h0; dq.init_t = true; dq.seg_state = seg_f;
  dq.out = share > 1 ? static_cast<void*>(ws + w.dq) : a.dq; dq.out_f32 = share > 1;
  Sweep dk = common(a, true);  // backwards, the state is D^T [Dv, Dk]
  dk.xq = a.v; dk.xk = a.dy; dk.xv = a.q; dk.gv = share;
  dk.KD = int(a.Dv); dk.VD = int(a.Dk);
  dk.wscale = a.scale; dk.reverse = true;
  dk.init = a.dlast; dk.init_t = true; dk.seg_state = seg_r;
  dk.out = share > 1 ? static_cast<void*>(ws + w.dk) : a.dk; dk.out_f32 = share > 1;
  Sweep dv = common(a, true);  // backwards, the state is D [Dk, Dv]
  dv.xq = a.k; dv.gq = share; dv.xk = a.q; dv.gk = share; dv.xv = a.dy;
  dv.KD = int(a.Dk); dv.VD = int(a.Dv);
  dv.wscale = a.scale; dv.reverse = true;
  dv.init = a.dlast; dv.seg_state = seg_r;
  dv.out = a.dv;
  dv.last = a.dh0; dv.final_decay = true;
  dv.exact = true;
  if (gate) {
    dq.xd = a.q; dk.xd = a.k;
    dq.gd = dk.gd = share;
    dq.dots = ws + w.dot_q;
    dk.dots = ws + w.dot_k;
    dq.dstate = a.dlast;
    dq.dstate_dot = end;
  }
  err = gate ? bwd_sizes<T, true>(dq, dk, dv) : bwd_sizes<T, false>(dq, dk, dv);
  if (err != hipSuccess || a.L == 0) return err;
  if (share > 1) {
    const int64_t n = a.b * a.L * a.G * a.Dk;
    for (int k = 0; k < 2; k++) {
      const float* in = reinterpret_cast<const float*>(ws + (k ? w.dk : w.dq));
      T* out = static_cast<T*>(k ? a.dk : a.dq);
      const bool vec = a.Dk % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0;
      err = vec ? launch_kind(kKindLinReduce, lin_group_sum_kernel<T, 4>, std::min(ceil_div(n, 1024), kSumBlocks), 256, a.stream, in, out, n, share, int(a.Dk))
                : launch_kind(kKindLinReduce, lin_group_sum_kernel<T, 1>, std::min(ceil_div(n, 256), kSumBlocks), 256, a.stream, in, out, n, share, int(a.Dk));
      if (err != hipSuccess) return err;
    }
  }
  if (gate) {
    const int h_blocks = int(ceil_div(a.H, kGateHeads));
    GateArgs<T> p{};
    p.a = reinterpret_cast<const Dot<T>*>(ws + w.dot_q); p.c = reinterpret_cast<const Dot<T>*>(ws + w.dot_k);
    p.sums = reinterpret_cast<double*>(ws + w.sums); p.resets = reinterpret_cast<uint8_t*>(ws + w.resets);
    p.end = end;
    p.g = static_cast<const T*>(a.g); p.A = a.A; p.lengths = a.lengths; p.dg = static_cast<T*>(a.dg);
    p.L = a.L; p.H = int(a.H); p.n_tiles = w.n_tiles; p.h_blocks = h_blocks;
    const int64_t blocks = a.b * w.n_tiles * h_blocks;
    err = launch_kind(kKindLinGate, lin_gate_tiles_kernel<T>, blocks, 256, a.stream, p);
    if (err != hipSuccess) return err;
    err = launch_kind(kKindLinGate, lin_gate_kernel<T>, blocks, 256, a.stream, p);
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
  if (a.b == 0 || a.H == 0) return 0;
  return plan_work(a, backward).total;
}

hipError_t launch_linattn_fwd(const LinAttnArgs& a, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  return a.dtype == 0 ? fwd_impl<float>(a, ws) : fwd_impl<bf16_bits>(a, ws);
}

hipError_t launch_linattn_bwd(const LinAttnArgs& a, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  return a.dtype == 0 ? bwd_impl<float>(a, ws) : bwd_impl<bf16_bits>(a, ws);
}

hipError_t launch_linattn_update(const LinAttnArgs& a) {
  return a.dtype == 0 ? update_impl<float>(a) : update_impl<bf16_bits>(a);
}

}  // namespace ssm
