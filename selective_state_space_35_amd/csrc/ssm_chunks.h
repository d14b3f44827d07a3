// Device code that the mixers computed in chunks of matrix products share (linear attention, the gated delta rule):
// operand fragments, tiles in LDS and their staging, decays of a chunk.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"

namespace ssm {

// A log decay below -10^4 counts as -10^4 (its factor is zero in float either way), so that
// minus infinity is a reset and differences of running sums stay numbers.
__device__ __forceinline__ float clamp_log(float x) { return x < -1e4f ? -1e4f : x; }

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
  // Params has the sweep's g, A, reverse, L and H
  template <typename Params>
  __device__ __forceinline__ void init(const Params& p, const Place& w, int c0) {
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

}  // namespace ssm
