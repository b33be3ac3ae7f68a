// Device-side building blocks of the block operators (linear, gated feed-forward,
// structure attention, norm): MFMA fragments, transposed fragment reads, activations.
//
// One 16x16 MFMA tile contracts CK values (bf16: 32, float32: 16 as four steps of 4).
// Lane l = 16 g + i holds, for both operands, index i and EV consecutive or grouped
// values of the contracted index; the result lane holds rows 4g .. 4g+3 of column i.
// Which EV contracted values a lane group g holds is free as long as both operands agree:
//   natural order   k = EV g + j                (rows of a matrix, EV consecutive channels)
//   tile order      k = 16 t + 4 g + r, j = 4 t + r   (bf16: tiles t = 0, 1; float32: t = 0)
// Tile order is how results of one product already sit in a lane, so a product's result
// (rounded to bf16 for bf16 features) is the next product's operand without any exchange
// between lanes; the other operand is then read in tile order too, transposed, from LDS.
// For float32 (EV = 4, one tile) the two orders are the same.
#pragma once
#include <type_traits>

#include "common.hpp"

namespace mdmp {
namespace ops {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

template <class T>
struct MF;  // T: storage type of the features (float, or uint16_t for bf16)
template <>
struct MF<uint16_t> {
  using F = s8;
  static constexpr int CK = 32, EV = 8, NT = 2;  // contracted length, values per lane, 16-row tiles of it
  static __device__ __forceinline__ f4 mma(f4 acc, F a, F b) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), acc, 0, 0,
                                                   0);
  }
  // two result tiles -> one operand, rounded to nearest even
  static __device__ __forceinline__ F pack(const f4* t) {
    u4 u{pk2bf(t[0].x, t[0].y), pk2bf(t[0].z, t[0].w), pk2bf(t[1].x, t[1].y), pk2bf(t[1].z, t[1].w)};
    return __builtin_bit_cast(F, u);
  }
  static __device__ __forceinline__ void unpack(F f, f4* t) {
    const u4 u = __builtin_bit_cast(u4, f);
#pragma unroll
    for (int z = 0; z < 2; ++z)
      t[z] = f4{__uint_as_float(u[2 * z] << 16), __uint_as_float(u[2 * z] & 0xffff0000u),
                __uint_as_float(u[2 * z + 1] << 16), __uint_as_float(u[2 * z + 1] & 0xffff0000u)};
  }
};
template <>
struct MF<float> {
  using F = f4;
  static constexpr int CK = 16, EV = 4, NT = 1;
  static __device__ __forceinline__ f4 mma(f4 acc, F a, F b) {
#pragma unroll
    for (int z = 0; z < 4; ++z) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[z], b[z], acc, 0, 0, 0);
    return acc;
  }
  static __device__ __forceinline__ F pack(const f4* t) { return t[0]; }
  static __device__ __forceinline__ void unpack(F f, f4* t) { t[0] = f; }
};

// 16 bytes of zeros, and a 16-byte load that reads zeros where !on
template <class F>
__device__ __forceinline__ F zero16() {
  return __builtin_bit_cast(F, u4{0u, 0u, 0u, 0u});
}
template <class F, class T>
__device__ __forceinline__ F ld16(const T* p, bool on) {
  return on ? *(const F*)p : zero16<F>();
}

// Padding of a row of a matrix in LDS, in elements.  bf16: 32 bytes, so that rows of C or of 32
// elements are 32 bytes off a multiple of 64 and both 16-byte reads of 16 consecutive rows and
// transposed reads of rows 4 g + r meet no bank twice (measured: 16 bytes of padding cost a
// conflict in every read); float32: 16 bytes, its transposed reads take single words.
template <class T>
constexpr int lds_pad() {
  return sizeof(T) == 2 ? 16 : 4;
}

// Transposed operand in tile order from an LDS matrix m[k][RS]: index = column col + i, contracted
// = rows k0 + 16 t + 4 g + r.  bf16: each group of 16 lanes reads four rows of 16 columns, lane
// 4 r + s the columns 4 s .. 4 s + 3 of row r, and lane i receives column i of the four rows
// (ds_read_b64_tr_b16).
template <int RS>
__device__ __forceinline__ s8 ldt(const uint16_t* m, int k0, int col, int lane) {
  const uint16_t* p = m + (k0 + 4 * (lane >> 4) + ((lane & 15) >> 2)) * RS + col + 4 * (lane & 3);
  const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p);
  const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(p + 16 * RS));
  return s8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
template <int RS>
__device__ __forceinline__ f4 ldt(const float* m, int k0, int col, int lane) {
  const float* p = m + (k0 + 4 * (lane >> 4)) * RS + col + (lane & 15);
  return f4{p[0], p[RS], p[2 * RS], p[3 * RS]};
}

// Row of a CK-row group that index i of result tile t stands for, such that the NT result
// tiles of a lane hold EV consecutive rows EV g .. EV g + EV - 1 (natural order)
template <class T>
__device__ __forceinline__ int nat_row(int t, int i) {
  if constexpr (sizeof(T) == 2)
    return 8 * (i >> 2) + 4 * t + (i & 3);
  else
    return i;
}
// Row 16 t + i in which row x = nat_row(t, i) of a group is stored: a group stored so is read by
// rows in the order nat_row, and transposed (ldt) with the contracted rows in natural order
template <class T>
__device__ __forceinline__ int nat_slot(int x) {
  if constexpr (sizeof(T) == 2)
    return x / 32 * 32 + 16 * ((x >> 2) & 1) + 4 * ((x >> 3) & 3) + (x & 3);
  else
    return x;
}

// A [ROWS][C] tile from global rows (stride ld) to LDS rows (stride RS), by NTH threads in
// 16-byte pieces: fetch() issues the loads into registers, put() stores them.  Rows at or
// past `rows` read as zeros.
template <class T, int ROWS, int C, int RS, int NTH>
struct Tile {
  static constexpr int EV = MF<T>::EV, VPR = C / EV, TOT = ROWS * VPR, IT = (TOT + NTH - 1) / NTH;
  u4 v[IT];
  __device__ __forceinline__ void fetch(const T* __restrict__ src, int64_t ld, int rows, int tid) {
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int x = tid + k * NTH, r = x / VPR, c = (x % VPR) * EV;
      v[k] = ld16<u4>(src + r * ld + c, (TOT % NTH == 0 || x < TOT) && r < rows);
    }
  }
  __device__ __forceinline__ void put(T* dst, int tid) const {
    put(dst, tid, [](int r) { return r; });
  }
  // row r stored as row slot(r)
  template <class SLOT>
  __device__ __forceinline__ void put(T* dst, int tid, SLOT slot) const {
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int x = tid + k * NTH, r = x / VPR, c = (x % VPR) * EV;
      if (TOT % NTH == 0 || x < TOT) *(u4*)(dst + slot(r) * RS + c) = v[k];
    }
  }
};

// What rounding left of the tiles that p packs, as a second operand: p and it are the tiles to 2^-17.
// Worth its products where few rows leave the matrix cores idle; float32 rounds nothing.
template <class T>
__device__ __forceinline__ typename MF<T>::F rest_of(typename MF<T>::F p, const f4* t) {
  using M = MF<T>;
  f4 r[M::NT];
  M::unpack(p, r);
#pragma unroll
  for (int z = 0; z < M::NT; ++z) r[z] = t[z] - r[z];
  return M::pack(r);
}

// EV consecutive elements of a row as float / from float
template <class T>
__device__ __forceinline__ void st_row(T* p, const f4* t) {
  *(typename MF<T>::F*)p = MF<T>::pack(t);
}

// the same, past the caches if STREAM (a compile-time choice: stores that differ in nothing else are
// merged, and lose the hint)
template <bool STREAM, class T>
__device__ __forceinline__ void st_row(T* p, const f4* t) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(__builtin_bit_cast(u4, MF<T>::pack(t)), (u4*)p);
  else
    st_row<T>(p, t);
}

// four consecutive elements
__device__ __forceinline__ void st4(float* p, f4 v) { *(f4*)p = v; }
__device__ __forceinline__ void st4(uint16_t* p, f4 v) { *(u2*)p = u2{pk2bf(v.x, v.y), pk2bf(v.z, v.w)}; }

// Sum over the four waves of a block of their [16 atoms][C] results, then rows out
template <class T, int C, class ROW>
__device__ __forceinline__ void join_waves(float* slab, int64_t a0, int64_t n, ROW row) {
  using M = MF<T>;
  constexpr int EV = M::EV, NT = M::NT, OS = C + 4;
  __syncthreads();
  for (int x = threadIdx.x; x < 16 * (C / EV); x += 256) {
    const int r = x / (C / EV), c = (x % (C / EV)) * EV;
    if (a0 + r >= n) break;
    f4 o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      o[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) o[t] += *(const f4*)(slab + (16 * w + r) * OS + c + 4 * t);
    }
    row(a0 + r, c, o);
  }
}

// orders the LDS accesses of one wave (its lanes exchange data through LDS it alone uses)
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// barrier of a block for its LDS accesses alone: loads from memory may stay in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Asks the scheduler to read operands from LDS ahead of their products: AHEAD reads first, then N
// times MFMAS products and READS reads, then REST products.  Left alone it reads each operand just
// before its products and waits out the LDS latency every time.
template <int AHEAD, int N, int MFMAS, int READS, int REST>
__device__ __forceinline__ void read_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
  for (int q = 0; q < N; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, REST, 0);
}

// sum over the four lane groups (lanes i, 16 + i, 32 + i, 48 + i)
__device__ __forceinline__ float gsum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float gmax(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}

constexpr float kLog2e = 1.4426950408889634f;

// Activations.  With s = sigmoid(z): value s (a z + b), derivative s (a + (a z + b)(1 - s));
// (a, b) = (1, 0) is SiLU, (0, 1) the sigmoid.
struct ActAB {
  float a, b;
};
__device__ __forceinline__ float act_val(float z, ActAB c) { return sigm(z) * (c.a * z + c.b); }
__device__ __forceinline__ void act_both(float z, ActAB c, float& v, float& d) {
  const float s = sigm(z), w = c.a * z + c.b;
  v = s * w;
  d = s * (c.a + w * (1.0f - s));
}

}  // namespace ops
}  // namespace mdmp
