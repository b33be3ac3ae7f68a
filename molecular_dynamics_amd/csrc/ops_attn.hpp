// Attention between all atoms of each structure: kernels (the calls: ops_attn.cpp).
//
// Scores are held in base 2: x = log2(e) (s - slope r), p = 2^(x - m).
//
// Layout.  A wave owns 16 atoms of one structure (queries in the forward and the row pass,
// keys in the column pass) as the columns of its MFMA tiles and walks the other side CK atoms
// at a time.  Scores are formed transposed, S[other][own] = K Q^T, so a lane holds scores of
// ONE own atom against 4 (x NT) others, in tile order: softmax weights and score gradients
// are the next product's operand without leaving their lanes, and the distance of a pair is
// formed once and used by every head (all C channels are in the wave).
//   NW = 1  short structures: a block is one wave, which stages what it needs for itself
//   NW = 4  long structures: the four waves of a block own 64 adjacent atoms of one structure and
//           share each step of the other side in LDS (two buffers, one barrier a step); few long
//           structures also split the other side over gridDim.y blocks, which leave float32
//           partial sums that a last kernel joins in order, so equal inputs give equal bits.
//
// A wave never straddles structures: slots of R = 16 NW atoms are numbered so that structure b
// owns slots s_b / R + b .. (floor), which needs no pass over the sizes; the structure of a slot
// is found by a 64-way search.  At most one slot per structure stays empty.
//
// Masked atoms and rows past the structure are staged as zeros and their scores set to -inf,
// so nothing they hold (NaN, infinities) reaches another atom.
//
// Bound: VALU.  A score costs one exp at a quarter of the rate and about a dozen plain operations
// beside 128 matrix operations (32 channels a head), 1/8 of its VALU time.  Measured, four heads of 32:
//   16,384 molecules of 8-32 atoms, bf16, forward     86 us  (its bytes at a copy's rate: 69)
//   16,411 atoms in one structure, bf16, capped, fwd 577 us  + join 14  (1.08e9 scores, 483 VALU
//                                                    instructions a wave for 16 x 32 pairs, four heads)
//   4,096 molecules of 1-40 atoms, bf16, capped: fwd 40-45, row pass 60, column pass 56 us
//   4,096 atoms, one periodic box, float32: fwd 123, row 177, col 206 us, joins 16 and 20
#pragma once
#include <algorithm>

#include "ops.hpp"

namespace mdmp {
namespace ops {

// A cap far above the scores does nothing, and 1 - 2 / (e^2y + 1) would spend its digits on it
inline bool cap_ok(float cap) { return cap == 0.f || (cap >= 1e-3f && cap <= 1e4f); }

struct AttnArgs {
  int n, n_struct;
  const int32_t* sptr;
  const float* pos;
  const float* slope;
  const uint8_t* mask;
  const void *q, *k, *v, *o, *dout;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
  double to_fix;    // 2^32 / box_L, 0: open
  float unit;       // length of one unit of a coordinate difference (box_L / 2^32, or 1)
  float scale;      // 1 / sqrt(d)
  // log-sums are held less lsub, about log2 of a structure's size, where it would take their digits:
  // with 4,096 atoms they are near 12, x - lse is rounded to 2^-21 before the exponential, and dpos
  // lost half of float32's quality (3.5e-6 off).  The backward passes' weights are then 2^lsub p, and
  // p_scale = 2^-lsub enters their results once.
  float lsub, p_scale;
  float cap;        // 0: none
  float tp[6], cap_near, cap_exp;  // the cap's polynomial, the scores it holds for, factor of the exponential beyond
  void *out, *dq, *dk, *dv;
  float *lse, *o32;    // saved: [n][H] base-2 log-sum, [n][C] unrounded output (bf16 only)
  float *dpos, *dslope_part, *dsum;  // [n][3]; [splits][slots][H]; [n][H] sum_c dout out
  // splits of the other side (gridDim.y) and, above 1, their partial sums: rows [splits][n][C] of
  // out, dq, dk, dv; (m, l) [splits][n][H][2]; position gradients [splits][n][3] of either pass
  int splits;
  float *p_out, *p_ml, *p_dq, *p_dk, *p_dv, *p_row, *p_col;
};

// Coordinates as 32-bit words.  Periodic: fixed point in units of box_L / 2^32, so the
// difference of two wraps into the minimum image by itself, with the border decided to 2^-32
// of the box; open: the floats themselves.
struct P3 {
  uint32_t x, y, z;
};
__device__ __forceinline__ uint32_t coord(float x, double to_fix) {
  return to_fix > 0 ? (uint32_t)(int64_t)rint((double)x * to_fix) : __float_as_uint(x);
}
__device__ __forceinline__ P3 load_pos(const AttnArgs& A, int i, bool on) {
  if (!on || !A.pos) return P3{0u, 0u, 0u};
  const float* p = A.pos + 3 * (int64_t)i;
  return P3{coord(p[0], A.to_fix), coord(p[1], A.to_fix), coord(p[2], A.to_fix)};
}
// other - own
__device__ __forceinline__ void diff(const P3& own, const u4& o, bool fix, float& dx, float& dy, float& dz) {
  if (fix) {
    dx = (float)(int32_t)(o.x - own.x);
    dy = (float)(int32_t)(o.y - own.y);
    dz = (float)(int32_t)(o.z - own.z);
  } else {
    dx = __uint_as_float(o.x) - __uint_as_float(own.x);
    dy = __uint_as_float(o.y) - __uint_as_float(own.y);
    dz = __uint_as_float(o.z) - __uint_as_float(own.z);
  }
}
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// a value that is equal in every lane, as a scalar
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Structure and row range of tile slot `slot` (R rows per slot); false: the slot is empty.
// Row bounds are clamped to [0, n], so no struct_ptr can lead out of the arrays.
// The first 64 entries looked at lie about where the slot is if sizes are even, which mostly holds
// them; they are read once and the structure's bounds taken from their lanes.
template <int R>
__device__ __forceinline__ bool find_slot(const AttnArgs& A, int slot, int lane, int& row0, int& s, int& e) {
  auto at = [&](int b) { return min(max(A.sptr[min(b, A.n_struct)], 0), A.n); };
  const int guess = (int)((int64_t)slot * A.n_struct / (A.n / R + A.n_struct));
  int base = max(0, min(guess - 32, A.n_struct - 63)), b, lo = 0, hi = A.n_struct - 1;
  int v = at(base + lane);
  int k = __popcll(__ballot(base + lane < A.n_struct && v / R + base + lane <= slot));
  if (k > 0 && k < 64) {
    b = base + k - 1;
    s = __builtin_amdgcn_readlane(v, k - 1);
    e = __builtin_amdgcn_readlane(v, k);
  } else {
    if (k == 0)
      hi = base - 1;
    else
      lo = base + 63;
    while (lo < hi) {
      const int step = (hi - lo + 64) / 64;  // ceil((hi - lo + 1) / 64)
      const int p = lo + lane * step;
      k = __popcll(__ballot(p <= hi && at(min(p, hi)) / R + p <= slot));
      if (k == 0) return false;
      lo += (k - 1) * step;
      hi = min(hi, lo + step - 1);
    }
    if (lo > hi) return false;
    b = lo;
    s = uniform(at(b));
    e = uniform(at(b + 1));
  }
  e = max(e, s);
  const int t = slot - (s / R + b);
  row0 = s + t * R;
  return t >= 0 && row0 < e;
}

// The CK atoms from k0 on of the other side: one bit each, whether they take part
template <int CK>
__device__ __forceinline__ uint64_t live(const AttnArgs& A, int k0, int e, int lane, bool masked) {
  const bool on = lane < CK && k0 + lane < e && (!masked || !A.mask || A.mask[k0 + lane] != 0);
  return __ballot(on);
}
template <int CK>
constexpr uint64_t all_live() {
  return (1ull << CK) - 1;
}

// CK rows of a matrix from row k0 on: a copy in LDS by NTH threads (rows of RS), or MFMA operands in
// natural order, frag[t][ch] = row 16 t + i.  Row k0 is the same for the wave, so an address is a
// scalar base and a 32-bit lane offset (rows are at most 2^24 elements long).  Rows past the
// structure (rows < CK of them left) are read as its last row, and cleared where their contents
// matter by the caller.
template <class T, int C, int RS, int NTH>
struct StepTile {
  static constexpr int CK = MF<T>::CK, EV = MF<T>::EV, VPR = C / EV, TOT = CK * VPR, IT = (TOT + NTH - 1) / NTH;
  static constexpr int RJ = NTH / VPR;
  static_assert(NTH % VPR == 0 && (TOT % NTH == 0 || TOT < NTH), "whole rows");
  u4 v[IT];
  static __device__ __forceinline__ bool in(int tid) { return TOT >= NTH || tid < TOT; }
  __device__ __forceinline__ void fetch(const T* src, int64_t ld, int64_t k0, int rows, int tid) {
    const T* p = src + k0 * ld;
    const uint32_t r = tid / VPR, c = (tid % VPR) * EV;
    if (!in(tid)) return;
    if (rows >= CK) {
      const uint32_t off = r * (uint32_t)ld + c;
#pragma unroll
      for (int j = 0; j < IT; ++j) v[j] = *(const u4*)(p + j * RJ * ld + off);
    } else {
#pragma unroll
      for (int j = 0; j < IT; ++j) v[j] = *(const u4*)(p + min(r + j * RJ, (uint32_t)rows - 1) * (uint32_t)ld + c);
    }
  }
  // rows without their bit become zeros
  __device__ __forceinline__ void clear(uint64_t on, int tid) {
    const uint32_t m = (uint32_t)on >> (tid / VPR % 32);
#pragma unroll
    for (int j = 0; j < IT; ++j)
      if (!((m >> (j * RJ % 32)) & 1)) v[j] = u4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void put(T* dst, int tid) const {
    if (!in(tid)) return;
#pragma unroll
    for (int j = 0; j < IT; ++j) *(u4*)(dst + (tid / VPR + j * RJ) * RS + (tid % VPR) * EV) = v[j];
  }
};
// chunks c0 .. c1 - 1 of the operands of NTL tiles
template <class T, int C, int NTL>
__device__ __forceinline__ void load_frags(typename MF<T>::F (&f)[NTL][C / MF<T>::CK], const T* src, int64_t ld,
                                           int64_t k0, int rows, int i, int g, int c0 = 0, int c1 = C / MF<T>::CK) {
  using M = MF<T>;
  const T* p = src + k0 * ld;
#pragma unroll
  for (int t = 0; t < NTL; ++t) {
    uint32_t r = 16 * t + i;
    if (rows < 16 * NTL) r = min(r, (uint32_t)rows - 1);
    const uint32_t off = r * (uint32_t)ld + M::EV * g;
#pragma unroll
    for (int ch = 0; ch < C / M::CK; ++ch)
      if (ch >= c0 && ch < c1) f[t][ch] = *(const typename M::F*)(p + off + ch * M::CK);
  }
}

// sum over head h's channels of the product of an operand pair: acc += A B over the channel
// chunks of the head.  Heads narrower than a chunk (bf16, 16 channels) take the chunk with
// the other head's lane groups of one operand zeroed.
template <class T, int DH, int NC>
__device__ __forceinline__ f4 head_mma(f4 acc, const typename MF<T>::F (&a)[NC], const typename MF<T>::F (&b)[NC],
                                       int h, int g) {
  using M = MF<T>;
  if constexpr (DH >= M::CK) {
#pragma unroll
    for (int c = 0; c < DH / M::CK; ++c) acc = M::mma(acc, a[h * (DH / M::CK) + c], b[h * (DH / M::CK) + c]);
  } else {
    static_assert(DH * 2 == M::CK, "two heads in a chunk");
    const typename M::F bh = (g >> 1) == (h & 1) ? b[h / 2] : zero16<typename M::F>();
    acc = M::mma(acc, a[h / 2], bh);
  }
  return acc;
}

// whether chunk ch of a row holds channels of head h in lane group g
template <class T, int DH>
__device__ __forceinline__ bool lane_in_head(int ch, int g, int h) {
  if constexpr (DH >= MF<T>::CK)
    return ch / (DH / MF<T>::CK) == h;
  else
    return 2 * ch + (g >> 1) == h;
}

// the channel chunks of head h: chunk_of(h) .. + chunks() - 1 (heads of half a chunk: the one it is in)
template <class T, int DH>
constexpr int chunks() {
  return DH >= MF<T>::CK ? DH / MF<T>::CK : 1;
}
template <class T, int DH>
constexpr int chunk_of(int h) {
  return DH >= MF<T>::CK ? h * (DH / MF<T>::CK) : h / 2;
}

// Scores in base 2: x = k f(S) + b with S the product of a query and a key: f = S without a cap, else
// f = tanh(y), y = S / (sqrt(d) cap).  Up to |y| = 0.75 tanh is S times a polynomial of NP terms in S^2,
// whose coefficients (tanh_terms, with the powers of S's factor and, in the forward, k in them) the
// host makes; beyond, in a step where a wave has any such score, 1 - 2 / (e^2y + 1) (an absolute error
// of 1e-7, 2e-7 of tanh there).  Neither exponential nor reciprocal, at a quarter of the rate, is needed for
// most steps: 16,411 atoms bf16, cap 20: a pass of 591 us against 657 with them.
constexpr float kCapNear = 0.75f;
template <int NP>
__device__ __forceinline__ float cap_near(const AttnArgs& A, float s) {  // the factor of s
  const float w = s * s;
  float f = A.tp[NP - 1];
#pragma unroll
  for (int z = NP - 2; z >= 0; --z) f = fmaf(w, f, A.tp[z]);
  return f;
}
__device__ __forceinline__ bool far_off(const AttnArgs& A, f4 x) {
  return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))) > A.cap_near;
}
// f such that s f = k tanh(y); a far score becomes 1 and f its value
template <int NP, int NT>
__device__ __forceinline__ void cap_factors(const AttnArgs& A, float k, f4 (&s)[NT], f4 (&f)[NT]) {
  bool far = false;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    far |= far_off(A, s[t]);
#pragma unroll
    for (int q = 0; q < 4; ++q) f[t][q] = cap_near<NP>(A, s[t][q]);
  }
  if (__any(far)) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float e = k * (1.0f - 2.0f * rcp(ex2(s[t][q] * A.cap_exp) + 1.0f));
        const bool on = fabsf(s[t][q]) > A.cap_near;
        f[t][q] = on ? e : f[t][q];
        s[t][q] = on ? 1.0f : s[t][q];
      }
  }
}
// tanh(y) = y (c_0 + c_1 y^2 + ...) up to 0.75 with the least relative error for so many terms: 3e-8, and
// 1.1e-5 in a forward pass over bf16 features that nothing follows: at a capped score of 20 that is
// 3e-4 of a weight, which is then rounded to 2^-9
template <int NP>
inline const double* tanh_terms() {
  static const double c4[4] = {0.99998898, -0.33269670, 0.12742689, -0.03545268};
  static const double c6[6] = {0.99999997, -0.33332959, 0.13325406, -0.05334442, 0.01958290, -0.00471625};
  return NP == 4 ? c4 : c6;
}
// the fields of A that the cap's polynomial takes (scale: of its result)
template <int NP>
void set_cap(AttnArgs& A, double scale) {
  const double f = (double)A.scale / A.cap;
  double pw = f * scale;
  for (int z = 0; z < NP; ++z, pw *= f * f) A.tp[z] = (float)(tanh_terms<NP>()[z] * pw);
  A.cap_near = (float)(kCapNear / f);
  A.cap_exp = (float)(2.0 * f * kLog2e);
}

// The distances of a step's pairs: float32 in lengths, so that the slope in base 2 is rounded once;
// bf16 in units of the coordinates, the unit in the slope
template <class T>
__device__ __forceinline__ float r_unit(const AttnArgs& A) {
  return sizeof(T) == 4 ? A.unit : 1.0f;
}
template <class T>
__device__ __forceinline__ float slope2(const AttnArgs& A, float slope) {
  return sizeof(T) == 4 ? slope * kLog2e : slope * (kLog2e * A.unit);
}
template <class T, int NT>
__device__ __forceinline__ void distances(f4 (&r)[NT], const AttnArgs& A, const P3& own, const u4* ps, bool fix, int g) {
  auto all = [&](auto periodic) {  // one branch a step: in each pair it would part every LDS read from the others
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float dx, dy, dz;
        diff(own, ps[16 * t + 4 * g + q], decltype(periodic)::value, dx, dy, dz);
        r[t][q] = __builtin_amdgcn_sqrtf(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
        if constexpr (sizeof(T) == 4) r[t][q] *= A.unit;
      }
  };
  if (fix)
    all(std::true_type{});
  else
    all(std::false_type{});
}
// Waves per SIMD that the register budgets aim at.  More heads hold more running sums and
// statistics: 8 heads at three waves (forward) or 4 heads of 16 channels at three (backward) spill
// (11,000 atoms bf16: 720 us against 577; 1,571 against 1,382).
#define ATTN_FWD_WAVES (C == 128 && (C / DH > 4 || sizeof(T) == 4) ? 2 : 3)
#define ATTN_BWD_WAVES (C == 128 || (C == 64 && C / DH > 1) ? 2 : 3)

// ------------------------------------------------------------------------------ forward
// CAP is a template parameter: with a branch in its place the uncapped form took 12% longer too (16,384
// molecules 105 us against 90), the capped scores being merged into its registers.
template <class T, int C, int DH, int NW, bool SAVE, bool CAP>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(ATTN_FWD_WAVES)))
void k_attn_fwd(AttnArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, NT = M::NT, CK = M::CK, H = C / DH, RS = C + lds_pad<T>(), EV = M::EV, NTH = 64 * NW;
  constexpr bool BF = sizeof(T) == 2, KL = NW > 1;  // KL: keys through LDS as well
  constexpr int NB = KL ? 2 : 1;
  __shared__ __align__(16) T s_v[NB][CK * RS];
  __shared__ __align__(16) T s_k[KL ? NB : 1][KL ? CK * RS : 8];
  __shared__ u4 s_pos[NB][CK];
  const int tid = threadIdx.x, lane = tid & 63, wave = NW > 1 ? uniform(tid >> 6) : 0, i = lane & 15, g = lane >> 4;
  int row0, s, e;
  if (!find_slot<16 * NW>(A, blockIdx.x, lane, row0, s, e)) return;
  const int own0 = row0 + 16 * wave, row = own0 + i;
  const bool fix = A.to_fix > 0, dist = A.pos != nullptr;
  typename M::F qf[1][NC];
  load_frags<T, C, 1>(qf, (const T*)A.q, A.ldq, min(own0, e - 1), max(e - own0, 1), i, g);
  const P3 own = load_pos(A, row, row < e);
  // thr: a score above it (in the reference m) raises the reference; -inf until there is one
  float m[H], thr[H];
  f4 l[H];  // bf16: every element the sum over all keys; float32: per-lane sums in l.x
#pragma unroll
  for (int h = 0; h < H; ++h) {
    m[h] = 0.f;
    thr[h] = -INFINITY;
    l[h] = f4{0.f, 0.f, 0.f, 0.f};
  }
  f4 acc[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) acc[ct] = f4{0.f, 0.f, 0.f, 0.f};
  constexpr int NP = BF && !SAVE ? 4 : 6;
  const float sc = A.scale * kLog2e;
  typename M::F ones;
  if constexpr (BF) ones = __builtin_bit_cast(typename M::F, u4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});

  // NW = 4: a step's loads are issued during the step before.  NW = 1: mostly a single step, the
  // registers of a step ahead are better left to more waves.
  StepTile<T, C, RS, NTH> tv, tk;
  typename M::F kf[NT][NC];
  P3 kp{0u, 0u, 0u};
  const int first = s + CK * (int)blockIdx.y, stride = CK * A.splits;
  uint64_t on = live<CK>(A, first, e, lane, true);
  auto fetch = [&](int k0, uint64_t b) {
    tv.fetch((const T*)A.v, A.ldv, k0, e - k0, tid);
    if constexpr (KL) tk.fetch((const T*)A.k, A.ldk, k0, e - k0, tid);
    if (dist && tid < CK) kp = load_pos(A, k0 + tid, (b >> tid) & 1);
  };
  auto put = [&](int b, uint64_t live_bits) {
    if (live_bits != all_live<CK>()) tv.clear(live_bits, tid);
    tv.put(s_v[b], tid);
    if constexpr (KL) tk.put(s_k[b], tid);
    if (dist && tid < CK) s_pos[b][tid] = u4{kp.x, kp.y, kp.z, 0u};
  };
  if constexpr (KL) {
    if (first < e) {
      fetch(first, on);
      put(0, on);
      lds_barrier();
    }
  }
  int b = 0;
  for (int k0 = first; k0 < e; k0 += stride) {
    const int kn = k0 + stride;
    const bool part = on != all_live<CK>();
    const uint64_t on_n = live<CK>(A, kn, e, lane, true);
    if constexpr (KL) {
      if (kn < e) fetch(kn, on_n);
    } else {
      fetch(k0, on);
      load_frags<T, C, NT>(kf, (const T*)A.k, A.ldk, k0, e - k0, i, g);
      put(0, on);
      wave_sync();
    }
    const T *vs = s_v[b], *ks = s_k[KL ? b : 0];
    const u4* ps = s_pos[b];
    if (own0 < e) {  // a wave past the structure only keeps step
      bool lv[NT][4];
      f4 r[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        r[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) lv[t][q] = ((uint32_t)on >> (4 * g)) >> (16 * t + q) & 1;
      }
      if (dist) distances<T, NT>(r, A, own, ps, fix, g);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        f4 x[NT], f[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (KL) {
#pragma unroll
            for (int ch = chunk_of<T, DH>(h); ch < chunk_of<T, DH>(h) + chunks<T, DH>(); ++ch)
              kf[t][ch] = *(const typename M::F*)(ks + (16 * t + i) * RS + ch * CK + EV * g);
          }
          x[t] = head_mma<T, DH, NC>(f4{0.f, 0.f, 0.f, 0.f}, kf[t], qf[0], h, g);
          f[t] = f4{sc, sc, sc, sc};
        }
        if constexpr (CAP) cap_factors<NP, NT>(A, A.cap * kLog2e, x, f);
        const float sl = dist ? slope2<T>(A, A.slope[h]) : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) x[t][q] = fmaf(x[t][q], f[t][q], fmaf(-sl, r[t][q], -m[h]));
        if (part) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[t][q] = lv[t][q] ? x[t][q] : -INFINITY;
        }
        // the reference is raised only when a score passes it by 8 (p <= 2^8): the sums are exact
        // relative to any reference, so most steps need no exchange and no rescale
        float lm = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t) lm = fmaxf(lm, fmaxf(fmaxf(x[t].x, x[t].y), fmaxf(x[t].z, x[t].w)));
        if (__any(lm > thr[h])) {
          const float mt = gmax(lm);
          const bool none = thr[h] == -INFINITY;
          const float d = none ? (mt == -INFINITY ? 0.f : mt) : fmaxf(mt, 0.f), al = ex2(-d);
          if (mt > -INFINITY) thr[h] = 8.0f;
          m[h] += d;
          if (!none) {
            l[h] *= al;
#pragma unroll
            for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct) acc[ct] *= al;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) x[t] -= d;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int q = 0; q < 4; ++q) x[t][q] = ex2(x[t][q]);
          if constexpr (!BF) l[h].x += (x[t].x + x[t].y) + (x[t].z + x[t].w);
        }
        const typename M::F p = M::pack(x);
        // bf16: the sum of the weights is a product with ones, off the VALU and of the same rounded
        // weights that the values get
        if constexpr (BF) l[h] = M::mma(l[h], ones, p);
        if constexpr (BF && SAVE) {
          // for a backward pass the weights enter as three bf16 values, p and its remainders (2^-27):
          // o32, and with it dsum and the float32 gradients, keep float32's quality
          f4 y[NT], z[NT];
          M::unpack(p, y);
#pragma unroll
          for (int t = 0; t < NT; ++t) y[t] = x[t] - y[t];
          const typename M::F p2 = M::pack(y);
          M::unpack(p2, z);
#pragma unroll
          for (int t = 0; t < NT; ++t) z[t] = y[t] - z[t];
          const typename M::F p3 = M::pack(z);
          l[h] = M::mma(M::mma(l[h], ones, p3), ones, p2);
#pragma unroll
          for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct) {
            const typename M::F f = ldt<RS>(vs, 0, 16 * ct, lane);
            acc[ct] = M::mma(M::mma(M::mma(acc[ct], f, p3), f, p2), f, p);
          }
        } else {
#pragma unroll
          for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct)
            acc[ct] = M::mma(acc[ct], ldt<RS>(vs, 0, 16 * ct, lane), p);
        }
      }
    }
    on = on_n;
    if constexpr (KL) {
      if (kn < e) put(b ^ 1, on_n);
      lds_barrier();
      b ^= 1;
    } else {
      wave_sync();
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if constexpr (!BF) l[h].x = gsum(l[h].x);
    if (thr[h] == -INFINITY) m[h] = -INFINITY;
  }
  if (row >= e) return;
  if (A.splits > 1) {
    const int64_t at = (int64_t)blockIdx.y * A.n + row;
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) *(f4*)(A.p_out + at * C + 16 * ct + 4 * g) = acc[ct];
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (g == 0) {
        A.p_ml[(at * H + h) * 2] = m[h];
        A.p_ml[(at * H + h) * 2 + 1] = l[h].x;
      }
    return;
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const bool any = l[h].x > 0.f || l[h].x != l[h].x;
    const float inv = any ? 1.0f / l[h].x : 0.f;
#pragma unroll
    for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct) {
      acc[ct] *= inv;
      const int c = 16 * ct + 4 * g;
      st4((T*)A.out + (int64_t)row * A.ldo + c, acc[ct]);
      if (A.o32) st4(A.o32 + (int64_t)row * C + c, acc[ct]);
    }
    if (A.lse && g == 0) A.lse[(int64_t)row * H + h] = any ? m[h] + (log2f(l[h].x) - A.lsub) : INFINITY;
  }
}

// Score, softmax weight and score gradient of one lane's 4 pairs:
//   p = 2^(x - lse) (2^lsub times the weight), dl = p (dp - dsum); ds = dl times the cap's slope 1 - tanh^2
template <bool CAP>
__device__ __forceinline__ void pair_grad(const AttnArgs& A, float kk, bool dist, f4 sraw, f4 dp, f4 r,
                                          float slope, f4 lse, f4 dsum, bool all, uint32_t on, f4& p, f4& dl, f4& ds) {
  f4 f;
  if constexpr (CAP) {
    f4 s1[1] = {sraw}, f1[1];
    cap_factors<6, 1>(A, 1.0f, s1, f1);
    sraw = s1[0] * f1[0];
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = fmaf(-sraw[q], sraw[q], 1.0f);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x = fmaf(kk, sraw[q], dist ? fmaf(-slope, r[q], -lse[q]) : -lse[q]);
    p[q] = ex2(x);
    dl[q] = p[q] * (dp[q] - dsum[q]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) ds[q] = CAP ? dl[q] * f[q] : dl[q];
  if (!all) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (!((on >> q) & 1)) p[q] = dl[q] = ds[q] = 0.f;
  }
}

// p += sum over the pairs of wgt (other - own) / r, nothing where r = 0 (other - own in units).
// Of the two images at exactly half a box the one towards the other atom's coordinate as wrapped is
// taken, so that the two atoms of a pair get opposite gradients (float32 coordinates meet there:
// about one pair in 2^24).  A lane looks for such pairs by the least of its differences.
template <int NT>
__device__ __forceinline__ void add_pairs(float (&p)[3], const f4 (&wgt)[NT], const f4 (&r)[NT], const P3& own,
                                          const u4* ps, bool fix, int g) {
  const int32_t kHalf = INT32_MIN;
  int32_t least = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u4 o = ps[16 * t + 4 * g + q];
      float dx, dy, dz;
      diff(own, o, fix, dx, dy, dz);
      least = min(least, min((int32_t)(o.x - own.x), min((int32_t)(o.y - own.y), (int32_t)(o.z - own.z))));
      const float f = r[t][q] > 0.f ? wgt[t][q] * rcp(r[t][q]) : 0.f;
      p[0] = fmaf(f, dx, p[0]), p[1] = fmaf(f, dy, p[1]), p[2] = fmaf(f, dz, p[2]);
    }
  if (fix && __any(least == kHalf)) {  // they were taken as -2^31: 2^32 more towards a larger coordinate
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u4 o = ps[16 * t + 4 * g + q];
        const float f = r[t][q] > 0.f ? wgt[t][q] * rcp(r[t][q]) * 4294967296.0f : 0.f;
        if ((int32_t)(o.x - own.x) == kHalf && o.x > own.x) p[0] += f;
        if ((int32_t)(o.y - own.y) == kHalf && o.y > own.y) p[1] += f;
        if ((int32_t)(o.z - own.z) == kHalf && o.z > own.z) p[2] += f;
      }
  }
}

// ------------------------------------------------------------------------------ row pass
// For 16 queries: dsum_i = sum_c dout out (per head), dq_i = scale sum_j ds_ij k_j, the queries'
// side of the position gradient, and the block's partial of dslope.  out enters unrounded (o32)
// so that dsum, and with it the float32 gradients, do not carry bf16's rounding.
template <class T, int C, int DH, int NW, bool CAP>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(ATTN_BWD_WAVES))) void k_attn_row(AttnArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, NT = M::NT, CK = M::CK, H = C / DH, RS = C + lds_pad<T>(), EV = M::EV, NTH = 64 * NW;
  constexpr bool VL = NW > 1;  // values through LDS as well
  constexpr int NB = VL ? 2 : 1;
  __shared__ __align__(16) T s_k[NB][CK * RS];
  __shared__ __align__(16) T s_v[VL ? NB : 1][VL ? CK * RS : 8];
  __shared__ u4 s_pos[NB][CK];
  __shared__ float s_s[NW][H];
  const int tid = threadIdx.x, lane = tid & 63, wave = NW > 1 ? uniform(tid >> 6) : 0, i = lane & 15, g = lane >> 4;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  int row0, s, e;
  if (!find_slot<16 * NW>(A, blockIdx.x, lane, row0, s, e)) {
    if (A.dslope_part && tid < H) A.dslope_part[block * H + tid] = 0.f;
    return;
  }
  const int own0 = row0 + 16 * wave, row = own0 + i;
  const bool fix = A.to_fix > 0, dist = A.pos != nullptr;
  typename M::F qf[1][NC], of[1][NC];
  load_frags<T, C, 1>(qf, (const T*)A.q, A.ldq, min(own0, e - 1), max(e - own0, 1), i, g);
  load_frags<T, C, 1>(of, (const T*)A.dout, A.lddo, min(own0, e - 1), max(e - own0, 1), i, g);
  const P3 own = load_pos(A, row, row < e);
  float lse[H], dsum[H], dsl[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    lse[h] = row < e ? A.lse[(int64_t)row * H + h] : INFINITY;
    dsum[h] = dsl[h] = 0.f;
  }
#pragma unroll
  for (int ch = 0; ch < NC; ++ch) {
    f4 a[NT];
    M::unpack(of[0][ch], a);
    float d = 0.f;
    if (row < e) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float* op = sizeof(T) == 2 ? A.o32 + (int64_t)row * C : (const float*)A.o + (int64_t)row * A.ldo;
        const f4 o = *(const f4*)(op + ch * CK + EV * g + 4 * t);
        d = fmaf(a[t].x, o.x, fmaf(a[t].y, o.y, fmaf(a[t].z, o.z, fmaf(a[t].w, o.w, d))));
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) dsum[h] += lane_in_head<T, DH>(ch, g, h) ? d : 0.f;
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    dsum[h] = gsum(dsum[h]);
    if (blockIdx.y == 0 && g == 0 && row < e) A.dsum[(int64_t)row * H + h] = dsum[h];
  }
  f4 acc[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) acc[ct] = f4{0.f, 0.f, 0.f, 0.f};
  float px[3] = {0.f, 0.f, 0.f};
  const float kk = (CAP ? A.cap : A.scale) * kLog2e;

  StepTile<T, C, RS, NTH> tk, tv;
  typename M::F vf[NT][NC];
  P3 kp{0u, 0u, 0u};
  const int first = s + CK * (int)blockIdx.y, stride = CK * A.splits;
  uint64_t on = live<CK>(A, first, e, lane, true);
  auto fetch = [&](int k0, uint64_t b) {
    tk.fetch((const T*)A.k, A.ldk, k0, e - k0, tid);
    if constexpr (VL) tv.fetch((const T*)A.v, A.ldv, k0, e - k0, tid);
    if (dist && tid < CK) kp = load_pos(A, k0 + tid, (b >> tid) & 1);
  };
  auto put = [&](int b, uint64_t live_bits) {
    if (live_bits != all_live<CK>()) tk.clear(live_bits, tid);
    tk.put(s_k[b], tid);
    if constexpr (VL) tv.put(s_v[b], tid);
    if (dist && tid < CK) s_pos[b][tid] = u4{kp.x, kp.y, kp.z, 0u};
  };
  if constexpr (VL) {
    if (first < e) {
      fetch(first, on);
      put(0, on);
      lds_barrier();
    }
  }
  int b = 0;
  for (int k0 = first; k0 < e; k0 += stride) {
    const int kn = k0 + stride;
    const uint64_t on_n = live<CK>(A, kn, e, lane, true);
    if constexpr (VL) {
      if (kn < e) fetch(kn, on_n);
    } else {  // mostly a single step: the registers of a step ahead are better left to the wave
      fetch(k0, on);
      load_frags<T, C, NT>(vf, (const T*)A.v, A.ldv, k0, e - k0, i, g);
      put(0, on);
      wave_sync();
    }
    const T *ks = s_k[b], *vs = s_v[VL ? b : 0];
    const u4* ps = s_pos[b];
    if (own0 < e) {  // a wave past the structure only keeps step
      f4 r[NT], wgt[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) wgt[t] = r[t] = f4{0.f, 0.f, 0.f, 0.f};
      if (dist) distances<T, NT>(r, A, own, ps, fix, g);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float sl = dist ? A.slope[h] : 0.f, sl2 = slope2<T>(A, sl);
        f4 ds[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          typename M::F kf[NC];
#pragma unroll
          for (int ch = chunk_of<T, DH>(h); ch < chunk_of<T, DH>(h) + chunks<T, DH>(); ++ch) {
            kf[ch] = *(const typename M::F*)(ks + (16 * t + i) * RS + ch * CK + EV * g);
            if constexpr (VL) vf[t][ch] = *(const typename M::F*)(vs + (16 * t + i) * RS + ch * CK + EV * g);
          }
          const f4 z = f4{0.f, 0.f, 0.f, 0.f};
          const f4 x = head_mma<T, DH, NC>(z, kf, qf[0], h, g), dp = head_mma<T, DH, NC>(z, vf[t], of[0], h, g);
          f4 p, dl;
          const f4 L = f4{lse[h], lse[h], lse[h], lse[h]}, S = f4{dsum[h], dsum[h], dsum[h], dsum[h]};
          pair_grad<CAP>(A, kk, dist, x, dp, r[t], sl2, L, S, on == all_live<CK>(), (uint32_t)on >> (4 * g) >> (16 * t), p, dl,
                       ds[t]);
          if (dist) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              wgt[t][q] = fmaf(sl, dl[q], wgt[t][q]);
              dsl[h] = fmaf(-dl[q], r[t][q], dsl[h]);
            }
          }
        }
        const typename M::F pd = M::pack(ds), pd2 = rest_of<T>(pd, ds);
#pragma unroll
        for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct) {
          const typename M::F f = ldt<RS>(ks, 0, 16 * ct, lane);
          if constexpr (sizeof(T) == 2) acc[ct] = M::mma(acc[ct], f, pd2);
          acc[ct] = M::mma(acc[ct], f, pd);
        }
      }
      if (A.dpos) add_pairs<NT>(px, wgt, r, own, ps, fix, g);
    }
    on = on_n;
    if constexpr (VL) {
      if (kn < e) put(b ^ 1, on_n);
      lds_barrier();
      b ^= 1;
    } else {
      wave_sync();
    }
  }
  if (A.dslope_part) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      dsl[h] = group_sum<64>(row < e ? dsl[h] : 0.f);
      if (lane == 0) s_s[wave][h] = dsl[h];
    }
    __syncthreads();
    if (tid < H) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += s_s[w][tid];
      A.dslope_part[block * H + tid] = (sizeof(T) == 4 ? v : v * A.unit) * A.p_scale;
    }
  }
#pragma unroll
  for (int a = 0; a < 3; ++a) px[a] = r_unit<T>(A) * A.p_scale * gsum(px[a]);
  if (row >= e) return;
  const int64_t at = (int64_t)blockIdx.y * A.n + row;
  const float gs = A.scale * A.p_scale;
  if (A.dpos && g < 3) (A.splits > 1 ? A.p_row + 3 * at : A.dpos + 3 * (int64_t)row)[g] = g == 0 ? px[0] : g == 1 ? px[1] : px[2];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) {
    const int c = 16 * ct + 4 * g;
    if (A.splits > 1)
      *(f4*)(A.p_dq + at * C + c) = acc[ct] * gs;
    else
      st4((T*)A.dq + (int64_t)row * A.lddq + c, acc[ct] * gs);
  }
}

// ------------------------------------------------------------------------------ column pass
// Here and in the row pass bf16 weights and score gradients enter as two operands (rest_of): dq, dk and
// dv carry the rounding of the output alone (4,096 molecules: 62 -> 62 and 55 -> 57 us).
// For 16 keys: dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i, and the keys' side of the
// position gradient, added to what the row pass wrote.
template <class T, int C, int DH, int NW, bool CAP>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(ATTN_BWD_WAVES))) void k_attn_col(AttnArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, NT = M::NT, CK = M::CK, H = C / DH, RS = C + lds_pad<T>(), EV = M::EV, NTH = 64 * NW;
  constexpr int NB = NW > 1 ? 2 : 1;
  __shared__ __align__(16) T s_q[NB][CK * RS];
  __shared__ __align__(16) T s_o[NB][CK * RS];
  __shared__ u4 s_pos[NB][CK];
  __shared__ __align__(16) float s_ls[NB][2][H][CK];  // log-sums and dsum of the step's queries
  const int tid = threadIdx.x, lane = tid & 63, wave = NW > 1 ? uniform(tid >> 6) : 0, i = lane & 15, g = lane >> 4;
  int row0, s, e;
  if (!find_slot<16 * NW>(A, blockIdx.x, lane, row0, s, e)) return;
  const int own0 = row0 + 16 * wave, row = own0 + i;
  const bool fix = A.to_fix > 0, dist = A.pos != nullptr;
  const uint64_t own_on = live<16>(A, own0, e, lane, true);
  const bool own_live = (own_on >> i) & 1, all_own = own_on == 0xffffull;
  const uint32_t own_bits = own_live ? ~0u : 0u;
  typename M::F kf[1][NC], vf[1][NC];
  load_frags<T, C, 1>(kf, (const T*)A.k, A.ldk, min(own0, e - 1), max(e - own0, 1), i, g);
  load_frags<T, C, 1>(vf, (const T*)A.v, A.ldv, min(own0, e - 1), max(e - own0, 1), i, g);
  const P3 own = load_pos(A, row, own_live);
  f4 ak[C / 16], av[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) ak[ct] = av[ct] = f4{0.f, 0.f, 0.f, 0.f};
  float px[3] = {0.f, 0.f, 0.f};
  const float kk = (CAP ? A.cap : A.scale) * kLog2e;

  StepTile<T, C, RS, NTH> tq, to;
  P3 kp{0u, 0u, 0u};
  float ln[H], sn[H];
  const int first = s + CK * (int)blockIdx.y, stride = CK * A.splits;
  auto fetch = [&](int k0) {
    tq.fetch((const T*)A.q, A.ldq, k0, e - k0, tid);
    to.fetch((const T*)A.dout, A.lddo, k0, e - k0, tid);
    if (tid < CK) {
      const bool l = k0 + tid < e;
      if (dist) kp = load_pos(A, k0 + tid, l);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        ln[h] = l ? A.lse[(int64_t)(k0 + tid) * H + h] : INFINITY;
        sn[h] = l ? A.dsum[(int64_t)(k0 + tid) * H + h] : 0.f;
      }
    }
  };
  auto put = [&](int b, int k0) {
    if (e - k0 < CK) {
      tq.clear((1ull << (e - k0)) - 1, tid);
      to.clear((1ull << (e - k0)) - 1, tid);
    }
    tq.put(s_q[b], tid);
    to.put(s_o[b], tid);
    if (tid < CK) {
      if (dist) s_pos[b][tid] = u4{kp.x, kp.y, kp.z, 0u};
#pragma unroll
      for (int h = 0; h < H; ++h) {
        s_ls[b][0][h][tid] = ln[h];
        s_ls[b][1][h][tid] = sn[h];
      }
    }
  };
  if constexpr (NW > 1) {
    if (first < e) {
      fetch(first);
      put(0, first);
      lds_barrier();
    }
  }
  int b = 0;
  for (int k0 = first; k0 < e; k0 += stride) {
    const int kn = k0 + stride;
    if constexpr (NW == 1) {
      fetch(k0);
      put(0, k0);
      wave_sync();
    } else {
      if (kn < e) fetch(kn);
    }
    const T *qs = s_q[b], *os = s_o[b];
    const u4* ps = s_pos[b];
    if (own_on != 0) {
      f4 r[NT], wgt[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) wgt[t] = r[t] = f4{0.f, 0.f, 0.f, 0.f};
      if (dist) distances<T, NT>(r, A, own, ps, fix, g);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float sl = dist ? A.slope[h] : 0.f, sl2 = slope2<T>(A, sl);
        f4 p[NT], ds[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          typename M::F qf[NC], of[NC];
#pragma unroll
          for (int ch = chunk_of<T, DH>(h); ch < chunk_of<T, DH>(h) + chunks<T, DH>(); ++ch) {
            qf[ch] = *(const typename M::F*)(qs + (16 * t + i) * RS + ch * CK + EV * g);
            of[ch] = *(const typename M::F*)(os + (16 * t + i) * RS + ch * CK + EV * g);
          }
          const f4 z = f4{0.f, 0.f, 0.f, 0.f};
          const f4 x = head_mma<T, DH, NC>(z, qf, kf[0], h, g), dp = head_mma<T, DH, NC>(z, of, vf[0], h, g);
          const f4 L = *(const f4*)(s_ls[b][0][h] + 16 * t + 4 * g), S = *(const f4*)(s_ls[b][1][h] + 16 * t + 4 * g);
          f4 dl;
          pair_grad<CAP>(A, kk, dist, x, dp, r[t], sl2, L, S, all_own, own_bits, p[t], dl, ds[t]);
          if (dist) {
#pragma unroll
            for (int q = 0; q < 4; ++q) wgt[t][q] = fmaf(sl, dl[q], wgt[t][q]);
          }
        }
        const typename M::F pp = M::pack(p), pd = M::pack(ds), pp2 = rest_of<T>(pp, p), pd2 = rest_of<T>(pd, ds);
#pragma unroll
        for (int ct = h * DH / 16; ct < (h + 1) * DH / 16; ++ct) {
          const typename M::F fo = ldt<RS>(os, 0, 16 * ct, lane), fq = ldt<RS>(qs, 0, 16 * ct, lane);
          if constexpr (sizeof(T) == 2) {
            av[ct] = M::mma(av[ct], fo, pp2);
            ak[ct] = M::mma(ak[ct], fq, pd2);
          }
          av[ct] = M::mma(av[ct], fo, pp);
          ak[ct] = M::mma(ak[ct], fq, pd);
        }
      }
      if (A.dpos) add_pairs<NT>(px, wgt, r, own, ps, fix, g);
    }
    if constexpr (NW > 1) {
      if (kn < e) put(b ^ 1, kn);
      lds_barrier();
      b ^= 1;
    } else {
      wave_sync();
    }
  }
#pragma unroll
  for (int a = 0; a < 3; ++a) px[a] = r_unit<T>(A) * A.p_scale * gsum(px[a]);
  if (row >= e) return;
  const int64_t at = (int64_t)blockIdx.y * A.n + row;
  const float gs = A.scale * A.p_scale;
  if (A.dpos && g < 3) {
    const float v = g == 0 ? px[0] : g == 1 ? px[1] : px[2];
    if (A.splits > 1)
      A.p_col[3 * at + g] = v;
    else
      A.dpos[3 * (int64_t)row + g] += v;
  }
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) {
    const int c = 16 * ct + 4 * g;
    if (A.splits > 1) {
      *(f4*)(A.p_dk + at * C + c) = ak[ct] * gs;
      *(f4*)(A.p_dv + at * C + c) = av[ct] * A.p_scale;
    } else {
      st4((T*)A.dk + (int64_t)row * A.lddk + c, ak[ct] * gs);
      st4((T*)A.dv + (int64_t)row * A.lddv + c, av[ct] * A.p_scale);
    }
  }
}

// ------------------------------------------------------------------------------ joins of splits
// rows of the structures: at or past struct_ptr[n_struct] nothing is written
__device__ __forceinline__ int rows_end(const AttnArgs& A) { return min(max(A.sptr[A.n_struct], 0), A.n); }

// out, saved log-sums: the splits' sums in one reference, in split order; EV channels a thread
template <class T>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs A, int C, int H) {
  using M = MF<T>;
  constexpr int EV = M::EV, NT = M::NT;
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, row = x / (C / EV);
  if (row >= rows_end(A)) return;
  const int c = (int)(x % (C / EV)) * EV, h = c / (C / H);
  float mm = -INFINITY, ll = 0.f;
  for (int s = 0; s < A.splits; ++s) mm = fmaxf(mm, A.p_ml[((s * (int64_t)A.n + row) * H + h) * 2]);
  f4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < A.splits; ++s) {
    const int64_t at = s * (int64_t)A.n + row;
    const float ms = A.p_ml[(at * H + h) * 2];
    const float f = mm == -INFINITY ? 1.0f : (ms == -INFINITY ? 0.f : ex2(ms - mm));
    ll = fmaf(f, A.p_ml[(at * H + h) * 2 + 1], ll);
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] += f * *(const f4*)(A.p_out + at * C + c + 4 * t);
  }
  const bool any = ll > 0.f || ll != ll;
  const float inv = any ? 1.0f / ll : 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    o[t] *= inv;
    if (A.o32) st4(A.o32 + row * C + c + 4 * t, o[t]);
  }
  st_row<T>((T*)A.out + row * A.ldo + c, o);
  if (A.lse && c % (C / H) == 0) A.lse[row * H + h] = any ? mm + (log2f(ll) - A.lsub) : INFINITY;
}

// dq, dk, dv (blockIdx.y 0, 1, 2) and dpos (3): sums over the splits, in split order
template <class T>
__global__ __launch_bounds__(256) void k_attn_join_bwd(AttnArgs A, int C) {
  using M = MF<T>;
  constexpr int EV = M::EV, NT = M::NT;
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int which = blockIdx.y, end = rows_end(A);
  if (which == 3) {
    if (x >= 3 * (int64_t)end) return;
    float v = 0.f;
    for (int s = 0; s < A.splits; ++s) v += A.p_row[3 * s * (int64_t)A.n + x];
    for (int s = 0; s < A.splits; ++s) v += A.p_col[3 * s * (int64_t)A.n + x];
    A.dpos[x] = v;
    return;
  }
  const int64_t row = x / (C / EV);
  if (row >= end) return;
  const int c = (int)(x % (C / EV)) * EV;
  const float* p = which == 0 ? A.p_dq : which == 1 ? A.p_dk : A.p_dv;
  f4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < A.splits; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] += *(const f4*)(p + (s * (int64_t)A.n + row) * C + c + 4 * t);
  if (which == 0)
    st_row<T>((T*)A.dq + row * A.lddq + c, o);
  else if (which == 1)
    st_row<T>((T*)A.dk + row * A.lddk + c, o);
  else
    st_row<T>((T*)A.dv + row * A.lddv + c, o);
}

template <class T>
int launch_join(const AttnArgs& A, int C, int H, bool bwd, hipStream_t st) {
  const unsigned blocks = (unsigned)cdiv((int64_t)A.n * (C / MF<T>::EV), 256);
  if (bwd)  // 3 n position gradients are at most as many as the pieces of one matrix times 3
    k_attn_join_bwd<T><<<dim3((unsigned)std::max<int64_t>(blocks, cdiv(3 * (int64_t)A.n, 256)), A.dpos ? 4 : 3), 256, 0, st>>>(A, C);
  else
    k_attn_join<T><<<blocks, 256, 0, st>>>(A, C, H);
  MP_CHECK_LAUNCH();
  return MP_OK;
}

// what: 0 forward, 1 row pass, 2 column pass
int launch_attn_bf16(const AttnArgs& A, int C, int dh, bool split, int what, hipStream_t st);
int launch_attn_f32(const AttnArgs& A, int C, int dh, bool split, int what, hipStream_t st);

template <class T, int C, int DH, int NW, bool CAP>
void launch_attn_k(AttnArgs A, int what, hipStream_t st) {
  const dim3 blocks((unsigned)(A.n / (16 * NW) + A.n_struct), (unsigned)A.splits);
  constexpr bool SAVES = sizeof(T) == 2;  // float32 has no second form
  if constexpr (CAP) {
    if (what > 0)
      set_cap<6>(A, 1.0);
    else if (A.lse || !SAVES)
      set_cap<6>(A, (double)A.cap * kLog2e);
    else
      set_cap<4>(A, (double)A.cap * kLog2e);
  }
  if (what == 1)
    k_attn_row<T, C, DH, NW, CAP><<<blocks, 64 * NW, 0, st>>>(A);
  else if (what == 2)
    k_attn_col<T, C, DH, NW, CAP><<<blocks, 64 * NW, 0, st>>>(A);
  else if (A.lse)
    k_attn_fwd<T, C, DH, NW, SAVES, CAP><<<blocks, 64 * NW, 0, st>>>(A);
  else
    k_attn_fwd<T, C, DH, NW, false, CAP><<<blocks, 64 * NW, 0, st>>>(A);
}

template <class T, int C, int DH>
int launch_attn_c(const AttnArgs& A, bool split, int what, hipStream_t st) {
  if (A.cap > 0)
    split ? launch_attn_k<T, C, DH, 4, true>(A, what, st) : launch_attn_k<T, C, DH, 1, true>(A, what, st);
  else
    split ? launch_attn_k<T, C, DH, 4, false>(A, what, st) : launch_attn_k<T, C, DH, 1, false>(A, what, st);
  MP_CHECK_LAUNCH();
  if (A.splits > 1 && what != 1) return launch_join<T>(A, C, C / DH, what == 2, st);
  return MP_OK;
}

}  // namespace ops
}  // namespace mdmp
