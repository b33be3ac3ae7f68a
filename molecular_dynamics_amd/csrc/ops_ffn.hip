// Gated feed-forward block y = residual + (act(x Wg^T) * (x Wu^T)) Wd^T and its gradients.
#include "ops_api.hpp"

namespace mdmp {
namespace ops {
namespace {

struct FfnArgs {
  int64_t n, ldx, ldr, ldy, lddx;  // ldy: stride of y (forward) or dy (backward)
  int hidden;
  ActAB ab;
  const void *x, *wg, *wu, *wd, *res, *dy;
  void *y, *dx;
  float* part;  // [splits][3 C hidden]: dWg [hidden][C], dWu [hidden][C], dWd [C][hidden]
  int64_t rows_per_split;
};

// One chunk of CK hidden units of the three matrices, in LDS: rows of Wg and Wu (CK x C) and
// columns of Wd (C x CK), staged by NTH threads.  Rows (hidden units of Wg and Wu, channels of Wd)
// are stored in the order nat_slot.  The backward pass reads Wd transposed, its hidden units as
// result rows: there hidden unit nat_row(t, i) is column 16 t + i.
template <class T, int C, int NTH, bool BWD>
struct Chunk {
  using M = MF<T>;
  static constexpr int CK = M::CK, RS = C + lds_pad<T>(), RD = CK + lds_pad<T>();
  static constexpr int SIZE = 2 * CK * RS + C * RD;
  Tile<T, CK, C, RS, NTH> g, u;
  Tile<T, C, CK, RD, NTH> d;
  __device__ __forceinline__ void fetch_gu(const FfnArgs& A, int h0, int tid) {
    g.fetch((const T*)A.wg + (int64_t)h0 * C, C, CK, tid);
    u.fetch((const T*)A.wu + (int64_t)h0 * C, C, CK, tid);
  }
  __device__ __forceinline__ void fetch_d(const FfnArgs& A, int h0, int tid) {
    d.fetch((const T*)A.wd + h0, A.hidden, C, tid);
  }
  __device__ __forceinline__ void fetch(const FfnArgs& A, int h0, int tid) {
    fetch_gu(A, h0, tid);
    fetch_d(A, h0, tid);
  }
  __device__ __forceinline__ void put(T* s, int tid) const {
    put_gu(s, tid);
    put_d(s + 2 * CK * RS, tid);
  }
  __device__ __forceinline__ void put_gu(T* s, int tid) const {
    auto slot = [](int r) { return nat_slot<T>(r); };
    g.put(s, tid, slot);
    u.put(s + CK * RS, tid, slot);
  }
  __device__ __forceinline__ void put_d(T* sd, int tid) const {
    auto slot = [](int r) { return nat_slot<T>(r); };
    if constexpr (!BWD || sizeof(T) == 4) {
      d.put(sd, tid, slot);
    } else {
      using TD = Tile<T, C, CK, RD, NTH>;
#pragma unroll
      for (int k = 0; k < TD::IT; ++k) {
        const int x = tid + k * NTH, r = x / TD::VPR, c = (x % TD::VPR) * M::EV;
        if (TD::TOT % NTH != 0 && x >= TD::TOT) break;
        T* q = sd + nat_slot<T>(r) * RD + c / 2;  // units c .. c + 3 of tile 0, c + 4 .. c + 7 of tile 1
        *(u2*)q = u2{d.v[k][0], d.v[k][1]};
        *(u2*)(q + 16) = u2{d.v[k][2], d.v[k][3]};
      }
    }
  }
};

template <class T, int C, int AT>
__device__ __forceinline__ void load_rows(typename MF<T>::F (&f)[AT][C / MF<T>::CK], const void* x, int64_t ld,
                                          int64_t a0, int64_t n, int i, int g) {
  using M = MF<T>;
#pragma unroll
  for (int at = 0; at < AT; ++at) {
    const int64_t a = a0 + 16 * at + i;
    const T* p = (const T*)x + a * ld + M::EV * g;
#pragma unroll
    for (int ch = 0; ch < C / M::CK; ++ch) f[at][ch] = ld16<typename M::F>(p + ch * M::CK, a < n);
  }
}

// One chunk of hidden units with 16 AT atoms' rows xf.  D[hid][a] = Wg x and Wu x with the hidden
// rows taken in the order nat_row, so a lane ends with EV consecutive hidden units of its atom,
// which after act(.) * (.) are the operand of D[c][a] += Wd h as they stand: hidden units live in
// registers only.  WG, WU, WD give the operand of (tile, channel chunk) of the three matrices.
template <class T, int C, int AT, class WG, class WU>
__device__ __forceinline__ void ffn_in(f4 (&zg)[AT][MF<T>::NT], f4 (&zu)[AT][MF<T>::NT],
                                       const typename MF<T>::F (&xf)[AT][C / MF<T>::CK], WG wg, WU wu) {
  using M = MF<T>;
#pragma unroll
  for (int t = 0; t < M::NT; ++t) {
#pragma unroll
    for (int at = 0; at < AT; ++at) zg[at][t] = zu[at][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ch = 0; ch < C / M::CK; ++ch) {
      const typename M::F fg = wg(t, ch), fu = wu(t, ch);
#pragma unroll
      for (int at = 0; at < AT; ++at) {
        zg[at][t] = M::mma(zg[at][t], fg, xf[at][ch]);
        zu[at][t] = M::mma(zu[at][t], fu, xf[at][ch]);
      }
    }
  }
}
template <class T, int AT>
__device__ __forceinline__ void ffn_act(typename MF<T>::F (&h)[AT], f4 (&zg)[AT][MF<T>::NT],
                                        const f4 (&zu)[AT][MF<T>::NT], ActAB ab) {
#pragma unroll
  for (int at = 0; at < AT; ++at) {
#pragma unroll
    for (int t = 0; t < MF<T>::NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) zg[at][t][r] = act_val(zg[at][t][r], ab) * zu[at][t][r];
    h[at] = MF<T>::pack(zg[at]);
  }
}
template <class T, int C, int AT, class WD>
__device__ __forceinline__ void ffn_down(f4 (&acc)[AT][C / MF<T>::CK][MF<T>::NT], const typename MF<T>::F (&h)[AT], WD wd) {
  using M = MF<T>;
#pragma unroll
  for (int p = 0; p < C / M::CK; ++p)
#pragma unroll
    for (int t = 0; t < M::NT; ++t) {
      const typename M::F f = wd(p, t);
#pragma unroll
      for (int at = 0; at < AT; ++at) acc[at][p][t] = M::mma(acc[at][p][t], f, h[at]);
    }
}

template <class T>
__device__ __forceinline__ void ffn_out(const FfnArgs& A, int64_t a, int c, f4* o) {
  using M = MF<T>;
  if (A.res) {
    f4 q[M::NT];
    M::unpack(*(const typename M::F*)((const T*)A.res + a * A.ldr + c), q);
#pragma unroll
    for (int t = 0; t < M::NT; ++t) o[t] += q[t];
  }
  st_row<T>((T*)A.y + a * A.ldy + c, o);
}

// Forward.  Eight waves of 16 AT atoms each share the weights in LDS and walk tiles of rows with a
// fixed stride.  A step of a wave is a phase of matrix products (the down product of the chunk
// before, then the two products of this chunk) and a phase of activations; waves 4-7, the second
// of each SIMD, run half a step behind waves 0-3, so that at any time one wave of a SIMD feeds the
// matrix cores and the other the VALU (in step, both would wait for the same unit).  A barrier
// separates the phases.  Weights have two buffers, a chunk's Wd used a step after its Wg and Wu;
// a half of the waves writes its half of a chunk in its activation phase: the first half what it
// needs next (Wg, Wu of chunk j + 1, Wd of chunk j), the second half, whose phase lies one barrier
// later, a chunk further, so both halves of a buffer are written between the same two barriers'
// last and first readers.  A wave's next rows of x arrive in LDS piece by piece during the chunks
// of the present ones, so no tile waits for memory.  Bound: the matrix products, their LDS operands and the
// sigmoid of every hidden unit (exp and reciprocal) on one SIMD: 1,048,576 rows of 128, 512 hidden,
// bf16 take 440 us, 940 TFLOP/s of the 1,300 that a large library product reaches; the products with
// their LDS reads and barriers alone take 340 us, the rows' way in and out alone 180.
template <class T, int C, int AT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_ffn(FfnArgs A) {
  using M = MF<T>;
  using CH = Chunk<T, C, 512, false>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, CK = M::CK, RS = CH::RS, RD = CH::RD, ROWS = 16 * AT;
  constexpr int GU = 2 * CK * RS, DN = C * RD, MPF = sizeof(T) == 2 ? 1 : 4;  // MPF: MFMAs per operand pair
  __shared__ __align__(16) T s[2 * (GU + DN) + 8 * ROWS * RS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  T *s_gu = s, *s_d = s + 2 * GU, *xs = s_d + 2 * DN + wave * ROWS * RS;
  constexpr int VPR = C / EV, PIECES = ROWS * VPR / 64, RJ = 64 / VPR;  // 16-byte pieces a lane moves per tile
  static_assert(ROWS * VPR % 64 == 0 && 64 % VPR == 0, "whole waves");
  const int pr = lane / VPR, pc = (lane % VPR) * EV;
  const int64_t tiles = (A.n + 8 * ROWS - 1) / (8 * ROWS);
  auto piece = [&](int64_t tile, int k) {  // rows past the end: the last row
    const int64_t a = min((tile * 8 + wave) * ROWS + pr + k * RJ, A.n - 1);
    return *(const u4*)((const T*)A.x + a * A.ldx + pc);
  };
  auto keep = [&](u4 v, int k) { *(u4*)(xs + (pr + k * RJ) * RS + pc) = v; };
  const int nk = A.hidden / CK, late = wave >> 2;
  // chunk k, modulo their number (the next tile starts over)
  auto chunk = [&](int k) { return (k < nk ? k : (k - nk) % nk) * CK; };
  {
    u4 v[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) v[k] = piece(blockIdx.x, k);
#pragma unroll
    for (int k = 0; k < PIECES; ++k) keep(v[k], k);
  }
  CH ck;
  ck.fetch_gu(A, 0, threadIdx.x);
  ck.put_gu(s_gu, threadIdx.x);
  if (late) {
    ck.fetch_gu(A, chunk(1), threadIdx.x);
    ck.fetch_d(A, 0, threadIdx.x);
    ck.put_gu(s_gu + GU, threadIdx.x);
    ck.put_d(s_d, threadIdx.x);
  }
  lds_barrier();
  if (late) lds_barrier();
  f4 zg[AT][NT], zu[AT][NT], acc[AT][NC][NT];
  typename M::F h[AT], xf[AT][NC], res[AT][NC];
  auto down = [&](int b) {
    const T* wd = s_d + b * DN + i * RD + EV * g;
    ffn_down<T, C, AT>(acc, h, [&](int p, int t) { return *(const typename M::F*)(wd + (p * CK + 16 * t) * RD); });
    constexpr int R = NT * NC, A0 = R < 8 ? R : 8;
    read_ahead<A0, R - A0, AT * MPF, 1, A0 * AT * MPF>();
  };
  int j = 0;  // steps taken
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t a0 = (tile * 8 + wave) * ROWS, next = tile + gridDim.x < tiles ? tile + gridDim.x : tile;
    wave_sync();
#pragma unroll
    for (int at = 0; at < AT; ++at)
#pragma unroll
      for (int ch = 0; ch < NC; ++ch) xf[at][ch] = *(const typename M::F*)(xs + (16 * at + i) * RS + ch * CK + EV * g);
    wave_sync();
#pragma unroll
    for (int at = 0; at < AT; ++at)
#pragma unroll
      for (int p = 0; p < NC; ++p)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[at][p][t] = f4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < nk; ++k, ++j) {
      ck.fetch_gu(A, chunk(k + 1 + late), threadIdx.x);
      ck.fetch_d(A, chunk(k + late), threadIdx.x);
      u4 xv;
      if (k < PIECES) xv = piece(next, k);
      if (k > 0) down((j - 1) & 1);
      if (A.res && k == nk - 1) {
#pragma unroll
        for (int at = 0; at < AT; ++at)
#pragma unroll
          for (int p = 0; p < NC; ++p)
            res[at][p] = *(const typename M::F*)((const T*)A.res + min(a0 + 16 * at + i, A.n - 1) * A.ldr + p * CK + EV * g);
      }
      const T *wg = s_gu + (j & 1) * GU + i * RS + EV * g, *wu = wg + CK * RS;
      ffn_in<T, C, AT>(zg, zu, xf, [&](int t, int ch) { return *(const typename M::F*)(wg + 16 * t * RS + ch * CK); },
                       [&](int t, int ch) { return *(const typename M::F*)(wu + 16 * t * RS + ch * CK); });
      constexpr int R = 2 * NT * NC, A0 = R < 8 ? R : 8;
      read_ahead<A0, R - A0, AT * MPF, 1, A0 * AT * MPF>();
      lds_barrier();
      ffn_act<T, AT>(h, zg, zu, A.ab);
      ck.put_gu(s_gu + ((j + 1 + late) & 1) * GU, threadIdx.x);
      ck.put_d(s_d + ((j + late) & 1) * DN, threadIdx.x);
      if (k < PIECES) keep(xv, k);
      lds_barrier();
    }
    down((j - 1) & 1);
    for (int k = nk; k < PIECES; ++k) keep(piece(next, k), k);  // fewer chunks than pieces
#pragma unroll
    for (int at = 0; at < AT; ++at) {
      const int64_t a = a0 + 16 * at + i;
      if (a >= A.n) continue;
#pragma unroll
      for (int p = 0; p < NC; ++p) {
        if (A.res) {
          f4 q[NT];
          M::unpack(res[at][p], q);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[at][p][t] += q[t];
        }
        st_row<T>((T*)A.y + a * A.ldy + p * CK + EV * g, acc[at][p]);
      }
    }
  }
  if (!late) lds_barrier();  // as many as the late half
}

// Forward for few rows: the four waves of a block take the same 16 atoms and every fourth chunk
// each, weights straight from L2, and their sums are joined in wave order.
template <class T, int C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_ffn_few(FfnArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, CK = M::CK, OS = C + 4;
  __shared__ __align__(16) float s_o[64 * OS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int64_t a0 = (int64_t)blockIdx.x * 16;
  typename M::F xf[1][NC];
  load_rows<T, C, 1>(xf, A.x, A.ldx, a0, A.n, i, g);
  f4 acc[1][NC][NT];
#pragma unroll
  for (int p = 0; p < NC; ++p)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][p][t] = f4{0.f, 0.f, 0.f, 0.f};
  for (int h0 = CK * wave; h0 < A.hidden; h0 += 4 * CK) {
    const T *wg = (const T*)A.wg + (int64_t)h0 * C + EV * g, *wu = (const T*)A.wu + (int64_t)h0 * C + EV * g;
    const T* wd = (const T*)A.wd + h0 + EV * g;
    f4 zg[1][NT], zu[1][NT];
    typename M::F h[1];
    ffn_in<T, C, 1>(zg, zu, xf, [&](int t, int ch) { return *(const typename M::F*)(wg + nat_row<T>(t, i) * C + ch * CK); },
                    [&](int t, int ch) { return *(const typename M::F*)(wu + nat_row<T>(t, i) * C + ch * CK); });
    ffn_act<T, 1>(h, zg, zu, A.ab);
    const typename M::F h2 = rest_of<T>(h[0], zg[0]);  // the hidden units as two operands
#pragma unroll
    for (int p = 0; p < NC; ++p)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const typename M::F f = *(const typename M::F*)(wd + (int64_t)(p * CK + nat_row<T>(t, i)) * A.hidden);
        if constexpr (sizeof(T) == 2) acc[0][p][t] = M::mma(acc[0][p][t], f, h2);
        acc[0][p][t] = M::mma(acc[0][p][t], f, h[0]);
      }
  }
  float* slab = s_o + (16 * wave + i) * OS;
#pragma unroll
  for (int p = 0; p < NC; ++p)
#pragma unroll
    for (int t = 0; t < NT; ++t) *(f4*)(slab + p * CK + EV * g + 4 * t) = acc[0][p][t];
  join_waves<T, C>(s_o, a0, A.n, [&](int64_t a, int c, f4* o) { ffn_out<T>(A, a, c, o); });
}

// gradients of the hidden pre-activations: with h = act(zg) zu,
//   dzu = dh act(zg),  dzg = dh zu act'(zg)
__device__ __forceinline__ void hidden_grad(float zg, float zu, float dh, ActAB ab, float& h, float& dzg, float& dzu) {
  float v, e;
  act_both(zg, ab, v, e);
  h = v * zu;
  dzu = dh * v;
  dzg = dh * zu * e;
}

// dx: the forward's first two products, dh = Wd^T dy (Wd read transposed from the same LDS
// chunk), the hidden gradients in registers, and D[c][a] += Wg^T dzg + Wu^T dzu (the same
// rows of Wg and Wu, read transposed).  SPLIT as in the forward, each wave with a chunk of its
// own in LDS.  Bound as the forward: 328,378 rows of 128, 512 hidden, bf16: five products, 255 us
// (840 TFLOP/s); with 512 threads a block 288.
template <class T, int C, bool SPLIT>
constexpr int ffn_dx_lds() {
  constexpr int SLAB = SPLIT ? 64 * (C + 4) * 4 : 0;
  constexpr int CHUNKS = (SPLIT ? 4 : 2) * Chunk<T, C, SPLIT ? 64 : 256, true>::SIZE * (int)sizeof(T);
  return SLAB > CHUNKS ? SLAB : CHUNKS;
}
template <class T, int C, int AT, bool SPLIT>
__device__ __forceinline__ void ffn_dx(const FfnArgs& A, int block, char* s_raw) {
  using M = MF<T>;
  using CH = Chunk<T, C, SPLIT ? 64 : 256, true>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, CK = M::CK, RS = CH::RS, RD = CH::RD, OS = C + 4;
  T* s = (T*)s_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int64_t a0 = SPLIT ? (int64_t)block * 16 : ((int64_t)block * 4 + wave) * (16 * AT);
  typename M::F xf[AT][NC], df[AT][NC];
  load_rows<T, C, AT>(xf, A.x, A.ldx, a0, A.n, i, g);
  load_rows<T, C, AT>(df, A.dy, A.ldy, a0, A.n, i, g);
  f4 acc[AT][C / 16];
#pragma unroll
  for (int at = 0; at < AT; ++at)
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) acc[at][ct] = f4{0.f, 0.f, 0.f, 0.f};
  CH ck;
  if constexpr (!SPLIT) {
    ck.fetch(A, 0, threadIdx.x);
    ck.put(s, threadIdx.x);
    __syncthreads();
  }
  int b = 0;
  for (int h0 = SPLIT ? CK * wave : 0; h0 < A.hidden; h0 += SPLIT ? 4 * CK : CK, b ^= 1) {
    T* buf = s + (SPLIT ? wave : b) * CH::SIZE;
    if constexpr (SPLIT) {
      ck.fetch(A, h0, lane);
      ck.put(buf, lane);
      wave_sync();
    } else {
      ck.fetch(A, min(h0 + CK, A.hidden - CK), threadIdx.x);
    }
    const T *wg = buf, *wu = wg + CK * RS, *wd = wu + CK * RS;
    f4 zg[AT][NT], zu[AT][NT], dh[AT][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int at = 0; at < AT; ++at) zg[at][t] = zu[at][t] = dh[at][t] = f4{0.f, 0.f, 0.f, 0.f};
      const int row = (16 * t + i) * RS + EV * g;
#pragma unroll
      for (int ch = 0; ch < NC; ++ch) {
        const typename M::F fg = *(const typename M::F*)(wg + row + ch * CK);
        const typename M::F fu = *(const typename M::F*)(wu + row + ch * CK);
        const typename M::F fd = ldt<RD>(wd, ch * CK, 16 * t, lane);
#pragma unroll
        for (int at = 0; at < AT; ++at) {
          zg[at][t] = M::mma(zg[at][t], fg, xf[at][ch]);
          zu[at][t] = M::mma(zu[at][t], fu, xf[at][ch]);
          dh[at][t] = M::mma(dh[at][t], fd, df[at][ch]);
        }
      }
    }
    typename M::F dg[AT], du[AT];
#pragma unroll
    for (int at = 0; at < AT; ++at) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float h, a, c;
          hidden_grad(zg[at][t][r], zu[at][t][r], dh[at][t][r], A.ab, h, a, c);
          zg[at][t][r] = a;
          zu[at][t][r] = c;
        }
      dg[at] = M::pack(zg[at]);
      du[at] = M::pack(zu[at]);
    }
    // hidden unit EV g + j of the operands is LDS row 16 t + 4 g + r: tile order
    constexpr bool FINE = SPLIT && sizeof(T) == 2;
    typename M::F dg2, du2;
    if constexpr (FINE) dg2 = rest_of<T>(dg[0], zg[0]), du2 = rest_of<T>(du[0], zu[0]);
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) {
      const typename M::F fg = ldt<RS>(wg, 0, 16 * ct, lane), fu = ldt<RS>(wu, 0, 16 * ct, lane);
      if constexpr (FINE) acc[0][ct] = M::mma(M::mma(acc[0][ct], fg, dg2), fu, du2);
#pragma unroll
      for (int at = 0; at < AT; ++at) acc[at][ct] = M::mma(M::mma(acc[at][ct], fg, dg[at]), fu, du[at]);
    }
    if constexpr (SPLIT) {
      wave_sync();
    } else {
      ck.put(s + (b ^ 1) * CH::SIZE, threadIdx.x);
      __syncthreads();
    }
  }
  if constexpr (SPLIT) {
    __syncthreads();  // the slabs lie over the chunks
    float* slab = (float*)s_raw + (16 * wave + i) * OS;
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) *(f4*)(slab + 16 * ct + 4 * g) = acc[0][ct];
    join_waves<T, C>((float*)s_raw, a0, A.n,
                     [&](int64_t a, int c, f4* o) { st_row<T>((T*)A.dx + a * A.lddx + c, o); });
  } else {
#pragma unroll
    for (int at = 0; at < AT; ++at) {
      const int64_t a = a0 + 16 * at + i;
      if (a >= A.n) continue;
#pragma unroll
      for (int ct = 0; ct < C / 16; ++ct) st4((T*)A.dx + a * A.lddx + 16 * ct + 4 * g, acc[at][ct]);
    }
  }
}

template <class T, int C, int AT, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(SPLIT ? 1 : 2, 2))) void k_ffn_dx(FfnArgs A) {
  __shared__ __align__(16) char s_raw[ffn_dx_lds<T, C, SPLIT>()];
  ffn_dx<T, C, AT, SPLIT>(A, blockIdx.x, s_raw);
}

// dWg, dWu, dWd over one split of the rows.  A wave owns 16 hidden units: their rows of Wg,
// Wu and Wd^T stay in registers, CK atoms' x and dy pass through LDS.  The hidden values are
// formed with the atoms as rows, which is tile order for the contraction over atoms:
//   dWg[hid][c] += dzg^T x,  dWu[hid][c] += dzu^T x,  dWd[c][hid] += dy^T h,
// x and dy read transposed from LDS.  Forming the hidden values a second time costs less than their way
// through memory would (672 MB written and read at 328,378 rows).  Bound as the forward: six products
// there in 285 us (905 TFLOP/s).
template <class T, int C>
constexpr int ffn_dw_lds() {
  return 4 * MF<T>::CK * (C + lds_pad<T>()) * (int)sizeof(T);
}
template <class T, int C, bool FEW>
__device__ __forceinline__ void ffn_dw(const FfnArgs& A, int bx, int by, char* s_raw) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, CK = M::CK, RS = C + lds_pad<T>();
  T *s_x = (T*)s_raw, *s_d = s_x + 2 * CK * RS;  // two buffers each
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int hw = bx * 64 + 16 * wave, hid = hw + i;
  const bool on = hw < A.hidden;
  typename M::F fg[NC], fu[NC], fd[NC];
  if (on) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
      const int c0 = ch * CK + EV * g;
      fg[ch] = *(const typename M::F*)((const T*)A.wg + (int64_t)hid * C + c0);
      fu[ch] = *(const typename M::F*)((const T*)A.wu + (int64_t)hid * C + c0);
      T t[EV];
#pragma unroll
      for (int j = 0; j < EV; ++j) t[j] = ((const T*)A.wd)[(int64_t)(c0 + j) * A.hidden + hid];
      fd[ch] = __builtin_bit_cast(typename M::F, t);
    }
  }
  f4 ag[C / 16], au[C / 16], ad[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) ag[ct] = au[ct] = ad[ct] = f4{0.f, 0.f, 0.f, 0.f};
  const int64_t r0 = (int64_t)by * A.rows_per_split, r1 = min(A.n, r0 + A.rows_per_split);
  Tile<T, CK, C, RS, 256> tx, td;
  auto fetch = [&](int64_t r) {
    const int rows = (int)min<int64_t>(CK, r1 - r);
    tx.fetch((const T*)A.x + r * A.ldx, A.ldx, rows, threadIdx.x);
    td.fetch((const T*)A.dy + r * A.ldy, A.ldy, rows, threadIdx.x);
  };
  if (r0 < r1) {
    fetch(r0);
    tx.put(s_x, threadIdx.x);
    td.put(s_d, threadIdx.x);
  }
  __syncthreads();
  int b = 0;
  for (int64_t r = r0; r < r1; r += CK, b ^= 1) {
    if (r + CK < r1) fetch(r + CK);
    if (on) {
      const T *xs = s_x + b * CK * RS, *ds = s_d + b * CK * RS;
      f4 h[NT], zg[NT], zu[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f4 dh = f4{0.f, 0.f, 0.f, 0.f};
        zg[t] = zu[t] = dh;
        const int row = (16 * t + i) * RS + EV * g;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
          const typename M::F fx = *(const typename M::F*)(xs + row + ch * CK);
          const typename M::F fy = *(const typename M::F*)(ds + row + ch * CK);
          zg[t] = M::mma(zg[t], fx, fg[ch]);
          zu[t] = M::mma(zu[t], fx, fu[ch]);
          dh = M::mma(dh, fy, fd[ch]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a, c, e;
          hidden_grad(zg[t][q], zu[t][q], dh[q], A.ab, e, a, c);
          h[t][q] = e;
          zg[t][q] = a;
          zu[t][q] = c;
        }
      }
      const typename M::F ph = M::pack(h), pg = M::pack(zg), pu = M::pack(zu);
      constexpr bool FINE = FEW && sizeof(T) == 2;
      typename M::F ph2, pg2, pu2;
      if constexpr (FINE) ph2 = rest_of<T>(ph, h), pg2 = rest_of<T>(pg, zg), pu2 = rest_of<T>(pu, zu);
#pragma unroll
      for (int ct = 0; ct < C / 16; ++ct) {
        const typename M::F fx = ldt<RS>(xs, 0, 16 * ct, lane), fy = ldt<RS>(ds, 0, 16 * ct, lane);
        if constexpr (FINE) {
          ag[ct] = M::mma(ag[ct], pg2, fx);
          au[ct] = M::mma(au[ct], pu2, fx);
          ad[ct] = M::mma(ad[ct], fy, ph2);
        }
        ag[ct] = M::mma(ag[ct], pg, fx);
        au[ct] = M::mma(au[ct], pu, fx);
        ad[ct] = M::mma(ad[ct], fy, ph);
      }
    }
    if (r + CK < r1) {
      tx.put(s_x + (b ^ 1) * CK * RS, threadIdx.x);
      td.put(s_d + (b ^ 1) * CK * RS, threadIdx.x);
    }
    __syncthreads();
  }
  if (!on) return;
  float* p = A.part + (int64_t)by * 3 * C * A.hidden;
  float* pu = p + (int64_t)C * A.hidden;
  float* pd = pu + (int64_t)C * A.hidden;
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      p[(int64_t)(hw + 4 * g + q) * C + 16 * ct + i] = ag[ct][q];
      pu[(int64_t)(hw + 4 * g + q) * C + 16 * ct + i] = au[ct][q];
      pd[(int64_t)(16 * ct + 4 * g + q) * A.hidden + hid] = ad[ct][q];
    }
}

template <class T, int C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_ffn_dw(FfnArgs A) {
  __shared__ __align__(16) char s_raw[ffn_dw_lds<T, C>()];
  ffn_dw<T, C, false>(A, blockIdx.x, blockIdx.y, s_raw);
}

// dx and the weight gradients of few rows in one launch: neither fills the card alone.  The first
// dx_blocks blocks form dx.
template <class T, int C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 2))) void k_ffn_bwd_few(FfnArgs A, int dx_blocks,
                                                                                               int nb) {
  constexpr int X = ffn_dx_lds<T, C, true>(), W = ffn_dw_lds<T, C>();
  __shared__ __align__(16) char s_raw[X > W ? X : W];
  const int b = (int)blockIdx.x - dx_blocks;
  if (b < 0)
    ffn_dx<T, C, 1, true>(A, blockIdx.x, s_raw);
  else
    ffn_dw<T, C, true>(A, b % nb, b / nb, s_raw);
}

// Splits of the rows for the weight gradients: about 512 blocks in all, each with at least
// 64 rows (a split costs three partial matrices written and read once; 4,096 rows of 64 float32,
// 256 hidden: 16.5 us and 6.4 for the sum, with at least 128 rows 20.4 and 5.3)
int64_t ffn_splits(int64_t n, int hidden) {
  const int64_t nb = cdiv(hidden, 64);
  return std::max<int64_t>(1, std::min<int64_t>(512 / nb, cdiv(n, 64)));
}

// Few rows: the hidden units are split over the waves of a block.  128 channels, 512 hidden
// units: bf16 27 us split and 28 not at 8,000 rows, 61 and 30 at 20,000; float32 50 and 108 at
// 8,000, 109 and 114 at 20,000.  There bf16's hidden units and their gradients enter the second
// products as two operands each (rest_of), so outputs carry one rounding and
// not three: 3 to 5 % of the backward, nothing of the forward.
bool ffn_few(int64_t n, bool bf16) { return n < (bf16 ? 8192 : 20480); }
// Whether dx and the weight gradients go in one launch, whose blocks all hold dx's LDS: float32, 256
// hidden of 64, with the sum: 17 us and 26 in two launches at 512 rows, 32 and 35 at 4,096; 512 of 128:
// 52 and 71 at 512, 62 and 78 at 2,048, but 160 and 155 at 8,000 (bf16 41 and 45, 65 and 60).
bool ffn_both(int64_t n, int C, bool bf16) { return n * C <= 384 << 10 && ffn_few(n, bf16); }
// what: 0 forward, 1 dx, 2 weight gradients, 3 both (few rows)
template <class T, int C>
int launch_ffn_c(FfnArgs A, int what, hipStream_t st) {
  constexpr int AT = sizeof(T) == 2 ? 2 : 1;
  const int64_t S = ffn_splits(A.n, A.hidden);
  A.rows_per_split = cdiv(cdiv(A.n, S), MF<T>::CK) * MF<T>::CK;
  if (what == 3) {
    const int nx = (int)cdiv(A.n, 16), nb = (int)cdiv(A.hidden, 64);
    k_ffn_bwd_few<T, C><<<(unsigned)(nx + nb * S), 256, 0, st>>>(A, nx, nb);
  } else if (what == 2) {
    k_ffn_dw<T, C><<<dim3((unsigned)cdiv(A.hidden, 64), (unsigned)S), 256, 0, st>>>(A);
  } else {
    const bool few = ffn_few(A.n, sizeof(T) == 2);
    const unsigned blocks = (unsigned)cdiv(A.n, few ? 16 : 64 * AT);
    if (what == 0) {
      if (few)
        k_ffn_few<T, C><<<blocks, 256, 0, st>>>(A);
      else
        k_ffn<T, C, AT><<<(unsigned)std::min<int64_t>(cdiv(A.n, 128 * AT), 256), 512, 0, st>>>(A);
    } else {
      if (few)
        k_ffn_dx<T, C, 1, true><<<blocks, 256, 0, st>>>(A);
      else
        k_ffn_dx<T, C, AT, false><<<blocks, 256, 0, st>>>(A);
    }
  }
  MP_CHECK_LAUNCH();
  return MP_OK;
}

int launch_ffn(const FfnArgs& A, int C, bool bf16, int what, hipStream_t st) {
  if (bf16) switch (C) {
      case 32: return launch_ffn_c<uint16_t, 32>(A, what, st);
      case 64: return launch_ffn_c<uint16_t, 64>(A, what, st);
      default: return launch_ffn_c<uint16_t, 128>(A, what, st);
    }
  switch (C) {
    case 16: return launch_ffn_c<float, 16>(A, what, st);
    case 32: return launch_ffn_c<float, 32>(A, what, st);
    case 64: return launch_ffn_c<float, 64>(A, what, st);
    default: return launch_ffn_c<float, 128>(A, what, st);
  }
}

int check_ffn(const char* who, int32_t n, int32_t channels, int32_t hidden, int32_t dt, int32_t act) {
  MP_TRY(check_width(who, channels, dt));
  if (n < 0 || n > kMaxRows) return arg_error(std::string(who) + ": n must be in 0..2^26");
  if (hidden < 32 || hidden > 4096 || hidden % 32)
    return arg_error(std::string(who) + ": hidden must be a multiple of 32 in 32..4096");
  if (act != MP_ACT_SILU && act != MP_ACT_SIGMOID) return arg_error(std::string(who) + ": act must be SiLU or sigmoid");
  return MP_OK;
}

FfnArgs ffn_args(int32_t n, int32_t hidden, int32_t act, const void* x, int64_t ldx, const void* wg, const void* wu,
                 const void* wd) {
  FfnArgs A{};
  A.n = n, A.hidden = hidden;
  A.ab = act == MP_ACT_SILU ? ActAB{1.f, 0.f} : ActAB{0.f, 1.f};
  A.x = x, A.ldx = ldx, A.wg = wg, A.wu = wu, A.wd = wd;
  return A;
}

}  // namespace
}  // namespace ops
}  // namespace mdmp

using namespace mdmp;

extern "C" int mp_gated_ffn(int32_t n, int32_t channels, int32_t hidden, int32_t dt, int32_t act, const void* x,
                            int64_t ldx, const void* wg, const void* wu, const void* wd, const void* residual,
                            int64_t ldr, void* y, int64_t ldy, hipStream_t st) {
  MP_TRY(ops::check_ffn("mp_gated_ffn", n, channels, hidden, dt, act));
  if (n == 0) return MP_OK;
  if (!x || !wg || !wu || !wd || !y) return arg_error("mp_gated_ffn: null x, weights or y");
  if (x == y) return arg_error("mp_gated_ffn: y must not be x");
  if (((uintptr_t)wg | (uintptr_t)wu | (uintptr_t)wd) & 15)
    return arg_error("mp_gated_ffn: weights must be 16-byte aligned");
  MP_ROWS("mp_gated_ffn", "x", x, ldx, channels, dt);
  MP_ROWS("mp_gated_ffn", "y", y, ldy, channels, dt);
  if (residual) MP_ROWS("mp_gated_ffn", "residual", residual, ldr, channels, dt);
  ops::FfnArgs A = ops::ffn_args(n, hidden, act, x, ldx, wg, wu, wd);
  A.res = residual, A.ldr = ldr, A.y = y, A.ldy = ldy;
  ProfScope p("gated_ffn", st);
  return ops::launch_ffn(A, channels, dt == 1, 0, st);
}

extern "C" int mp_gated_ffn_bwd_ws(int32_t n, int32_t channels, int32_t hidden, int32_t dt, size_t* bytes) {
  MP_TRY(ops::check_ffn("mp_gated_ffn_bwd_ws", n, channels, hidden, dt, MP_ACT_SILU));
  if (!bytes) return arg_error("mp_gated_ffn_bwd_ws: null bytes");
  *bytes = align_up(sizeof(float) * 3 * (size_t)channels * hidden * ops::ffn_splits(n, hidden));
  return MP_OK;
}

extern "C" int mp_gated_ffn_bwd(int32_t n, int32_t channels, int32_t hidden, int32_t dt, int32_t act, const void* x,
                                int64_t ldx, const void* wg, const void* wu, const void* wd, const void* dy,
                                int64_t lddy, void* dx, int64_t lddx, void* dwg, void* dwu, void* dwd, void* ws,
                                size_t ws_bytes, hipStream_t st) {
  MP_TRY(ops::check_ffn("mp_gated_ffn_bwd", n, channels, hidden, dt, act));
  const bool grads = dwg || dwu || dwd;
  if (grads && !(dwg && dwu && dwd)) return arg_error("mp_gated_ffn_bwd: give all three weight gradients or none");
  if (n > 0) {
    if (!x || !wg || !wu || !wd || !dy) return arg_error("mp_gated_ffn_bwd: null x, weights or dy");
    if (dx && (dx == x || dx == dy)) return arg_error("mp_gated_ffn_bwd: dx must not be x or dy");
    if (((uintptr_t)wg | (uintptr_t)wu | (uintptr_t)wd) & 15)
      return arg_error("mp_gated_ffn_bwd: weights must be 16-byte aligned");
    MP_ROWS("mp_gated_ffn_bwd", "x", x, ldx, channels, dt);
    MP_ROWS("mp_gated_ffn_bwd", "dy", dy, lddy, channels, dt);
    if (dx) MP_ROWS("mp_gated_ffn_bwd", "dx", dx, lddx, channels, dt);
  }
  ops::FfnArgs A = ops::ffn_args(n, hidden, act, x, ldx, wg, wu, wd);
  A.dy = dy, A.ldy = lddy, A.dx = dx, A.lddx = lddx;
  if (grads) {
    size_t need = 0;
    MP_TRY(mp_gated_ffn_bwd_ws(n, channels, hidden, dt, &need));
    if (!ws || ((uintptr_t)ws & 15)) return arg_error("mp_gated_ffn_bwd: workspace null or not 16-byte aligned");
    if (ws_bytes < need) return arg_error("mp_gated_ffn_bwd: workspace too small");
    A.part = (float*)ws;
  }
  ProfScope p("gated_ffn_bwd", st);
  if (n > 0 && dx && grads && ops::ffn_both(n, channels, dt == 1)) {
    MP_TRY(ops::launch_ffn(A, channels, dt == 1, 3, st));
  } else {
    if (n > 0 && dx) MP_TRY(ops::launch_ffn(A, channels, dt == 1, 1, st));
    if (!grads) return MP_OK;
    if (n > 0) MP_TRY(ops::launch_ffn(A, channels, dt == 1, 2, st));
  }
  const int64_t S = n > 0 ? ops::ffn_splits(n, hidden) : 0, N = (int64_t)channels * hidden;
  const ops::Segment seg[3] = {{0, N, dwg, dt == 1}, {N, N, dwu, dt == 1}, {2 * N, N, dwd, dt == 1}};
  return ops::reduce_rows(A.part, S, 3 * N, seg, 3, st);
}
