// y = residual + act(x W^T + bias) on atom rows, and its gradients.
#include "ops_api.hpp"

namespace mdmp {
namespace ops {
namespace {

struct LinArgs {
  int64_t n, ldx, ldr, ldy, lddx;  // ldy: stride of y (forward) or dy (backward)
  int out;
  bool act;
  ActAB ab;
  const void *x, *w, *res, *dy;
  const float* bias;
  void *y, *dx;
  float* part;           // [splits][out C + out]: dW, then dbias
  int64_t rows_per_split;
  bool stream;  // y past the caches
};

// EV outputs of one atom: bias, activation, residual, 16-byte store
template <class T, bool STREAM>
__device__ __forceinline__ void lin_out(const LinArgs& A, int64_t a, int oe, const f4* bias, f4* o) {
  using M = MF<T>;
#pragma unroll
  for (int t = 0; t < M::NT; ++t) o[t] += bias[t];
  if (A.act) {
#pragma unroll
    for (int t = 0; t < M::NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[t][r] = act_val(o[t][r], A.ab);
  }
  if (A.res) {
    f4 q[M::NT];
    M::unpack(*(const typename M::F*)((const T*)A.res + a * A.ldr + oe), q);
#pragma unroll
    for (int t = 0; t < M::NT; ++t) o[t] += q[t];
  }
  st_row<STREAM>((T*)A.y + a * A.ldy + oe, o);
}
template <int NT>
__device__ __forceinline__ void lin_bias(const LinArgs& A, int oe, f4* b) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    b[t] = f4{0.f, 0.f, 0.f, 0.f};
    if (A.bias && oe < A.out)
      b[t] = f4{A.bias[oe + 4 * t], A.bias[oe + 4 * t + 1], A.bias[oe + 4 * t + 2], A.bias[oe + 4 * t + 3]};
  }
}

// Forward, few rows: D[o][a] = sum_c W[o][c] x[a][c].  A wave keeps 16 atoms' rows in registers as
// one operand and walks the outputs CK at a time, the other operand read straight from W.  W's
// rows are taken in the order nat_row, which leaves EV consecutive outputs of an atom in each
// lane: bias, activation, residual and the 16-byte stores follow without an exchange.
// gridDim.y splits the outputs.  Bound: latency of its two reads (512 rows of 128 float32: 4.3 us).
template <class T, int C>
__global__ __launch_bounds__(256) void k_linear_few(LinArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, OG = M::CK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t a = ((int64_t)blockIdx.x * 4 + wave) * 16 + i;
  if (a - i >= A.n) return;
  typename M::F xf[NC];
  const T* p = (const T*)A.x + a * A.ldx + EV * g;
#pragma unroll
  for (int ch = 0; ch < NC; ++ch) xf[ch] = ld16<typename M::F>(p + ch * M::CK, a < A.n);
  const int ngr = (A.out + OG - 1) / OG;
  const int per = (ngr + gridDim.y - 1) / gridDim.y;
  const int g0 = blockIdx.y * per, g1 = min(ngr, g0 + per);
  for (int og = g0; og < g1; ++og) {
    const int oe = og * OG + EV * g;
    f4 acc[NT], bias[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const T* wp = (const T*)A.w + (int64_t)min(og * OG + nat_row<T>(t, i), A.out - 1) * C + EV * g;
      acc[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ch = 0; ch < NC; ++ch) acc[t] = M::mma(acc[t], *(const typename M::F*)(wp + ch * M::CK), xf[ch]);
    }
    lin_bias<NT>(A, oe, bias);
    if (a < A.n && oe < A.out) lin_out<T, false>(A, a, oe, bias, acc);
  }
}

// Forward, many rows: the same product with OB outputs' rows of W resident in LDS (in the order
// nat_slot) for the whole walk of a block over its rows; each of the eight waves walks tiles of
// 16 AT atoms by itself, the next tile's rows on their way.  gridDim.y covers the outputs.
// Bound: HBM (the y rows): 328,378 rows of 128 -> 384 in bf16 take 87 us, 3.9 TB/s of the 4.9 that a
// large copy reaches.  W read from L2 by every wave instead: 115 us (the traffic of L1).
template <class T, int C, int OB, int AT, bool STREAM>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_linear(LinArgs A) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, OG = M::CK, RS = C + lds_pad<T>(), VPR = C / EV;
  __shared__ __align__(16) T s_w[OB * RS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int ob = blockIdx.y * OB, no = min(OB, A.out - ob);
  const int64_t tiles = (A.n + 16 * AT - 1) / (16 * AT), step = (int64_t)gridDim.x * 8;
  int64_t tile = (int64_t)blockIdx.x * 8 + wave;
  typename M::F xf[AT][NC], xn[AT][NC];
  auto fetch = [&](int64_t tl) {  // rows past the end: the last row
#pragma unroll
    for (int at = 0; at < AT; ++at) {
      const int64_t a = min(tl * (16 * AT) + 16 * at + i, A.n - 1);
      const T* p = (const T*)A.x + a * A.ldx + EV * g;
#pragma unroll
      for (int ch = 0; ch < NC; ++ch) xn[at][ch] = *(const typename M::F*)(p + ch * M::CK);
    }
  };
  fetch(tile);
  for (int x = threadIdx.x; x < no * VPR; x += 512) {
    const int r = x / VPR, c = (x % VPR) * EV;
    *(u4*)(s_w + nat_slot<T>(r) * RS + c) = *(const u4*)((const T*)A.w + (int64_t)(ob + r) * C + c);
  }
  __syncthreads();
  for (; tile < tiles; tile += step) {
#pragma unroll
    for (int at = 0; at < AT; ++at)
#pragma unroll
      for (int ch = 0; ch < NC; ++ch) xf[at][ch] = xn[at][ch];
    fetch(tile + step);
    for (int o0 = 0; o0 < no; o0 += OG) {
      const int oe = ob + o0 + EV * g;
      f4 acc[AT][NT], bias[NT];
      lin_bias<NT>(A, oe, bias);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const T* wp = s_w + (o0 + 16 * t + i) * RS + EV * g;
#pragma unroll
        for (int at = 0; at < AT; ++at) acc[at][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
          const typename M::F f = *(const typename M::F*)(wp + ch * M::CK);
#pragma unroll
          for (int at = 0; at < AT; ++at) acc[at][t] = M::mma(acc[at][t], f, xf[at][ch]);
        }
      }
#pragma unroll
      for (int at = 0; at < AT; ++at) {
        const int64_t a = tile * (16 * AT) + 16 * at + i;
        if (a < A.n && oe < A.out) lin_out<T, STREAM>(A, a, oe, bias, acc[at]);
      }
    }
  }
}

// dx: D[c][a] = sum_o W[o][c] dz[a][o], dz = dy act'(z), z formed again by the forward's
// product.  Both operands of dz sit as EV consecutive outputs per lane (natural order), so
// dz goes from result to operand in registers.  W passes through LDS CK rows at a time,
// output nat_row(t, i) in row 16 t + i, read there by rows (z) and transposed (dx).
// SPLIT (few rows): the four waves take the same 16 atoms and every fourth group of outputs,
// each with rows of its own in LDS, and their sums are joined.
// Bound: HBM (dy rows) without an activation.
template <class T, int C, bool SPLIT>
constexpr int linear_dx_lds() {
  constexpr int ROWS = (SPLIT ? 4 : 2) * MF<T>::CK * (C + lds_pad<T>()) * (int)sizeof(T), SLAB = SPLIT ? 64 * (C + 4) * 4 : 0;
  return ROWS > SLAB ? ROWS : SLAB;
}
template <class T, int C, bool SPLIT>
__device__ __forceinline__ void linear_dx(const LinArgs& A, int block, char* s_raw) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, OG = M::CK, RS = C + lds_pad<T>(), OS = C + 4;
  T* s = (T*)s_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int64_t a0 = SPLIT ? (int64_t)block * 16 : ((int64_t)block * 4 + wave) * 16;
  const int64_t a = a0 + i;
  typename M::F xf[NC];
  if (A.act) {
    const T* p = (const T*)A.x + a * A.ldx + EV * g;
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) xf[ch] = ld16<typename M::F>(p + ch * M::CK, a < A.n);
  }
  f4 dx[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) dx[ct] = f4{0.f, 0.f, 0.f, 0.f};
  const int ngr = (A.out + OG - 1) / OG, tid = SPLIT ? lane : (int)threadIdx.x, step = SPLIT ? 4 : 1;
  auto slot = [](int r) { return nat_slot<T>(r); };
  Tile<T, OG, C, RS, SPLIT ? 64 : 256> tw;
  typename M::F dz, dzn;
  auto fetch = [&](int og) {
    const int o0 = og * OG, oe = o0 + EV * g;
    tw.fetch((const T*)A.w + (int64_t)o0 * C, C, A.out - o0, tid);
    dzn = ld16<typename M::F>((const T*)A.dy + a * A.ldy + oe, a < A.n && oe < A.out);
  };
  const int og0 = SPLIT ? wave : 0;
  if (og0 < ngr) fetch(og0);
  int b = 0;
  for (int og = og0; og < ngr; og += step, b ^= 1) {
    const int oe = og * OG + EV * g;
    T* w = s + (SPLIT ? wave : b) * OG * RS;
    tw.put(w, tid, slot);
    dz = dzn;
    // two buffers: a wave that is a step ahead writes the one that the others have left
    if constexpr (SPLIT)
      wave_sync();
    else
      __syncthreads();
    if (og + step < ngr) fetch(og + step);
    if (A.act) {
      f4 z[NT], d[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        z[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
          z[t] = M::mma(z[t], *(const typename M::F*)(w + (16 * t + i) * RS + ch * M::CK + EV * g), xf[ch]);
      }
      M::unpack(dz, d);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float bias = A.bias && oe < A.out ? A.bias[oe + 4 * t + r] : 0.f;
          float v, e;
          act_both(z[t][r] + bias, A.ab, v, e);
          d[t][r] *= e;
        }
      dz = M::pack(d);
      if constexpr (SPLIT && sizeof(T) == 2) {  // few rows: dz as two operands
        const typename M::F dz2 = rest_of<T>(dz, d);
#pragma unroll
        for (int ct = 0; ct < C / 16; ++ct) dx[ct] = M::mma(dx[ct], ldt<RS>(w, 0, 16 * ct, lane), dz2);
      }
    }
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) dx[ct] = M::mma(dx[ct], ldt<RS>(w, 0, 16 * ct, lane), dz);
    if constexpr (SPLIT) wave_sync();
  }
  if constexpr (SPLIT) {
    __syncthreads();  // the slabs lie over the rows of W
    float* slab = (float*)s_raw + (16 * wave + i) * OS;
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) *(f4*)(slab + 16 * ct + 4 * g) = dx[ct];
    join_waves<T, C>((float*)s_raw, a0, A.n,
                     [&](int64_t r, int c, f4* o) { st_row<T>((T*)A.dx + r * A.lddx + c, o); });
  } else {
    if (a >= A.n) return;
#pragma unroll
    for (int ct = 0; ct < C / 16; ++ct) st4((T*)A.dx + a * A.lddx + 16 * ct + 4 * g, dx[ct]);
  }
}

template <class T, int C, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_linear_dx(LinArgs A) {
  __shared__ __align__(16) char s_raw[linear_dx_lds<T, C, SPLIT>()];
  linear_dx<T, C, SPLIT>(A, blockIdx.x, s_raw);
}

// dW, dbias: D[o][c] = sum_a dz[a][o] x[a][c] over one split of the rows.  A wave owns 16
// outputs and all C channels; CK atoms at a time pass through LDS.  z is formed with the
// atoms as rows, which is tile order for the contraction over atoms, the order in which dy
// and x are read transposed.  Each split writes its own partial, added up in split order.
// Bound: HBM (x and dy rows).
constexpr int kDwOut = 64;  // outputs of a block
template <class T, int C>
constexpr int linear_dw_lds() {
  return 2 * MF<T>::CK * (C + kDwOut + 2 * lds_pad<T>()) * (int)sizeof(T);
}
template <class T, int C, bool FEW>
__device__ __forceinline__ void linear_dw(const LinArgs& A, int bx, int by, char* s_raw) {
  using M = MF<T>;
  constexpr int NC = C / M::CK, EV = M::EV, NT = M::NT, CK = M::CK, RS = C + lds_pad<T>();
  constexpr int OB = kDwOut, RO = OB + lds_pad<T>();
  T *s_x = (T*)s_raw, *s_d = s_x + 2 * CK * RS;  // two buffers each
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int ob = bx * OB, o = ob + 16 * wave + i;
  const bool on = ob + 16 * wave < A.out;
  typename M::F wf[NC];
  float bias = 0.f, db = 0.f;
  if (on && A.act) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
      wf[ch] = *(const typename M::F*)((const T*)A.w + (int64_t)o * C + ch * CK + EV * g);
    if (A.bias) bias = A.bias[o];
  }
  f4 acc[C / 16];
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct) acc[ct] = f4{0.f, 0.f, 0.f, 0.f};
  const int64_t r0 = (int64_t)by * A.rows_per_split, r1 = min(A.n, r0 + A.rows_per_split);
  Tile<T, CK, C, RS, 256> tx;
  // the block's 64 columns of dy; columns past the last output read as zeros
  constexpr int VPD = OB / EV, ITD = (CK * VPD + 255) / 256;
  u4 vd[ITD];
  auto fetch = [&](int64_t r) {
    tx.fetch((const T*)A.x + r * A.ldx, A.ldx, (int)min<int64_t>(CK, r1 - r), threadIdx.x);
#pragma unroll
    for (int k = 0; k < ITD; ++k) {
      const int x = threadIdx.x + k * 256, rr = x / VPD, c = (x % VPD) * EV;
      vd[k] = ld16<u4>((const T*)A.dy + (r + rr) * A.ldy + ob + c, x < CK * VPD && r + rr < r1 && ob + c < A.out);
    }
  };
  auto put = [&](int b) {
    tx.put(s_x + b * CK * RS, threadIdx.x);
#pragma unroll
    for (int k = 0; k < ITD; ++k) {
      const int x = threadIdx.x + k * 256, rr = x / VPD, c = (x % VPD) * EV;
      if (x < CK * VPD) *(u4*)(s_d + b * CK * RO + rr * RO + c) = vd[k];
    }
  };
  if (r0 < r1) {
    fetch(r0);
    put(0);
  }
  __syncthreads();
  int b = 0;
  for (int64_t r = r0; r < r1; r += CK, b ^= 1) {
    if (r + CK < r1) fetch(r + CK);
    if (on) {
      const T *xs = s_x + b * CK * RS, *ds = s_d + b * CK * RO;
      typename M::F dz = ldt<RO>(ds, 0, 16 * wave, lane);
      f4 d[NT];
      M::unpack(dz, d);
      if (A.act) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          f4 z = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ch = 0; ch < NC; ++ch)
            z = M::mma(z, *(const typename M::F*)(xs + (16 * t + i) * RS + ch * CK + EV * g), wf[ch]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v, e;
            act_both(z[q] + bias, A.ab, v, e);
            d[t][q] *= e;
          }
        }
        dz = M::pack(d);
        if constexpr (FEW && sizeof(T) == 2) {
          const typename M::F dz2 = rest_of<T>(dz, d);
#pragma unroll
          for (int ct = 0; ct < C / 16; ++ct) acc[ct] = M::mma(acc[ct], dz2, ldt<RS>(xs, 0, 16 * ct, lane));
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) db += (d[t].x + d[t].y) + (d[t].z + d[t].w);
#pragma unroll
      for (int ct = 0; ct < C / 16; ++ct) acc[ct] = M::mma(acc[ct], dz, ldt<RS>(xs, 0, 16 * ct, lane));
    }
    if (r + CK < r1) put(b ^ 1);
    __syncthreads();
  }
  if (!on) return;
  float* ps = A.part + (int64_t)by * A.out * (C + 1);
  float* p = ps + (int64_t)(ob + 16 * wave) * C;
#pragma unroll
  for (int ct = 0; ct < C / 16; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) p[(4 * g + q) * C + 16 * ct + i] = acc[ct][q];
  db = gsum(db);
  if (g == 0) ps[(int64_t)A.out * C + o] = db;
}

template <class T, int C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3))) void k_linear_dw(LinArgs A) {
  __shared__ __align__(16) char s_raw[linear_dw_lds<T, C>()];
  linear_dw<T, C, false>(A, blockIdx.x, blockIdx.y, s_raw);
}

// dx and dW of few rows in one launch: neither fills the card alone.  The first dx_blocks blocks
// form dx.
template <class T, int C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_linear_bwd_few(LinArgs A, int dx_blocks,
                                                                                               int nb) {
  constexpr int X = linear_dx_lds<T, C, true>(), W = linear_dw_lds<T, C>();
  __shared__ __align__(16) char s_raw[X > W ? X : W];
  const int b = (int)blockIdx.x - dx_blocks;
  if (b < 0)
    linear_dx<T, C, true>(A, blockIdx.x, s_raw);
  else
    linear_dw<T, C, true>(A, b % nb, b / nb, s_raw);
}

// Splits of the rows for dW: about 512 blocks in all, each with at least 32 rows (a split
// costs a partial matrix written and read once)
int64_t dw_splits(int64_t n, int out) {
  const int64_t nb = cdiv(out, 64);
  return std::max<int64_t>(1, std::min<int64_t>(512 / nb, cdiv(n, 32)));
}

template <class T, int C, int OB>
void launch_linear_big(const LinArgs& A, dim3 grid, hipStream_t st) {
  auto* k = A.stream ? k_linear<T, C, OB, 2, true> : k_linear<T, C, OB, 2, false>;
  k<<<grid, 512, 0, st>>>(A);
}

// Few rows: dx splits its outputs over the waves of a block, and goes in one launch with dW (float32,
// 128 -> 128, with the sum: 9.8 us and 15.4 in two launches at 512 rows, 36 and 39 at 16,000).
bool linear_both(int64_t n) { return n < 32768; }
// what: 0 forward, 1 dx, 2 dW and dbias, 3 both (few rows)
template <class T>
int launch_linear(const LinArgs& A0, int C, int what, hipStream_t st) {
  LinArgs A = A0;
  constexpr int BIG = sizeof(T) == 2 ? 512 : 256;  // outputs whose rows fit LDS at C = 128
  // Few rows: every wave takes one 16-atom tile, and the outputs are split too.  128 -> 384: bf16
  // 16 us so and 19 with W in LDS at 8,000 rows, 33 and 23 at 32,000; float32 21 and 48 at 8,000,
  // 60 and 53 at 32,000.
  const bool few = A.n < (sizeof(T) == 2 ? 16384 : 28672);
  const int64_t bx = few ? cdiv(A.n, 64) : std::min<int64_t>(cdiv(A.n, 256), A.out <= 128 ? 512 : 256);
  const int by = few ? (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(A.out, MF<T>::CK), 512 / bx))
                     : (int)cdiv(A.out, A.out <= 128 ? 128 : BIG);
  const int64_t S = dw_splits(A.n, A.out);
  A.rows_per_split = cdiv(cdiv(A.n, S), MF<T>::CK) * MF<T>::CK;
#define MP_CASE(CC)                                                                         \
  case CC:                                                                                  \
    if (what == 0) {                                                                        \
      if (few)                                                                              \
        k_linear_few<T, CC><<<dim3((unsigned)bx, by), 256, 0, st>>>(A);                     \
      else if (A.out <= 128)                                                                \
        launch_linear_big<T, CC, 128>(A, dim3((unsigned)bx, by), st);                       \
      else                                                                                  \
        launch_linear_big<T, CC, BIG>(A, dim3((unsigned)bx, by), st);                       \
    } else if (what == 1) {                                                                 \
      if (linear_both(A.n))                                                                  \
        k_linear_dx<T, CC, true><<<(unsigned)cdiv(A.n, 16), 256, 0, st>>>(A);               \
      else                                                                                  \
        k_linear_dx<T, CC, false><<<(unsigned)cdiv(A.n, 64), 256, 0, st>>>(A);              \
    } else if (what == 3) {                                                                 \
      const int nx = (int)cdiv(A.n, 16), nb = (int)cdiv(A.out, kDwOut);                     \
      k_linear_bwd_few<T, CC><<<(unsigned)(nx + nb * S), 256, 0, st>>>(A, nx, nb);          \
    } else {                                                                                \
      k_linear_dw<T, CC><<<dim3((unsigned)cdiv(A.out, 64), (unsigned)S), 256, 0, st>>>(A);  \
    }                                                                                       \
    break;
  switch (C) {
    MP_CASE(32)
    MP_CASE(64)
    MP_CASE(128)
    default:
      if constexpr (sizeof(T) == 4) {
        switch (C) { MP_CASE(16) }
      }
  }
#undef MP_CASE
  MP_CHECK_LAUNCH();
  return MP_OK;
}

int check_linear(const char* who, int32_t n, int32_t in, int32_t out, int32_t dt, int32_t act) {
  MP_TRY(check_width(who, in, dt));
  if (n < 0 || n > kMaxRows) return arg_error(std::string(who) + ": n must be in 0..2^26");
  if (out < 16 || out > 1024 || out % 16) return arg_error(std::string(who) + ": out must be a multiple of 16 in 16..1024");
  if (act < MP_ACT_NONE || act > MP_ACT_SIGMOID) return arg_error(std::string(who) + ": unknown activation");
  return MP_OK;
}

LinArgs lin_args(int32_t n, int32_t out, int32_t act, const void* x, int64_t ldx, const void* w, const float* bias) {
  LinArgs A{};
  A.n = n, A.out = out;
  A.act = act != MP_ACT_NONE;
  A.ab = act == MP_ACT_SILU ? ActAB{1.f, 0.f} : ActAB{0.f, 1.f};
  A.x = x, A.ldx = ldx, A.w = w, A.bias = bias;
  return A;
}

}  // namespace
}  // namespace ops
}  // namespace mdmp

using namespace mdmp;

extern "C" int mp_linear(int32_t n, int32_t in, int32_t out, int32_t dt, int32_t act, const void* x, int64_t ldx,
                         const void* w, const float* bias, const void* residual, int64_t ldr, void* y, int64_t ldy,
                         hipStream_t st) {
  MP_TRY(ops::check_linear("mp_linear", n, in, out, dt, act));
  if (n == 0) return MP_OK;
  if (!x || !w || !y) return arg_error("mp_linear: null x, w or y");
  if (x == y) return arg_error("mp_linear: y must not be x");
  if ((uintptr_t)w & 15) return arg_error("mp_linear: w must be 16-byte aligned");
  MP_ROWS("mp_linear", "x", x, ldx, in, dt);
  MP_ROWS("mp_linear", "y", y, ldy, out, dt);
  if (residual) MP_ROWS("mp_linear", "residual", residual, ldr, out, dt);
  ops::LinArgs A = ops::lin_args(n, out, act, x, ldx, w, bias);
  A.res = residual, A.ldr = ldr, A.y = y, A.ldy = ldy;
  A.stream = ops::streams((int64_t)n * (in + (int64_t)out * (residual ? 2 : 1)) * (dt == 1 ? 2 : 4));
  ProfScope p("linear", st);
  return dt == 1 ? ops::launch_linear<uint16_t>(A, in, 0, st) : ops::launch_linear<float>(A, in, 0, st);
}

extern "C" int mp_linear_bwd_ws(int32_t n, int32_t in, int32_t out, int32_t dt, size_t* bytes) {
  MP_TRY(ops::check_linear("mp_linear_bwd_ws", n, in, out, dt, 0));
  if (!bytes) return arg_error("mp_linear_bwd_ws: null bytes");
  const int64_t S = ops::dw_splits(n, out);
  *bytes = align_up(sizeof(float) * (size_t)(S * out * (in + 1)));
  return MP_OK;
}

extern "C" int mp_linear_bwd(int32_t n, int32_t in, int32_t out, int32_t dt, int32_t act, const void* x, int64_t ldx,
                             const void* w, const float* bias, const void* dy, int64_t lddy, void* dx, int64_t lddx,
                             void* dw, float* dbias, void* ws, size_t ws_bytes, hipStream_t st) {
  MP_TRY(ops::check_linear("mp_linear_bwd", n, in, out, dt, act));
  if (n > 0) {
    if (!x || !w || !dy) return arg_error("mp_linear_bwd: null x, w or dy");
    if (dx && (dx == x || dx == dy)) return arg_error("mp_linear_bwd: dx must not be x or dy");
    if ((uintptr_t)w & 15) return arg_error("mp_linear_bwd: w must be 16-byte aligned");
    MP_ROWS("mp_linear_bwd", "x", x, ldx, in, dt);
    MP_ROWS("mp_linear_bwd", "dy", dy, lddy, out, dt);
    if (dx) MP_ROWS("mp_linear_bwd", "dx", dx, lddx, in, dt);
  }
  ops::LinArgs A = ops::lin_args(n, out, act, x, ldx, w, bias);
  A.dy = dy, A.ldy = lddy, A.dx = dx, A.lddx = lddx;
  int64_t S = 0;
  if (dw || dbias) {
    if (!ws || ((uintptr_t)ws & 15)) return arg_error("mp_linear_bwd: workspace null or not 16-byte aligned");
    size_t need = 0;
    MP_TRY(mp_linear_bwd_ws(n, in, out, dt, &need));
    if (ws_bytes < need) return arg_error("mp_linear_bwd: workspace too small");
    S = ops::dw_splits(n, out);
    A.part = (float*)ws;
  }
  ProfScope p("linear_bwd", st);
  auto go = [&](int what) {
    return dt == 1 ? ops::launch_linear<uint16_t>(A, in, what, st) : ops::launch_linear<float>(A, in, what, st);
  };
  if (n > 0 && dx && A.part && ops::linear_both(n)) {
    MP_TRY(go(3));
  } else {
    if (n > 0 && dx) MP_TRY(go(1));
    if (!A.part) return MP_OK;
    if (n > 0) MP_TRY(go(2));
  }
  if (n == 0) S = 0;  // no rows: sums over nothing, zeros
  const int64_t N = (int64_t)out * in;
  const ops::Segment seg[2] = {{0, N, dw, dt == 1}, {N, out, dbias, false}};
  return ops::reduce_rows(A.part, S, N + out, seg, 2, st);
}
