// Norm after a block, its gate and residual scale, and the norm before the next block.
#include <cmath>

#include "ops_api.hpp"

namespace mdmp {
namespace ops {
namespace {

// With ms(t) = mean_c t^2 + eps, per row:
//   bn = b ms(b)^-1/2          (bn = b without w_post)
//   y  = x + scale sigmoid(gate) w_post bn
//   u  = w_pre y ms(y)^-1/2    (from y before it is rounded to the feature type)
// A row lives in LR = C / V adjacent lanes, V values (16 bytes) each, so the two means are
// exchanges inside those lanes and every tensor is read or written once, 16 bytes a lane.
// Bound: HBM.  1,048,576 rows of 128 bf16 without a gate: 192-204 us, 5.3-5.6 TB/s; 131,072 of float32 with one:
// forward 53 us (6.3 TB/s), backward 87 (6.2).
template <class T, int V>
struct Row {
  float v[V];
  __device__ __forceinline__ void load(const T* p) {
    typename MF<T>::F f = *(const typename MF<T>::F*)p;
    f4 t[2];
    MF<T>::unpack(f, t);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = t[j / 4][j % 4];
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(T* p) const {
    f4 t[2];
#pragma unroll
    for (int j = 0; j < V; ++j) t[j / 4][j % 4] = v[j];
    st_row<STREAM>(p, t);
  }
};

// V consecutive float32 parameters (16-byte aligned), or a constant where there are none
template <int V>
__device__ __forceinline__ void ldp(float* v, const float* p, float other) {
#pragma unroll
  for (int q = 0; q < V / 4; ++q) {
    const f4 t = p ? *(const f4*)(p + 4 * q) : f4{other, other, other, other};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * q + j] = t[j];
  }
}

// x^-1/2 to float32 rounding: the hardware value and one Newton step
__device__ __forceinline__ float rsq(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  const float e = fmaf(-x * r, r, 1.0f);
  return x < 3.0e38f ? fmaf(0.5f * r, e, r) : r;
}

struct NormPtrs {
  int64_t n, ldx, ldb, ldg, ldy, ldu, lddx, lddb, lddg;
  const void *x, *b, *gate;
  const float *scale, *w_post, *w_pre;
  float eps;
  void *y, *u;                    // forward outputs (u may be null)
  const void *dy, *du;            // backward inputs (either may be null); strides ldy, ldu
  void *dx, *db, *dg;             // backward outputs (nullable)
  float* part;                    // [blocks][3][C]
  bool stream;                    // outputs past the caches
};

template <class T, int C, bool STREAM>
__global__ __launch_bounds__(256) void k_norm_block(NormPtrs A) {
  constexpr int V = MF<T>::EV, LR = C / V, RPB = 256 / LR;
  const int rl = threadIdx.x / LR, c0 = (threadIdx.x % LR) * V;
  float sc[V], wp[V], wq[V];
  ldp<V>(sc, A.scale ? A.scale + c0 : nullptr, 1.0f);
  ldp<V>(wp, A.w_post ? A.w_post + c0 : nullptr, 1.0f);
  ldp<V>(wq, A.w_pre ? A.w_pre + c0 : nullptr, 0.0f);
  // rows past the end leave the loop as a whole group of LR lanes, so every exchange runs
  // inside one group
  for (int64_t row = (int64_t)blockIdx.x * RPB + rl; row < A.n; row += (int64_t)gridDim.x * RPB) {
    Row<T, V> x, b, g;
    x.load((const T*)A.x + row * A.ldx + c0);
    b.load((const T*)A.b + row * A.ldb + c0);
    if (A.gate) g.load((const T*)A.gate + row * A.ldg + c0);
    float ib = 1.0f;
    if (A.w_post) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(b.v[j], b.v[j], s);
      ib = rsq(group_sum<LR>(s) * (1.0f / C) + A.eps);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float gs = A.gate ? sc[j] * sigm(g.v[j]) : sc[j];
      x.v[j] = fmaf(gs, wp[j] * (b.v[j] * ib), x.v[j]);
    }
    x.template store<STREAM>((T*)A.y + row * A.ldy + c0);
    if (A.u) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(x.v[j], x.v[j], s);
      const float iy = rsq(group_sum<LR>(s) * (1.0f / C) + A.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) x.v[j] = wq[j] * (x.v[j] * iy);
      x.template store<STREAM>((T*)A.u + row * A.ldu + c0);
    }
  }
}

// Backward: y is formed again from x, b and gate (cheaper than reading it back), the row's
// gradients follow the chain above, and each lane keeps the sums over its rows of the three
// parameter gradients of its channels.  Blocks walk rows with a fixed stride and write one
// partial row each, added up in block order afterwards, so repeated calls give equal bits.
template <class T, int C, bool STREAM>
__global__ __launch_bounds__(256) void k_norm_block_bwd(NormPtrs A) {
  constexpr int V = MF<T>::EV, LR = C / V, RPB = 256 / LR;
  __shared__ float s_p[RPB][3 * C];
  const int rl = threadIdx.x / LR, c0 = (threadIdx.x % LR) * V;
  float sc[V], wp[V], wq[V], a_s[V], a_p[V], a_q[V];
  ldp<V>(sc, A.scale ? A.scale + c0 : nullptr, 1.0f);
  ldp<V>(wp, A.w_post ? A.w_post + c0 : nullptr, 1.0f);
  ldp<V>(wq, A.w_pre ? A.w_pre + c0 : nullptr, 0.0f);
#pragma unroll
  for (int j = 0; j < V; ++j) a_s[j] = a_p[j] = a_q[j] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * RPB + rl; row < A.n; row += (int64_t)gridDim.x * RPB) {
    Row<T, V> x, b, g, dy, du;
    x.load((const T*)A.x + row * A.ldx + c0);
    b.load((const T*)A.b + row * A.ldb + c0);
    if (A.gate) g.load((const T*)A.gate + row * A.ldg + c0);
    if (A.dy) dy.load((const T*)A.dy + row * A.ldy + c0);
    if (A.du) du.load((const T*)A.du + row * A.ldu + c0);
    float ib = 1.0f;
    if (A.w_post) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(b.v[j], b.v[j], s);
      ib = rsq(group_sum<LR>(s) * (1.0f / C) + A.eps);
    }
    float gs[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      gs[j] = A.gate ? sigm(g.v[j]) : 1.0f;
      b.v[j] *= ib;  // bn
      if (!A.dy) dy.v[j] = 0.f;
    }
    if (A.du) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x.v[j] = fmaf(sc[j] * gs[j], wp[j] * b.v[j], x.v[j]);  // y
        s = fmaf(x.v[j], x.v[j], s);
      }
      const float iy = rsq(group_sum<LR>(s) * (1.0f / C) + A.eps);
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x.v[j] *= iy;  // y / rms(y)
        a_q[j] = fmaf(du.v[j], x.v[j], a_q[j]);
        du.v[j] *= wq[j];
        t = fmaf(du.v[j], x.v[j], t);
      }
      t = group_sum<LR>(t) * (1.0f / C);
#pragma unroll
      for (int j = 0; j < V; ++j) dy.v[j] = fmaf(iy, fmaf(-x.v[j], t, du.v[j]), dy.v[j]);
    }
    if (A.dx) dy.template store<STREAM>((T*)A.dx + row * A.lddx + c0);
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float bw = wp[j] * b.v[j], ds = dy.v[j] * gs[j];
      a_s[j] = fmaf(ds, bw, a_s[j]);
      if (A.gate) g.v[j] = dy.v[j] * sc[j] * bw * gs[j] * (1.0f - gs[j]);
      dy.v[j] = ds * sc[j];
      a_p[j] = fmaf(dy.v[j], b.v[j], a_p[j]);
      dy.v[j] *= wp[j];
      t = fmaf(dy.v[j], b.v[j], t);
    }
    if (A.dg) g.template store<STREAM>((T*)A.dg + row * A.lddg + c0);
    if (A.db) {
      if (A.w_post) {
        t = group_sum<LR>(t) * (1.0f / C);
#pragma unroll
        for (int j = 0; j < V; ++j) dy.v[j] = ib * fmaf(-b.v[j], t, dy.v[j]);
      }
      dy.template store<STREAM>((T*)A.db + row * A.lddb + c0);
    }
  }
  if (!A.part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    s_p[rl][c0 + j] = a_s[j];
    s_p[rl][C + c0 + j] = a_p[j];
    s_p[rl][2 * C + c0 + j] = a_q[j];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 3 * C; k += 256) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < RPB; ++r) s += s_p[r][k];
    A.part[(size_t)blockIdx.x * 3 * C + k] = s;
  }
}

template <class T, int C>
void launch_norm_c(const NormPtrs& A, bool bwd, int blocks, hipStream_t st) {
  auto* k = bwd ? (A.stream ? k_norm_block_bwd<T, C, true> : k_norm_block_bwd<T, C, false>)
                : (A.stream ? k_norm_block<T, C, true> : k_norm_block<T, C, false>);
  k<<<blocks, 256, 0, st>>>(A);
}

template <class T>
int launch_norm(const NormPtrs& A, int C, bool bwd, int blocks, hipStream_t st) {
#define MP_CASE(CC)                            \
  case CC:                                     \
    launch_norm_c<T, CC>(A, bwd, blocks, st);  \
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

// one partial row of parameter gradients per block of the backward pass: enough blocks to
// fill the 256 CUs four times, no more than there are rows for
int norm_blocks(int64_t n, int C, bool bf16, int most = 1024) {
  const int rpb = 256 / (C / (bf16 ? 8 : 4));
  return (int)std::min<int64_t>(cdiv(n, rpb), most);
}

struct Segments {
  Segment s[3];
};
// A block of 1024 threads takes NCOL columns, its thread rows every (1024 / NCOL)-th partial row,
// joined pairwise.  Few columns (the distance slopes) take 8: with 32, three quarters of the
// threads would idle over thousands of partial rows (9,300 rows of 4: 48 us against 6).
template <int NCOL>
__global__ __launch_bounds__(1024) void k_reduce_rows(const float* __restrict__ part, int64_t S, int64_t ldp, Segments G) {
  constexpr int NR = 1024 / NCOL;
  __shared__ float sh[NR][NCOL];
  const Segment sg = G.s[blockIdx.y];
  const int c = threadIdx.x % NCOL, r = threadIdx.x / NCOL;
  const int64_t j = (int64_t)blockIdx.x * NCOL + c;
  if ((int64_t)blockIdx.x * NCOL >= sg.N) return;
  float s = 0.f;
  if (j < sg.N) {
#pragma unroll 8
    for (int64_t k = r; k < S; k += NR) s += part[k * ldp + sg.off + j];
  }
  sh[r][c] = s;
  __syncthreads();
#pragma unroll
  for (int o = NR / 2; o > 0; o >>= 1) {
    if (r < o) sh[r][c] += sh[r + o][c];
    __syncthreads();
  }
  if (r == 0 && j < sg.N) {
    if (sg.bf16)
      ((uint16_t*)sg.out)[j] = f2bf(sh[0][c]);
    else
      ((float*)sg.out)[j] = sh[0][c];
  }
}

}  // namespace

int reduce_rows(const float* part, int64_t S, int64_t ldp, const Segment* seg, int nseg, hipStream_t st) {
  Segments G{};
  int k = 0;
  int64_t most = 0;
  for (int q = 0; q < nseg; ++q)
    if (seg[q].out) {
      most = std::max(most, seg[q].N);
      G.s[k++] = seg[q];
    }
  if (k == 0) return MP_OK;
  if (most <= 8)
    k_reduce_rows<8><<<dim3(1, k), 1024, 0, st>>>(part, S, ldp, G);
  else
    k_reduce_rows<32><<<dim3((unsigned)cdiv(most, 32), k), 1024, 0, st>>>(part, S, ldp, G);
  MP_CHECK_LAUNCH();
  return MP_OK;
}

}  // namespace ops

static int check_norm(const mp_norm_args* a, ops::NormPtrs& A) {
  if (!a) return arg_error("mp_norm_block: null arguments");
  MP_TRY(ops::check_width("mp_norm_block", a->channels, a->feat_dtype));
  if (a->n < 0 || a->n > ops::kMaxRows) return arg_error("mp_norm_block: n must be in 0..2^26");
  // below that the hardware's reciprocal square root takes a zero row to infinity
  if (!(a->eps >= 1e-30f) || !std::isfinite(a->eps)) return arg_error("mp_norm_block: eps must be finite and >= 1e-30");
  if (((uintptr_t)a->scale | (uintptr_t)a->w_post | (uintptr_t)a->w_pre) & 15)
    return arg_error("mp_norm_block: scale, w_post and w_pre must be 16-byte aligned");
  A = ops::NormPtrs{};
  A.n = a->n;
  A.x = a->x, A.b = a->b, A.gate = a->gate;
  A.ldx = a->ldx, A.ldb = a->ldb, A.ldg = a->ldg;
  A.scale = a->scale, A.w_post = a->w_post, A.w_pre = a->w_pre;
  A.eps = a->eps;
  if (a->n == 0) return MP_OK;
  if (!a->x || !a->b) return arg_error("mp_norm_block: null x or b");
  MP_ROWS("mp_norm_block", "x", a->x, a->ldx, a->channels, a->feat_dtype);
  MP_ROWS("mp_norm_block", "b", a->b, a->ldb, a->channels, a->feat_dtype);
  if (a->gate) MP_ROWS("mp_norm_block", "gate", a->gate, a->ldg, a->channels, a->feat_dtype);
  return MP_OK;
}

}  // namespace mdmp

using namespace mdmp;

extern "C" int mp_norm_block(const mp_norm_args* a, void* y, int64_t ldy, void* u, int64_t ldu, hipStream_t st) {
  ops::NormPtrs A;
  MP_TRY(check_norm(a, A));
  if ((u != nullptr) != (a->w_pre != nullptr) && a->n > 0)
    return arg_error("mp_norm_block: u is written if and only if w_pre is given");
  if (a->n == 0) return MP_OK;
  if (!y) return arg_error("mp_norm_block: null y");
  MP_ROWS("mp_norm_block", "y", y, ldy, a->channels, a->feat_dtype);
  if (u) MP_ROWS("mp_norm_block", "u", u, ldu, a->channels, a->feat_dtype);
  A.y = y, A.ldy = ldy, A.u = u, A.ldu = ldu;
  A.stream = ops::streams((int64_t)a->n * a->channels * (a->feat_dtype == 1 ? 2 : 4) * (3 + !!a->gate + !!u));
  ProfScope p("norm_block", st);
  const int blocks = ops::norm_blocks(a->n, a->channels, a->feat_dtype == 1, 8192);
  return a->feat_dtype == 1 ? ops::launch_norm<uint16_t>(A, a->channels, false, blocks, st)
                            : ops::launch_norm<float>(A, a->channels, false, blocks, st);
}

extern "C" int mp_norm_block_bwd_ws(int32_t n, int32_t channels, int32_t feat_dtype, size_t* bytes) {
  MP_TRY(ops::check_width("mp_norm_block_bwd_ws", channels, feat_dtype));
  if (n < 0 || n > ops::kMaxRows || !bytes) return arg_error("mp_norm_block_bwd_ws: bad arguments");
  *bytes = align_up(sizeof(float) * 3 * channels * (size_t)std::max(1, ops::norm_blocks(n, channels, feat_dtype == 1)));
  return MP_OK;
}

extern "C" int mp_norm_block_bwd(const mp_norm_args* a, const void* dy, int64_t lddy, const void* du, int64_t lddu,
                                 void* dx, int64_t lddx, void* db, int64_t lddb, void* dgate, int64_t lddg,
                                 float* dscale, float* dw_post, float* dw_pre, void* ws, size_t ws_bytes,
                                 hipStream_t st) {
  ops::NormPtrs A;
  MP_TRY(check_norm(a, A));
  const int C = a->channels, dt = a->feat_dtype;
  if (dgate && !a->gate && a->n > 0) return arg_error("mp_norm_block_bwd: dgate without a gate");
  if (dw_post && !a->w_post) return arg_error("mp_norm_block_bwd: dw_post without w_post");
  if (dw_pre && !a->w_pre) return arg_error("mp_norm_block_bwd: dw_pre without w_pre");
  const bool params = dscale || dw_post || dw_pre;
  if (a->n > 0) {
    if (!dy && !du) return arg_error("mp_norm_block_bwd: dy and du are both null");
    if (du && !a->w_pre) return arg_error("mp_norm_block_bwd: du without w_pre");
    if (dy) MP_ROWS("mp_norm_block_bwd", "dy", dy, lddy, C, dt);
    if (du) MP_ROWS("mp_norm_block_bwd", "du", du, lddu, C, dt);
    if (dx) MP_ROWS("mp_norm_block_bwd", "dx", dx, lddx, C, dt);
    if (db) MP_ROWS("mp_norm_block_bwd", "db", db, lddb, C, dt);
    if (dgate) MP_ROWS("mp_norm_block_bwd", "dgate", dgate, lddg, C, dt);
  }
  A.dy = dy, A.ldy = lddy, A.du = du, A.ldu = lddu;
  A.dx = dx, A.lddx = lddx, A.db = db, A.lddb = lddb, A.dg = dgate, A.lddg = lddg;
  A.stream = ops::streams((int64_t)a->n * C * (dt == 1 ? 2 : 4) *
                          (2 + !!a->gate + !!dy + !!du + !!dx + !!db + !!dgate));
  int blocks = 0;
  if (params) {
    size_t need = 0;
    MP_TRY(mp_norm_block_bwd_ws(a->n, C, dt, &need));
    if (!ws || ws_bytes < need) return arg_error("mp_norm_block_bwd: workspace too small");
    if ((uintptr_t)ws & 15) return arg_error("mp_norm_block_bwd: workspace must be 16-byte aligned");
    A.part = (float*)ws;
  }
  ProfScope p("norm_block_bwd", st);
  if (a->n > 0) {
    blocks = ops::norm_blocks(a->n, C, dt == 1);
    MP_TRY(dt == 1 ? ops::launch_norm<uint16_t>(A, C, true, blocks, st)
                   : ops::launch_norm<float>(A, C, true, blocks, st));
  }
  // no rows: sums over nothing, zeros
  const ops::Segment seg[3] = {{0, C, dscale, false}, {C, C, dw_post, false}, {2 * C, C, dw_pre, false}};
  return ops::reduce_rows(A.part, blocks, 3 * C, seg, 3, st);
}
