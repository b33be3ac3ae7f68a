// Energy and forces with global blocks (attention beyond the cutoff, feed-forward) between
// the last layer and the readout: the block operators in sequence, forward and backward.
#include <algorithm>
#include <vector>

#include "model.hpp"
#include "ops.hpp"

struct mp_mixer {
  int32_t C = 0, B = 0, H = 0, F = 0, dt = 0;
  float cap = 0.f;
  void* dev = nullptr;  // one allocation for the arrays below
  struct Block {
    const void *wqkv, *wo, *wg, *wu, *wd;                    // feature type
    const float *w1, *slope, *p1, *s1, *w2, *p2, *s2;        // float32
  } blk[MP_MAX_BLOCKS];
  const float* zero;  // [C], the scale of a norm without a block
};

namespace mdmp {
namespace {

constexpr float kEps = 1e-6f;

// what one block keeps for its backward pass: the streams before the attention (x0) and the
// feed-forward (x1), both norms' outputs, queries | keys | values, attention and block outputs
struct Saved {
  void *x0, *u1, *qkv, *att, *o, *x1, *u2, *f;
  float *stat, *dpos;
};
struct Carve {
  Saved s[MP_MAX_BLOCKS];
  void *dx, *du, *db, *da, *dqkv;  // gradients, one block's at a time
  void* ws;                        // of the attention calls, one at a time
  size_t ws_bytes;
};

int carve(Arena& a, const mp_mixer* M, int32_t n, int32_t n_struct, Carve& w) {
  const int es = M->dt == 1 ? 2 : 4;
  auto rows = [&](int c) { return (void*)a.take<char>((int64_t)n * c * es); };
  int64_t stat = 0;
  MP_TRY(mp_structure_attention_saved(n, M->C, M->H, M->dt, &stat));
  for (int t = 0; t < M->B; ++t) {
    Saved& s = w.s[t];
    s.x0 = rows(M->C), s.u1 = rows(M->C), s.qkv = rows(3 * M->C), s.att = rows(M->C), s.o = rows(M->C);
    s.x1 = rows(M->C), s.u2 = rows(M->C), s.f = rows(M->C);
    s.stat = a.take<float>(stat);
    s.dpos = a.take<float>((int64_t)n * 3);
  }
  w.dx = rows(M->C), w.du = rows(M->C), w.db = rows(M->C), w.da = rows(M->C), w.dqkv = rows(3 * M->C);
  size_t fwd = 0;
  MP_TRY(mp_structure_attention_ws(n, n_struct, M->C, M->H, &fwd));
  MP_TRY(mp_structure_attention_bwd_ws(n, n_struct, M->C, M->H, &w.ws_bytes));
  w.ws_bytes = std::max(w.ws_bytes, fwd);
  w.ws = a.take<char>((int64_t)w.ws_bytes);
  return MP_OK;
}

mp_norm_args norm_args(const mp_mixer* M, int n, const void* x, int64_t ldx, const void* b, int64_t ldb,
                       const float* scale, const float* post, const float* pre) {
  return mp_norm_args{n, M->C, M->dt, kEps, x, ldx, b, ldb, nullptr, 0, scale, post, pre};
}

const void* col(const void* p, int c, int dt) { return (const char*)p + (size_t)c * (dt == 1 ? 2 : 4); }
void* col(void* p, int c, int dt) { return (char*)p + (size_t)c * (dt == 1 ? 2 : 4); }

mp_attention_args attention_args(const MixRun& R, const mp_mixer* M, const mp_mixer::Block& W, const mp_graph* g,
                                 const void* qkv) {
  mp_attention_args a{};
  a.n = g->n, a.n_struct = R.n_struct, a.channels = M->C, a.heads = M->H, a.feat_dtype = M->dt;
  a.cap = M->cap, a.box_L = g->box_L;
  a.struct_ptr = R.struct_ptr, a.pos = g->pos, a.slope = W.slope;
  a.q = qkv, a.k = col(qkv, M->C, M->dt), a.v = col(qkv, 2 * M->C, M->dt);
  a.ldq = a.ldk = a.ldv = 3 * M->C;
  return a;
}

// rows 0 of g_h (float32, stride K C) to bf16 rows and back, 4 channels a thread
__global__ __launch_bounds__(256) void k_grad_rows(float* __restrict__ g_h, int64_t n, int C, int64_t ld,
                                                   uint16_t* __restrict__ rows, bool back) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, r = x / (C / 4);
  if (r >= n) return;
  const int c = (int)(x % (C / 4)) * 4;
  float* p = g_h + r * ld + c;
  uint16_t* q = rows + r * C + c;
  if (back)
    ops::st4(p, ops::f4{bf2f(q[0]), bf2f(q[1]), bf2f(q[2]), bf2f(q[3])});
  else
    ops::st4(q, *(const ops::f4*)p);
}

struct DposList {
  const float* p[MP_MAX_BLOCKS];
};
// forces[perm] -= the blocks' position gradients, in block order; non-finite sums set the flag's
// first bit, a struct_ptr that does not go from 0 to n in ascending order its second (rows outside
// the structures have no attention, so their sums mean nothing)
__global__ __launch_bounds__(256) void k_mixer_forces(DposList L, int B, int n, const int32_t* __restrict__ perm,
                                                      const int32_t* __restrict__ sptr, int n_struct,
                                                      float* __restrict__ F, int32_t* __restrict__ flag) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  bool bad = x == 0 && (sptr[0] != 0 || sptr[n_struct] != n);
  for (int64_t b = x; b < n_struct; b += (int64_t)gridDim.x * 256) bad |= sptr[b] > sptr[b + 1];
  if (bad) atomicOr(flag, 2);
  if (x >= 3 * (int64_t)n) return;
  float s = 0.f;
  for (int t = 0; t < B; ++t) s += L.p[t][x];
  const int i = (int)(x / 3);
  const int64_t o = 3 * (int64_t)(perm ? perm[i] : i) + x % 3;
  const float f = F[o] - s;
  F[o] = f;
  if (!isfinite(f)) atomicOr(flag, 1);
}

int64_t count(const mp_model* m, int32_t B, int32_t H, int32_t F) {
  const int64_t C = m->cfg.channels;
  return B * (4 * C * C + 3 * C * (int64_t)F + 6 * C + H);
}

int check_shape(const mp_model* m, int32_t B, int32_t H, int32_t F) {
  if (!m) return arg_error("mixer: null model");
  if (B < 1 || B > MP_MAX_BLOCKS) return arg_error("mixer: n_blocks out of range");
  // the operators' own checks of the shape (no rows: nothing is launched)
  int64_t s = 0;
  MP_TRY(mp_structure_attention_saved(0, m->cfg.channels, H, m->cfg.feat_dtype, &s));
  size_t b = 0;
  return mp_gated_ffn_bwd_ws(0, m->cfg.channels, F, m->cfg.feat_dtype, &b);
}

uint16_t round_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

}  // namespace

int mixer_forward(const MixRun& R, const Plan& P, const mp_graph* g, void* h, hipStream_t st) {
  const mp_mixer* M = R.mixer;
  const int n = P.n, C = M->C, F = M->F, dt = M->dt;
  const int64_t ldh = (int64_t)P.K * C;
  Arena a(R.ws, R.ws_bytes);
  Carve w;
  MP_TRY(carve(a, M, n, R.n_struct, w));
  if (!a.ok()) return arg_error("mp_energy_forces_mixer: workspace too small");
  // x0 = h^0 (a scale of zero: nothing is added), u = its norm
  mp_norm_args na = norm_args(M, n, h, ldh, h, ldh, M->zero, nullptr, M->blk[0].w1);
  MP_TRY(mp_norm_block(&na, w.s[0].x0, C, w.s[0].u1, C, st));
  for (int t = 0; t < M->B; ++t) {
    const mp_mixer::Block& W = M->blk[t];
    Saved& s = w.s[t];
    MP_TRY(mp_linear(n, C, 3 * C, dt, MP_ACT_NONE, s.u1, C, W.wqkv, nullptr, nullptr, 0, s.qkv, 3 * C, st));
    const mp_attention_args aa = attention_args(R, M, W, g, s.qkv);
    MP_TRY(mp_structure_attention(&aa, s.att, C, s.stat, w.ws, w.ws_bytes, st));
    MP_TRY(mp_linear(n, C, C, dt, MP_ACT_NONE, s.att, C, W.wo, nullptr, nullptr, 0, s.o, C, st));
    na = norm_args(M, n, s.x0, C, s.o, C, W.s1, W.p1, W.w2);
    MP_TRY(mp_norm_block(&na, s.x1, C, s.u2, C, st));
    MP_TRY(mp_gated_ffn(n, C, F, dt, MP_ACT_SILU, s.u2, C, W.wg, W.wu, W.wd, nullptr, 0, s.f, C, st));
    const bool last = t == M->B - 1;
    na = norm_args(M, n, s.x1, C, s.f, C, W.s2, W.p2, last ? nullptr : M->blk[t + 1].w1);
    MP_TRY(last ? mp_norm_block(&na, h, ldh, nullptr, 0, st)
                : mp_norm_block(&na, w.s[t + 1].x0, C, w.s[t + 1].u1, C, st));
  }
  return MP_OK;
}

int mixer_backward(const MixRun& R, const Plan& P, const mp_graph* g, float* g_h, hipStream_t st) {
  const mp_mixer* M = R.mixer;
  const int n = P.n, C = M->C, F = M->F, dt = M->dt;
  const int64_t ldg = (int64_t)P.K * C;
  Arena a(R.ws, R.ws_bytes);
  Carve w;
  MP_TRY(carve(a, M, n, R.n_struct, w));
  if (!a.ok()) return arg_error("mp_energy_forces_mixer: workspace too small");
  const int blocks = (int)cdiv((int64_t)n * (C / 4), 256);
  void* dx = g_h;  // the gradient of the stream, in place; bf16 features: in bf16 rows
  int64_t ldx = ldg;
  if (dt == 1) {
    dx = w.dx, ldx = C;
    k_grad_rows<<<blocks, 256, 0, st>>>(g_h, n, C, ldg, (uint16_t*)dx, false);
    MP_CHECK_LAUNCH();
  }
  for (int t = M->B - 1; t >= 0; --t) {
    const mp_mixer::Block& W = M->blk[t];
    const Saved& s = w.s[t];
    const bool last = t == M->B - 1;
    mp_norm_args na = norm_args(M, n, s.x1, C, s.f, C, W.s2, W.p2, last ? nullptr : M->blk[t + 1].w1);
    MP_TRY(mp_norm_block_bwd(&na, dx, ldx, last ? nullptr : w.du, C, dx, ldx, w.db, C, nullptr, 0, nullptr, nullptr,
                             nullptr, nullptr, 0, st));
    MP_TRY(mp_gated_ffn_bwd(n, C, F, dt, MP_ACT_SILU, s.u2, C, W.wg, W.wu, W.wd, w.db, C, w.du, C, nullptr, nullptr,
                            nullptr, nullptr, 0, st));
    na = norm_args(M, n, s.x0, C, s.o, C, W.s1, W.p1, W.w2);
    MP_TRY(mp_norm_block_bwd(&na, dx, ldx, w.du, C, dx, ldx, w.db, C, nullptr, 0, nullptr, nullptr, nullptr, nullptr,
                             0, st));
    MP_TRY(mp_linear_bwd(n, C, C, dt, MP_ACT_NONE, s.att, C, W.wo, nullptr, w.db, C, w.da, C, nullptr, nullptr, nullptr,
                         0, st));
    const mp_attention_args aa = attention_args(R, M, W, g, s.qkv);
    MP_TRY(mp_structure_attention_bwd(&aa, s.att, C, s.stat, w.da, C, w.dqkv, 3 * C, col(w.dqkv, C, dt), 3 * C,
                                      col(w.dqkv, 2 * C, dt), 3 * C, s.dpos, nullptr, w.ws, w.ws_bytes, st));
    MP_TRY(mp_linear_bwd(n, C, 3 * C, dt, MP_ACT_NONE, s.u1, C, W.wqkv, nullptr, w.dqkv, 3 * C, w.du, C, nullptr,
                         nullptr, nullptr, 0, st));
  }
  mp_norm_args na = norm_args(M, n, w.s[0].x0, C, w.s[0].x0, C, M->zero, nullptr, M->blk[0].w1);
  MP_TRY(mp_norm_block_bwd(&na, dx, ldx, w.du, C, dx, ldx, nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr, nullptr,
                           0, st));
  if (dt == 1) {
    k_grad_rows<<<blocks, 256, 0, st>>>(g_h, n, C, ldg, (uint16_t*)dx, true);
    MP_CHECK_LAUNCH();
  }
  return MP_OK;
}

int mixer_forces(const MixRun& R, const Plan& P, const int32_t* perm, float* forces, int32_t* flag, hipStream_t st) {
  Arena a(R.ws, R.ws_bytes);
  Carve w;
  MP_TRY(carve(a, R.mixer, P.n, R.n_struct, w));
  DposList L{};
  for (int t = 0; t < R.mixer->B; ++t) L.p[t] = w.s[t].dpos;
  k_mixer_forces<<<(int)cdiv(3 * (int64_t)P.n, 256), 256, 0, st>>>(L, R.mixer->B, P.n, perm, R.struct_ptr, R.n_struct,
                                                                 forces, flag);
  MP_CHECK_LAUNCH();
  return MP_OK;
}

}  // namespace mdmp

using namespace mdmp;

extern "C" int mp_mixer_num_weights(const mp_model* m, int32_t n_blocks, int32_t heads, int32_t hidden, int64_t* n) {
  MP_TRY(check_shape(m, n_blocks, heads, hidden));
  if (!n) return arg_error("mp_mixer_num_weights: null n");
  *n = count(m, n_blocks, heads, hidden);
  return MP_OK;
}

extern "C" int mp_mixer_create(const mp_model* m, int32_t n_blocks, int32_t heads, int32_t hidden, float cap,
                               const float* w, int64_t nw, mp_mixer** out) {
  MP_TRY(check_shape(m, n_blocks, heads, hidden));
  if (!w || !out) return arg_error("mp_mixer_create: null weights or out");
  if (!(cap == 0.f || (cap >= 1e-3f && cap <= 1e4f))) return arg_error("mp_mixer_create: cap must be 0 or in 1e-3..1e4");
  if (nw != count(m, n_blocks, heads, hidden)) return arg_error("mp_mixer_create: weight count does not match");
  const int C = m->cfg.channels, dt = m->cfg.feat_dtype, es = dt == 1 ? 2 : 4;
  const int64_t CC = (int64_t)C * C, CF = (int64_t)C * hidden;
  mp_mixer* M = nullptr;
  std::vector<char> buf;
  std::vector<size_t> off;
  try {
    M = new mp_mixer();
    auto add = [&](const float* src, int64_t k, bool matrix) {
      const size_t o = align_up(buf.size());
      off.push_back(o);
      buf.resize(o + (size_t)k * (matrix ? es : 4));
      if (matrix && dt == 1)
        for (int64_t q = 0; q < k; ++q) ((uint16_t*)(buf.data() + o))[q] = round_bf16(src[q]);
      else
        std::copy(src, src + k, (float*)(buf.data() + o));
    };
    const float* p = w;
    auto next = [&](int64_t k, bool matrix) {
      add(p, k, matrix);
      p += k;
    };
    for (int t = 0; t < n_blocks; ++t) {
      next(C, false), next(3 * CC, true), next(heads, false), next(CC, true), next(C, false), next(C, false);
      next(C, false), next(CF, true), next(CF, true), next(CF, true), next(C, false), next(C, false);
    }
    const std::vector<float> z(C, 0.f);
    add(z.data(), C, false);
  } catch (const std::exception&) {
    delete M;
    return arg_error("mp_mixer_create: out of host memory");
  }
  hipError_t e = hipMalloc(&M->dev, buf.size());
  if (e == hipSuccess) e = hipMemcpy(M->dev, buf.data(), buf.size(), hipMemcpyHostToDevice);
  if (e != hipSuccess) {
    if (M->dev) (void)hipFree(M->dev);
    delete M;
    set_error(std::string("mp_mixer_create: ") + hipGetErrorString(e));
    return MP_ERR_HIP;
  }
  M->C = C, M->B = n_blocks, M->H = heads, M->F = hidden, M->dt = dt, M->cap = cap;
  auto at = [&](size_t k) { return (const float*)((const char*)M->dev + off[k]); };
  for (int t = 0; t < n_blocks; ++t) {
    mp_mixer::Block& b = M->blk[t];
    const size_t k = 12 * (size_t)t;
    b.w1 = at(k), b.wqkv = at(k + 1), b.slope = at(k + 2), b.wo = at(k + 3), b.p1 = at(k + 4), b.s1 = at(k + 5);
    b.w2 = at(k + 6), b.wg = at(k + 7), b.wu = at(k + 8), b.wd = at(k + 9), b.p2 = at(k + 10), b.s2 = at(k + 11);
  }
  M->zero = at(12 * (size_t)n_blocks);
  *out = M;
  return MP_OK;
}

extern "C" int mp_mixer_destroy(mp_mixer* M) {
  if (!M) return MP_OK;
  (void)hipFree(M->dev);
  delete M;
  return MP_OK;
}

static int check_run(const mp_model* m, const mp_mixer* M, int32_t n, int32_t n_struct) {
  if (!m || !M) return arg_error("mp_energy_forces_mixer: null model or mixer");
  if (M->C != m->cfg.channels || M->dt != m->cfg.feat_dtype)
    return arg_error("mp_energy_forces_mixer: the mixer was made for another model's channels or feature type");
  if (n < 1 || n_struct < 1) return arg_error("mp_energy_forces_mixer: n and n_struct must be >= 1");
  return MP_OK;
}

extern "C" int mp_energy_forces_mixer_ws(const mp_model* m, const mp_mixer* M, int32_t n, int32_t n_struct,
                                         int64_t n_edges, size_t* bytes) {
  MP_TRY(check_run(m, M, n, n_struct));
  if (!bytes || n_edges < 0) return arg_error("mp_energy_forces_mixer_ws: bad arguments");
  Arena a(nullptr, 0, true);
  Carve w;
  MP_TRY(carve(a, M, n, n_struct, w));
  *bytes = ef_bytes(m, n, n_edges) + a.off;
  return MP_OK;
}

extern "C" int mp_energy_forces_mixer(const mp_model* m, const mp_mixer* M, const mp_graph* g,
                                      const int32_t* struct_ptr, int32_t n_struct, const int32_t* perm, double* energy,
                                      float* forces, float* atom_energy, void* ws, size_t ws_bytes, hipStream_t st) {
  if (!g) return arg_error("mp_energy_forces_mixer: null graph");
  MP_TRY(check_run(m, M, g->n, n_struct));
  if (!struct_ptr) return arg_error("mp_energy_forces_mixer: null struct_ptr");
  size_t need = 0;
  MP_TRY(mp_energy_forces_mixer_ws(m, M, g->n, n_struct, g->n_edges, &need));
  if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need)
    return arg_error("mp_energy_forces_mixer: workspace null, not 256-byte aligned or too small");
  const size_t own = ef_bytes(m, g->n, g->n_edges);
  const MixRun R{M, struct_ptr, n_struct, (char*)ws + own, ws_bytes - own};
  return ef_enqueue(m, g, g->n_edges, perm, energy, forces, atom_energy, ws, own, nullptr, st, nullptr, nullptr, &R);
}
