// C ABI of the attention between all atoms of each structure.
#include <algorithm>
#include <cmath>

#include "ops_api.hpp"
#include "ops_attn.hpp"

namespace mdmp {
namespace ops {
namespace {

// Structures of up to this many atoms on average: a block is one wave, 16 atoms of a structure.
// Longer ones: blocks of four waves own 64 atoms and share their way along the other side.
constexpr int kLongAbove = 64;
bool long_ones(int64_t n, int64_t n_struct) { return n > kLongAbove * n_struct; }

// Slots of rows in the grid
int64_t slots_of(int64_t n, int64_t n_struct) { return n / (long_ones(n, n_struct) ? 64 : 16) + n_struct; }

// Splits of the other side over blocks, for few long structures: towards 2,048 blocks (the chip
// holds 768 at a time, and a last round that is not full should be a small part of the whole),
// each with at least 128 atoms of the other side, at most 16 (each costs a float32 partial of the
// rows, written and read once).
int splits_of(int64_t n, int64_t n_struct) {
  if (!long_ones(n, n_struct)) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>({cdiv(2048, slots_of(n, n_struct)), n / n_struct / 128, 16}));
}

constexpr int32_t kMaxStruct = 1 << 25;  // with kMaxRows: slots of 64 threads in 32 bits

// the kernels address the rows of one step by 32-bit offsets from a 64-bit base
constexpr int64_t kMaxLd = 1 << 24;

int check_shape(const char* who, int32_t n, int32_t channels, int32_t heads, int32_t dt) {
  MP_TRY(check_width(who, channels, dt));
  if (n < 0 || n > kMaxRows) return arg_error(std::string(who) + ": n must be in 0..2^26");
  const int dh = heads >= 1 && channels % heads == 0 ? channels / heads : 0;
  if (dh != 16 && dh != 32 && dh != 64) return arg_error(std::string(who) + ": channels / heads must be 16, 32 or 64");
  return MP_OK;
}

int attn_args(const char* who, const mp_attention_args* a, AttnArgs& A) {
  if (!a) return arg_error(std::string(who) + ": null arguments");
  MP_TRY(check_shape(who, a->n, a->channels, a->heads, a->feat_dtype));
  if (a->n_struct < 0 || a->n_struct > kMaxStruct) return arg_error(std::string(who) + ": n_struct must be in 0..2^25");
  if (!cap_ok(a->cap)) return arg_error(std::string(who) + ": cap must be 0 or in 1e-3..1e4");
  if (!(a->box_L >= 0) || !std::isfinite(a->box_L))
    return arg_error(std::string(who) + ": box_L must be finite and >= 0 (0: open boundary)");
  if (a->n > 0 && (a->pos != nullptr) != (a->slope != nullptr))  // no atoms: pos may be null
    return arg_error(std::string(who) + ": give both pos and slope, or neither");
  A = AttnArgs{};
  A.n = a->n, A.n_struct = a->n_struct;
  A.sptr = a->struct_ptr, A.pos = a->pos, A.slope = a->slope, A.mask = a->mask;
  A.q = a->q, A.k = a->k, A.v = a->v;
  A.ldq = a->ldq, A.ldk = a->ldk, A.ldv = a->ldv;
  A.to_fix = a->box_L > 0 ? 4294967296.0 / (double)a->box_L : 0.0;
  A.unit = a->box_L > 0 ? (float)((double)a->box_L / 4294967296.0) : 1.0f;
  A.scale = (float)(1.0 / std::sqrt((double)(a->channels / a->heads)));
  A.cap = a->cap;
  A.splits = 1;
  if (a->n == 0 || a->n_struct == 0) return MP_OK;
  const int size = std::max(1, a->n / a->n_struct), lsub = 31 - __builtin_clz(size);
  A.lsub = (float)lsub, A.p_scale = std::ldexp(1.0f, -lsub);
  if (!a->struct_ptr) return arg_error(std::string(who) + ": null struct_ptr");
  if (!a->q || !a->k || !a->v) return arg_error(std::string(who) + ": null q, k or v");
  const int C = a->channels, es = a->feat_dtype == 1 ? 2 : 4;
  if (a->ldq > kMaxLd || a->ldk > kMaxLd || a->ldv > kMaxLd) return arg_error(std::string(who) + ": row stride above 2^24");
  if (!rows_ok(a->q, a->ldq, C, es) || !rows_ok(a->k, a->ldk, C, es) || !rows_ok(a->v, a->ldv, C, es))
    return arg_error(std::string(who) +
                     ": rows of q, k and v must be 16-byte aligned, with a row stride of at least their width and a "
                     "multiple of 16 bytes");
  return MP_OK;
}

int launch(const mp_attention_args* a, const AttnArgs& A, int what, hipStream_t st) {
  const bool split = long_ones(a->n, a->n_struct);
  const int dh = a->channels / a->heads;
  return a->feat_dtype == 1 ? launch_attn_bf16(A, a->channels, dh, split, what, st)
                            : launch_attn_f32(A, a->channels, dh, split, what, st);
}

// workspace of the backward passes
struct BwdWs {
  int splits;
  int64_t blocks;  // of the row pass: partials of dslope
  float *dsum, *slope, *dq, *dk, *dv, *row, *col;
};
void carve_bwd(Arena& ar, int64_t n, int64_t n_struct, int C, int H, BwdWs& w) {
  w.splits = n > 0 && n_struct > 0 ? splits_of(n, n_struct) : 1;
  w.blocks = n_struct > 0 ? w.splits * slots_of(n, n_struct) : 0;
  w.dsum = ar.take<float>(n * H);
  w.slope = ar.take<float>(w.blocks * H);
  w.dq = w.dk = w.dv = w.row = w.col = nullptr;
  if (w.splits == 1) return;
  w.dq = ar.take<float>(w.splits * n * C), w.dk = ar.take<float>(w.splits * n * C);
  w.dv = ar.take<float>(w.splits * n * C);
  w.row = ar.take<float>(w.splits * n * 3), w.col = ar.take<float>(w.splits * n * 3);
}

// saved: [n][C] unrounded output (bf16 features only), then [n][H] base-2 log-sums
int64_t saved_o32(int64_t n, int C, int dt) { return dt == 1 ? n * C : 0; }

}  // namespace
}  // namespace ops
}  // namespace mdmp

using namespace mdmp;

extern "C" int mp_structure_attention_saved(int32_t n, int32_t channels, int32_t heads, int32_t dt, int64_t* floats) {
  MP_TRY(ops::check_shape("mp_structure_attention_saved", n, channels, heads, dt));
  if (!floats) return arg_error("mp_structure_attention_saved: null floats");
  *floats = ops::saved_o32(n, channels, dt) + (int64_t)n * heads;
  return MP_OK;
}

extern "C" int mp_structure_attention_ws(int32_t n, int32_t n_struct, int32_t channels, int32_t heads, size_t* bytes) {
  MP_TRY(ops::check_shape("mp_structure_attention_ws", n, channels, heads, 0));
  if (n_struct < 0 || n_struct > ops::kMaxStruct || !bytes)
    return arg_error("mp_structure_attention_ws: bad arguments");
  const int64_t S = n > 0 && n_struct > 0 ? ops::splits_of(n, n_struct) : 1;
  *bytes = S > 1 ? align_up(sizeof(float) * (size_t)(S * n * (channels + 2 * heads))) : 0;
  return MP_OK;
}

extern "C" int mp_structure_attention(const mp_attention_args* a, void* out, int64_t ldo, float* saved, void* ws,
                                      size_t ws_bytes, hipStream_t st) {
  ops::AttnArgs A;
  MP_TRY(ops::attn_args("mp_structure_attention", a, A));
  if (a->n == 0 || a->n_struct == 0) return MP_OK;
  if (!out) return arg_error("mp_structure_attention: null out");
  MP_ROWS("mp_structure_attention", "out", out, ldo, a->channels, a->feat_dtype);
  if ((uintptr_t)saved & 15) return arg_error("mp_structure_attention: saved must be 16-byte aligned");
  A.out = out, A.ldo = ldo;
  if (saved) {
    A.o32 = a->feat_dtype == 1 ? saved : nullptr;
    A.lse = saved + ops::saved_o32(a->n, a->channels, a->feat_dtype);
  }
  size_t need = 0;
  MP_TRY(mp_structure_attention_ws(a->n, a->n_struct, a->channels, a->heads, &need));
  if (need > 0) {
    if (!ws || ((uintptr_t)ws & 15)) return arg_error("mp_structure_attention: workspace null or not 16-byte aligned");
    if (ws_bytes < need) return arg_error("mp_structure_attention: workspace too small");
    A.splits = ops::splits_of(a->n, a->n_struct);
    A.p_out = (float*)ws;
    A.p_ml = A.p_out + (int64_t)A.splits * a->n * a->channels;
  }
  if (out == a->q || out == a->k || out == a->v) return arg_error("mp_structure_attention: out must not be q, k or v");
  ProfScope p("structure_attention", st);
  return ops::launch(a, A, 0, st);
}

extern "C" int mp_structure_attention_bwd_ws(int32_t n, int32_t n_struct, int32_t channels, int32_t heads,
                                             size_t* bytes) {
  MP_TRY(ops::check_shape("mp_structure_attention_bwd_ws", n, channels, heads, 0));
  if (n_struct < 0 || n_struct > ops::kMaxStruct || !bytes)
    return arg_error("mp_structure_attention_bwd_ws: bad arguments");
  Arena ar(nullptr, 0, true);
  ops::BwdWs w;
  ops::carve_bwd(ar, n, n_struct, channels, heads, w);
  *bytes = ar.off;
  return MP_OK;
}

extern "C" int mp_structure_attention_bwd(const mp_attention_args* a, const void* out, int64_t ldo, const float* saved,
                                          const void* dout, int64_t lddo, void* dq, int64_t lddq, void* dk,
                                          int64_t lddk, void* dv, int64_t lddv, float* dpos, float* dslope, void* ws,
                                          size_t ws_bytes, hipStream_t st) {
  ops::AttnArgs A;
  MP_TRY(ops::attn_args("mp_structure_attention_bwd", a, A));
  if ((dpos || dslope) && !a->slope) return arg_error("mp_structure_attention_bwd: dpos and dslope need pos and slope");
  const int C = a->channels, H = a->heads, dt = a->feat_dtype;
  if (a->n == 0 || a->n_struct == 0) {  // no pair: the sum over nothing
    const ops::Segment none{0, H, dslope, false};
    return ops::reduce_rows(nullptr, 0, H, &none, 1, st);
  }
  if (!out || !saved || !dout || !dq || !dk || !dv)
    return arg_error("mp_structure_attention_bwd: null out, saved, dout, dq, dk or dv");
  if (lddo > ops::kMaxLd) return arg_error("mp_structure_attention_bwd: row stride above 2^24");
  MP_ROWS("mp_structure_attention_bwd", "out", out, ldo, C, dt);
  MP_ROWS("mp_structure_attention_bwd", "dout", dout, lddo, C, dt);
  MP_ROWS("mp_structure_attention_bwd", "dq", dq, lddq, C, dt);
  MP_ROWS("mp_structure_attention_bwd", "dk", dk, lddk, C, dt);
  MP_ROWS("mp_structure_attention_bwd", "dv", dv, lddv, C, dt);
  if ((uintptr_t)saved & 15) return arg_error("mp_structure_attention_bwd: saved must be 16-byte aligned");
  if (!ws || ((uintptr_t)ws & 15)) return arg_error("mp_structure_attention_bwd: workspace null or not 16-byte aligned");
  Arena ar(ws, ws_bytes);
  ops::BwdWs w;
  ops::carve_bwd(ar, a->n, a->n_struct, C, H, w);
  A.dsum = w.dsum, A.splits = w.splits;
  A.p_dq = w.dq, A.p_dk = w.dk, A.p_dv = w.dv, A.p_row = w.row, A.p_col = w.col;
  if (!ar.ok()) return arg_error("mp_structure_attention_bwd: workspace too small");
  const void* const grads[3] = {dq, dk, dv};
  for (int i = 0; i < 3; ++i)  // the column pass reads what the row pass read
    for (const void* p : {a->q, a->k, a->v, dout, out, (const void*)grads[(i + 1) % 3]})
      if (grads[i] == p) return arg_error("mp_structure_attention_bwd: dq, dk and dv must not be each other or an input");
  A.o = out, A.ldo = ldo, A.dout = dout, A.lddo = lddo;
  A.dq = dq, A.lddq = lddq, A.dk = dk, A.lddk = lddk, A.dv = dv, A.lddv = lddv;
  A.o32 = const_cast<float*>(dt == 1 ? saved : nullptr);
  A.lse = const_cast<float*>(saved + ops::saved_o32(a->n, C, dt));
  A.dpos = dpos;
  A.dslope_part = dslope ? w.slope : nullptr;
  ProfScope p("structure_attention_bwd", st);
  MP_TRY(ops::launch(a, A, 1, st));
  MP_TRY(ops::launch(a, A, 2, st));
  const ops::Segment seg{0, H, dslope, false};
  return ops::reduce_rows(w.slope, w.blocks, H, &seg, 1, st);
}
