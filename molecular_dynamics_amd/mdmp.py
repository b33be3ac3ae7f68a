"""ctypes binding of libmdmp (the C ABI in include/mdmp.h).

Argument marshalling only: every step of the path runs in the HIP library.
PyTorch supplies device memory and the current stream.  Importing this module
fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import numpy as np
import torch  # noqa: F401  before the library, which then shares PyTorch's HIP runtime; after it there would be two

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmdmp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libmdmp.so not found at {LIB_PATH}; run `python -m molecular_dynamics_amd.build`")

_lib = ctypes.CDLL(LIB_PATH)

ORDERS = {"hilbert": 0, "morton": 1, "input": 2}  # MP_ORDER_* of mdmp.h

NOALLOC_SCRATCH_BYTES = 64 << 20  # MP_NOALLOC_SCRATCH_BYTES of mdmp.h

MP_OK, MP_ERR_ARG, MP_ERR_BOX, MP_ERR_CAPACITY, MP_ERR_HIP, MP_ERR_NUMERIC, MP_ERR_STATE = 0, -1, -2, -3, -4, -5, -6
_NAMES = {-1: "MP_ERR_ARG", -2: "MP_ERR_BOX", -3: "MP_ERR_CAPACITY", -4: "MP_ERR_HIP", -5: "MP_ERR_NUMERIC",
          -6: "MP_ERR_STATE"}

EXPORTS = ["mp_version", "mp_last_error", "mp_model_num_weights", "mp_model_create", "mp_model_destroy",
           "mp_cg_table", "mp_build_neighbors_ws", "mp_build_neighbors", "mp_build_neighbors_ordered",
           "mp_build_neighbors_batched_ws", "mp_build_neighbors_batched", "mp_structure_energies",
           "mp_layer_forward_ws",
           "mp_layer_forward", "mp_embed", "mp_energy_forces_ws", "mp_energy_forces", "mp_energy_forces_status",
           "mp_energy_forces_noalloc", "mp_heads_create",
           "mp_heads_destroy", "mp_energy_forces_heads", "mp_md_create",
           "mp_md_set_state", "mp_md_step", "mp_md_use_graphs", "mp_md_set_langevin", "mp_md_step_nvt",
           "mp_md_get_state", "mp_md_destroy",
           "mp_linear", "mp_linear_bwd_ws", "mp_linear_bwd", "mp_gated_ffn", "mp_gated_ffn_bwd_ws",
           "mp_gated_ffn_bwd", "mp_norm_block", "mp_norm_block_bwd_ws", "mp_norm_block_bwd",
           "mp_structure_attention_saved", "mp_structure_attention_ws", "mp_structure_attention",
           "mp_structure_attention_bwd_ws",
           "mp_structure_attention_bwd", "mp_mixer_num_weights", "mp_mixer_create", "mp_mixer_destroy",
           "mp_energy_forces_mixer_ws", "mp_energy_forces_mixer",
           "mp_profile_enable",
           "mp_profile_reset", "mp_profile_read"]


class MPError(RuntimeError):
    def __init__(self, code, where):
        msg = _lib.mp_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_NAMES.get(code, code)}: {msg}")
        self.code = code


class mp_model_config(ctypes.Structure):
    _fields_ = [("n_species", ctypes.c_int32), ("channels", ctypes.c_int32), ("lmax", ctypes.c_int32),
                ("n_bessel", ctypes.c_int32), ("radial_hidden", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("layers", ctypes.c_int32), ("feat_dtype", ctypes.c_int32), ("cutoff", ctypes.c_float)]


class mp_graph(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("box_L", ctypes.c_float), ("pos", ctypes.c_void_p),
                ("species", ctypes.c_void_p), ("row_ptr", ctypes.c_void_p), ("col", ctypes.c_void_p),
                ("rev", ctypes.c_void_p), ("n_edges", ctypes.c_int64)]


class mp_norm_args(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("channels", ctypes.c_int32), ("feat_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("b", ctypes.c_void_p),
                ("ldb", ctypes.c_int64), ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p)]


class mp_attention_args(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("n_struct", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("feat_dtype", ctypes.c_int32), ("cap", ctypes.c_float),
                ("box_L", ctypes.c_float), ("struct_ptr", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("slope", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("ldq", ctypes.c_int64), ("k", ctypes.c_void_p), ("ldk", ctypes.c_int64), ("v", ctypes.c_void_p),
                ("ldv", ctypes.c_int64)]


_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_P = ctypes.POINTER
_sig = {
    "mp_version": ([], ctypes.c_int),
    "mp_last_error": ([], ctypes.c_char_p),
    "mp_model_num_weights": ([_P(mp_model_config), _P(_i64)], ctypes.c_int),
    "mp_model_create": ([_P(mp_model_config), _vp, _i64, _P(_vp)], ctypes.c_int),
    "mp_model_destroy": ([_vp], ctypes.c_int),
    "mp_cg_table": ([_i32, _vp, _i64, _P(_i64)], ctypes.c_int),
    "mp_build_neighbors_ws": ([_i32, _f32, _f32, _f32, _P(_sz)], ctypes.c_int),
    "mp_build_neighbors": ([_vp, _vp, _i32, _f32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _P(_i64), _vp,
                            _sz, _vp], ctypes.c_int),
    "mp_build_neighbors_ordered": ([_vp, _vp, _i32, _f32, _f32, _f32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                    _P(_i64), _vp, _sz, _vp], ctypes.c_int),
    "mp_build_neighbors_batched_ws": ([_i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_build_neighbors_batched": ([_vp, _i32, _vp, _i32, _f32, _f32, _vp, _vp, _vp, _i64, _P(_i64), _vp, _sz, _vp],
                                   ctypes.c_int),
    "mp_structure_energies": ([_vp, _vp, _i32, _vp, _vp], ctypes.c_int),
    "mp_layer_forward_ws": ([_vp, _i32, _i64, _P(_sz)], ctypes.c_int),
    "mp_layer_forward": ([_vp, _i32, _P(mp_graph), _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_embed": ([_vp, _P(mp_graph), _vp, _vp], ctypes.c_int),
    "mp_energy_forces_ws": ([_vp, _i32, _i64, _P(_sz)], ctypes.c_int),
    "mp_energy_forces": ([_vp, _P(mp_graph), _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_energy_forces_status": ([_vp, _vp], ctypes.c_int),
    "mp_energy_forces_noalloc": ([_vp, _P(mp_graph), _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mp_heads_create": ([_vp, _i32, _vp, _vp, _vp, _P(_vp)], ctypes.c_int),
    "mp_heads_destroy": ([_vp], ctypes.c_int),
    "mp_energy_forces_heads": ([_vp, _vp, _P(mp_graph), _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_md_create": ([_vp, _i32, _f32, _f32, _f32, _vp, _P(_vp)], ctypes.c_int),
    "mp_md_set_state": ([_vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mp_md_step": ([_vp, _i32, _vp, _vp], ctypes.c_int),
    "mp_md_use_graphs": ([_vp, _i32], ctypes.c_int),
    "mp_md_set_langevin": ([_vp, _f32, _f32], ctypes.c_int),
    "mp_md_step_nvt": ([_vp, _i32, _vp, _vp, _vp], ctypes.c_int),
    "mp_md_get_state": ([_vp, _vp, _vp, _P(_i64), _P(_i32), _P(_i32), _P(_f32), _vp], ctypes.c_int),
    "mp_md_destroy": ([_vp], ctypes.c_int),
    "mp_linear": ([_i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mp_linear_bwd_ws": ([_i32, _i32, _i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_linear_bwd": ([_i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _sz,
                       _vp], ctypes.c_int),
    "mp_gated_ffn": ([_i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp],
                     ctypes.c_int),
    "mp_gated_ffn_bwd_ws": ([_i32, _i32, _i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_gated_ffn_bwd": ([_i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp,
                          _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_norm_block": ([_P(mp_norm_args), _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mp_norm_block_bwd_ws": ([_i32, _i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_norm_block_bwd": ([_P(mp_norm_args), _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                           _vp, _sz, _vp], ctypes.c_int),
    "mp_structure_attention_saved": ([_i32, _i32, _i32, _i32, _P(_i64)], ctypes.c_int),
    "mp_structure_attention_ws": ([_i32, _i32, _i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_structure_attention": ([_P(mp_attention_args), _vp, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_structure_attention_bwd_ws": ([_i32, _i32, _i32, _i32, _P(_sz)], ctypes.c_int),
    "mp_structure_attention_bwd": ([_P(mp_attention_args), _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                                    _i64, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_mixer_num_weights": ([_vp, _i32, _i32, _i32, _P(_i64)], ctypes.c_int),
    "mp_mixer_create": ([_vp, _i32, _i32, _i32, _f32, _vp, _i64, _P(_vp)], ctypes.c_int),
    "mp_mixer_destroy": ([_vp], ctypes.c_int),
    "mp_energy_forces_mixer_ws": ([_vp, _vp, _i32, _i32, _i64, _P(_sz)], ctypes.c_int),
    "mp_energy_forces_mixer": ([_vp, _vp, _P(mp_graph), _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mp_profile_enable": ([ctypes.c_int], ctypes.c_int),
    "mp_profile_reset": ([], ctypes.c_int),
    "mp_profile_read": ([ctypes.c_char_p, _P(ctypes.c_double), _P(_i64)], ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def _check(rc, where):
    if rc != MP_OK:
        raise MPError(rc, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ws(nbytes):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")


def cg_table(lmax):
    """Host-only: the library's real CG rows (l1, l2, l3, m1+l1, m2+l2, m3+l3, value)."""
    n = ctypes.c_int64(0)
    _check(_lib.mp_cg_table(lmax, None, 0, ctypes.byref(n)), "mp_cg_table")
    out = np.zeros((n.value, 7), np.float64)
    _check(_lib.mp_cg_table(lmax, out.ctypes.data, n.value, ctypes.byref(n)), "mp_cg_table")
    return out


def config_struct(cfg):
    return mp_model_config(cfg.n_species, cfg.channels, cfg.lmax, cfg.n_bessel, cfg.radial_hidden, cfg.heads,
                           cfg.layers, 1 if cfg.feat_bf16 else 0, cfg.cutoff)


def num_weights(cfg):
    n = ctypes.c_int64(0)
    c = config_struct(cfg)
    _check(_lib.mp_model_num_weights(ctypes.byref(c), ctypes.byref(n)), "mp_model_num_weights")
    return n.value


class Model:
    def __init__(self, cfg, weights):
        self.cfg = cfg
        w = np.ascontiguousarray(weights, np.float32)
        self._c = config_struct(cfg)
        h = ctypes.c_void_p(0)
        _check(_lib.mp_model_create(ctypes.byref(self._c), w.ctypes.data, w.size, ctypes.byref(h)),
               "mp_model_create")
        self.h = h

    @property
    def K(self):
        return (self.cfg.lmax + 1) ** 2

    def close(self):
        if self.h:
            _lib.mp_model_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Graph:
    """Sorted-slot neighbour graph on the device (owns its tensors)."""

    def __init__(self, n, L, pos, species, row_ptr, col, rev, n_edges, perm=None):
        self.n, self.L = n, float(L)
        self.pos, self.species, self.row_ptr, self.col, self.rev = pos, species, row_ptr, col, rev
        self.n_edges, self.perm = int(n_edges), perm

    def struct(self):
        return mp_graph(self.n, self.L, _ptr(self.pos), _ptr(self.species), _ptr(self.row_ptr), _ptr(self.col),
                        _ptr(self.rev), self.n_edges)


def estimate_capacity(n, L, cutoff, skin, slack=1.25):
    R = float(cutoff) + float(skin)
    rho = n / float(L) ** 3
    return int(math.ceil(slack * n * rho * 4.0 / 3.0 * math.pi * R ** 3)) + 4096


def build_neighbors(pos, species, L, cutoff, skin, capacity=None, order="hilbert"):
    """pos: cuda float32 [n,3]; species: cuda int32 [n].  Returns Graph (with perm).
    order: "hilbert" (default), "morton" or "input" (ORDERS)."""
    import torch
    n = pos.shape[0]
    dev = pos.device
    nbytes = ctypes.c_size_t(0)
    _check(_lib.mp_build_neighbors_ws(n, L, cutoff, skin, ctypes.byref(nbytes)), "mp_build_neighbors_ws")
    ws = _ws(nbytes.value)
    perm = torch.empty(n, dtype=torch.int32, device=dev)
    pos_s = torch.empty(n, 3, dtype=torch.float32, device=dev)
    sp_s = torch.empty(n, dtype=torch.int32, device=dev)
    row_ptr = torch.empty(n + 1, dtype=torch.int32, device=dev)
    cap = capacity if capacity is not None else estimate_capacity(n, L, cutoff, skin)
    for _ in range(2):
        col = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
        rev = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
        ne = ctypes.c_int64(0)
        rc = _lib.mp_build_neighbors_ordered(_ptr(pos), _ptr(species), n, L, cutoff, skin, ORDERS[order], _ptr(perm),
                                             _ptr(pos_s), _ptr(sp_s), _ptr(row_ptr), _ptr(col), _ptr(rev), cap,
                                             ctypes.byref(ne), _ptr(ws), ws.numel(), _stream())
        if rc == MP_ERR_CAPACITY and capacity is None:
            cap = ne.value
            continue
        _check(rc, "mp_build_neighbors")
        return Graph(n, L, pos_s, sp_s, row_ptr, col, rev, ne.value, perm)
    raise MPError(MP_ERR_CAPACITY, "mp_build_neighbors")


def build_neighbors_batched(pos, species, struct_ptr, cutoff, skin=0.0, capacity=None):
    """Open-boundary graph of many small structures concatenated in input order.
    pos: cuda float32 [n,3]; species: cuda int32 [n]; struct_ptr: cuda int32 [B+1].
    Returns Graph with L = 0 (open boundary) and perm = None."""
    import torch
    n, nst = pos.shape[0], struct_ptr.shape[0] - 1
    nbytes = ctypes.c_size_t(0)
    _check(_lib.mp_build_neighbors_batched_ws(n, nst, ctypes.byref(nbytes)), "mp_build_neighbors_batched_ws")
    ws = _ws(nbytes.value)
    row_ptr = torch.empty(n + 1, dtype=torch.int32, device=pos.device)
    cap = capacity if capacity is not None else 64 * n
    for _ in range(2):
        col = torch.empty(max(cap, 1), dtype=torch.int32, device=pos.device)
        rev = torch.empty(max(cap, 1), dtype=torch.int32, device=pos.device)
        ne = ctypes.c_int64(0)
        rc = _lib.mp_build_neighbors_batched(_ptr(pos), n, _ptr(struct_ptr), nst, cutoff, skin, _ptr(row_ptr),
                                             _ptr(col), _ptr(rev), cap, ctypes.byref(ne), _ptr(ws), ws.numel(),
                                             _stream())
        if rc == MP_ERR_CAPACITY and capacity is None:
            cap = ne.value
            continue
        _check(rc, "mp_build_neighbors_batched")
        return Graph(n, 0.0, pos, species, row_ptr, col, rev, ne.value, None)
    raise MPError(MP_ERR_CAPACITY, "mp_build_neighbors_batched")


def structure_energies(atom_energy, struct_ptr, out=None):
    """float64 [B] per-structure sums of the float32 atom energies (device)."""
    import torch
    nst = struct_ptr.shape[0] - 1
    out = torch.empty(nst, dtype=torch.float64, device=atom_energy.device) if out is None else out
    _check(_lib.mp_structure_energies(_ptr(atom_energy), _ptr(struct_ptr), nst, _ptr(out), _stream()),
           "mp_structure_energies")
    return out


def feat_dtype(model):
    import torch
    return torch.int16 if model.cfg.feat_bf16 else torch.float32


def embed(model, g):
    import torch
    h = torch.empty(g.n, model.K, model.cfg.channels, dtype=feat_dtype(model), device="cuda")
    gs = g.struct()
    _check(_lib.mp_embed(model.h, ctypes.byref(gs), _ptr(h), _stream()), "mp_embed")
    return h


def layer_forward(model, layer, g, h_in):
    import torch
    nbytes = ctypes.c_size_t(0)
    _check(_lib.mp_layer_forward_ws(model.h, g.n, max(g.n_edges, 1), ctypes.byref(nbytes)), "mp_layer_forward_ws")
    ws = _ws(nbytes.value)
    h_out = torch.empty_like(h_in)
    gs = g.struct()
    _check(_lib.mp_layer_forward(model.h, layer, ctypes.byref(gs), _ptr(h_in), _ptr(h_out), _ptr(ws), ws.numel(),
                                 _stream()), "mp_layer_forward")
    return h_out


class EnergyForces:
    """Reusable workspace for repeated mp_energy_forces calls on one graph size."""

    def __init__(self, model, n, capacity):
        import torch
        self.model = model
        nbytes = ctypes.c_size_t(0)
        _check(_lib.mp_energy_forces_ws(model.h, n, max(int(capacity), 1), ctypes.byref(nbytes)),
               "mp_energy_forces_ws")
        self.nbytes = nbytes.value
        self.ws = _ws(nbytes.value)
        self.energy = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.n, self.capacity = n, capacity

    def __call__(self, g, perm=None, forces=None, atom_energy=None, stream=None, check=True):
        """Enqueue mp_energy_forces; check: then wait for it and raise MPError (MP_ERR_NUMERIC)
        if the energy or a force is non-finite (mp_energy_forces_status)."""
        import torch
        if g.n != self.n or g.n_edges > self.capacity:
            raise ValueError("graph does not fit this workspace")
        if forces is None:
            forces = torch.empty(g.n, 3, dtype=torch.float32, device="cuda")
        gs = g.struct()
        st = ctypes.c_void_p(stream) if stream is not None else _stream()
        _check(_lib.mp_energy_forces(self.model.h, ctypes.byref(gs), _ptr(perm), _ptr(self.energy), _ptr(forces),
                                     _ptr(atom_energy), _ptr(self.ws), self.ws.numel(), st), "mp_energy_forces")
        if check:
            self.status(st)
        return self.energy, forces

    def status(self, stream=None):
        st = ctypes.c_void_p(stream) if isinstance(stream, int) else (stream or _stream())
        _check(_lib.mp_energy_forces_status(_ptr(self.ws), st), "mp_energy_forces_status")


def energy_forces_noalloc(model, g, energy, forces, perm=None, atom_energy=None, nonfinite=None):
    """mp_energy_forces_noalloc into caller tensors (energy float64 [1], forces float32 [n][3],
    atom_energy float32 [n] or None, nonfinite int32 [1] or None); enqueues only."""
    gs = g.struct()
    _check(_lib.mp_energy_forces_noalloc(model.h, ctypes.byref(gs), _ptr(perm), _ptr(energy), _ptr(forces),
                                         _ptr(atom_energy), _ptr(nonfinite), _stream()), "mp_energy_forces_noalloc")


def energy_forces(model, g, perm=None, atom_energy=None):
    ef = EnergyForces(model, g.n, max(g.n_edges, 1))
    E, F = ef(g, perm=perm, atom_energy=atom_energy)
    return float(E.item()), F


class Heads:
    """R readout heads on one model's encoder (mp_heads_create): wr [R][C][C] (out, in),
    wout [R][C], lam [R], host arrays."""

    def __init__(self, model, wr, wout, lam):
        wr = np.ascontiguousarray(wr, np.float32)
        wout = np.ascontiguousarray(wout, np.float32)
        lam = np.ascontiguousarray(lam, np.float32)
        R, C = lam.size, model.cfg.channels
        if wr.shape != (R, C, C) or wout.shape != (R, C):
            raise ValueError(f"heads: want wr [{R}][{C}][{C}] and wout [{R}][{C}]")
        h = ctypes.c_void_p(0)
        _check(_lib.mp_heads_create(model.h, R, wr.ctypes.data, wout.ctypes.data, lam.ctypes.data, ctypes.byref(h)),
               "mp_heads_create")
        self.h, self.R, self.model = h, R, model

    def close(self):
        if self.h:
            _lib.mp_heads_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def energy_forces_heads(model, heads, g, perm=None, ws=None):
    """mp_energy_forces_heads: returns (head energies float64 [R] (device), E = sum_k lam_k E_k
    (float), forces [n][3], per-head atom energies [R][n] (device, slot order))."""
    import torch
    if ws is None:
        nbytes = ctypes.c_size_t(0)
        _check(_lib.mp_energy_forces_ws(model.h, g.n, max(g.n_edges, 1), ctypes.byref(nbytes)),
               "mp_energy_forces_ws")
        ws = _ws(nbytes.value)
    e_heads = torch.zeros(heads.R, dtype=torch.float64, device="cuda")
    energy = torch.zeros(1, dtype=torch.float64, device="cuda")
    forces = torch.empty(g.n, 3, dtype=torch.float32, device="cuda")
    e_atoms = torch.empty(heads.R, g.n, dtype=torch.float32, device="cuda")
    gs = g.struct()
    _check(_lib.mp_energy_forces_heads(model.h, heads.h, ctypes.byref(gs), _ptr(perm), _ptr(e_heads), _ptr(energy),
                                       _ptr(forces), _ptr(e_atoms), _ptr(ws), ws.numel(), _stream()),
           "mp_energy_forces_heads")
    _check(_lib.mp_energy_forces_status(_ptr(ws), _stream()), "mp_energy_forces_status")
    return e_heads, float(energy.item()), forces, e_atoms


# ---------------------------------------------------------------- block operators
# Rows are 2-d cuda tensors of float32 or bfloat16 (torch.bfloat16, or its bits as int16, as in
# feat_dtype), unit stride in the second dimension and any row stride of a multiple of 16 bytes:
# h[:, 0] of a feature tensor [n, K, C] is such a matrix.  Outputs are of the rows' dtype unless
# said otherwise, allocated here when not given.  All calls enqueue on the current stream of the
# current device, where every tensor has to be.

ACTS = {"none": 0, "silu": 1, "sigmoid": 2}  # MP_ACT_* of mdmp.h


def _need(ok, where, what):
    if not ok:
        raise ValueError(f"{where}: {what}")


def _raw_stream(dev):
    import torch
    return torch.cuda.current_stream(dev).cuda_stream


class _Rows:
    """Checks of one call: its rows' number, dtype and device, taken from the first matrix."""

    def __init__(self, where, x):
        import torch
        _need(isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda, where, "rows must be 2-d cuda tensors")
        self.dt = x.dtype
        self.bf16 = 0 if x.dtype == torch.float32 else 1
        _need(self.dt in (torch.float32, torch.bfloat16, torch.int16), where, "rows must be float32 or bfloat16")
        self.dev = torch.cuda.current_device()
        self.where, self.n, self.c, self.f32 = where, x.shape[0], x.shape[1], torch.float32

    def rows(self, name, t, width=None):
        """(pointer, row stride) of an [n][width] matrix of rows; (None, 0) for None"""
        if t is None:
            return None, 0
        w = self.c if width is None else width
        if t.get_device() == self.dev and t.dtype == self.dt and t.dim() == 2 and t.shape[0] == self.n and t.shape[1] == w:
            s0, s1 = t.stride()
            if s1 == 1:
                return t.data_ptr(), s0 if self.n > 1 else w
        _need(t.get_device() == self.dev, self.where, f"{name} must be on the current device")
        _need(t.dtype == self.dt, self.where, f"{name} must have the dtype of the other rows")
        _need(tuple(t.shape) == (self.n, w), self.where, f"{name} must have {self.n} rows of {w}")
        raise ValueError(f"{self.where}: {name} must have unit stride along a row")

    def vec(self, name, t, shape, dtype=None):
        """pointer of a contiguous float32 (or given dtype) array, None for None"""
        if t is None:
            return None
        if (t.get_device() == self.dev and t.dtype == (dtype or self.f32) and t.shape == shape and t.is_contiguous()):
            return t.data_ptr()
        _need(t.get_device() == self.dev and t.is_contiguous(), self.where,
              f"{name} must be a contiguous tensor on the current device")
        _need(t.dtype == (dtype or self.f32), self.where, f"{name} must be {dtype or self.f32}")
        raise ValueError(f"{self.where}: {name} must have shape {tuple(shape)}")

    def new(self, width=None, dtype=None):
        import torch
        return torch.empty(self.n, self.c if width is None else width, dtype=dtype or self.dt, device=self.dev)

    def vec_new(self, size):
        import torch
        return torch.empty(size, dtype=self.f32, device=self.dev)

    def ws(self, nbytes):
        import torch
        return torch.empty(nbytes, dtype=torch.uint8, device=self.dev)


@functools.lru_cache(maxsize=512)
def _size_of(fn, ctype, *args):
    """what a size query of the library answers for a shape"""
    n = ctype(0)
    _check(getattr(_lib, fn)(*args, ctypes.byref(n)), fn)
    return n.value


def _act_id(where, act):
    _need(act in ACTS, where, f"unknown activation {act!r}")
    return ACTS[act]


def linear(x, weight, bias=None, act="none", residual=None, out=None):
    """residual + act(x weight^T + bias): x [n][in], weight [out][in], bias float32 [out] -> [n][out].
    out may be residual."""
    r = _Rows("linear", x)
    o = weight.shape[0]
    out = r.new(o) if out is None else out
    _check(_lib.mp_linear(r.n, r.c, o, r.bf16, _act_id("linear", act), *r.rows("x", x),
                          r.vec("weight", weight, (o, r.c), r.dt), r.vec("bias", bias, (o,)),
                          *r.rows("residual", residual, o), *r.rows("out", out, o), _raw_stream(r.dev)), "mp_linear")
    return out


def linear_bwd(x, weight, dy, bias=None, act="none", weight_grads=True):
    """(dx, dweight, dbias) of linear for dy [n][out]; the residual's gradient is dy.  dbias is
    float32, None without a bias; without weight_grads (forces only) dweight and dbias are None."""
    import torch
    r = _Rows("linear_bwd", x)
    o = weight.shape[0]
    dx = r.new()
    dw = db = ws = None
    nws = 0
    if weight_grads:
        dw = torch.empty_like(weight)
        db = r.vec_new(o) if bias is not None else None
        nws = _size_of("mp_linear_bwd_ws", ctypes.c_size_t, r.n, r.c, o, r.bf16)
        ws = r.ws(nws)
    _check(_lib.mp_linear_bwd(r.n, r.c, o, r.bf16, _act_id("linear_bwd", act), *r.rows("x", x),
                              r.vec("weight", weight, (o, r.c), r.dt), r.vec("bias", bias, (o,)),
                              *r.rows("dy", dy, o), dx.data_ptr(), r.c, _ptr(dw), _ptr(db), _ptr(ws), nws,
                              _raw_stream(r.dev)), "mp_linear_bwd")
    return dx, dw, db


def gated_ffn(x, w_gate, w_up, w_down, act="silu", residual=None, out=None):
    """residual + (act(x w_gate^T) * (x w_up^T)) w_down^T: x [n][C], w_gate and w_up [hidden][C],
    w_down [C][hidden] -> [n][C].  out may be residual."""
    r = _Rows("gated_ffn", x)
    f = w_gate.shape[0]
    out = r.new() if out is None else out
    _check(_lib.mp_gated_ffn(r.n, r.c, f, r.bf16, _act_id("gated_ffn", act), *r.rows("x", x),
                             r.vec("w_gate", w_gate, (f, r.c), r.dt), r.vec("w_up", w_up, (f, r.c), r.dt),
                             r.vec("w_down", w_down, (r.c, f), r.dt), *r.rows("residual", residual),
                             *r.rows("out", out), _raw_stream(r.dev)), "mp_gated_ffn")
    return out


def gated_ffn_bwd(x, w_gate, w_up, w_down, dy, act="silu", weight_grads=True):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn for dy [n][C]; the residual's gradient is dy.
    Without weight_grads (forces only) the last three are None."""
    import torch
    r = _Rows("gated_ffn_bwd", x)
    f = w_gate.shape[0]
    dx = r.new()
    g, ws, nws = [None] * 3, None, 0
    if weight_grads:
        g = [torch.empty_like(t) for t in (w_gate, w_up, w_down)]
        nws = _size_of("mp_gated_ffn_bwd_ws", ctypes.c_size_t, r.n, r.c, f, r.bf16)
        ws = r.ws(nws)
    _check(_lib.mp_gated_ffn_bwd(r.n, r.c, f, r.bf16, _act_id("gated_ffn_bwd", act), *r.rows("x", x),
                                 r.vec("w_gate", w_gate, (f, r.c), r.dt), r.vec("w_up", w_up, (f, r.c), r.dt),
                                 r.vec("w_down", w_down, (r.c, f), r.dt), *r.rows("dy", dy), dx.data_ptr(), r.c,
                                 *[_ptr(t) for t in g], _ptr(ws), nws, _raw_stream(r.dev)), "mp_gated_ffn_bwd")
    return (dx, *g)


def _norm_args(r, x, b, scale, gate, w_post, w_pre, eps):
    c = (r.c,)
    return mp_norm_args(r.n, r.c, r.bf16, eps, *r.rows("x", x), *r.rows("b", b), *r.rows("gate", gate),
                        r.vec("scale", scale, c), r.vec("w_post", w_post, c), r.vec("w_pre", w_pre, c))


def norm_block(x, b, scale=None, gate=None, w_post=None, w_pre=None, eps=1e-6, out=None):
    """(y, u): y = x + scale * sigmoid(gate) * (w_post * b / rms(b)) and u = w_pre * y / rms(y), the
    norm after a block with its gate and residual scale and the norm before the next block.
    scale, w_post, w_pre float32 [C] or None (no factor; no norm of b; u = None); gate rows or None.
    out (for y) may be x or b."""
    r = _Rows("norm_block", x)
    a = _norm_args(r, x, b, scale, gate, w_post, w_pre, eps)
    y = r.new() if out is None else out
    u = r.new() if w_pre is not None else None
    _check(_lib.mp_norm_block(ctypes.byref(a), *r.rows("out", y), _ptr(u), r.c, _raw_stream(r.dev)), "mp_norm_block")
    return y, u


def norm_block_bwd(x, b, dy, du=None, scale=None, gate=None, w_post=None, w_pre=None, eps=1e-6, param_grads=True):
    """Gradients of norm_block for dy and du (either may be None: zero) as a dict: dx, db, dgate
    (rows) and dscale, dw_post, dw_pre (float32); None for what was not given."""
    r = _Rows("norm_block_bwd", x)
    a = _norm_args(r, x, b, scale, gate, w_post, w_pre, eps)
    g = {"dx": r.new(), "db": r.new(), "dgate": r.new() if gate is not None else None}
    ws, nws = None, 0
    for k, p in (("dscale", scale), ("dw_post", w_post), ("dw_pre", w_pre)):
        g[k] = r.vec_new(r.c) if p is not None and param_grads else None
        if g[k] is not None and ws is None:
            nws = _size_of("mp_norm_block_bwd_ws", ctypes.c_size_t, r.n, r.c, r.bf16)
            ws = r.ws(nws)
    _check(_lib.mp_norm_block_bwd(ctypes.byref(a), *r.rows("dy", dy), *r.rows("du", du), _ptr(g["dx"]), r.c,
                                  _ptr(g["db"]), r.c, _ptr(g["dgate"]), r.c, _ptr(g["dscale"]), _ptr(g["dw_post"]),
                                  _ptr(g["dw_pre"]), _ptr(ws), nws, _raw_stream(r.dev)), "mp_norm_block_bwd")
    return g


def _attention_args(r, q, k, v, struct_ptr, heads, pos, slope, L, mask, cap):
    import torch
    nst = struct_ptr.numel() - 1
    _need(nst >= 0, r.where, "struct_ptr must hold n_struct + 1 entries")
    if mask is not None and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    return mp_attention_args(r.n, nst, r.c, heads, r.bf16, cap, L, r.vec("struct_ptr", struct_ptr, (nst + 1,), torch.int32),
                             r.vec("pos", pos, (r.n, 3)), r.vec("slope", slope, (heads,)),
                             r.vec("mask", mask, (r.n,), torch.uint8), *r.rows("q", q), *r.rows("k", k),
                             *r.rows("v", v))


def structure_attention(q, k, v, struct_ptr, heads, pos=None, slope=None, L=0.0, mask=None, cap=0.0, out=None,
                        save=False):
    """Softmax attention between all atoms of each structure (rows struct_ptr[b] .. struct_ptr[b+1]-1 of
    q, k, v [n][C]; int32, device): scores q.k / sqrt(C / heads), capped by cap tanh(./cap) if cap > 0,
    minus slope[head] times the distance of the pair (pos float32 [n][3], slope float32 [heads]; minimum
    image if L > 0), over the atoms with mask != 0 (bool or uint8 [n]).  Rows past the last structure are
    not written (an out allocated here holds anything there).  save: returns (out, saved), saved for
    structure_attention_bwd."""
    r = _Rows("structure_attention", q)
    a = _attention_args(r, q, k, v, struct_ptr, heads, pos, slope, L, mask, cap)
    out = r.new() if out is None else out
    saved = r.vec_new(_size_of("mp_structure_attention_saved", ctypes.c_int64, r.n, r.c, heads, r.bf16)) if save else None
    nws = _size_of("mp_structure_attention_ws", ctypes.c_size_t, r.n, a.n_struct, r.c, heads)
    ws = r.ws(nws) if nws else None
    _check(_lib.mp_structure_attention(ctypes.byref(a), *r.rows("out", out), _ptr(saved), _ptr(ws), nws,
                                       _raw_stream(r.dev)), "mp_structure_attention")
    return (out, saved) if save else out


def structure_attention_bwd(q, k, v, struct_ptr, heads, out, saved, dout, pos=None, slope=None, L=0.0, mask=None,
                            cap=0.0, dq=None, dk=None, dv=None, dpos=None):
    """Gradients of structure_attention for dout as a dict: dq, dk, dv (rows), dpos float32 [n][3] and
    dslope float32 [heads] (None without pos).  out, saved: what the forward call returned.  dq, dk, dv
    and dpos may be given to be written into (column slices of one matrix, say).  Rows past the last
    structure are not written (tensors allocated here hold anything there)."""
    r = _Rows("structure_attention_bwd", q)
    a = _attention_args(r, q, k, v, struct_ptr, heads, pos, slope, L, mask, cap)
    _need(dpos is None or pos is not None, r.where, "dpos without pos")
    m = _size_of("mp_structure_attention_saved", ctypes.c_int64, r.n, r.c, heads, r.bf16)
    g = {"dq": r.new() if dq is None else dq, "dk": r.new() if dk is None else dk, "dv": r.new() if dv is None else dv,
         "dpos": r.new(3, r.f32) if pos is not None and dpos is None else dpos,
         "dslope": r.vec_new(heads) if pos is not None else None}
    nws = _size_of("mp_structure_attention_bwd_ws", ctypes.c_size_t, r.n, a.n_struct, r.c, heads)
    ws = r.ws(nws)
    _check(_lib.mp_structure_attention_bwd(ctypes.byref(a), *r.rows("out", out), r.vec("saved", saved, (m,)),
                                           *r.rows("dout", dout), *r.rows("dq", g["dq"]), *r.rows("dk", g["dk"]),
                                           *r.rows("dv", g["dv"]), r.vec("dpos", g["dpos"], (r.n, 3)),
                                           _ptr(g["dslope"]), _ptr(ws), nws, _raw_stream(r.dev)),
           "mp_structure_attention_bwd")
    return g


class Mixer:
    """Global blocks (structure attention and a gated feed-forward) between a model's last layer and
    its readout (mp_mixer_create); weights: host float32 blob in the order of mdmp.h."""

    def __init__(self, model, n_blocks, heads, hidden, weights, cap=0.0):
        w = np.ascontiguousarray(weights, np.float32)
        h = ctypes.c_void_p(0)
        _check(_lib.mp_mixer_create(model.h, n_blocks, heads, hidden, cap, w.ctypes.data, w.size, ctypes.byref(h)),
               "mp_mixer_create")
        self.h, self.model, self.n_blocks = h, model, n_blocks

    @staticmethod
    def num_weights(model, n_blocks, heads, hidden):
        n = ctypes.c_int64(0)
        _check(_lib.mp_mixer_num_weights(model.h, n_blocks, heads, hidden, ctypes.byref(n)), "mp_mixer_num_weights")
        return n.value

    def close(self):
        if self.h:
            _lib.mp_mixer_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def energy_forces_mixer(model, mixer, g, struct_ptr=None, perm=None, atom_energy=None, ws=None):
    """mp_energy_forces_mixer: (energy (float), forces [n][3]).  struct_ptr: cuda int32 [B + 1], the
    structures of the graph (None: the whole graph is one)."""
    import torch
    if struct_ptr is None:
        struct_ptr = torch.tensor([0, g.n], dtype=torch.int32, device="cuda")
    nst = struct_ptr.numel() - 1
    if ws is None:
        nbytes = ctypes.c_size_t(0)
        _check(_lib.mp_energy_forces_mixer_ws(model.h, mixer.h, g.n, nst, max(g.n_edges, 1), ctypes.byref(nbytes)),
               "mp_energy_forces_mixer_ws")
        ws = _ws(nbytes.value)
    _need(struct_ptr.is_cuda and struct_ptr.is_contiguous() and struct_ptr.dtype == torch.int32 and struct_ptr.dim() == 1,
          "energy_forces_mixer", "struct_ptr must be a contiguous 1-d int32 cuda tensor")
    sp = struct_ptr.data_ptr()
    energy = torch.zeros(1, dtype=torch.float64, device="cuda")
    forces = torch.empty(g.n, 3, dtype=torch.float32, device="cuda")
    gs = g.struct()
    _check(_lib.mp_energy_forces_mixer(model.h, mixer.h, ctypes.byref(gs), sp, nst, _ptr(perm), _ptr(energy),
                                       _ptr(forces), _ptr(atom_energy), _ptr(ws), ws.numel(), _stream()),
           "mp_energy_forces_mixer")
    _check(_lib.mp_energy_forces_status(_ptr(ws), _stream()), "mp_energy_forces_status")
    return float(energy.item()), forces


class MD:
    """Velocity-Verlet NVE handle (mp_md_*).  masses: per species, amu."""

    def __init__(self, model, n, L, skin, dt_fs, masses):
        self.model, self.n = model, n
        m = np.ascontiguousarray(masses, np.float32)
        h = ctypes.c_void_p(0)
        _check(_lib.mp_md_create(model.h, n, L, skin, dt_fs, m.ctypes.data, ctypes.byref(h)), "mp_md_create")
        self.h = h

    def set_state(self, pos, vel, species):
        _check(_lib.mp_md_set_state(self.h, _ptr(pos), _ptr(vel), _ptr(species), _stream()), "mp_md_set_state")

    def use_graphs(self, enable=True):
        """replay captured step graphs (default) or enqueue each step's kernels"""
        _check(_lib.mp_md_use_graphs(self.h, 1 if enable else 0), "mp_md_use_graphs")

    def set_langevin(self, temperature_K, gamma_per_ps):
        """BAOAB Langevin thermostat (gamma > 0), or back to NVE (gamma = 0)"""
        _check(_lib.mp_md_set_langevin(self.h, float(temperature_K), float(gamma_per_ps)), "mp_md_set_langevin")

    def step_nvt(self, noise, e_log=True):
        """Advance len(noise) Langevin steps; noise: cuda float32 [n_steps][n][3] standard normals
        in input-atom order.  Returns numpy [n_steps][2] (kinetic, potential) or None."""
        import torch
        n_steps = noise.shape[0]
        assert noise.dtype == torch.float32 and noise.is_cuda and noise.is_contiguous()
        assert tuple(noise.shape[1:]) == (self.n, 3)
        log = torch.zeros(max(n_steps, 1), 2, dtype=torch.float64, device="cuda") if e_log else None
        _check(_lib.mp_md_step_nvt(self.h, n_steps, _ptr(noise), _ptr(log), _stream()), "mp_md_step_nvt")
        return log[:n_steps].cpu().numpy() if e_log else None

    def step(self, n_steps, e_log=True):
        """Advance n_steps; returns numpy [n_steps][2] (kinetic, potential) in eV, or None."""
        import torch
        log = torch.zeros(max(n_steps, 1), 2, dtype=torch.float64, device="cuda") if e_log else None
        _check(_lib.mp_md_step(self.h, n_steps, _ptr(log), _stream()), "mp_md_step")
        return log[:n_steps].cpu().numpy() if e_log else None

    def state(self):
        import torch
        pos = torch.empty(self.n, 3, dtype=torch.float32, device="cuda")
        vel = torch.empty(self.n, 3, dtype=torch.float32, device="cuda")
        step, nreb, ncap, dmin = ctypes.c_int64(0), ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_float(0)
        _check(_lib.mp_md_get_state(self.h, _ptr(pos), _ptr(vel), ctypes.byref(step), ctypes.byref(nreb),
                                    ctypes.byref(ncap), ctypes.byref(dmin), _stream()), "mp_md_get_state")
        return {"pos": pos.cpu().numpy(), "vel": vel.cpu().numpy(), "step": step.value, "n_rebuilds": nreb.value,
                "n_captures": ncap.value, "min_pair": dmin.value}

    def close(self):
        if self.h:
            _lib.mp_md_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def profile_enable(on=True):
    _check(_lib.mp_profile_enable(1 if on else 0), "mp_profile_enable")


def profile_reset():
    _check(_lib.mp_profile_reset(), "mp_profile_reset")


def profile_read(name):
    """(total_ms, launches) for kernel `name` since the last reset."""
    ms, n = ctypes.c_double(0), ctypes.c_int64(0)
    _check(_lib.mp_profile_read(name.encode(), ctypes.byref(ms), ctypes.byref(n)), "mp_profile_read")
    return ms.value, n.value


def bf16_to_f32(t):
    """int16 bit patterns of bfloat16 -> float32 tensor."""
    import torch
    return (t.to(torch.int32) << 16).view(torch.float32)
