"""Refusals of the block operators (mp_linear, mp_gated_ffn, mp_norm_block,
mp_structure_attention and their backward calls) that need no GPU: every argument the C ABI
checks is checked before any device work, so these calls return MP_ERR_ARG here too."""
import ctypes

import pytest

from molecular_dynamics_amd import mdmp

L = mdmp._lib
P = 0x1000          # an aligned address; never dereferenced by a refused call
Y = 0x2000
ODD = 0x1008        # 8-byte aligned only


def refused(rc, *words):
    assert rc == mdmp.MP_ERR_ARG
    msg = L.mp_last_error().decode()
    assert all(w in msg for w in words), msg


def lin(n=8, k=64, o=64, dt=0, act=0, x=P, ldx=64, w=P, bias=None, res=None, ldr=64, y=Y, ldy=64):
    return L.mp_linear(n, k, o, dt, act, x, ldx, w, bias, res, ldr, y, ldy, None)


def test_linear_refusals():
    refused(lin(n=-1), "n must")
    refused(lin(n=2 ** 26 + 1), "n must")
    refused(lin(y=P), "y must not be x")
    refused(lin(k=48), "channels")
    refused(lin(k=16, dt=1), "16 channels")
    refused(lin(dt=2), "feat_dtype")
    for o in (0, 8, 24, 1040):
        refused(lin(o=o), "out")
    refused(lin(act=3), "activation")
    refused(lin(x=None), "null")
    refused(lin(w=None), "null")
    refused(lin(y=None), "null")
    refused(lin(w=ODD), "aligned")
    refused(lin(x=ODD), "rows of x")
    refused(lin(ldx=60), "rows of x")
    refused(lin(ldx=66), "rows of x")
    refused(lin(ldy=0), "rows of y")
    refused(lin(res=P, ldr=63), "residual")
    assert lin(n=0, x=None, w=None, y=None) == mdmp.MP_OK


def test_linear_bwd_refusals():
    n = ctypes.c_size_t(0)
    assert L.mp_linear_bwd_ws(1000, 64, 96, 0, ctypes.byref(n)) == mdmp.MP_OK and n.value > 96 * 64 * 4
    refused(L.mp_linear_bwd_ws(1000, 64, 90, 0, ctypes.byref(n)), "out")
    refused(L.mp_linear_bwd_ws(1000, 64, 96, 0, None), "null")

    def bwd(x=P, w=P, dy=P, lddy=96, dx=None, dw=P, db=None, ws=P, nb=n.value):
        return L.mp_linear_bwd(1000, 64, 96, 0, 0, x, 64, w, None, dy, lddy, dx, 64, dw, db, ws, nb, None)
    refused(bwd(nb=n.value - 1), "workspace too small")
    refused(bwd(ws=None), "workspace")
    refused(bwd(ws=ODD), "workspace")
    refused(bwd(dy=None), "null")
    refused(bwd(lddy=95), "rows of dy")
    refused(bwd(dx=ODD, dw=None), "rows of dx")


def ffn(n=8, c=64, f=64, dt=0, act=1, x=P, ldx=64, g=P, u=P, d=P, y=Y, ldy=64):
    return L.mp_gated_ffn(n, c, f, dt, act, x, ldx, g, u, d, None, 0, y, ldy, None)


def test_gated_ffn_refusals():
    refused(ffn(c=100), "channels")
    refused(ffn(c=16, dt=1), "16 channels")
    for f in (0, 16, 48, 4128):
        refused(ffn(f=f), "hidden")
    refused(ffn(act=0), "act")
    refused(ffn(x=None), "null")
    refused(ffn(y=P), "y must not be x")
    refused(ffn(d=None), "null")
    refused(ffn(u=ODD), "aligned")
    refused(ffn(ldx=62), "rows of x")
    assert ffn(n=0, x=None) == mdmp.MP_OK
    n = ctypes.c_size_t(0)
    assert L.mp_gated_ffn_bwd_ws(500, 64, 96, 1, ctypes.byref(n)) == mdmp.MP_OK and n.value >= 3 * 96 * 64 * 4

    def bwd(dg=P, du=P, dd=P, ws=P, nb=n.value):
        return L.mp_gated_ffn_bwd(500, 64, 96, 1, 1, P, 64, P, P, P, P, 64, None, 64, dg, du, dd, ws, nb, None)
    refused(bwd(du=None), "all three")
    refused(bwd(nb=n.value - 256), "workspace")
    refused(bwd(ws=None), "workspace")


def norm_args(n=8, c=64, dt=0, eps=1e-6, x=P, ldx=64, b=P, ldb=64, gate=None, ldg=64, scale=None, post=None, pre=None):
    return ctypes.byref(mdmp.mp_norm_args(n, c, dt, eps, x, ldx, b, ldb, gate, ldg, scale, post, pre))


def test_norm_block_refusals():
    def norm(y=P, u=None, **kw):
        return L.mp_norm_block(norm_args(**kw), y, 64, u, 64, None)
    refused(norm(c=8), "channels")
    refused(norm(n=-5), "n must")
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-37):
        refused(norm(eps=eps), "eps")
    refused(norm(x=None), "null")
    refused(norm(y=None), "null")
    refused(norm(u=P), "w_pre")
    refused(norm(pre=P), "w_pre")
    refused(norm(scale=0x1004), "aligned")
    refused(norm(gate=ODD), "rows of gate")
    refused(norm(ldb=63), "rows of b")
    refused(L.mp_norm_block(None, P, 64, None, 64, None), "null")
    n = ctypes.c_size_t(0)
    assert L.mp_norm_block_bwd_ws(8, 64, 0, ctypes.byref(n)) == mdmp.MP_OK

    def bwd(dy=P, du=None, dgate=None, ds=P, dpost=None, dpre=None, ws=P, nb=n.value, **kw):
        return L.mp_norm_block_bwd(norm_args(**kw), dy, 64, du, 64, P, 64, P, 64, dgate, 64, ds, dpost, dpre, ws, nb,
                                   None)
    refused(bwd(dy=None), "both null")
    refused(bwd(du=P), "du without")
    refused(bwd(dgate=P), "dgate without")
    refused(bwd(dpost=P), "dw_post without")
    refused(bwd(dpre=P), "dw_pre without")
    refused(bwd(nb=0), "workspace")
    refused(bwd(ws=ODD), "workspace")


def attn_args(n=40, ns=2, c=64, h=2, dt=0, cap=0.0, box=0.0, sp=P, pos=None, slope=None, mask=None, q=P, ldq=64, k=P,
              ldk=64, v=P, ldv=64):
    return ctypes.byref(mdmp.mp_attention_args(n, ns, c, h, dt, cap, box, sp, pos, slope, mask, q, ldq, k, ldk, v, ldv))


def test_structure_attention_refusals():
    def attn(out=P, ldo=64, saved=None, ws=None, nb=0, **kw):
        return L.mp_structure_attention(attn_args(**kw), out, ldo, saved, ws, nb, None)
    for h in (0, -1, 3, 8, 64):   # 64 channels: 16, 32 or 64 per head
        refused(attn(h=h), "channels / heads")
    refused(attn(c=128, h=1), "channels / heads")
    refused(attn(c=40), "channels")
    refused(attn(n=-1), "n must")
    refused(attn(ns=-1), "n_struct")
    for cap in (-1.0, float("nan"), float("inf"), 1e-4, 1e5):
        refused(attn(cap=cap), "cap")
    for box in (-1.0, float("nan"), float("inf")):
        refused(attn(box=box), "box_L")
    refused(attn(pos=P), "both pos and slope")
    refused(attn(slope=P), "both pos and slope")
    refused(attn(n=2 ** 26 + 1), "n must")
    refused(attn(ns=2 ** 25 + 1), "n_struct")
    refused(attn(sp=None), "struct_ptr")
    refused(attn(k=None), "null")
    refused(attn(ldv=60), "row")
    refused(attn(q=ODD), "row")
    refused(attn(out=None), "null out")
    refused(attn(ldo=63), "rows of out")
    refused(attn(saved=ODD), "saved")
    n = ctypes.c_size_t(0)   # few long structures need a workspace, many short ones none
    assert L.mp_structure_attention_ws(40, 2, 64, 2, ctypes.byref(n)) == mdmp.MP_OK and n.value == 0
    assert L.mp_structure_attention_ws(5000, 1, 64, 2, ctypes.byref(n)) == mdmp.MP_OK and n.value > 5000 * 64 * 4
    refused(attn(n=5000, ns=1), "workspace")
    refused(attn(n=5000, ns=1, ws=P, nb=n.value - 1), "workspace too small")
    refused(attn(n=5000, ns=1, ws=ODD, nb=n.value), "workspace")
    refused(attn(ldq=(1 << 24) + 64), "2^24")
    assert attn(n=0, q=None, sp=None) == mdmp.MP_OK and attn(ns=0, q=None, sp=None) == mdmp.MP_OK
    n = ctypes.c_size_t(0)
    assert L.mp_structure_attention_bwd_ws(40, 2, 64, 2, ctypes.byref(n)) == mdmp.MP_OK
    m = ctypes.c_int64(0)
    assert L.mp_structure_attention_saved(40, 64, 2, 1, ctypes.byref(m)) == mdmp.MP_OK and m.value == 40 * 66
    assert L.mp_structure_attention_saved(40, 64, 2, 0, ctypes.byref(m)) == mdmp.MP_OK and m.value == 40 * 2

    def bwd(out=P, saved=P, do=P, dq=P, dpos=None, dsl=None, ws=P, nb=n.value, **kw):
        return L.mp_structure_attention_bwd(attn_args(**kw), out, 64, saved, do, 64, dq, 64, P, 64, P, 64, dpos, dsl,
                                            ws, nb, None)
    refused(bwd(dpos=P), "need pos")
    refused(bwd(dsl=P), "need pos")
    refused(bwd(saved=None), "null")
    refused(bwd(dq=None), "null")
    refused(bwd(dq=ODD), "rows of dq")
    refused(bwd(ws=None), "workspace")
    refused(bwd(nb=n.value - 1), "workspace too small")


def test_one_hip_runtime_whatever_is_imported_first():
    """The binding imported before torch must not bring a second HIP runtime into the process (device
    calls of one of the two then find no device)."""
    import subprocess
    import sys
    code = ("from molecular_dynamics_amd import mdmp; import torch; "
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1] == "1", r.stdout + r.stderr
