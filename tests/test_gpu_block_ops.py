"""Block operators (mp_linear, mp_gated_ffn, mp_norm_block, mp_structure_attention and their
backward calls) against float64 definitions on the CPU (tests/block_ops_ref.py, whose bounds
are derived there from the kernels' arithmetic)."""
import math

import pytest
import torch

from tests import block_ops_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def strided(g, n, c, pad, dtype):
    """rows of a wider matrix: row stride c + pad"""
    return randn(g, max(n, 1), c + pad, dtype=dtype)[:n, :c] if pad else randn(g, n, c, dtype=dtype)


def m():
    from molecular_dynamics_amd import mdmp
    return mdmp


# ------------------------------------------------------------------------------ linear
LINEAR = [
    # n, in, out, dtype, act, bias, residual, pad
    (1, 128, 384, "bf16", "none", True, False, 0),
    (17, 32, 16, "bf16", "silu", True, True, 8),
    (300, 64, 48, "bf16", "sigmoid", False, True, 64),
    (1025, 128, 1024, "bf16", "silu", True, False, 0),
    (1, 16, 16, "f32", "silu", True, False, 0),
    (63, 16, 48, "f32", "none", True, True, 4),
    (129, 32, 80, "f32", "sigmoid", True, False, 0),
    (700, 64, 208, "f32", "silu", False, True, 12),
    (515, 128, 144, "f32", "none", False, False, 128),
    (70001, 128, 400, "bf16", "silu", True, True, 8),
    (66000, 64, 96, "f32", "none", True, False, 4),
    (65537, 32, 304, "f32", "sigmoid", False, False, 0),
    (65999, 32, 16, "bf16", "none", False, True, 0),
]


@pytest.mark.parametrize("n,k,o,dt,act,bias,res,pad", LINEAR)
def test_linear(n, k, o, dt, act, bias, res, pad):
    g, t = gen(n + o), DT[dt]
    print(f"linear n={n} {k}->{o} {dt} {act} bias={bias} res={res} pad={pad}", flush=True)
    x, w = strided(g, n, k, pad, t), randn(g, o, k, scale=k ** -0.5, dtype=t)
    b = randn(g, o) if bias else None
    r = strided(g, n, o, pad, t) if res else None
    dy = strided(g, n, o, pad, t)
    ref = R.linear(x, w, b, act, r, dy)
    y = m().linear(x, w, bias=b, act=act, residual=r)
    dx, dw, db = m().linear_bwd(x, w, dy, bias=b, act=act)
    torch.cuda.synchronize()
    assert y.dtype == t and dx.dtype == t and dw.dtype == t and (db is None) == (b is None)
    for name, got in (("y", y), ("dx", dx), ("dw", dw)) + ((("db", db),) if bias else ()):
        R.check(name, got, *ref[name])
    # forces only: the same dx, no weight gradients
    dx2, dw2, db2 = m().linear_bwd(x, w, dy, bias=b, act=act, weight_grads=False)
    assert torch.equal(dx, dx2) and dw2 is None and db2 is None
    # residual updated in place
    if res:
        buf = r.clone()
        out = m().linear(x, w, bias=b, act=act, residual=buf, out=buf)
        assert out is buf and torch.equal(buf, y)


# ------------------------------------------------------------------------------ feed-forward
FFN = [
    # n, channels, hidden, dtype, act, residual, pad
    (1, 128, 512, "bf16", "silu", True, 0),
    (77, 32, 32, "bf16", "sigmoid", False, 8),
    (500, 64, 224, "bf16", "silu", False, 64),
    (33000, 128, 96, "bf16", "silu", True, 0),
    (1, 16, 32, "f32", "silu", True, 0),
    (65, 16, 96, "f32", "sigmoid", False, 4),
    (300, 32, 160, "f32", "silu", True, 16),
    (131, 64, 256, "f32", "silu", False, 0),
    (260, 128, 512, "f32", "sigmoid", True, 128),
]


@pytest.mark.parametrize("n,c,f,dt,act,res,pad", FFN)
def test_gated_ffn(n, c, f, dt, act, res, pad):
    g, t = gen(n + f), DT[dt]
    print(f"ffn n={n} C={c} F={f} {dt} {act} res={res} pad={pad}", flush=True)
    x, dy = strided(g, n, c, pad, t), strided(g, n, c, pad, t)
    wg, wu = randn(g, f, c, scale=c ** -0.5, dtype=t), randn(g, f, c, scale=c ** -0.5, dtype=t)
    wd = randn(g, c, f, scale=f ** -0.5, dtype=t)
    r = strided(g, n, c, pad, t) if res else None
    ref = R.ffn(x, wg, wu, wd, act, r, dy)
    y = m().gated_ffn(x, wg, wu, wd, act=act, residual=r)
    grads = m().gated_ffn_bwd(x, wg, wu, wd, dy, act=act)
    torch.cuda.synchronize()
    R.check("y", y, *ref["y"])
    for name, got in zip(("dx", "dwg", "dwu", "dwd"), grads):
        assert got.dtype == t
        R.check(name, got, *ref[name])
    only = m().gated_ffn_bwd(x, wg, wu, wd, dy, act=act, weight_grads=False)
    assert torch.equal(only[0], grads[0]) and only[1:] == (None, None, None)
    if res:
        buf = r.clone()
        m().gated_ffn(x, wg, wu, wd, act=act, residual=buf, out=buf)
        assert torch.equal(buf, y)


# ------------------------------------------------------------------------------ norms
NORM = [
    # n, channels, dtype, scale, gate, post, pre, pad
    (1, 128, "bf16", True, True, True, True, 0),
    (33, 32, "bf16", True, False, False, True, 8),
    (1027, 64, "bf16", False, True, True, False, 16),
    (40000, 128, "bf16", True, False, True, True, 0),
    (1, 16, "f32", True, False, True, True, 0),
    (130, 16, "f32", False, True, False, True, 4),
    (77, 32, "f32", True, True, True, False, 0),
    (513, 64, "f32", False, False, False, False, 64),
    (9001, 128, "f32", True, True, True, True, 12),
]


@pytest.mark.parametrize("n,c,dt,sc,gate,post,pre,pad", NORM)
def test_norm_block(n, c, dt, sc, gate, post, pre, pad):
    g, t = gen(n + c), DT[dt]
    print(f"norm n={n} C={c} {dt} scale={sc} gate={gate} post={post} pre={pre} pad={pad}", flush=True)
    eps = 1e-6
    x, b = strided(g, n, c, pad, t), strided(g, n, c, pad, t)
    ga = strided(g, n, c, pad, t) if gate else None
    scale = randn(g, c) if sc else None
    w_post, w_pre = (randn(g, c) if post else None), (randn(g, c) if pre else None)
    dy, du = strided(g, n, c, pad, t), (strided(g, n, c, pad, t) if pre else None)
    # a row of zeros: rms is sqrt(eps)
    if n > 30:
        x[7] = 0
        b[7] = 0
    kw = dict(scale=scale, gate=ga, w_post=w_post, w_pre=w_pre, eps=eps)
    ref = R.norm(x, b, scale, ga, w_post, w_pre, eps, dy, du)
    y, u = m().norm_block(x, b, **kw)
    gr = m().norm_block_bwd(x, b, dy, du=du, **kw)
    torch.cuda.synchronize()
    R.check("y", y, *ref["y"])
    assert (u is None) == (not pre)
    if pre:
        R.check("u", u, *ref["u"])
    for name in ("dx", "db", "dgate", "dscale", "dw_post", "dw_pre"):
        assert (gr[name] is not None) == (name in ref), name
        if name in ref:
            R.check(name, gr[name], *ref[name])
    # only one of the two incoming gradients
    if pre:
        ref = R.norm(x, b, scale, ga, w_post, w_pre, eps, None, du)
        gr = m().norm_block_bwd(x, b, None, du=du, param_grads=False, **kw)
        R.check("dx (du only)", gr["dx"], *ref["dx"])
        R.check("db (du only)", gr["db"], *ref["db"])
        assert gr["dw_pre"] is None
    buf = x.clone()
    y2, _ = m().norm_block(buf, b, out=buf, **kw)
    assert torch.equal(y2, y)


# ------------------------------------------------------------------------------ attention
def structure_case(sizes, c, heads, dt, bias, cap, mask, L, seed, tail=0, pad=0):
    g, t = gen(seed), DT[dt]
    n = sum(sizes) + tail
    q, k, v, do = (strided(g, n, c, pad, t) for _ in range(4))
    sptr = torch.tensor([0] + sizes).cumsum(0).to(torch.int32).cuda()
    kw = dict(cap=cap)
    if bias:
        kw["pos"] = (torch.rand(n, 3, generator=g) * (L or 9.0)).cuda()
        if L:   # unwrapped positions are allowed
            kw["pos"] += (torch.randint(-1, 2, (n, 3), generator=g) * L).cuda().float()
        kw["slope"] = (torch.rand(heads, generator=g) - 0.2).cuda()
        kw["L"] = L
    if mask is not None:
        kw["mask"] = (torch.rand(n, generator=g) < mask).cuda()
    return n, q, k, v, do, sptr, kw


ATTN = [
    # sizes, channels, heads, dtype, distance term, cap, mask, L, pad
    ([1], 128, 4, "bf16", True, 20.0, None, 0.0, 0),
    ([1, 2, 0, 3, 15, 16, 17, 31, 32, 33, 47, 48, 49, 0, 0, 64, 1], 128, 4, "bf16", True, 0.0, None, 0.0, 0),
    ([0, 0, 5, 40, 0], 64, 2, "bf16", False, 5.0, 0.5, 0.0, 64),
    ([23, 9], 64, 4, "bf16", True, 5.0, 0.7, 0.0, 8),
    ([300], 128, 8, "bf16", True, 20.0, 0.8, 14.0, 0),
    ([129, 200], 32, 1, "bf16", True, 0.0, None, 0.0, 0),
    ([70, 131], 32, 2, "bf16", False, 0.0, 0.9, 0.0, 0),
    ([257], 128, 2, "bf16", True, 3.0, None, 13.0, 128),
    ([90], 64, 1, "bf16", True, 0.0, 0.02, 0.0, 0),
    ([1], 16, 1, "f32", True, 0.0, None, 0.0, 0),
    ([1, 2, 0, 3, 15, 16, 17, 31, 32, 33, 47, 48, 49, 0, 0, 64, 1], 128, 4, "f32", True, 20.0, 0.6, 0.0, 0),
    ([5, 40, 0, 7], 64, 2, "f32", False, 5.0, 0.5, 0.0, 4),
    ([300], 128, 8, "f32", True, 0.0, None, 14.0, 0),
    ([150, 201], 32, 2, "f32", True, 2.0, 0.8, 0.0, 0),
    ([333], 16, 1, "f32", True, 0.0, None, 15.0, 16),
    ([140], 64, 4, "f32", False, 0.0, None, 0.0, 0),
    ([100, 0, 99], 64, 1, "f32", True, 0.0, 0.05, 0.0, 0),
    ([70], 32, 1, "f32", True, 30.0, None, 0.0, 0),
    ([131], 128, 2, "f32", True, 0.0, None, 12.0, 0),
    # long enough for the other side to be split over blocks; one structure without it among them
    ([1100, 7, 0, 1301], 32, 2, "bf16", True, 8.0, 0.7, 0.0, 0),
    ([1500], 64, 2, "f32", True, 0.0, 0.9, 25.0, 8),
    ([1600], 128, 4, "bf16", True, 0.0, None, 26.0, 0),
    ([1030, 1029], 16, 1, "f32", False, 5.0, None, 0.0, 0),
    # sizes far from even: the structure of a slot is far from where even sizes would put it
    ([900] + [1] * 300 + [0] * 90 + [3] * 100, 32, 1, "bf16", True, 0.0, None, 0.0, 0),
    ([2] * 150 + [0] * 200 + [1] * 200 + [700, 1], 16, 1, "f32", True, 0.0, 0.8, 0.0, 0),
    ([1] * 70 + [6500], 16, 1, "f32", False, 0.0, None, 0.0, 0),
]


@pytest.mark.parametrize("sizes,c,heads,dt,bias,cap,mask,L,pad", ATTN)
def test_structure_attention(sizes, c, heads, dt, bias, cap, mask, L, pad):
    tail = 5
    n, q, k, v, do, sptr, kw = structure_case(sizes, c, heads, dt, bias, cap, mask, L, sum(sizes) + c, tail, pad)
    print(f"attention {sizes} C={c} H={heads} {dt} bias={bias} cap={cap} mask={mask} L={L} pad={pad}", flush=True)
    # rows behind the last structure, and what masked keys hold, are nobody's business
    nan = math.nan
    last = n - tail
    k[last:] = nan
    v[last:] = nan
    q[last:] = nan
    if mask is not None:
        dead = ~kw["mask"]
        k[dead] = nan
        v[dead] = math.inf
    out0 = torch.full((n, c), 7.0, dtype=q.dtype, device="cuda")
    ref = R.attention(q, k, v, sptr, heads, dout=None, **kw)
    out = m().structure_attention(q, k, v, sptr, heads, out=out0, **kw)
    torch.cuda.synchronize()
    assert out is out0 and bool((out[last:] == 7.0).all())
    R.check("out", out[:last], ref["out"][0][:last], ref["out"][1][:last])
    # gradients
    ref = R.attention(q, k, v, sptr, heads, dout=do, save=True, **kw)
    out, saved = m().structure_attention(q, k, v, sptr, heads, save=True, **kw)
    R.check("out (saving)", out[:last], ref["out"][0][:last], ref["out"][1][:last])
    buf = torch.full((n, 3 * c), 7.0, dtype=q.dtype, device="cuda")   # one matrix for the three
    dpos = torch.full((n, 3), 7.0, device="cuda") if bias else None
    g = m().structure_attention_bwd(q, k, v, sptr, heads, out, saved, do, dq=buf[:, :c], dk=buf[:, c:2 * c],
                                    dv=buf[:, 2 * c:], dpos=dpos, **kw)
    torch.cuda.synchronize()
    assert bool((buf[last:] == 7.0).all()) and (dpos is None or bool((dpos[last:] == 7.0).all()))
    for name in ("dq", "dk", "dv") + (("dpos",) if bias else ()):
        R.check(name, g[name][:last], ref[name][0][:last], ref[name][1][:last])
    if bias:
        R.check("dslope", g["dslope"], *ref["dslope"])
    else:
        assert g["dpos"] is None and g["dslope"] is None


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_structure_attention_no_key_left(dt):
    """A structure without any unmasked atom: zero rows and zero gradients."""
    n, q, k, v, do, sptr, kw = structure_case([20, 150, 33], 64, 2, dt, True, 4.0, 1.0, 0.0, 3)
    kw["mask"][20:170] = False
    out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
    g = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
    torch.cuda.synchronize()
    for t in (out, g["dq"], g["dk"], g["dv"], g["dpos"]):
        assert bool((t[20:170] == 0).all()) and bool(torch.isfinite(t).all()) and float(t[:20].float().abs().max()) > 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_structure_attention_huge_scores(dt):
    """Scores of several hundred: the weights are one-hot, nothing overflows; capped, they stay soft."""
    n, q, k, v, do, sptr, kw = structure_case([40, 100], 64, 2, dt, True, 0.0, None, 0.0, 11)
    q, k = (q.float() * 30).to(q.dtype), (k.float() * 30).to(k.dtype)
    for cap in (0.0, 2.0):
        kw["cap"] = cap
        ref = R.attention(q, k, v, sptr, 2, dout=do, save=True, **kw)
        out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
        g = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
        R.check("out", out, *ref["out"])
        for name in ("dq", "dk", "dv", "dpos", "dslope"):
            R.check(name, g[name], *ref[name])


def test_structure_attention_coincident_atoms():
    """r = 0 between distinct atoms: the position gradient of that pair is zero, not NaN."""
    n, q, k, v, do, sptr, kw = structure_case([12], 32, 2, "f32", True, 0.0, None, 0.0, 5)
    kw["pos"][4] = kw["pos"][9]
    ref = R.attention(q, k, v, sptr, 2, dout=do, save=True, **kw)
    out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
    g = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
    for name in ("dq", "dk", "dv", "dpos", "dslope"):
        R.check(name, g[name], *ref[name])


@pytest.mark.parametrize("dt,sizes", [("f32", [50, 64, 3]), ("f32", [700]), ("bf16", [40, 40]), ("bf16", [300])])
def test_structure_attention_half_a_box(dt, sizes):
    """Coordinates on a grid of an eighth of the box: many pairs exactly half a box apart in some
    direction.  The gradient points along the coordinates' own difference there, so a pair's two are
    opposite, and equal positions have none."""
    n, q, k, v, do, sptr, kw = structure_case(sizes, 64, 2, dt, True, 0.0, None, 0.0, 41)
    kw["pos"] = torch.randint(0, 8, (n, 3), generator=gen(42)).float().cuda()
    kw["slope"], kw["L"] = torch.tensor([0.3, 0.7], device="cuda"), 8.0
    ref = R.attention(q, k, v, sptr, 2, dout=do, save=True, **kw)
    out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
    g = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
    R.check("out", out, *ref["out"])
    for name in ("dq", "dk", "dv", "dpos", "dslope"):
        R.check(name, g[name], *ref[name])


@pytest.mark.parametrize("cap", [1e-3, 0.3, 200.0, 1e4])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_structure_attention_caps(dt, cap):
    """The ends of the cap's range: every score past the polynomial, scores on both sides of its end, none."""
    n, q, k, v, do, sptr, kw = structure_case([90, 33], 64, 2, dt, True, cap, None, 0.0, 31)
    ref = R.attention(q, k, v, sptr, 2, **kw)
    R.check("out", m().structure_attention(q, k, v, sptr, 2, **kw), *ref["out"])
    ref = R.attention(q, k, v, sptr, 2, dout=do, save=True, **kw)
    out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
    g = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
    R.check("out", out, *ref["out"])
    for name in ("dq", "dk", "dv", "dpos", "dslope"):
        R.check(name, g[name], *ref[name])


# ------------------------------------------------------------------------------ how they are called
def _one_of_each(dt, seed, n=700, c=64, sizes=(300, 21, 0, 350)):
    """Closures over fixed inputs: every operator and its backward, as lists of tensors."""
    g, t = gen(seed), DT[dt]
    x, b, dy, gate = (randn(g, n, c, dtype=t) for _ in range(4))
    w, wg, wu, wd = (randn(g, *s, scale=0.1, dtype=t) for s in ((96, c), (128, c), (128, c), (c, 128)))
    bias, sc, wp, wq = randn(g, 96), randn(g, c), randn(g, c), randn(g, c)
    dyw = randn(g, n, 96, dtype=t)
    n2, q, k, v, do, sptr, kw = structure_case(list(sizes), c, 2, dt, True, 5.0, 0.8, 0.0, seed, n - sum(sizes))
    nk = dict(scale=sc, gate=gate, w_post=wp, w_pre=wq)

    def attn():
        out = torch.zeros_like(q)
        out, saved = m().structure_attention(q, k, v, sptr, 2, out=out, save=True, **kw)
        g = [torch.zeros_like(q) for _ in range(3)] + [torch.zeros(n, 3, device="cuda")]
        gr = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, dq=g[0], dk=g[1], dv=g[2], dpos=g[3], **kw)
        return [out, *g, gr["dslope"]]
    return {
        "linear": lambda: [m().linear(x, w, bias=bias, act="silu"), *m().linear_bwd(x, w, dyw, bias=bias, act="silu")],
        "ffn": lambda: [m().gated_ffn(x, wg, wu, wd), *m().gated_ffn_bwd(x, wg, wu, wd, dy)],
        "norm": lambda: [*m().norm_block(x, b, **nk), *[v for v in m().norm_block_bwd(x, b, dy, du=dy, **nk).values()]],
        "attention": attn,
    }


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeats_streams_and_graphs_give_the_same_bits(dt):
    """A second call, a call on another stream, and replays of a captured call (with the program's
    own work between them) give the bits of the first call."""
    for name, f in _one_of_each(dt, 77).items():
        print(f"{name} {dt}", flush=True)
        ref = [t.clone() for t in f()]
        torch.cuda.synchronize()
        same = lambda got: all(torch.equal(a, b) for a, b in zip(ref, got))  # noqa: E731
        assert same(f())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = f()
        torch.cuda.current_stream().wait_stream(side)
        assert same(got), (name, "another stream")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = f()
        for k in range(3):
            for h in held:
                h.fill_(3)
            graph.replay()
            f()                       # the program's own work beside the replays
            torch.cuda.synchronize()
            assert same(held), (name, "replay", k)


def test_two_calls_at_once():
    """The same operators enqueued on two streams at a time, each with its own scratch, keep their bits."""
    a, b = _one_of_each("bf16", 78), _one_of_each("f32", 79, n=900, sizes=(800, 40))
    for name in a:
        ra, rb = [t.clone() for t in a[name]()], [t.clone() for t in b[name]()]
        torch.cuda.synchronize()
        s = [torch.cuda.Stream() for _ in range(2)]
        got = [None, None]
        for st, k, f in ((s[0], 0, a[name]), (s[1], 1, b[name])):
            with torch.cuda.stream(st):
                for _ in range(3):
                    got[k] = f()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ra, got[0])), name
        assert all(torch.equal(x, y) for x, y in zip(rb, got[1])), name


def test_offsets_past_32_bits():
    """Rows so far apart that the last ones lie past 2^32 elements."""
    g, n, ld = gen(9), 530, 1 << 23
    big = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda").as_strided((n, ld), (ld, 1))
    assert (n - 1) * ld > 2 ** 32
    x, y = big[:, :64], big[:, 128:192]
    x.copy_(randn(g, n, 64, dtype=torch.bfloat16))
    xc = x.contiguous()
    w, wg = randn(g, 64, 64, scale=0.1, dtype=torch.bfloat16), randn(g, 96, 64, scale=0.1, dtype=torch.bfloat16)
    wd, s = randn(g, 64, 96, scale=0.1, dtype=torch.bfloat16), randn(g, 64)
    same = lambda got: torch.equal(got.contiguous(), ref)  # noqa: E731
    ref = m().linear(xc, w, residual=xc)
    assert same(m().linear(x, w, residual=x, out=y))
    ref = m().gated_ffn(xc, wg, wg, wd)
    assert same(m().gated_ffn(x, wg, wg, wd, out=y))
    ref = m().norm_block(xc, xc, gate=xc, w_post=s)[0]
    assert same(m().norm_block(x, x, gate=x, w_post=s, out=y)[0])
    pairs = [(m().linear_bwd(xc, w, xc), m().linear_bwd(x, w, x)),
             (m().gated_ffn_bwd(xc, wg, wg, wd, xc), m().gated_ffn_bwd(x, wg, wg, wd, x)),
             (list(m().norm_block_bwd(xc, xc, xc, w_post=s).values()), list(m().norm_block_bwd(x, x, x, w_post=s).values()))]
    for a, b in pairs:
        assert all((u is None and v is None) or torch.equal(u, v) for u, v in zip(a, b))
    for sizes in ([n], [25, 30] * 9 + [35]):   # long structures, short ones
        sptr = torch.tensor([0, *torch.tensor(sizes).cumsum(0)], dtype=torch.int32, device="cuda")
        assert int(sptr[-1]) == n
        kw = dict(pos=randn(g, n, 3, scale=3.0), slope=torch.tensor([0.2, 0.4], device="cuda"))
        ref, saved = m().structure_attention(xc, xc, xc, sptr, 2, save=True, **kw)
        got, saved2 = m().structure_attention(x, x, x, sptr, 2, save=True, out=y, **kw)
        assert same(got) and torch.equal(saved, saved2)
        ga = m().structure_attention_bwd(xc, xc, xc, sptr, 2, ref, saved, xc, **kw)
        d = [big[:, 256 + 64 * k:320 + 64 * k] for k in range(3)]
        gb = m().structure_attention_bwd(x, x, x, sptr, 2, y, saved, x, dq=d[0], dk=d[1], dv=d[2], **kw)
        assert all(torch.equal(ga[k], gb[k].contiguous()) for k in ga)


def test_bf16_bits_as_int16():
    """Rows as int16 bit patterns (the feature tensors' form) give the same bits as bfloat16."""
    g = gen(5)
    x, w = randn(g, 100, 64, dtype=torch.bfloat16), randn(g, 48, 64, dtype=torch.bfloat16)
    y = m().linear(x, w)
    y2 = m().linear(x.view(torch.int16), w.view(torch.int16))
    assert y2.dtype == torch.int16 and torch.equal(y2.view(torch.bfloat16), y)


def test_scalar_rows_of_a_feature_tensor():
    """h[:, 0] of a [n, K, C] feature tensor in place: the other rows stay as they are."""
    g = gen(6)
    h = randn(g, 333, 9, 128)
    before = h.clone()
    b, sc, wp = randn(g, 333, 128), randn(g, 128), randn(g, 128)
    y, u = m().norm_block(h[:, 0], b, scale=sc, w_post=wp, w_pre=wp, out=h[:, 0])
    ref = R.norm(before[:, 0], b, sc, None, wp, wp, 1e-6, None, None)
    R.check("y", h[:, 0], *ref["y"])
    R.check("u", u, *ref["u"])
    assert torch.equal(h[:, 1:], before[:, 1:])


def test_no_rows_and_no_structures():
    t = torch.float32
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(32, 64, device="cuda")
    b = torch.ones(32, device="cuda")
    assert m().linear(x, w, bias=b).shape == (0, 32)
    dx, dw, db = m().linear_bwd(x, w, torch.empty(0, 32, device="cuda"), bias=b)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    wg, wd = torch.ones(96, 64, device="cuda"), torch.ones(64, 96, device="cuda")
    assert m().gated_ffn(x, wg, wg, wd).shape == (0, 64)
    g = m().gated_ffn_bwd(x, wg, wg, wd, x)
    assert g[0].shape == (0, 64) and all(bool((v == 0).all()) for v in g[1:])
    s = torch.ones(64, device="cuda")
    y, u = m().norm_block(x, x, scale=s, w_post=s, w_pre=s)
    assert y.shape == u.shape == (0, 64)
    g = m().norm_block_bwd(x, x, x, du=x, scale=s, w_post=s, w_pre=s)
    assert all(bool((g[k] == 0).all()) for k in ("dscale", "dw_post", "dw_pre"))
    kw = dict(pos=torch.empty(0, 3, device="cuda"), slope=torch.ones(2, device="cuda"))
    for n, sp in ((0, [0]), (0, [0, 0, 0]), (5, [0]), (5, [0, 0])):
        q = torch.randn(n, 64, device="cuda", dtype=t)
        kw["pos"] = torch.zeros(n, 3, device="cuda")
        sptr = torch.tensor(sp, dtype=torch.int32, device="cuda")
        keep, *d = [torch.full((n, 64), 2.0, device="cuda") for _ in range(4)]
        out, saved = m().structure_attention(q, q, q, sptr, 2, out=keep, save=True, **kw)
        g = m().structure_attention_bwd(q, q, q, sptr, 2, out, saved, q, dq=d[0], dk=d[1], dv=d[2], **kw)
        assert all(bool((v == 2).all()) for v in (keep, *d)) and bool((g["dslope"] == 0).all())


def test_python_refusals():
    x, w = torch.zeros(8, 64, device="cuda"), torch.zeros(32, 64, device="cuda")
    sp = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    bad = [
        lambda: m().linear(x.cpu(), w), lambda: m().linear(x, w.bfloat16()), lambda: m().linear(x.half(), w.half()),
        lambda: m().linear(x, w, act="gelu"), lambda: m().linear(x, w, bias=torch.zeros(31, device="cuda")),
        lambda: m().linear(x, w, residual=torch.zeros(7, 32, device="cuda")), lambda: m().linear(x.t().contiguous().t(), w),
        lambda: m().linear(x, w[:, :32]), lambda: m().linear(x[0], w),
        lambda: m().gated_ffn(x, w, w[:16], w.t().contiguous()),
        lambda: m().norm_block(x, x[:4]), lambda: m().norm_block(x, x, scale=torch.ones(64)),
        lambda: m().structure_attention(x, x, x, sp.long(), 2), lambda: m().structure_attention(x, x[:4], x, sp, 2),
        lambda: m().structure_attention(x, x, x, sp, 2, mask=torch.ones(7, dtype=torch.bool, device="cuda")),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", k, flush=True)
    odd = [
        lambda: m().linear(torch.zeros(8, 66, device="cuda")[:, :64], w),           # row stride of 264 bytes
        lambda: m().linear(torch.zeros(8, 65, device="cuda")[:, 1:], w),            # rows not 16-byte aligned
        lambda: m().linear(x[:1].expand(8, 64), w),                                 # row stride 0
        lambda: m().gated_ffn(x, w, w, w.t().contiguous(), act="none"),
        lambda: m().structure_attention(x, x, x, sp, 8), lambda: m().structure_attention(x, x, x, sp, 2, cap=-1.0),
        lambda: m().structure_attention(x, x, x, sp, 2, pos=torch.zeros(8, 3, device="cuda")),
    ]
    t = torch.zeros(64, 64, device="cuda")
    sv = torch.zeros(8 * 2, device="cuda")
    odd += [  # outputs that another part of the call still reads
        lambda: m().linear(x, t, out=x), lambda: m().gated_ffn(x, t, t, t, out=x),
        lambda: m().structure_attention(x, x, x, sp, 2, out=x),
        lambda: m().structure_attention_bwd(x, x, x, sp, 2, x, sv, x, dq=x),
        lambda: m().structure_attention_bwd(x, x, x, sp, 2, x, sv, x, dk=t[:8], dv=t[:8]),
    ]
    for k, f in enumerate(odd):
        with pytest.raises(m().MPError) as e:
            f()
            print("not refused:", k, flush=True)
        assert e.value.code == m().MP_ERR_ARG


# ------------------------------------------------------------------------------ gradients as differences
def test_gradients_against_differences():
    """<gradient, direction> against central differences of the float64 definitions along the
    direction (step h: the difference is off by O(h^2) of the third derivative, here below 1e-6
    of the value at h = 1e-4; the float32 gradients' own bounds are far below 1e-4)."""
    g, h = gen(9), 1e-4

    def along(f, args, grads, dirs):
        lo, hi = ([None if a is None else a.cpu().double() + s * h * d for a, d in zip(args, dirs)] for s in (-1, 1))
        num = (f(*hi) - f(*lo)) / (2 * h)
        got = sum(float((gr.cpu().double() * d).sum()) for gr, d in zip(grads, dirs) if gr is not None)
        size = sum(float((gr.cpu().double().abs() * d.abs()).sum()) for gr, d in zip(grads, dirs) if gr is not None)
        print(f"  difference {float(num):.8f}, gradient {got:.8f}", flush=True)
        assert abs(float(num) - got) <= 1e-5 * size

    def dirs(*ts):
        return [torch.zeros(()) if t is None else torch.randn(t.shape, generator=g, dtype=torch.float64) for t in ts]

    n, c = 50, 32
    x, dy = randn(g, n, c), randn(g, n, c)
    wg, wu, wd = randn(g, 64, c, scale=0.2), randn(g, 64, c, scale=0.2), randn(g, c, 64, scale=0.2)
    dy64 = dy.cpu().double()
    along(lambda *a: (R.ffn(*a, "silu", None, None)["y"][0] * dy64).sum(), (x, wg, wu, wd),
          m().gated_ffn_bwd(x, wg, wu, wd, dy), dirs(x, wg, wu, wd))
    w, b = randn(g, c, c, scale=0.2), randn(g, c)
    along(lambda *a: (R.linear(*a, "sigmoid", None, None)["y"][0] * dy64).sum(), (x, w, b),
          m().linear_bwd(x, w, dy, bias=b, act="sigmoid"), dirs(x, w, b))
    gate, sc, wp, wq, bb, du = randn(g, n, c), randn(g, c), randn(g, c), randn(g, c), randn(g, n, c), randn(g, n, c)
    du64 = du.cpu().double()

    def fnorm(x_, b_, s_, g_, p_, q_):
        r = R.norm(x_, b_, s_, g_, p_, q_, 1e-6, None, None)
        return (r["y"][0] * dy64).sum() + (r["u"][0] * du64).sum()
    gr = m().norm_block_bwd(x, bb, dy, du=du, scale=sc, gate=gate, w_post=wp, w_pre=wq)
    along(fnorm, (x, bb, sc, gate, wp, wq), [gr[k] for k in ("dx", "db", "dscale", "dgate", "dw_post", "dw_pre")],
          dirs(x, bb, sc, gate, wp, wq))
    n, q, k, v, do, sptr, kw = structure_case([20, 75], c, 2, "f32", True, 3.0, None, 0.0, 21)
    do64 = do.cpu().double()
    out, saved = m().structure_attention(q, k, v, sptr, 2, save=True, **kw)
    gr = m().structure_attention_bwd(q, k, v, sptr, 2, out, saved, do, **kw)
    along(lambda q_, k_, v_, p_, s_: (R.attention(q_, k_, v_, sptr, 2, pos=p_, slope=s_, cap=3.0)["out"][0] * do64).sum(),
          (q, k, v, kw["pos"], kw["slope"]), [gr[t] for t in ("dq", "dk", "dv", "dpos", "dslope")],
          dirs(q, k, v, kw["pos"], kw["slope"]))
