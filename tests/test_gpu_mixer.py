"""Energy and forces with global blocks (mp_energy_forces_mixer: the block operators run
together, forward and backward, between the layers and the readout) vs the oracle
(oracle.model.energy_mixer, float64 CPU), to the bars of the other energy paths: float32 1e-4,
bf16 2e-2 of sum_i |E_i| and of the largest force."""
import numpy as np
import pytest

from tests import mixer_case as MC
from tests.helpers import energy_error, force_error

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.tensor(a, device="cuda")


@pytest.mark.parametrize("C,lmax,heads,T,bf16,H,hidden,B,cap", [
    (16, 1, 2, 1, False, 1, 32, 2, 3.0), (64, 2, 4, 2, False, 2, 96, 1, 0.0), (128, 2, 4, 2, True, 4, 256, 2, 10.0)])
def test_batch_parity(C, lmax, heads, T, bf16, H, hidden, B, cap):
    import torch
    from molecular_dynamics_amd import mdmp
    from oracle import model as OM
    from oracle import neighbors as NB
    print(f"mixer batch C={C} bf16={bf16} blocks={B} H={H} hidden={hidden} cap={cap}", flush=True)
    pos, sp, sptr, cfg, w = MC.batch(20, 1, 40, 50 + C, C, lmax, heads, T, bf16)
    mw = MC.weights(C, B, H, hidden, 60 + C)
    g = mdmp.build_neighbors_batched(dev(pos), dev(sp), dev(sptr), cfg.cutoff, 0.5)
    model = mdmp.Model(cfg, w)
    assert mdmp.Mixer.num_weights(model, B, H, hidden) == mw.size
    mixer = mdmp.Mixer(model, B, H, hidden, mw, cap=cap)
    e_at = torch.empty(len(pos), dtype=torch.float32, device="cuda")
    E, F = mdmp.energy_forces_mixer(model, mixer, g, dev(sptr), atom_energy=e_at)
    rp, col = NB.csr_open_batched(pos, sptr, cfg.cutoff, 0.5)
    ref = OM.energy_mixer(cfg, w, mw, B, H, hidden, cap, pos, sp, None, rp, col, sptr)
    ee, fe = energy_error(E, ref["E"], ref["E_atoms"]), force_error(F.cpu().numpy(), ref["F"])
    ae = np.abs(e_at.cpu().numpy() - ref["E_atoms"]).max() / np.abs(ref["E_atoms"]).max()
    print(f"  energy err {ee:.2e}, force err {fe:.2e}, atom-energy err {ae:.2e}", flush=True)
    tol = 2e-2 if bf16 else 1e-4
    assert ee <= tol and fe <= tol and ae <= tol
    # the blocks matter: without them the forces are others; and the same call gives the same bits
    _, F0 = mdmp.energy_forces(model, g)
    assert force_error(F0.cpu().numpy(), ref["F"]) > 10 * tol
    E2, F2 = mdmp.energy_forces_mixer(model, mixer, g, dev(sptr))
    assert E2 == E and torch.equal(F, F2)
    mixer.close()


@pytest.mark.parametrize("bf16", [False, True])
def test_periodic_box_parity(bf16):
    """One periodic box as one structure: sorted slots, un-permuted forces, minimum image."""
    from molecular_dynamics_amd import inputs, mdmp
    from oracle import model as OM
    from oracle import neighbors as NB
    box = inputs.box_uniform(400, 16.0, 3, 91)
    cfg = inputs.ModelConfig(n_species=3, channels=64, lmax=2, n_bessel=8, heads=4, layers=2, cutoff=5.0,
                             feat_bf16=bf16)
    w = inputs.make_weights(cfg, np.random.SeedSequence(92).spawn(3)[2])
    mw = MC.weights(64, 2, 4, 128, 93)
    g = mdmp.build_neighbors(dev(box.pos), dev(box.species), box.L, cfg.cutoff, 1.0)
    model = mdmp.Model(cfg, w)
    mixer = mdmp.Mixer(model, 2, 4, 128, mw, cap=5.0)
    E, F = mdmp.energy_forces_mixer(model, mixer, g, perm=g.perm)
    nb = NB.build_neighbors(box.pos, box.L, cfg.cutoff, 1.0)
    ref = OM.energy_mixer(cfg, w, mw, 2, 4, 128, 5.0, nb["pos_sorted"], box.species[nb["perm"]], box.L, nb["row_ptr"],
                          nb["col"], [0, 400])
    Fref = np.empty_like(ref["F"])
    Fref[nb["perm"]] = ref["F"]
    ee, fe = energy_error(E, ref["E"], ref["E_atoms"]), force_error(F.cpu().numpy(), Fref)
    print(f"mixer box bf16={bf16}: energy err {ee:.2e}, force err {fe:.2e}", flush=True)
    tol = 2e-2 if bf16 else 1e-4
    assert ee <= tol and fe <= tol


def test_mixer_errors():
    from molecular_dynamics_amd import mdmp
    pos, sp, sptr, cfg, w = MC.batch(4, 3, 9, 70, 64, 2, 4, 1, False)
    model = mdmp.Model(cfg, w)
    mw = MC.weights(64, 1, 2, 64, 71)

    def bad(n_blocks=1, heads=2, hidden=64, weights=mw, cap=0.0):
        with pytest.raises(mdmp.MPError) as e:
            mdmp.Mixer(model, n_blocks, heads, hidden, weights, cap=cap)
        assert e.value.code == mdmp.MP_ERR_ARG
    bad(n_blocks=0)
    bad(n_blocks=17)
    bad(heads=3)
    bad(hidden=40)
    bad(weights=mw[:-1])
    bad(cap=-1.0)
    mixer = mdmp.Mixer(model, 1, 2, 64, mw)
    g = mdmp.build_neighbors_batched(dev(pos), dev(sp), dev(sptr), cfg.cutoff, 0.0)
    import torch
    small = torch.empty(4096, dtype=torch.uint8, device="cuda")
    with pytest.raises(mdmp.MPError) as e:
        mdmp.energy_forces_mixer(model, mixer, g, dev(sptr), ws=small)
    assert e.value.code == mdmp.MP_ERR_ARG
    # a mixer made for another model's channels
    pos2, sp2, sptr2, cfg2, w2 = MC.batch(4, 3, 9, 70, 128, 2, 4, 1, False)
    with pytest.raises(mdmp.MPError) as e:
        mdmp.energy_forces_mixer(mdmp.Model(cfg2, w2), mixer, g, dev(sptr))
    assert e.value.code == mdmp.MP_ERR_ARG


@pytest.mark.parametrize("bf16", [False, True])
def test_captured_evaluation_replays(bf16):
    """The whole evaluation captured once and replayed, with other work between, gives the same bits."""
    import ctypes
    import torch
    from molecular_dynamics_amd import mdmp
    pos, sp, sptr, cfg, w = MC.batch(12, 1, 70, 54, 64, 2, 4, 2, bf16)
    mw = MC.weights(64, 2, 2, 96, 66)
    g = mdmp.build_neighbors_batched(dev(pos), dev(sp), dev(sptr), cfg.cutoff, 0.5)
    model = mdmp.Model(cfg, w)
    mixer = mdmp.Mixer(model, 2, 2, 96, mw, cap=4.0)
    ptr = dev(sptr)
    E, F = mdmp.energy_forces_mixer(model, mixer, g, ptr)
    nb = ctypes.c_size_t(0)
    mdmp._check(mdmp._lib.mp_energy_forces_mixer_ws(model.h, mixer.h, g.n, len(sptr) - 1, g.n_edges,
                                                    ctypes.byref(nb)), "ws")
    ws = mdmp._ws(nb.value)
    e2, f2 = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(g.n, 3, device="cuda")
    gs = g.struct()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdmp._check(mdmp._lib.mp_energy_forces_mixer(model.h, mixer.h, ctypes.byref(gs), ptr.data_ptr(), len(sptr) - 1,
                                                     None, e2.data_ptr(), f2.data_ptr(), None, ws.data_ptr(),
                                                     ws.numel(), mdmp._stream()), "mp_energy_forces_mixer")
    for _ in range(3):
        e2.fill_(1)
        f2.fill_(1)
        graph.replay()
        mdmp.energy_forces(model, g)
        torch.cuda.synchronize()
        assert float(e2.item()) == E and torch.equal(f2, F)


def test_structures_that_do_not_cover_the_atoms_are_refused():
    import torch
    from molecular_dynamics_amd import mdmp
    pos, sp, sptr, cfg, w = MC.batch(6, 2, 20, 55, 16, 1, 2, 1, False)
    g = mdmp.build_neighbors_batched(dev(pos), dev(sp), dev(sptr), cfg.cutoff, 0.5)
    model = mdmp.Model(cfg, w)
    mixer = mdmp.Mixer(model, 1, 1, 64, MC.weights(16, 1, 1, 64, 67))
    n = len(pos)
    E, F = mdmp.energy_forces_mixer(model, mixer, g, dev(sptr))
    for bad in ([0, n - 1], [1, n], [0, n + 1], [0, n // 2 + 1, n // 2, n]):
        with pytest.raises(mdmp.MPError) as e:
            mdmp.energy_forces_mixer(model, mixer, g, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert e.value.code == mdmp.MP_ERR_ARG
    E2, F2 = mdmp.energy_forces_mixer(model, mixer, g, dev(sptr))
    assert E2 == E and torch.equal(F2, F)
