"""Seeded mixers (global blocks) and small batched structures for the mixer tests."""
import numpy as np


def weights(C, n_blocks, heads, hidden, seed):
    """Float32 blob: matrices N(0, 1/fan_in), norm weights about 1, residual scales about 0.5,
    slopes per angstrom halved from head to head."""
    from oracle import model as OM
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(n_blocks):
        for name, r, c in OM.mixer_layout(C, heads, hidden):
            if name == "slope":
                out.append(0.5 ** np.arange(heads) * (1 + 0.1 * rng.random(heads)))
            elif name in ("w1", "w2", "p1", "p2"):
                out.append(1 + 0.1 * rng.standard_normal(c))
            elif name in ("s1", "s2"):
                out.append(0.5 + 0.1 * rng.standard_normal(c))
            else:
                out.append((rng.standard_normal((r, c)) / np.sqrt(c)).ravel())
    return np.concatenate(out).astype(np.float32)


def batch(n_struct, n_min, n_max, seed, C, lmax, heads, T, bf16, cutoff=4.5):
    from molecular_dynamics_amd import inputs
    pos, sp, sptr = inputs.batch_molecules(n_struct, n_min, n_max, seed, n_species=3)
    cfg = inputs.ModelConfig(n_species=3, channels=C, lmax=lmax, n_bessel=8, heads=heads, layers=T, cutoff=cutoff,
                             feat_bf16=bf16)
    w = inputs.make_weights(cfg, np.random.SeedSequence(seed).spawn(3)[2])
    return pos, sp, sptr, cfg, w
