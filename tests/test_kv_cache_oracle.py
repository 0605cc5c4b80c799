"""What the 8-bit cache oracle returns for tolerances, without a GPU."""
import numpy as np

from oracle import kv_cache as oracle


def test_forward_tolerances_know_only_the_keys_that_a_row_sees():
    """A page of far larger values that the first queries end before, or that the
    last ones' windows begin behind, enters no other row's largest |v|."""
    rng = np.random.default_rng(0)
    P, HKV, D, L, m = 16, 2, 64, 40, 12
    kc, vc = (oracle.to_e4m3(rng.standard_normal((3, P, HKV, D)) * 50) for _ in range(2))
    ks = np.full((3, HKV), 2.0 ** -6)
    q = rng.standard_normal((m, 2 * HKV, D))
    for big, window in ((2, -1), (1, 5)):
        vs = np.full((3, HKV), 2.0 ** -6)
        vs[big] *= 2.0 ** 20
        o, lse, mag, dots, seen, vmax = oracle.forward(q, kc, vc, ks, vs, np.arange(3)[None], [0, m], [L], 0.1, True,
                                                       window)
        for f in range(2 * HKV):
            v = np.abs(oracle.E4M3[vc] * vs[:, None, :, None])[:, :, f // 2].reshape(3 * P, D).max(1)
            for i in range(m):
                at = L - m + i
                j = np.arange(max(0, at - window + 1) if window > 0 else 0, at + 1)
                assert vmax[f, i] == v[j].max() and seen[f, i] == len(j)
        assert vmax.min() < 2.0 ** 4 < vmax.max()
