"""Drafted trees on the GPU: infinities in held rows and in tokens, expired waits, table entries that are left alone."""
import numpy as np
import pytest
import torch

from parity import f64
from test_gpu_tree import BF16, DEV, F32, Problem, config, random_parents

rat = pytest.importorskip("recurrence_augmented_dilated_gated_b200")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4, 20, 40])
def test_runs_that_begin_with_keys_left_out(N):
    # The persistent form deals whole tiles of 128 rows out, three or four to a CTA here.  Three tiles of every four
    # hold keys that every node scores -inf, so most runs begin with one; the other held rows and the nodes score
    # about -300: weights that vanish beside a reference of 0, and are all there is.
    parent = random_parents(np.random.default_rng(N), 1, N, 4, pad=False)
    cfg = config(1, N, 1, 128, BF16, [1], [0], [0], scale=1.0)
    p = Problem(cfg, 800000, [60000], parent, std=0.3)
    p.q[..., 0], p.k[..., 0], p.hk[..., 0] = 1.0, -300.0, -300.0
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.hk[:, torch.arange(60000) // 128 % 4 != 3, :, 5] = -float("inf")
    p.to_gpu()
    p.check(*p.step())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("D,W,N", [(1, 0, 3), (1, 0, 20), (1, 0, 40), (3, 9, 20), (4, 0, 40)])
def test_infinities_in_held_rows(dtype, d, D, W, N):
    # a key that scores -inf drops out; a value that is infinite reaches the nodes that see its row, in its channel
    # and with its sign, and nothing else
    parent = random_parents(np.random.default_rng(N), 2, N, 4, pad=False)
    cfg = config(2, N, 1, d, dtype, [D], [W], scale=0.2)
    p = Problem(cfg, 400, [300, 41], parent)
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.hk[0, 150:160, 0, 5] = -float("inf")
    p.hk[1, 30:35, 0, 5] = -float("inf")
    p.hv[0, 20, 0, 7], p.hv[0, 296, 0, 9], p.hv[1, 40, 0, 11] = float("inf"), -float("inf"), float("inf")
    p.to_gpu()
    o, lse = p.step()
    ro, rl = p.reference()
    got = f64(o)
    assert np.array_equal(np.isnan(got), np.isnan(ro)) and not np.isnan(ro).any()
    hit = np.isinf(ro)
    assert hit.any() and np.array_equal(got[~np.isfinite(got)], ro[hit]) and np.array_equal(np.isinf(got), hit)
    off = got[~hit] - ro[~hit]
    assert np.abs(f64(lse) - rl).max() <= (1e-4 if dtype == F32 else 1e-3)
    if dtype == F32:
        assert np.abs(off).max() <= 1e-4
    else:
        assert np.linalg.norm(off) <= 1e-2 * np.linalg.norm(ro[~hit])
