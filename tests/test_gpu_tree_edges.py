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
