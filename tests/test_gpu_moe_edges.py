"""Edges of the mixture-of-experts operators on a B200, beside test_gpu_moe.py
(whose problems, references and tolerances are used here)."""
import numpy as np
import pytest

import test_gpu_moe as base

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

q4k = base.q4k     # the module's fixture


# ------------------------------------------------------------------ routing

@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,top_k", [(1, 2, 1), (2, 2, 1), (64, 8, 3), (65, 8, 3), (24, 33, 4), (300, 33, 4),
                                       (64, 100, 16), (200, 256, 16)])
def test_route_signed_zeros_tie(q4k, t, e, top_k, renorm):
    """-0.0 and +0.0 are equal logits: the lower expert comes first, in the one-launch
    (up to 64 tokens) and the two-launch path, wherever the tie lies."""
    rng = np.random.default_rng(t * 100 + e)
    zeros = np.where(rng.random((t, e)) < 0.5, np.float32(-0.0), np.float32(0.0))
    logits = np.where(rng.random((t, e)) < 0.7, zeros, rng.choice(np.float32([-1, 1, 2]), (t, e)))
    logits[0] = 0.0
    logits[0, 0] = -0.0                       # the first expert wins over every +0.0
    logits[-1] = np.where(np.arange(e) % 2 == 0, np.float32(-0.0), np.float32(0.0))    # across the cut at top_k
    logits = logits.astype(np.float32)
    assert np.signbit(logits[0, 0])
    base.check_route(base.gpu_route(q4k, logits, top_k, renorm), logits, top_k, renorm, f"{t}x{e} top {top_k}")
