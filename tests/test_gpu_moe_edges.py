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


# ------------------------------------------------------------------ products

def slot_rows(p, e, a, b):
    """Rows of y that expert e's slots a .. b - 1 write, their values and bounds in 64 bits."""
    alone = np.zeros(p.experts + 1, np.int32)      # the list in which only expert e has pairs
    alone[:e + 1], alone[e + 1:] = a, b
    kept, p.offsets = p.offsets, alone
    want, tol = base.reference(p)
    p.offsets = kept
    rows = np.arange(a, b) if len(p.ws) == 2 else p.order[a:b]
    return rows, want[a:b], tol[a:b]


@pytest.mark.parametrize("bad", [[0, 8, 30, 20, 20], [0, 8, 15, 20, 10], [0, 12, 25, 30, -7], [0, 30, -2 ** 31, 5, 5],
                                 [0, 8, -1, 20, 30], [40, 8, 15, 20, 30], [0, 8, 15, 20, 31]])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("per_row", [0, 1, 3])
def test_experts_with_sound_offsets_survive_bad_ones(q4k, per_row, mats, half, bad):
    """Where some expert's offsets do not ascend within the pairs, the others' rows
    are computed all the same, also behind the last entry of the offsets; whatever
    an earlier call left in the library's workspace does not show."""
    assert q4k.q4k_device_fault_flags() == 0
    p = base.Problem(30, 4, 1, 60, 512, 23, mats=mats, half=half, per_row=per_row)
    x = p.dx.clone()
    p.dx.copy_(torch.full_like(x, 3.0))
    base.run_product(q4k, p)                       # leaves other rows in the workspace
    p.dx.copy_(x)
    p.offsets = np.array(bad).astype(np.int32)
    p.doff = base.dev(p.offsets)
    y = base.run_product(q4k, p).float().cpu().numpy()
    assert q4k.q4k_device_fault_flags() == q4k.Q4K_FAULT_ROUTE_RANGE
    skipped = np.ones(p.pairs, bool)
    for e in range(p.experts):
        a, b = bad[e], bad[e + 1]
        if not 0 <= a < b <= p.pairs:
            continue
        rows, want, tol = slot_rows(p, e, a, b)
        assert (np.abs(y[rows] - want) <= tol).all(), f"expert {e}"
        skipped[rows] = False
    assert (y[skipped] == base.FILL).all()
