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


def test_route_of_the_most_tokens(q4k):
    """The largest batch the call accepts (2^31 - 1 tokens of one expert): token
    indexes plus a grid's stride pass 2^31. Every 1000003rd token, and the last, has
    no expert left."""
    t, gap = 2 ** 31 - 1, 1000003
    if torch.cuda.mem_get_info()[0] < 44e9:
        pytest.skip("needs 44 GB of device memory")
    logits = torch.zeros(t, device="cuda")
    logits[::gap] = -float("inf")
    logits[-1] = -float("inf")
    ids, order = (torch.full((t,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    w = torch.full((t,), 99.0, device="cuda")
    off = torch.full((2,), 99, dtype=torch.int32, device="cuda")
    q4k.q4k_moe_route(logits, ids, w, off, order, t, 1, 1)
    torch.cuda.synchronize()
    lost = torch.cat([torch.arange(0, t, gap, device="cuda"), torch.tensor([t - 1], device="cuda")])
    live = t - lost.numel()
    assert off.tolist() == [0, live]
    slot0 = 0
    for a in range(0, t, 2 ** 27):
        b = min(a + 2 ** 27, t)
        want = torch.zeros(b - a, dtype=torch.int32, device="cuda")
        want[lost[(lost >= a) & (lost < b)] - a] = -1
        assert torch.equal(ids[a:b], want)
        assert torch.equal(w[a:b], (want + 1).float())
        pairs = torch.nonzero(want == 0).view(-1) + a
        assert torch.equal(order[slot0:slot0 + pairs.numel()].long(), pairs)
        slot0 += pairs.numel()
    assert slot0 == live and bool((order[live:] == -1).all())
    del logits, ids, order, w, want, pairs
    torch.cuda.empty_cache()


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
