"""The mixture-of-experts operators through the C ABI on a B200, against the
64-bit reference of moe_reference.py (the products through the CPU oracle).

Tolerances: routing lists are equal; routing weights within the f32 error of
exp, sum and quotient (moe_reference.route); q4k_moe_gemv* within the q4k_gemv /
q4k_gemv_swiglu bounds, q4k_moe_gemm_f16 within oracle.gemm_f16_tolerance, the
fp16 output of q4k_moe_gemm_swiglu_f16 half a binary16 step (2^-11 relative,
2^-25 at the subnormals) beyond that; the combination within top_k + 1 f32
roundings of the sum of magnitudes."""
import os

import numpy as np
import pytest

import moe_reference as ref
import oracle
import q4k_synth
import special_blocks

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NTHREADS = max(1, len(os.sched_getaffinity(0)))
FILL = 7.25     # what output buffers hold before a call


@pytest.fixture(scope="module")
def q4k():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gguf_quant_dequant_q4k_b200 as lib
    return lib


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ routing

def gpu_route(q4k, logits, top_k, renorm, stream=None):
    t, e = logits.shape
    lg = dev(logits)
    ids = torch.full((t, top_k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((t, top_k), float("nan"), device="cuda")
    off = torch.full((e + 1,), 99, dtype=torch.int32, device="cuda")
    order = torch.full((t * top_k,), 99, dtype=torch.int32, device="cuda")
    q4k.q4k_moe_route(lg, ids, w, off, order, t, e, top_k, renorm=renorm, stream=stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), off.cpu().numpy(), order.cpu().numpy()


def check_route(got, logits, top_k, renorm, what=""):
    ids, w, off, order = got
    rids, rw, tol = ref.route(logits, top_k, renorm)
    assert np.array_equal(ids, rids), f"{what}: ids"
    err = np.abs(w.astype(np.float64) - rw)
    assert (err <= tol).all(), f"{what}: weights, worst {np.nanmax(err / tol):.3g}"
    roff, rorder = ref.group(rids, logits.shape[1])
    assert np.array_equal(off, roff), f"{what}: offsets"
    assert np.array_equal(order, rorder), f"{what}: order"


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,top_k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (7, 31, 3), (24, 64, 8), (33, 32, 16),
                                       (65, 33, 1), (130, 65, 5), (200, 128, 8), (257, 129, 4), (64, 256, 16),
                                       (1000, 16, 2), (2049, 100, 6), (5000, 255, 8), (50000, 16, 2)])
def test_route(q4k, t, e, top_k, renorm):
    rng = np.random.default_rng(t * 1000 + e)
    logits = rng.standard_normal((t, e)).astype(np.float32)
    logits = np.round(logits * 8) / 8                       # many ties
    logits += np.where(rng.random(e) < 0.2, 3, 0)[None, :]  # favoured experts
    logits = logits.astype(np.float32)
    check_route(gpu_route(q4k, logits, top_k, renorm), logits, top_k, renorm, f"{t}x{e} top {top_k}")


@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(q4k, renorm):
    rng = np.random.default_rng(5)
    t, e, top_k = 300, 40, 4
    logits = (rng.standard_normal((t, e)) * 30).astype(np.float32)
    logits[rng.random((t, e)) < 0.5] = -np.inf
    logits[rng.random((t, e)) < 0.05] = np.nan
    logits[rng.random((t, e)) < 0.05] = np.finfo(np.float32).min
    logits[rng.random((t, e)) < 0.02] = -0.0
    logits[10] = -np.inf
    logits[11] = np.nan
    logits[12, 1:] = -np.inf                # one expert left
    logits[13] = np.finfo(np.float32).min   # the lowest finite value is a value
    logits[14] = np.finfo(np.float32).max
    logits[15, 3:6] = np.inf
    logits[16] = 0.0
    logits[16, 7] = -0.0                    # equal to the other zeros
    got = gpu_route(q4k, logits, top_k, renorm)
    check_route(got, logits, top_k, renorm, "special values")
    assert not np.isnan(got[1]).any()


def test_route_all_to_one_expert_and_none(q4k):
    logits = np.full((700, 9), -np.inf, np.float32)
    check_route(gpu_route(q4k, logits, 2, True), logits, 2, True, "nobody")
    logits[:, 8] = 1.0
    check_route(gpu_route(q4k, logits, 2, True), logits, 2, True, "all to the last")
    logits[:] = 0.0
    check_route(gpu_route(q4k, logits, 2, True), logits, 2, True, "all equal")


def test_route_no_tokens(q4k):
    off = torch.full((9,), 99, dtype=torch.int32, device="cuda")
    q4k.q4k_moe_route(None, None, None, off, None, 0, 8, 2)
    torch.cuda.synchronize()
    assert (off.cpu().numpy() == 0).all()


# ------------------------------------------------------------------ products

class Problem:
    """One routed batch on the host and the device."""

    def __init__(self, tokens, experts, top_k, n, k, seed, pad=0, skew=0.7, mats=1, half=False, per_row=None, ids=None):
        rng = np.random.default_rng(seed)
        self.n, self.k, self.experts, self.half = n, k, experts, half
        self.ids = ref.random_ids(rng, tokens, experts, top_k, pad, skew) if ids is None else ids
        self.pairs = self.ids.size
        self.offsets, self.order = ref.group(self.ids, experts)
        self.per_row = top_k if per_row is None else per_row
        rows = self.pairs if self.per_row == 0 else -(-self.pairs // self.per_row)
        self.ws = [ref.expert_matrices(experts, n, k, seed + 1000 * (i + 1)) for i in range(mats)]
        x = q4k_synth.x_vectors(k, rows, seed + 7)
        if half:
            # weights are up to ~19 here: keep fp16 outputs in range
            x = x * np.float32(2.0 ** -6)
        self.x = oracle.floats_to_half(x) if half else x
        self.dw = [dev(w) for w in self.ws]
        self.dx = dev(self.x).view(torch.float16) if half else dev(self.x)
        self.doff, self.dorder = dev(self.offsets), dev(self.order)

    def sizes(self):
        return (self.experts, self.pairs, self.per_row, self.n, self.k)

    def out(self, dtype):
        return torch.full((self.pairs, self.n), FILL, dtype=dtype, device="cuda")

    def live(self):
        return int(self.offsets[-1])


def run_product(q4k, p, out=None, stream=None):
    gated = len(p.ws) == 2
    fn = {(False, False): q4k.q4k_moe_gemv, (False, True): q4k.q4k_moe_gemv_swiglu,
          (True, False): q4k.q4k_moe_gemm_f16, (True, True): q4k.q4k_moe_gemm_swiglu_f16}[(p.half, gated)]
    y = p.out(torch.float16 if p.half and gated else torch.float32) if out is None else out
    fn(*p.dw, p.dx, p.doff, p.dorder, y, *p.sizes(), stream=stream)
    return y


def reference(p):
    """(values, bounds) per slot."""
    if len(p.ws) == 1:
        if p.half:
            return ref.gemm(p.ws, p.x, p.offsets, p.order, p.per_row, p.n, p.k)
        return ref.gemv(p.ws, p.x, p.offsets, p.order, p.per_row, p.n, p.k, NTHREADS)
    part = [ref.gemm([w], p.x, p.offsets, p.order, p.per_row, p.n, p.k) if p.half else
            ref.gemv([w], p.x, p.offsets, p.order, p.per_row, p.n, p.k, NTHREADS) for w in p.ws]
    h, tol = ref.swiglu(part[0][0], part[1][0], part[0][1], part[1][1])
    return (h, tol + 2.0 ** -11 * (np.abs(h) + tol) + 2.0 ** -25) if p.half else (h, tol)


def check_product(p, y, what=""):
    torch.cuda.synchronize()
    y = y.float().cpu().numpy()
    want, tol = reference(p)
    live = p.live()
    if len(p.ws) == 2:      # rows in slot order
        got, untouched = y[:live], y[live:]
    else:                   # rows in pair order
        got = y[p.order[:live]]
        untouched = np.delete(y, p.order[:live], axis=0)
    assert (untouched == FILL).all(), f"{what}: rows without a pair were written"
    err = np.abs(got.astype(np.float64) - want[:live])
    bad = ~(err <= tol[:live])
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, worst "
                           f"{np.nanmax(err / tol[:live]):.3g}")


GEMV_CASES = [  # tokens, experts, top_k, n, k, pad
    (1, 1, 1, 1, 256, 0), (1, 4, 2, 3, 512, 0), (2, 3, 1, 15, 768, 0), (3, 8, 2, 16, 1024, 0), (5, 4, 3, 17, 2048, 1),
    (1, 8, 8, 130, 1536, 0), (9, 4, 2, 257, 2304, 2), (24, 16, 4, 96, 1280, 3), (33, 2, 2, 64, 512, 0),
    (70, 3, 1, 40, 256, 5), (1, 8, 2, 1000, 4096, 0), (4, 8, 2, 300, 14336, 0), (2, 2, 1, 70, 20736, 0),
    (16, 40, 6, 200, 1024, 1), (5, 2, 1, 17, 28672, 0), (4, 2, 1, 16, 43008, 0), (30, 3, 1, 1030, 2048, 0),
    (1, 3, 1, 5, 1024, 0), (2, 6, 2, 2400, 1280, 0), (500, 4, 3, 40, 256, 9), (10, 256, 16, 20, 256, 1), (9, 2, 1, 5000, 512, 0), (3, 2, 2, 777, 4096, 0),
]


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("tokens,experts,top_k,n,k,pad", GEMV_CASES)
def test_gemv_matches_oracle(q4k, tokens, experts, top_k, n, k, pad, mats):
    p = Problem(tokens, experts, top_k, n, k, 40 + tokens + n, pad, mats=mats)
    check_product(p, run_product(q4k, p), f"{tokens} tokens {experts}x{n}x{k}")


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("per_row", [0, 1, 3])
def test_gemv_row_maps(q4k, per_row, mats):
    """x rows by slot, by pair, and by three pairs at a time (their number no multiple of 3)."""
    p = Problem(11, 5, 2, 50, 512, 77, pad=2, mats=mats, per_row=per_row)
    check_product(p, run_product(q4k, p), f"per_row {per_row}")


GEMM_CASES = [
    (1, 1, 1, 1, 256, 0), (1, 4, 2, 3, 512, 0), (3, 3, 1, 15, 768, 0), (17, 2, 2, 63, 512, 1), (40, 8, 2, 64, 1024, 3),
    (100, 4, 3, 65, 256, 0), (129, 1, 1, 128, 512, 0), (300, 3, 2, 130, 768, 7), (257, 2, 1, 200, 1280, 0),
    (600, 4, 2, 257, 512, 11), (64, 40, 6, 100, 1024, 1), (260, 2, 2, 96, 4096, 0), (150, 2, 1, 70, 14336, 0),
    (1100, 2, 1, 129, 256, 0), (257, 1, 1, 300, 512, 0), (70, 256, 8, 30, 256, 3), (192, 1, 1, 260, 2304, 0), (193, 1, 1, 130, 1280, 1),
]


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("tokens,experts,top_k,n,k,pad", GEMM_CASES)
def test_gemm_matches_oracle(q4k, tokens, experts, top_k, n, k, pad, mats):
    p = Problem(tokens, experts, top_k, n, k, 90 + tokens + n, pad, mats=mats, half=True)
    check_product(p, run_product(q4k, p), f"{tokens} tokens {experts}x{n}x{k}")


@pytest.mark.parametrize("mats", [1, 2])
def test_gemv_long_rows_in_slot_order(q4k, mats):
    """Rows of x by slot where K is shared by the CTAs of a cluster."""
    p = Problem(9, 3, 2, 50, 14336, 79, pad=1, mats=mats, per_row=0)
    check_product(p, run_product(q4k, p), "long rows")


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("n,k", [(600, 1792), (2600, 256), (40, 512), (300, 14336)])
def test_gemv_uneven_groups(q4k, n, k, mats):
    """Experts of no, one to five, nine and seventeen vectors: groups of unequal cost shared out to the clusters,
    rows of an odd number of superblocks cut between warps; every row of every pair is written."""
    counts = [0, 5, 1, 0, 17, 2, 3, 9, 4, 0]
    ids = np.repeat(np.arange(10), counts).astype(np.int32)
    ids = np.random.default_rng(5).permutation(ids).reshape(-1, 1)
    p = Problem(len(ids), 10, 1, n, k, 82 + n, mats=mats, ids=ids)
    check_product(p, run_product(q4k, p), f"{n}x{k}")


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("k", [512, 14336])
def test_nobody_routed(q4k, k, mats, half):
    """Every pair without an expert: nothing is written, nothing faults."""
    p = Problem(6, 3, 2, 20, k, 80, mats=mats, half=half, ids=np.full((6, 2), -1, np.int32))
    y = run_product(q4k, p)
    torch.cuda.synchronize()
    assert (y == FILL).all()
    assert q4k.q4k_device_fault_flags() == 0


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_nonfinite_weights_stay_in_their_row(q4k, mats, half):
    """A row of W whose d is NaN, and one whose dmin is inf: that output feature
    of that expert's pairs is not finite, everything else keeps its bits."""
    p = Problem(40, 3, 1, 70, 768, 81, mats=mats, half=half)
    clean = run_product(q4k, p).float().cpu().numpy()
    w = p.ws[-1].copy()
    blocks = w.reshape(3, 70, 3, 144)
    blocks[1, 17, 2, 0:2] = (0x00, 0x7E)      # d = NaN
    blocks[1, 33, 0, 2:4] = (0x00, 0x7C)      # dmin = inf
    blocks[1, 33, 0, 8:12] = 0x3F             # its first mins are not 0
    p.dw[-1] = dev(w)
    y = run_product(q4k, p).float().cpu().numpy()
    slots = slice(int(p.offsets[1]), int(p.offsets[2]))
    rows = np.arange(p.pairs)[slots] if mats == 2 else p.order[slots]
    assert rows.size and not np.isfinite(y[np.ix_(rows, [17, 33])]).any()
    keep = np.ones(y.shape, bool)
    keep[np.ix_(rows, [17, 33])] = False
    assert np.array_equal(y[keep], clean[keep])


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("per_row", [0, 1, 3])
def test_gemm_row_maps(q4k, per_row, mats):
    p = Problem(211, 5, 2, 150, 512, 78, pad=20, mats=mats, half=True, per_row=per_row)
    check_product(p, run_product(q4k, p), f"per_row {per_row}")


def test_gemm_equals_the_mirror_product_on_integers(q4k):
    """Integer weights and activations: every partial sum is exact in f32, so
    the grouped product must equal the sum (a decode, layout or descriptor
    mistake cannot)."""
    n, k, experts, tokens = 140, 1024, 3, 333
    rng = np.random.default_rng(3)
    p = Problem(tokens, experts, 1, n, k, 5, half=True)
    blocks = np.empty((experts * n * (k // 256), 144), np.uint8)
    for i in range(len(blocks)):   # d = 1, dmin = 1: weight sc*q - m, |.| <= 45 - 20
        blocks[i] = oracle.pack(0x3C00, 0x3C00, rng.integers(0, 4, 8), rng.integers(0, 20, 8), rng.integers(0, 16, 256))
    p.ws = [blocks.reshape(experts, -1)]
    p.dw = [dev(p.ws[0])]
    p.x = rng.integers(-4, 5, (tokens, k)).astype(np.float16).view(np.uint16)
    p.dx = dev(p.x).view(torch.float16)
    y = run_product(q4k, p).cpu().numpy()
    want, _ = reference(p)
    assert np.array_equal(y[p.order].astype(np.float64), want)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("matrix", ["zero_quants", "near_cancelling"])
def test_cancelling_weights(q4k, matrix, half):
    """Weights that are differences of nearly equal terms."""
    n, k, experts, tokens = 33, 1024, 2, 6
    p = Problem(tokens, experts, 1, n, k, 6, half=half)
    w = (special_blocks.zero_quant_matrix(n, k) if matrix == "zero_quants"
         else special_blocks.near_cancelling_matrix(n, k, 8))
    p.ws = [np.stack([w, w])]
    p.dw = [dev(p.ws[0])]
    check_product(p, run_product(q4k, p), matrix)


@pytest.mark.parametrize("half", [False, True])
def test_unit_vectors_give_columns(q4k, half):
    """x = unit vectors: y is the decoded weight (f32 for the gemv's bound, the
    fp16 mirror's exactly)."""
    n, k, experts = 37, 512, 2
    p = Problem(k, experts, 1, n, k, 9, half=half, ids=np.arange(k, dtype=np.int32).reshape(k, 1) % 2)
    eye = np.eye(k, dtype=np.float32)
    p.x = oracle.floats_to_half(eye) if half else eye
    p.dx = dev(p.x).view(torch.float16) if half else dev(p.x)
    y = run_product(q4k, p).cpu().numpy()
    for e in range(experts):
        cols = np.arange(e, k, 2)
        if half:
            m = oracle.half_values(oracle.dequant_f16(p.ws[0][e], n, k))
            assert np.array_equal(y[cols], m.T[cols].astype(np.float32))
        else:
            m = oracle.dequant_f32(p.ws[0][e], n, k).astype(np.float64)
            assert (np.abs(y[cols] - m.T[cols]) <= oracle.tolerance(np.abs(m.T[cols]))).all()


def test_gemv_nonfinite_x_stays_in_its_row(q4k):
    """An inf or NaN in one row of x makes that row's outputs NaN (or inf) and
    changes no other row, whichever rows share a pass with it."""
    p = Problem(12, 2, 1, 40, 768, 12)
    clean = run_product(q4k, p).cpu().numpy()
    x = p.x.copy()
    x[3, 100] = np.nan
    x[8, 700] = np.inf
    p.dx = dev(x)
    y = run_product(q4k, p).cpu().numpy()
    bad = [3, 8]
    assert not np.isfinite(y[bad]).any()
    keep = [i for i in range(12) if i not in bad]
    assert np.array_equal(y[keep], clean[keep])


def test_gemm_nonfinite_x_stays_in_its_row(q4k):
    p = Problem(40, 2, 1, 40, 768, 13, half=True)
    clean = run_product(q4k, p).cpu().numpy()
    x = p.dx.clone()
    x[3, 100] = float("nan")
    p.dx = x
    y = run_product(q4k, p).cpu().numpy()
    assert np.isnan(y[3]).all()
    keep = [i for i in range(40) if i != 3]
    assert np.array_equal(y[keep], clean[keep])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_products_repeat_bit_for_bit(q4k, half, mats):
    p = Problem(50, 6, 2, 300, 2048, 15, pad=3, mats=mats, half=half)
    a = run_product(q4k, p)
    for _ in range(3):
        b = run_product(q4k, p)
        assert torch.equal(a, b)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_offsets_inside_larger_buffers(q4k, half, mats):
    """Operands at 16-byte offsets, y inside a guard band, on a side stream."""
    p = Problem(9, 3, 2, 70, 512, 17, mats=mats, half=half)
    dt = torch.float16 if half and mats == 2 else torch.float32
    size = p.pairs * p.n
    buf = torch.full((size + 64,), FILL, dtype=dt, device="cuda")
    xb = torch.zeros(p.dx.numel() + 32, dtype=p.dx.dtype, device="cuda")
    xoff = 16 // p.dx.element_size()
    xb[xoff:xoff + p.dx.numel()] = p.dx.reshape(-1)
    wb = [torch.zeros(w.numel() + 64, dtype=torch.uint8, device="cuda") for w in p.dw]
    for b, w in zip(wb, p.dw):
        b[16:16 + w.numel()] = w.reshape(-1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fn = (q4k.q4k_moe_gemm_swiglu_f16 if mats == 2 else q4k.q4k_moe_gemm_f16) if half else (
        q4k.q4k_moe_gemv_swiglu if mats == 2 else q4k.q4k_moe_gemv)
    fn(*(b.data_ptr() + 16 for b in wb), xb.data_ptr() + 16, p.doff.data_ptr(), p.dorder.data_ptr(),
       buf.data_ptr() + 32 * buf.element_size(), *p.sizes(), stream=s)
    s.synchronize()
    assert (buf[:32] == FILL).all() and (buf[32 + size:] == FILL).all()
    check_product(p, buf[32:32 + size].view(p.pairs, p.n), "offset buffers")


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_graph_capture_and_two_streams(q4k, half, mats):
    """Captured calls replay with new routing and inputs in the same buffers;
    two streams at once do not disturb each other."""
    p = Problem(20, 4, 2, 200, 1024, 18, mats=mats, half=half)
    q = Problem(20, 4, 2, 200, 1024, 19, mats=mats, half=half)
    dt = torch.float16 if half and mats == 2 else torch.float32
    y = p.out(dt)
    run_product(q4k, p, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_product(q4k, p, y)
    eager = run_product(q4k, q)
    y.fill_(FILL)
    for a, b in zip([p.dx, p.doff, p.dorder] + p.dw, [q.dx, q.doff, q.dorder] + q.dw):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, eager)

    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    p2 = Problem(13, 4, 2, 500, 768, 21, mats=mats, half=half)
    want = run_product(q4k, p2)
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(s1):
            outs.append((run_product(q4k, q, q.out(dt)), eager))
        with torch.cuda.stream(s2):
            outs.append((run_product(q4k, p2, p2.out(dt)), want))
    torch.cuda.synchronize()
    for got, wanted in outs:
        assert torch.equal(got, wanted)


FIRST_CALL_IN_CAPTURE = """
import sys
sys.path[:0] = [%r, %r]
import torch
import gguf_quant_dequant_q4k_b200 as q4k
import test_gpu_moe as t
p = t.Problem(20, 4, 2, 200, 1024, 18, mats=2, half=True)
d = t.Problem(20, 4, 2, 96, 1024, 19, mats=1, half=False)
y, z = p.out(torch.float16), d.out(torch.float32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    t.run_product(q4k, p, y)
    t.run_product(q4k, d, z)
g.replay()
g.replay()
t.check_product(p, y, "captured first call")
t.check_product(d, z, "captured first call")
print("captured ok")
"""


def test_first_call_of_a_process_is_captured():
    """Nothing the first call sets up (attributes, the workspace pool) breaks a capture."""
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_CAPTURE % (os.path.dirname(here), here)], timeout=300,
                         capture_output=True, text=True)
    assert out.returncode == 0 and "captured ok" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_bad_lists_are_skipped_and_flagged(q4k, half, mats):
    """Order entries outside the pairs: their slots are skipped, the others
    right; offsets that do not ascend within the pairs: the expert is skipped."""
    assert q4k.q4k_device_fault_flags() == 0
    p = Problem(30, 4, 1, 60, 512, 22, mats=mats, half=half)
    good = run_product(q4k, p).cpu().numpy()
    order = p.order.copy()
    order[4], order[11] = -5, p.pairs
    p.dorder = dev(order)
    y = run_product(q4k, p).cpu().numpy()
    assert q4k.q4k_device_fault_flags() == q4k.Q4K_FAULT_ROUTE_RANGE
    lost = [4, 11] if mats == 2 else [p.order[4], p.order[11]]
    keep = np.setdiff1d(np.arange(p.pairs), lost)
    assert (y[lost] == FILL).all() and np.array_equal(y[keep], good[keep])

    p.dorder = dev(p.order)
    for bad in (np.array([0, 8, 5, 20, 30]), np.array([0, 8, 15, 20, 31]), np.array([-1, 8, 15, 20, 30]),
                np.array([2 ** 31 - 1, 8, -2 ** 31, 20, 30])):
        offsets = bad.astype(np.int32)
        p.doff = dev(offsets)
        y = run_product(q4k, p).cpu().numpy()
        assert q4k.q4k_device_fault_flags() == q4k.Q4K_FAULT_ROUTE_RANGE
        rows = np.ones(p.pairs, bool)
        for e in range(4):
            a, b = int(offsets[e]), int(offsets[e + 1])
            if 0 <= a <= b <= p.pairs:
                rows[np.arange(a, b) if mats == 2 else p.order[a:b]] = False
        assert (y[rows] == FILL).all(), "an expert with bad offsets was computed"
    p.doff = dev(p.offsets)
    assert np.array_equal(run_product(q4k, p).cpu().numpy(), good)
    assert q4k.q4k_device_fault_flags() == 0


# ------------------------------------------------------------------ combination

@pytest.mark.parametrize("t,top_k,hidden,residual", [(1, 1, 4, False), (1, 2, 4096, True), (3, 3, 260, True),
                                                     (24, 8, 2048, True), (77, 4, 1028, False), (500, 16, 64, True),
                                                     (1200, 5, 512, False)])
def test_combine(q4k, t, top_k, hidden, residual):
    rng = np.random.default_rng(t + hidden)
    z = rng.standard_normal((t * top_k, hidden)).astype(np.float32)
    ids = rng.integers(-1, 6, (t, top_k)).astype(np.int32)
    w = rng.random((t, top_k)).astype(np.float32)
    res = rng.standard_normal((t, hidden)).astype(np.float32) if residual else None
    z[(ids < 0).reshape(-1)] = np.nan      # rows without an expert are never read
    y = torch.full((t, hidden), FILL, device="cuda")
    q4k.q4k_moe_combine(dev(z), dev(ids), dev(w), dev(res) if residual else None, y, t, top_k, hidden)
    torch.cuda.synchronize()
    live = (ids >= 0)[..., None]
    zz = np.where(live, z.reshape(t, top_k, hidden).astype(np.float64), 0.0) * w[..., None]
    want = zz.sum(1) + (res if residual else 0.0)
    tol = (top_k + 1) * 2.0 ** -24 * (np.abs(zz).sum(1) + (np.abs(res) if residual else 0.0)) + 1e-37
    err = np.abs(y.cpu().numpy().astype(np.float64) - want)
    assert (err <= tol).all()


def test_combine_in_place_on_the_residual(q4k):
    t, top_k, hidden = 19, 2, 300
    rng = np.random.default_rng(0)
    z = dev(rng.standard_normal((t * top_k, hidden)).astype(np.float32))
    ids = torch.zeros((t, top_k), dtype=torch.int32, device="cuda")
    w = torch.rand((t, top_k), device="cuda")
    res = dev(rng.standard_normal((t, hidden)).astype(np.float32))
    y = torch.empty_like(res)
    q4k.q4k_moe_combine(z, ids, w, res, y, t, top_k, hidden)
    q4k.q4k_moe_combine(z, ids, w, res, res, t, top_k, hidden)
    assert torch.equal(y, res)


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("prompt", [False, True])
def test_layer(q4k, prompt):
    """route -> gate/up with SwiGLU -> down -> combine, as a layer uses them,
    with padded tokens, against the same layer in 64 bits. The bound follows the
    error through the chain: h's own bound enters the down product through
    sum |w| |dh|, that sum through the routing weights."""
    tokens, experts, top_k, hidden, inter, pad = (150, 4, 2, 512, 768, 9) if prompt else (7, 8, 2, 512, 768, 2)
    rng = np.random.default_rng(31)
    logits = rng.standard_normal((tokens, experts)).astype(np.float32)
    logits[tokens - pad:] = -np.inf
    res = rng.standard_normal((tokens, hidden)).astype(np.float32)
    x = (rng.standard_normal((tokens, hidden)) * 2.0 ** -6).astype(np.float32)
    wg, wu, wd = (ref.expert_matrices(experts, *s, seed) for s, seed in
                  (((inter, hidden), 100), ((inter, hidden), 400), ((hidden, inter), 700)))
    pairs = tokens * top_k
    ids = torch.empty((tokens, top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((tokens, top_k), device="cuda")
    off = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(pairs, dtype=torch.int32, device="cuda")
    z = torch.full((pairs, hidden), float("nan"), device="cuda")
    y = torch.full((tokens, hidden), FILL, device="cuda")
    dx, dres = dev(x), dev(res)
    if prompt:
        xin = torch.empty((tokens, hidden), dtype=torch.float16, device="cuda")
        h = torch.full((pairs, inter), float("nan"), dtype=torch.float16, device="cuda")
    else:
        xin, h = dx, torch.full((pairs, inter), float("nan"), device="cuda")
    dwg, dwu, dwd, lg = dev(wg), dev(wu), dev(wd), dev(logits)

    def layer():
        q4k.q4k_moe_route(lg, ids, w, off, order, tokens, experts, top_k)
        if prompt:
            q4k.q4k_f32_to_f16(dx, xin, tokens * hidden)
            q4k.q4k_moe_gemm_swiglu_f16(dwg, dwu, xin, off, order, h, experts, pairs, top_k, inter, hidden)
            q4k.q4k_moe_gemm_f16(dwd, h, off, order, z, experts, pairs, 0, hidden, inter)
        else:
            q4k.q4k_moe_gemv_swiglu(dwg, dwu, xin, off, order, h, experts, pairs, top_k, inter, hidden)
            q4k.q4k_moe_gemv(dwd, h, off, order, z, experts, pairs, 0, hidden, inter)
        q4k.q4k_moe_combine(z, ids, w, dres, y, tokens, top_k, hidden)

    layer()
    torch.cuda.synchronize()
    rids, rw, wtol = ref.route(logits, top_k, True)
    assert np.array_equal(ids.cpu().numpy(), rids)
    roff, rorder = ref.group(rids, experts)
    live = int(roff[-1])
    xr = oracle.floats_to_half(x) if prompt else x
    mk = (lambda m, a, rows, per, n, k: ref.gemm([m], a, roff, rorder, per, n, k)) if prompt else (
        lambda m, a, rows, per, n, k: ref.gemv([m], a, roff, rorder, per, n, k, NTHREADS))
    (g, tg), (u, tu) = mk(wg, xr, tokens, top_k, inter, hidden), mk(wu, xr, tokens, top_k, inter, hidden)
    hr, ht = ref.swiglu(g, u, tg, tu)
    if prompt:
        ht = ht + 2.0 ** -11 * (np.abs(hr) + ht) + 2.0 ** -25
    want = res.astype(np.float64).copy()
    tol = 2.0 ** -22 * np.abs(want) + 1e-30
    for e in range(experts):
        if prompt:
            m = oracle.half_values(oracle.dequant_f16(wd[e], hidden, inter)).astype(np.float64)
        else:
            m = oracle.dequant_f32(wd[e], hidden, inter).astype(np.float64)
        for s in range(roff[e], roff[e + 1]):
            pr = rorder[s]
            t, j = pr // top_k, pr % top_k
            v = m @ hr[s]
            a = np.abs(m) @ (np.abs(hr[s]) + ht[s])
            dv = np.abs(m) @ ht[s] + (oracle.gemm_f16_tolerance(a, inter) if prompt else oracle.tolerance(a))
            want[t] += rw[t, j] * v
            tol[t] += (rw[t, j] + wtol[t, j]) * dv + wtol[t, j] * np.abs(v) + 4 * 2.0 ** -24 * rw[t, j] * np.abs(v)
    got = y.cpu().numpy().astype(np.float64)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol):.3g}"
    assert np.array_equal(got[tokens - pad:], res[tokens - pad:].astype(np.float64)), "padded tokens"
    assert live == int((rids >= 0).sum())

    # the same layer captured into a graph, replayed twice, gives the same bits
    first = y.clone()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        layer()
    for _ in range(2):
        y.fill_(FILL)
        gph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)


def test_moe_no_fault_flags(q4k):
    assert q4k.q4k_device_fault_flags() == 0
