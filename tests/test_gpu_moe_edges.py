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
    (small batches) and the two-launch path, wherever the tie lies."""
    rng = np.random.default_rng(t * 100 + e)
    zeros = np.where(rng.random((t, e)) < 0.5, np.float32(-0.0), np.float32(0.0))
    logits = np.where(rng.random((t, e)) < 0.7, zeros, rng.choice(np.float32([-1, 1, 2]), (t, e)))
    logits[0] = 0.0
    logits[0, 0] = -0.0                       # the first expert wins over every +0.0
    logits[-1] = np.where(np.arange(e) % 2 == 0, np.float32(-0.0), np.float32(0.0))    # across the cut at top_k
    logits = logits.astype(np.float32)
    assert np.signbit(logits[0, 0])
    base.check_route(base.gpu_route(q4k, logits, top_k, renorm), logits, top_k, renorm, f"{t}x{e} top {top_k}")


@pytest.mark.parametrize("t", [31, 32, 33])
@pytest.mark.parametrize("e,top_k", [(8, 2), (64, 8), (256, 16)])
def test_route_around_the_one_launch_limit(q4k, t, e, top_k):
    logits = np.random.default_rng(t + e).standard_normal((t, e)).astype(np.float32)
    logits[3] = -np.inf
    base.check_route(base.gpu_route(q4k, logits, top_k, True), logits, top_k, True, f"{t}x{e} top {top_k}")


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


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(4096, 2, 1, 20, 256), (256, 256, 16, 17, 512), (2048, 5, 2, 33, 4096)])
def test_gemv_of_the_most_pairs(q4k, tokens, experts, top_k, n, k, mats):
    assert tokens * top_k == q4k.Q4K_MOE_GEMV_MAX_PAIRS
    p = base.Problem(tokens, experts, top_k, n, k, 500 + tokens, pad=7, mats=mats)
    base.check_product(p, base.run_product(q4k, p), f"{tokens} tokens {experts}x{n}x{k}")


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mats", [1, 2])
def test_one_row_for_all_pairs(q4k, mats, half):
    """pairs_per_row beyond the pairs: x is one row."""
    p = base.Problem(150, 3, 1, 70, 768, 510, mats=mats, half=half, per_row=1000)
    assert p.dx.shape[0] == 1
    base.check_product(p, base.run_product(q4k, p), "one row")


# The 64-bit product on the device: every output of cases that are too large for the CPU oracle's loops.

def reference64(q4k, p):
    """(values, sums of magnitudes) per slot and matrix, float64 on the device, of the
    weights that q4k_dequant_f16 gives (test_gpu_prefill.py: the oracle's bits)."""
    rows = torch.from_numpy(np.ascontiguousarray(base.ref.x_row(p.order, p.per_row))).cuda()
    x = p.dx.double()
    out = []
    mirror = torch.empty((p.n, p.k), dtype=torch.float16, device="cuda")
    for w in p.dw:
        y, a = (torch.zeros((p.pairs, p.n), dtype=torch.float64, device="cuda") for _ in range(2))
        for e in range(p.experts):
            s0, s1 = int(p.offsets[e]), int(p.offsets[e + 1])
            if s0 == s1:
                continue
            q4k.q4k_dequant_f16(w[e].contiguous(), mirror, p.n, p.k)
            m = mirror.double()
            xe = x[rows[s0:s1]]
            y[s0:s1], a[s0:s1] = xe @ m.T, xe.abs() @ m.abs().T
        out.append((y, a))
    return out


def plain_tolerance(a, k):
    """q4k_moe_gemm_f16: the q4k_gemm_f16 bound of sums of at most 768 products
    (768 * 2^-23 sum|w x|, 1e-6), then one f32 addition, rounded to nearest, for each
    such sum (2^-24 of a partial sum, itself at most 1.0001 sum|w x|)."""
    return (min(k, 768) * 2.0 ** -23 + 1.0001 * -(-k // 768) * 2.0 ** -24) * a + 1e-6


def check64(q4k, p, y, what):
    got = y.double()
    live = int(p.offsets[-1])
    ref64 = reference64(q4k, p)
    if len(p.ws) == 1:
        (want, a), = ref64
        tol = plain_tolerance(a, p.k)
        got = got[torch.from_numpy(p.order[:live].astype(np.int64)).cuda()]
    else:
        (g, ag), (u, au) = ref64
        tg, tu = (p.k * 2.0 ** -23 * a + 1e-6 for a in (ag, au))
        s = g * torch.sigmoid(g)
        want = s * u
        tol = 1.1 * tg * (u.abs() + tu) + (s.abs() + 1.1 * tg) * tu + 1e-6 * want.abs() + 1e-30
        tol = tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25      # the rounding to binary16
        got = got[:live]
    err = (got - want[:live]).abs()
    bad = ~(err <= tol[:live])
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance"


MANY_TILES = [  # pairs per expert, rows of the plain and of the gate/up form, k: two or more tiles per pair of CTAs
    ([700, 13, 0, 487], 7300, 3700, 1280),                                 # large groups, blocks of up to 192 / 256 slots
    ([1025], 10100, 5000, 1024),                                           # one expert
    ([500, 130, 1, 0, 64, 33] + [20] * 10, 4900, 2500, 1280),              # small groups, one of them in four blocks
]


@pytest.mark.parametrize("counts", [[96], [97], [128], [129], [192], [193], [256], [257], [384], [385], [513], [500, 14], [0, 514]])
@pytest.mark.parametrize("mats", [1, 2])
def test_gemm_block_limits(q4k, counts, mats):
    """Numbers of pairs around the limits of the shapes and of their blocks."""
    ids = np.random.default_rng(7).permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32).reshape(-1, 1)
    p = base.Problem(len(ids), len(counts), 1, 290, 1280, 310 + len(ids), mats=mats, half=True, ids=ids)
    y = base.run_product(q4k, p)
    check64(q4k, p, y, f"{counts}")
    assert torch.equal(base.run_product(q4k, p), y)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("counts,n_plain,n_gated,k", MANY_TILES)
def test_gemm_many_tiles_per_pair(q4k, counts, n_plain, n_gated, k, mats):
    """Every pair of CTAs takes several tiles of several superblocks: accumulators,
    rings and decoded weights are reused across tiles. Every output is compared."""
    ids = np.random.default_rng(6).permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32).reshape(-1, 1)
    n = n_plain if mats == 1 else n_gated
    slots = (192 if mats == 1 else 256) if len(ids) > (128 if mats == 1 else 96) * len(counts) else 128
    tiles = sum(-(-c // slots) for c in counts) * -(-n // (256 if mats == 1 else 128))
    assert tiles > 2 * 74
    p = base.Problem(len(ids), len(counts), 1, n, k, 300 + n, mats=mats, half=True, ids=ids)
    y = base.run_product(q4k, p)
    check64(q4k, p, y, f"{len(ids)} pairs {len(counts)}x{n}x{k}")
    assert torch.equal(base.run_product(q4k, p), y)
    assert q4k.q4k_device_fault_flags() == 0


def test_gemm_long_sums_of_one_sign(q4k):
    """Sums of positive terms, where an accumulator that cuts off instead of rounding
    drifts one way, over rows of 1024 superblocks: the plain form keeps the bound of
    sums of 768 products."""
    n, k, experts, tokens = 24, 262144, 2, 5
    rng = np.random.default_rng(8)
    some = np.stack([base.oracle.pack(0x0C00, 0, rng.integers(8, 64, 8), np.zeros(8, int), rng.integers(1, 16, 256))
                     for _ in range(64)])                                  # d = 2^-12, no minimum
    p = base.Problem(tokens, experts, 1, n, 256, 24, half=True)
    p.k = k
    p.ws = [some[rng.integers(0, 64, experts * n * (k // 256))].reshape(experts, -1)]
    p.dw = [base.dev(p.ws[0])]
    p.x = rng.uniform(0.5, 1.0, (tokens, k)).astype(np.float16).view(np.uint16)
    p.dx = base.dev(p.x).view(torch.float16)
    check64(q4k, p, base.run_product(q4k, p), "long sums")


# ------------------------------------------------------------------ combination

@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("top_k", range(1, 17))
def test_combine_every_top_k(q4k, top_k, residual):
    """Tokens with all, some and no choices; rows of z without an expert hold NaN and
    are not read."""
    t, hidden = 37, 132
    rng = np.random.default_rng(top_k)
    ids = rng.integers(-1, 6, (t, top_k)).astype(np.int32)
    ids[0], ids[1] = -1, 0
    z = rng.standard_normal((t, top_k, hidden)).astype(np.float32)
    z[ids < 0] = np.nan
    w = rng.random((t, top_k)).astype(np.float32)
    res = rng.standard_normal((t, hidden)).astype(np.float32)
    y = torch.full((t, hidden), base.FILL, device="cuda")
    q4k.q4k_moe_combine(base.dev(z), base.dev(ids), base.dev(w), base.dev(res) if residual else None, y, t, top_k, hidden)
    live = (ids >= 0)[..., None]
    terms = np.where(live, z, 0).astype(np.float64) * np.where(live, w[..., None], 0)
    start = res.astype(np.float64) if residual else np.zeros((t, hidden))
    # each fma rounds once: half a step, 2^-24, of a partial sum of at most the sum of magnitudes
    tol = top_k * 2.0 ** -24 * 1.0001 * (np.abs(start) + np.abs(terms).sum(1)) + 1e-37
    err = np.abs(y.cpu().numpy().astype(np.float64) - (start + terms.sum(1)))
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol):.3g}"
    assert np.array_equal(y[0].cpu().numpy(), start[0].astype(np.float32))


# ------------------------------------------------------------------ large buffers, graphs, threads

def device_weights(experts, n, k, seed):
    """Random superblocks made on the device: d = 2^-12, dmin = 2^-9, other bytes at random."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    w = torch.randint(0, 256, (experts, n * (k // 256), 144), dtype=torch.uint8, device="cuda", generator=gen)
    w[..., 0:4] = torch.tensor([0x00, 0x0C, 0x00, 0x18], dtype=torch.uint8, device="cuda")
    return w


@pytest.mark.parametrize("name", ["gemv", "gemv_swiglu", "gemm", "gemm_swiglu"])
def test_weights_beyond_4_gib(q4k, name):
    """Experts whose matrices lie behind 2^32 bytes of the operand."""
    experts, n, k = 160, 14336, 4096
    if torch.cuda.mem_get_info()[0] < 16e9:
        pytest.skip("needs 16 GB of device memory")
    half, gated = name.startswith("gemm"), name.endswith("swiglu")
    w = device_weights(experts, n, k, 1)
    assert w.numel() > 2 ** 32 and (experts - 1) * n * (k // 256) * 144 > 2 ** 32
    ids = np.array([159, 0, 158, 159, 127, 159], np.int32).reshape(-1, 1)     # 127: across 2^32
    off, order = base.ref.group(ids, experts)
    x = torch.randn(6, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) / 64
    x = x.half() if half else x
    y = torch.full((6, n), base.FILL, device="cuda", dtype=torch.float16 if half and gated else torch.float32)
    fn = getattr(q4k, "q4k_moe_" + name + ("_f16" if half else ""))
    fn(*([w, w] if gated else [w]), x, base.dev(off), base.dev(order), y, experts, 6, 1, n, k)
    m16 = torch.empty((n, k), dtype=torch.float16, device="cuda")
    m32 = torch.empty((n, k), device="cuda")
    for slot, pair in enumerate(order):
        e = int(ids[pair, 0])
        if half:
            q4k.q4k_dequant_f16(w[e], m16, n, k)
        else:
            q4k.q4k_dequant_f32(w[e], m32, n, k)
        m, xr = (m16 if half else m32).double(), x[int(pair)].double()
        v, a = m @ xr, m.abs() @ xr.abs()
        tol = plain_tolerance(a, k) if half and not gated else k * 2.0 ** -23 * a + 1e-6 if half else 1e-4 * a + 1e-6
        if gated:
            s = v * torch.sigmoid(v)
            tol = 1.1 * tol * (v.abs() + tol) + (s.abs() + 1.1 * tol) * tol + 1e-6 * (s * v).abs() + 1e-30
            v = s * v
            if half:
                tol = tol + 2.0 ** -11 * (v.abs() + tol) + 2.0 ** -25
        got = y[slot if gated else int(pair)].double()
        assert bool(((got - v).abs() <= tol).all()), f"expert {e}"
    assert q4k.q4k_device_fault_flags() == 0


@pytest.mark.parametrize("mats", [1, 2])
def test_outputs_beyond_2_31_elements(q4k, mats):
    """More than 2^31 outputs: rows at the start, around 2^31 elements and at the end."""
    pairs, n, k = 70001, 31000, 256
    if torch.cuda.mem_get_info()[0] < 16e9:
        pytest.skip("needs 16 GB of device memory")
    assert pairs * n > 2 ** 31
    ids = (np.arange(pairs, dtype=np.int32) % 2).reshape(-1, 1)
    off, order = base.ref.group(ids, 2)
    ws = [device_weights(2, n, k, 3 + i) for i in range(mats)]
    x = (torch.randn(pairs, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) / 8).half()
    y = torch.full((pairs, n), base.FILL, device="cuda", dtype=torch.float16 if mats == 2 else torch.float32)
    fn = q4k.q4k_moe_gemm_swiglu_f16 if mats == 2 else q4k.q4k_moe_gemm_f16
    fn(*ws, x, base.dev(off), base.dev(order), y, 2, pairs, 1, n, k)
    mirror = torch.empty((n, k), dtype=torch.float16, device="cuda")
    at = 2 ** 31 // n
    for row in (0, 1, at - 1, at, at + 1, pairs - 2, pairs - 1):
        pair = int(order[row]) if mats == 2 else row
        xr, vs, ts = x[pair].double(), [], []
        for w in ws:
            q4k.q4k_dequant_f16(w[pair % 2], mirror, n, k)
            m = mirror.double()
            vs.append(m @ xr)
            ts.append(plain_tolerance(m.abs() @ xr.abs(), k))
        v, tol = vs[0], ts[0]
        if mats == 2:
            s = v * torch.sigmoid(v)
            tol = 1.1 * ts[0] * (vs[1].abs() + ts[1]) + (s.abs() + 1.1 * ts[0]) * ts[1] + 1e-6 * (s * vs[1]).abs() + 1e-30
            v = s * vs[1]
            tol = tol + 2.0 ** -11 * (v.abs() + tol) + 2.0 ** -25
        assert bool(((y[row].double() - v).abs() <= tol).all()), f"row {row}"
    assert bool((y[:, 0] != base.FILL).all()) and bool((y[:, n - 1] != base.FILL).all())
    del x, y
    torch.cuda.empty_cache()


def test_combine_beyond_2_31_elements(q4k):
    t, top_k, hidden = 70001, 8, 4096
    if torch.cuda.mem_get_info()[0] < 16e9:
        pytest.skip("needs 16 GB of device memory")
    z = torch.randn(t * top_k, hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    assert z.numel() > 2 ** 31
    ids = torch.zeros((t, top_k), dtype=torch.int32, device="cuda")
    w = torch.rand((t, top_k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    y = torch.full((t, hidden), float("nan"), device="cuda")
    q4k.q4k_moe_combine(z, ids, w, None, y, t, top_k, hidden)
    at = 2 ** 31 // (hidden * top_k)
    for rows in (slice(0, 3), slice(at - 2, at + 2), slice(t - 3, t)):
        terms = z.view(t, top_k, hidden)[rows].double() * w[rows].double().unsqueeze(-1)
        tol = top_k * 2.0 ** -24 * 1.0001 * terms.abs().sum(1) + 1e-37
        assert bool(((y[rows].double() - terms.sum(1)).abs() <= tol).all())
    assert not bool(torch.isnan(y).any())
    del z, y
    torch.cuda.empty_cache()


def test_captured_products_at_once(q4k):
    """Two captured graphs whose calls copy x into a workspace, replayed on two streams
    at once, beside eager calls on a third: each has its own rows."""
    problems = [base.Problem(300 + 50 * i, 4, 2, 500, 1024, 400 + i, mats=2, half=True) for i in range(3)]
    want = [base.run_product(q4k, p) for p in problems]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = []
    for p, y in zip(problems[:2], outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            base.run_product(q4k, p, y)
            base.run_product(q4k, p, y)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for y in outs:
            y.fill_(base.FILL)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            base.run_product(q4k, problems[2], outs[2], stream=streams[2])
        torch.cuda.synchronize()
        for y, w in zip(outs, want):
            assert torch.equal(y, w)


def test_calls_of_several_threads(q4k):
    """Host threads with a stream each."""
    from concurrent.futures import ThreadPoolExecutor
    problems = [base.Problem(40, 4, 2, 300, 1024, 410 + i, mats=1 + i % 2, half=i >= 2) for i in range(4)]
    want = [base.run_product(q4k, p) for p in problems]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        outs = [torch.full_like(want[i], base.FILL) for _ in range(20)]
        torch.cuda.synchronize()
        for y in outs:
            base.run_product(q4k, problems[i], y, stream=s)
        s.synchronize()
        return all(torch.equal(y, want[i]) for y in outs)

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))


def test_no_memory_for_the_workspace(q4k):
    """A call whose copy of x no device holds (2^28 pairs of one row) is refused with
    the allocation's error, and the calls after it are answered."""
    if torch.cuda.mem_get_info()[0] < 8e9:
        pytest.skip("needs 8 GB of device memory")
    p = base.Problem(40, 4, 2, 300, 1024, 420, half=True)
    want = base.run_product(q4k, p)
    pairs, k = 2 ** 28, 2048
    assert pairs * k * 2 > 1e12
    w = device_weights(1, 1, k, 7)
    x = torch.zeros((1, k), dtype=torch.float16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    order = torch.full((pairs,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((pairs, 1), base.FILL, device="cuda")
    status = q4k.q4k_moe_gemm_f16_status(w, x, off, order, y, 1, pairs, pairs, 1, k)
    assert status == q4k.Q4K_ERR_CUDA and q4k.q4k_last_cuda_error() == 2      # cudaErrorMemoryAllocation
    assert torch.equal(base.run_product(q4k, p), want)
    torch.cuda.synchronize()
    assert bool((y == base.FILL).all())


def test_a_refused_allocation_is_not_the_next_call_s_error(q4k):
    """The dense calls look for a launch error of their own; what an earlier call has
    reported is not one."""
    pairs, k = 2 ** 28, 2048
    if torch.cuda.mem_get_info()[0] < 8e9:
        pytest.skip("needs 8 GB of device memory")
    w = device_weights(1, 2, k, 9)
    x = torch.zeros((1, k), dtype=torch.float16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    order = torch.full((pairs,), -1, dtype=torch.int32, device="cuda")
    y = torch.empty((pairs, 1), device="cuda")
    out = torch.empty((2, k), device="cuda")
    for _ in range(2):
        assert q4k.q4k_moe_gemm_f16_status(w, x, off, order, y, 1, pairs, pairs, 1, k) == q4k.Q4K_ERR_CUDA
        assert q4k.q4k_dequant_f32_status(w, out, 2, k) == q4k.Q4K_OK
    torch.cuda.synchronize()


def test_longest_row_of_the_gated_gemm(q4k):
    """No wait gives up on the longest row that is accepted."""
    n, k = 2, q4k.Q4K_MOE_GEMM_SWIGLU_MAX_K
    w = device_weights(1, n, k, 8)
    x = torch.zeros((1, k), dtype=torch.float16, device="cuda")
    off, order = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [0]))
    y = torch.full((1, n), base.FILL, dtype=torch.float16, device="cuda")
    q4k.q4k_moe_gemm_swiglu_f16(w, w, x, off, order, y, 1, 1, 1, n, k)
    torch.cuda.synchronize()
    assert q4k.q4k_device_fault_flags() == 0 and bool((y == 0).all())
