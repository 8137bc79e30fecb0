"""Argument checks of the mixture-of-experts operators on the CPU: every call
here is refused (or has nothing to do) before any CUDA call."""
import numpy as np
import pytest

import gguf_quant_dequant_q4k_b200 as q4k
import moe_reference as ref

A = 1 << 20    # plausible device addresses, 1 MiB apart, never dereferenced


def route_args(**kw):
    a = dict(logits=A, ids=2 * A, weights=3 * A, offsets=4 * A, order=5 * A, n_tokens=3, n_experts=8, top_k=2)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(offsets=0), q4k.Q4K_ERR_NULL),
    (dict(logits=0), q4k.Q4K_ERR_NULL),
    (dict(ids=0), q4k.Q4K_ERR_NULL),
    (dict(weights=0), q4k.Q4K_ERR_NULL),
    (dict(order=0), q4k.Q4K_ERR_NULL),
    (dict(n_tokens=-1), q4k.Q4K_ERR_SHAPE),
    (dict(n_experts=0), q4k.Q4K_ERR_SHAPE),
    (dict(n_experts=257), q4k.Q4K_ERR_SHAPE),
    (dict(top_k=0), q4k.Q4K_ERR_SHAPE),
    (dict(top_k=9), q4k.Q4K_ERR_SHAPE),                       # more than the experts
    (dict(n_experts=64, top_k=17), q4k.Q4K_ERR_SHAPE),
    (dict(n_tokens=2 ** 30, top_k=2), q4k.Q4K_ERR_SHAPE),     # 2^31 pairs
    (dict(logits=A + 2), q4k.Q4K_ERR_ALIGN),
    (dict(order=5 * A + 1), q4k.Q4K_ERR_ALIGN),
    (dict(ids=A + 8), q4k.Q4K_ERR_OVERLAP),                   # inside logits
    (dict(order=3 * A + 4), q4k.Q4K_ERR_OVERLAP),             # inside weights
    (dict(offsets=2 * A), q4k.Q4K_ERR_OVERLAP),               # on ids
])
def test_route_refusals(kw, expect):
    assert q4k.q4k_moe_route_status(stream=0, **route_args(**kw)) == expect


def test_route_refuses_unknown_flags():
    lib = q4k.capi.library()
    assert lib.q4k_moe_route(A, 2 * A, 3 * A, 4 * A, 5 * A, 3, 8, 2, 2, None) == q4k.Q4K_ERR_SHAPE


GATED = ("q4k_moe_gemv_swiglu", "q4k_moe_gemm_swiglu_f16")
PLAIN = ("q4k_moe_gemv", "q4k_moe_gemm_f16")


def product_status(name, w=A, w2=2 * A, x=3 * A, offsets=4 * A, order=5 * A, y=6 * A, n_experts=4, n_pairs=6,
                   pairs_per_row=2, n=8, k=256):
    ws = (w, w2) if name in GATED else (w,)
    return getattr(q4k, name + "_status")(*ws, x, offsets, order, y, n_experts, n_pairs, pairs_per_row, n, k, stream=0)


@pytest.mark.parametrize("name", GATED + PLAIN)
@pytest.mark.parametrize("kw,expect", [
    (dict(w=0), q4k.Q4K_ERR_NULL),
    (dict(x=0), q4k.Q4K_ERR_NULL),
    (dict(offsets=0), q4k.Q4K_ERR_NULL),
    (dict(order=0), q4k.Q4K_ERR_NULL),
    (dict(y=0), q4k.Q4K_ERR_NULL),
    (dict(k=0), q4k.Q4K_ERR_SHAPE),
    (dict(k=100), q4k.Q4K_ERR_SHAPE),
    (dict(n=0), q4k.Q4K_ERR_SHAPE),
    (dict(n=-4), q4k.Q4K_ERR_SHAPE),
    (dict(n_experts=0), q4k.Q4K_ERR_SHAPE),
    (dict(n_experts=257), q4k.Q4K_ERR_SHAPE),
    (dict(n_experts=256, n=2 ** 23), q4k.Q4K_ERR_SHAPE),       # 2^31 rows
    (dict(n_pairs=-1), q4k.Q4K_ERR_SHAPE),
    (dict(pairs_per_row=-1), q4k.Q4K_ERR_SHAPE),
    (dict(w=A + 8), q4k.Q4K_ERR_ALIGN),
    (dict(x=3 * A + 8), q4k.Q4K_ERR_ALIGN),
    (dict(y=6 * A + 2), q4k.Q4K_ERR_ALIGN),
    (dict(offsets=4 * A + 2), q4k.Q4K_ERR_ALIGN),
    (dict(y=A + 144), q4k.Q4K_ERR_OVERLAP),                    # inside the matrices
    (dict(y=A + 3 * 8 * 144 + 16), q4k.Q4K_ERR_OVERLAP),       # inside the last expert's
    (dict(y=3 * A + 512), q4k.Q4K_ERR_OVERLAP),                # inside x
    (dict(y=5 * A), q4k.Q4K_ERR_OVERLAP),                      # on order
    (dict(n_pairs=0), q4k.Q4K_OK),                             # nothing to do
    (dict(n_pairs=0, x=0, order=0, y=0), q4k.Q4K_OK),
])
def test_product_refusals(name, kw, expect):
    assert product_status(name, **kw) == expect


@pytest.mark.parametrize("name", GATED)
def test_gated_refusals(name):
    assert product_status(name, w2=0) == q4k.Q4K_ERR_NULL
    assert product_status(name, w2=2 * A + 4) == q4k.Q4K_ERR_ALIGN
    assert product_status(name, y=2 * A + 16) == q4k.Q4K_ERR_OVERLAP


@pytest.mark.parametrize("name", ("q4k_moe_gemv", "q4k_moe_gemv_swiglu"))
def test_gemv_refuses_prompt_sizes(name):
    big = 1 << 30
    assert product_status(name, n_pairs=q4k.Q4K_MOE_GEMV_MAX_PAIRS + 1, y=big) == q4k.Q4K_ERR_UNSUPPORTED_M
    assert product_status(name, k=q4k.Q4K_MOE_GEMV_MAX_K + 256, y=big) == q4k.Q4K_ERR_SHAPE


def combine_args(**kw):
    a = dict(z=A, ids=2 * A, weights=3 * A, residual=4 * A, y=5 * A, n_tokens=3, top_k=2, hidden=8)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(z=0), q4k.Q4K_ERR_NULL),
    (dict(ids=0), q4k.Q4K_ERR_NULL),
    (dict(weights=0), q4k.Q4K_ERR_NULL),
    (dict(y=0), q4k.Q4K_ERR_NULL),
    (dict(n_tokens=-1), q4k.Q4K_ERR_SHAPE),
    (dict(hidden=0), q4k.Q4K_ERR_SHAPE),
    (dict(hidden=6), q4k.Q4K_ERR_SHAPE),
    (dict(top_k=0), q4k.Q4K_ERR_SHAPE),
    (dict(top_k=17), q4k.Q4K_ERR_SHAPE),
    (dict(n_tokens=2 ** 30), q4k.Q4K_ERR_SHAPE),
    (dict(z=A + 4), q4k.Q4K_ERR_ALIGN),
    (dict(y=5 * A + 8), q4k.Q4K_ERR_ALIGN),
    (dict(residual=4 * A + 4), q4k.Q4K_ERR_ALIGN),
    (dict(y=A + 16), q4k.Q4K_ERR_OVERLAP),                     # inside z
    (dict(y=4 * A + 16), q4k.Q4K_ERR_OVERLAP),                 # shifted against the residual
    (dict(y=3 * A), q4k.Q4K_ERR_OVERLAP),                      # on the weights
    (dict(n_tokens=0), q4k.Q4K_OK),
    (dict(n_tokens=0, z=0, ids=0, weights=0, y=0), q4k.Q4K_OK),
])
def test_combine_refusals(kw, expect):
    assert q4k.q4k_moe_combine_status(stream=0, **combine_args(**kw)) == expect


def test_raising_forms():
    for call in (lambda: q4k.q4k_moe_route(stream=0, **route_args(top_k=9)),
                 lambda: q4k.q4k_moe_gemv(A, 3 * A, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 100, stream=0),
                 lambda: q4k.q4k_moe_gemv_swiglu(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 100, stream=0),
                 lambda: q4k.q4k_moe_gemm_f16(A, 3 * A, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 100, stream=0),
                 lambda: q4k.q4k_moe_gemm_swiglu_f16(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 100, stream=0),
                 lambda: q4k.q4k_moe_combine(stream=0, **combine_args(hidden=6))):
        with pytest.raises(q4k.Q4KError) as e:
            call()
        assert e.value.status == q4k.Q4K_ERR_SHAPE


def test_binding_checks_tensors():
    """Element types and host tensors raise before the C call."""
    torch = pytest.importorskip("torch")
    f32, f16 = torch.zeros(4096), torch.zeros(4096, dtype=torch.float16)
    i64 = torch.zeros(64, dtype=torch.int64)
    with pytest.raises(TypeError):
        q4k.q4k_moe_route_status(stream=0, **route_args(ids=i64))
    with pytest.raises(TypeError):
        q4k.q4k_moe_gemm_f16_status(A, f32, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 256, stream=0)
    with pytest.raises(TypeError):
        q4k.q4k_moe_gemv_status(A, f16, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 256, stream=0)
    with pytest.raises(ValueError):
        q4k.q4k_moe_gemv_status(A, f32, 4 * A, 5 * A, 6 * A, 4, 6, 2, 8, 256, stream=0)
    with pytest.raises(TypeError):
        q4k.q4k_moe_combine_status(stream=0, **combine_args(y=f16))


# ------------------------------------------------------------------ the reference itself

def test_reference_route_and_group():
    logits = np.array([[0.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [np.nan, 1.0, -np.inf, -np.inf],
                       [np.inf, np.inf, 0.0, 1.0]], np.float32)
    ids, w, _ = ref.route(logits, 3, True)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [1, -1, -1], [0, 1, 3]]
    assert np.allclose(w[0], np.array([1, 1, np.exp(-2)]) / (2 + np.exp(-2)))
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [1, 0, 0]
    assert w[3].tolist() == [0.5, 0.5, 0.0]
    offsets, order = ref.group(ids, 4)
    assert offsets.tolist() == [0, 2, 5, 6, 7]
    assert order.tolist() == [2, 9, 0, 6, 10, 1, 11] + [-1] * 5
    _, w_all, _ = ref.route(logits, 1, False)
    assert np.allclose(w_all[0], 1 / (2 + np.exp(-2)))
