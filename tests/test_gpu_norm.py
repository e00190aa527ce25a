"""The residual update with its norms on the GPU against the 64-bit oracle.

Bound per value: the fp32 mean of K squares (per-thread chains of at most 32 terms, two halving
trees and K's reciprocal) is off by less than 48 2^-24 relative, its inverse root by half of that
plus 2^-23, and the products and the division by s add under 8 roundings of 2^-24; together below
2^-18 of t and of x. h adds t's error, a rounding of 2^-24 of h, and x carries h's error through the
norm (its own share of the mean included, at most sqrt(mean square) again). fp16 outputs add 2^-11,
or 2^-25 below the normal range.
"""
import numpy as np
import pytest

from oracle import block_oracle as B
from gpu_util import dev, host, lib, torch_mod

pytestmark = pytest.mark.gpu
E32, E16, SUB = 2.0 ** -18, 2.0 ** -11, 2.0 ** -25


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch_mod().cuda.is_available():
        pytest.skip("no CUDA device")
    lib()


def inputs(M, K, post, gates, scaled, seed=0):
    rng = np.random.default_rng([M, K, seed])
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    y = n(M, K)
    y[:, rng.permutation(K)[: max(1, K // 100)]] *= 20
    return dict(y=y.astype(np.float16), residual=(2 * n(M, K)).astype(np.float16), weight=(1 + 0.1 * n(K)).astype(np.float16),
                post_weight=(1 + 0.1 * n(K)).astype(np.float16) if post else None,
                gate=n(gates, K).astype(np.float16) if gates else None,
                s=np.exp(rng.uniform(-1.5, 1.5, K)).astype(np.float32) if scaled else None)


def to_dev(a):
    return {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in a.items()}


def check(got, a, what="", **kw):
    h, x, t = B.residual_norm(**a, **kw)
    eh = E32 * np.abs(t) + 2.0 ** -24 * np.abs(h)
    gain = np.abs(np.asarray(a["weight"], np.float64)) / (1.0 if a["s"] is None else a["s"])
    root = np.sqrt((h * h).mean(1, keepdims=True) + kw.get("eps", 1e-6))
    ex = E32 * np.abs(x) + gain / root * (eh + np.abs(h) / root * np.sqrt((eh * eh).mean(1, keepdims=True)))
    for out, ref, e, name in ((got[0], h, eh, "h"), (got[1], x, ex, "x")):
        if out is None:
            continue
        d = np.abs(host(out).astype(np.float64) - ref)
        bad = ~(d <= e * (1 + E16) + E16 * np.abs(ref) + SUB)
        assert not bad.any(), f"{what} {name}: {bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 264), (5, 4104), (2, 8192), (4, 11016), (2, 16384), (3, 16392),
                                 (1, 28672), (2, 32768), (300, 512)])
@pytest.mark.parametrize("post,gate,scaled", [(False, "none", False), (True, "one", True), (False, "row", True), (True, "row", False)])
def test_norm(M, K, post, gate, scaled):
    P = lib()
    a = inputs(M, K, post, {"none": 0, "one": 1, "row": M}[gate], scaled)
    check(P.awq_residual_norm(**to_dev(a), alpha=0.7, eps=1e-5), a, f"M={M} K={K}", alpha=0.7, eps=1e-5)


def test_gate_per_sequence_no_residual_and_no_h():
    P = lib()
    a = inputs(12, 1024, True, 3, True)
    check(P.awq_residual_norm(**to_dev(a), alpha=-1.5), a, "3 sequences of 4 rows", alpha=-1.5)
    a["residual"] = None
    h, x = P.awq_residual_norm(**to_dev(a), want_h=False)
    assert h is None
    check((h, x), a, "no residual")


def test_rows_of_zeros_and_large_values():
    P = lib()
    a = inputs(4, 512, True, 1, False)
    a["y"][1] = 0
    a["residual"][1] = 0                         # h = 0: x = 0
    a["y"][2] = 60000 * np.sign(a["y"][2].astype(np.float32)).astype(np.float16)
    a["residual"][3] = 30000                     # squares beyond the fp16 range
    got = P.awq_residual_norm(**to_dev(a))
    check(got, a, "zeros and large values")
    assert (host(got[0])[1] == 0).all() and (host(got[1])[1] == 0).all()
    a["y"][0, 3] = np.nan
    h, x = (host(v) for v in P.awq_residual_norm(**to_dev(a)))
    assert np.isnan(h[0]).all() and np.isnan(x[0]).all() and np.isfinite(x[1:]).all()
    a["post_weight"] = None
    h, x = (host(v) for v in P.awq_residual_norm(**to_dev(a)))
    assert np.isnan(h[0]).sum() == 1 and np.isnan(x[0]).all()


def test_zero_rows_without_eps_and_alpha_zero():
    P = lib()
    a = inputs(2, 64, False, 0, False)
    check(P.awq_residual_norm(**to_dev(a), alpha=0.0, eps=0.0), a, "alpha 0", alpha=0.0, eps=0.0)


def test_rows_do_not_depend_on_the_batch_and_repeat():
    torch, P = torch_mod(), lib()
    a = inputs(64, 4096, True, 64, True)
    d = to_dev(a)
    h, x = P.awq_residual_norm(**d)
    h2, x2 = P.awq_residual_norm(**d)
    assert torch.equal(h, h2) and torch.equal(x, x2)
    one = {k: v[5:6].contiguous() if k in ("y", "residual", "gate") else v for k, v in d.items()}
    h1, x1 = P.awq_residual_norm(**one)
    assert torch.equal(h1[0], h[5]) and torch.equal(x1[0], x[5])


def test_captured_chain_into_a_quantized_layer():
    """norm -> int8 layer -> norm in a CUDA graph, replayed with new inputs, equals the eager calls."""
    torch, P = torch_mod(), lib()
    K, M = 1024, 9
    rng = np.random.default_rng(3)
    W = (rng.standard_normal((K, K)) * 0.02).astype(np.float16)
    layer = P.AWQInt8Linear.from_float(dev(W), dev(rng.standard_normal((32, K)).astype(np.float16)))
    w = torch.ones(K, dtype=torch.float16, device="cuda")
    y, r = (torch.zeros((M, K), dtype=torch.float16, device="cuda") for _ in range(2))

    def block():
        h, x = P.awq_residual_norm(y, r, w)       # the layer divides by its own s
        return (h, *P.awq_residual_norm(layer(x), h, w, post_weight=w, alpha=0.5))

    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block()
    for seed in range(3):
        y.copy_(dev(np.random.default_rng([seed, 0]).standard_normal((M, K)).astype(np.float16)))
        r.copy_(dev(np.random.default_rng([seed, 1]).standard_normal((M, K)).astype(np.float16)))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, block()))


def test_rows_past_2_31_elements():
    torch, P = torch_mod(), lib()
    K, M = 32768, 65540
    y = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    r = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    assert y.numel() > 2 ** 31
    a = inputs(3, K, True, 0, True)
    y[-3:], r[-3:] = dev(a["y"]), dev(a["residual"])
    d = to_dev(a)
    h, x = P.awq_residual_norm(y, r, d["weight"], post_weight=d["post_weight"], s=d["s"])
    check((h[-3:], x[-3:]), a, "last rows")
    assert not h[:-3].any() and not x[:-3].any()


def test_refusals_on_the_device():
    torch, P = torch_mod(), lib()
    y = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    P.awq_residual_norm(y, y, w)
    for args, kw, error in (((y.t(), None, w), {}, ValueError), ((y, y[:2], w), {}, ValueError), ((y, y, w[:32]), {}, ValueError),
                            ((y.float(), None, w), {}, TypeError), ((y, y.cpu(), w), {}, ValueError),
                            ((y[:, :12].contiguous(), None, w[:12]), {}, ValueError), ((y, y, w), dict(gate=w), ValueError),
                            ((y, y, w), dict(eps=-1.0), ValueError), ((y, y, w), dict(alpha=float("inf")), ValueError),
                            ((y, y, w), dict(s=w), TypeError), ((y, y, w), dict(out=(None, None)), ValueError),
                            ((None, y, w), {}, TypeError), ((y, y, None), {}, TypeError)):
        with pytest.raises(error):
            P.awq_residual_norm(*args, **kw)


def test_gate_and_post_weight_refusals_on_the_device():
    torch, P = torch_mod(), lib()
    half = lambda *shape: torch.ones(shape, dtype=torch.float16, device="cuda")  # noqa: E731
    y = half(4, 64)
    for bad in (dict(gate=half(3, 64)), dict(gate=half(0, 64)), dict(gate=half(2, 72)), dict(gate=half(64)),
                dict(gate=half(2, 64).float()), dict(gate=half(64, 2).t()), dict(gate=half(2, 64).cpu()),
                dict(post_weight=half(63)), dict(post_weight=half(1, 64)), dict(post_weight=half(64).float())):
        with pytest.raises((ValueError, TypeError)):
            P.awq_residual_norm(y, y, half(64), **bad)


@pytest.mark.parametrize("M,K", [(1, 4096), (3, 12296), (600, 4104), (2400, 4104), (2, 32768)])
@pytest.mark.parametrize("post,gates", [(False, 0), (True, -1)])
def test_in_place(M, K, post, gates):
    """h in the residual's buffer and x in y's, or the other way round: the bits of the call with buffers of its own."""
    torch, P = torch_mod(), lib()
    gen = torch.Generator("cuda").manual_seed(M + K)
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=gen).half()  # noqa: E731
    y, r, w = rand(M, K), rand(M, K), rand(K)
    kw = dict(post_weight=w if post else None, gate=rand(M, K) if gates else None, alpha=0.7, s=rand(K).float().abs() + 0.1)
    h, x = P.awq_residual_norm(y, r, w, **kw)
    for swap in (False, True):
        a, b = y.clone(), r.clone()
        out = (a, b) if swap else (b, a)
        got = P.awq_residual_norm(a, b, w, out=out, **kw)
        assert got[0] is out[0] and torch.equal(out[0], h) and torch.equal(out[1], x)
    b = r.clone()
    _, x2 = P.awq_residual_norm(y, b, w, out=(b, torch.empty_like(y)), **kw)
    assert torch.equal(b, h) and torch.equal(x2, x)


def test_largest_inputs_and_alpha():
    """The largest alpha, gate, y and K: h is past fp16, and x is still the normalised row."""
    P = lib()
    K = P.NORM_MAX_K
    a = inputs(2, K, False, 1, False)
    sign = np.sign(a["y"].astype(np.float32))
    sign[sign == 0] = 1
    a["y"], a["gate"] = (65504 * sign).astype(np.float16), np.full((1, K), 65504, np.float16)
    h, x = P.awq_residual_norm(**to_dev(a), alpha=P.NORM_MAX_ALPHA)
    assert np.isinf(host(h)).all()
    check((None, x), a, "largest alpha", alpha=P.NORM_MAX_ALPHA)
