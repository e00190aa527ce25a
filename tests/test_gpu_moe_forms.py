"""The mixture-of-experts layer in every form that its kernel takes, against the definition in 64 bits on
the GPU: layers whose gate/up sums go over several stages, whose intermediate is cut into several parts, and
whose last units are drawn by whoever is done first; and the precision of the intermediate.

Tolerances. The output is rounded to fp16 once: half a step per element, 2^-11 relative at most, and in the
mean square at most a step's 1 / sqrt(12), 2^-11 / sqrt(3) of the value where the mantissa is smallest. The
rest is fp32: sums of products within 2^-18 of the sum of magnitudes, SiLU, p and the division by h_scale
within 2^-16, and the intermediate's integers within 2^-20 of the largest of 256 neighbours."""
import math

import numpy as np
import pytest

from oracle import awq_oracle as O
from gpu_util import dev, host, lib, torch_mod

pytestmark = pytest.mark.gpu

REL = 2.0 ** -11 / math.sqrt(3.0) + 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch_mod().cuda.is_available():
        pytest.skip("no CUDA device")
    lib()


def dequantize(packed, N, K):
    """One packed layer in 64 bits, code by code from the layout's index rule."""
    torch = torch_mod()
    words, S, Z = packed
    G2 = -(-(K // 128) // 2)
    n, k = torch.arange(N, device="cuda")[:, None], torch.arange(K, device="cuda")[None, :]
    T, h, r = n // 16, (n // 8) % 2, n % 8
    word = (T * 4 * G2 + k // 64) * 128 + (4 * r + (k // 16) % 4) * 4 + (k // 4) % 4
    q = (words[word] >> (4 * (h + 2 * ((k // 2) % 2) + 4 * (k % 2)))) & 15
    g = torch.arange(K // 128, device="cuda")[None, :]
    s = S[(T * 2 * G2 + g) * 16 + 2 * r + h].double()
    z = (Z[(T * 2 * G2 + g) * 8 + r].int() >> (4 * h)) & 15
    return ((q.view(N, -1, 128) - z[..., None]).double() * s[..., None]).view(N, K)


def cut(groups):
    """(strips per stage, chunks) of a layer with this many groups along K."""
    q = -(-groups // 2)
    shift = 4 if q <= 1 else 3 if q <= 2 else 2 if q <= 4 else 1 if q <= 8 else 0
    return 1 << shift, -(-q // 16)


class Layer:
    def __init__(self, T, E, top, K, I, renorm=True, h_scale=None, gu_std=0.05, dn_std=0.05, seed=0):
        torch, P = torch_mod(), lib()
        self.shape = T, E, top, K, I
        gen = torch.Generator("cuda").manual_seed(1000003 * seed + 7919 * T + 101 * E + top + K * 31 + I)
        rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        self.x, self.router = rand(T, K).half(), (rand(E, K) * 0.05).half()
        stack = lambda layers: tuple(torch.stack(t) for t in zip(*layers))  # noqa: E731
        self.gu = stack([P.awq_quantize_g128((rand(2 * I, K) * gu_std).half()) for _ in range(E)])
        self.dn = stack([P.awq_quantize_g128((rand(K, I) * dn_std).half()) for _ in range(E)])
        self.hs = None if h_scale is None else (rand(E, I).abs() + 0.5) * h_scale
        self.renorm = renorm
        self.layer = P.AWQMoE(self.router, self.gu, self.dn, I, top, renorm, self.hs)

    def __call__(self, **kw):
        return self.layer(self.x, **kw)

    def reference(self):
        """(y, bound, blocks) in 64 bits, an expert at a time; a block is up to 8 tokens of one expert."""
        torch = torch_mod()
        T, E, top, K, I = self.shape
        x = self.x.double()
        logits = x @ self.router.double().t()
        order = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = order[1][:, :top]
        if top < E:
            assert (order[0][:, top - 1] - order[0][:, top]).min() > 1e-4, "too close to call"
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e.gather(1, ids)
        p = p / (p if self.renorm else e).sum(1, keepdim=True)
        y, err, blocks = torch.zeros_like(x), torch.zeros_like(x), 0
        for k in range(E):
            rows, rank = (ids == k).nonzero(as_tuple=True)
            if len(rows) == 0:
                continue
            blocks += -(-len(rows) // 8)
            w = dequantize([t[k] for t in self.gu], 2 * I, K)
            gu, mag = x[rows] @ w.t(), x[rows].abs() @ w.abs().t()
            g, u = gu[:, :I], gu[:, I:]
            sig = torch.sigmoid(g)
            s = 1.0 if self.hs is None else self.hs[k].double()
            h = g * sig * u / s
            slope = (sig * (1 + g * (1 - sig))).abs()
            dh = 2.0 ** -18 * (slope * u.abs() * mag[:, :I] + (g * sig).abs() * mag[:, I:]) / s + 2.0 ** -16 * h.abs()
            for a in range(0, I, 256):
                dh[:, a:a + 256] += 2.0 ** -20 * h[:, a:a + 256].abs().amax(1, keepdim=True)
            w = dequantize([t[k] for t in self.dn], K, I)
            share = p[rows, rank][:, None]
            y[rows] += share * (h @ w.t())
            err[rows] += share * ((dh + 2.0 ** -18 * h.abs()) @ w.abs().t())
        return y, err + 2.0 ** -11 * (y.abs() + err) + 2.0 ** -25, blocks

    def check(self, y, ref=None, what=""):
        ref, bound, _ = ref or self.reference()
        bad = ~((y.double() - ref).abs() <= bound)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {bad.nonzero()[0].tolist()}"
        rel = float((y.double() - ref).norm() / ref.norm())
        # below fp16's normal range (h near 1e-8: 1e-8 p sqrt(8 512) 1000 = 5e-6) half a step is 2^-25
        limit = REL + 2.0 ** -25 * math.sqrt(ref.numel()) / float(ref.norm())
        assert rel <= limit, f"{what}: relative Frobenius error {rel:.3e}"


def test_the_layout_rule_agrees_with_the_oracle():
    rng = np.random.default_rng(0)
    q, S, z = O.quantize_groups((rng.standard_normal((48, 384)) * 0.05).astype(np.float16))
    qw, sc, zb = O.pack(q, S, z)
    w = dequantize((dev(qw.view(np.int32)), dev(sc), dev(zb)), 48, 384)
    assert np.array_equal(host(w), O.dequantize(q, S, z).astype(np.float64))


# ---------------------------------------------------------------------------- precision of the intermediate
@pytest.mark.parametrize("shape", [(1, 8, 2, 512, 1024), (5, 16, 4, 512, 384), (9, 8, 2, 384, 640), (32, 8, 2, 1024, 512)])
@pytest.mark.parametrize("h_scale", [None, 1.0])
def test_only_the_output_is_rounded(shape, h_scale):
    c = Layer(*shape, h_scale=h_scale)
    c.check(c())


@pytest.mark.parametrize("what,gu_std,dn_std,h_scale", [
    ("p h near 1e-5", 0.002, 1.0, None), ("h near 1e-8", 0.002, 1000.0, 1e5), ("h past 65504", 20.0, 1e-3, None)])
def test_small_and_large_intermediates(what, gu_std, dn_std, h_scale):
    """128 experts without renormalization: every p is near 1/100. h has fp32's range."""
    c = Layer(6, 128, 8, 512, 512, renorm=False, h_scale=h_scale, gu_std=gu_std, dn_std=dn_std)
    c.router.mul_(0.2)
    y = c()
    assert bool(y.isfinite().all())
    c.check(y, what=what)


# ---------------------------------------------------------------------------- forms
# (T, E, top, K, I), then whether the last units are drawn in phase 1 and in phase 2, and the chunks of K that
# they have there. 9 and 10 pairs of groups a chunk where a chunk holds up to 16; stages of one strip and of two.
FORMS = [((17, 2, 2, 4224, 4736), (True, True), (2, 2)), ((9, 4, 4, 8192, 4096), (True, True), (2, 1)),
         ((32, 4, 2, 4096, 14336), (True, True), (1, 4)), ((1, 3, 1, 6144, 2048), (False, False), (2, 1)),
         ((32, 4, 4, 2048, 4736), (True, True), (1, 2)), ((32, 4, 4, 8192, 2048), (True, True), (2, 1))]


def form(shape, blocks):
    """((drawn in phase 1, in phase 2), (chunks of each)) by the kernel's rules for this device."""
    _, _, _, K, I = shape
    ctas = torch_mod().cuda.get_device_properties(0).multi_processor_count
    (strips1, chunks1), (strips2, chunks2) = cut(K // 128), cut(I // 128)
    drawn = (blocks * (I // 16) >= 8 * ctas * strips1, blocks * chunks2 * (K // 32) >= 8 * ctas * strips2)
    return drawn, (chunks1, chunks2)


@pytest.mark.parametrize("shape,drawn,chunks", FORMS)
def test_forms(shape, drawn, chunks):
    torch, P = torch_mod(), lib()
    c = Layer(*shape)
    ref = c.reference()
    assert form(shape, ref[2]) == (drawn, chunks)
    y = c()
    c.check(y, ref)
    assert all(torch.equal(y, c()) for _ in range(5))      # whoever draws a unit, the sums are the same
    assert P.awq_poll_device_status() == P.AWQ_OK


def test_forms_with_scales_and_without_renormalization():
    c = Layer(17, 2, 2, 4224, 4736, renorm=False, h_scale=1.0)
    c.check(c())


def test_drawn_units_replayed_and_beside_another_stream():
    """Launches that draw units follow and overlap one another: each starts from the tickets that the last left."""
    torch, P = torch_mod(), lib()
    c, d = Layer(17, 2, 2, 4224, 4736), Layer(9, 4, 4, 8192, 4096)
    rc, rd = c.reference(), d.reference()
    yc, yd = c(), d()
    c.check(yc, rc)
    d.check(yd, rd)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zc, zd = c(), d()
    for _ in range(3):
        zc.zero_()
        zd.zero_()
        g.replay()
        assert torch.equal(zc, yc) and torch.equal(zd, yd)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(12):
        for layer, s in zip((c, d), streams):
            with torch.cuda.stream(s):
                out.append(layer())
    torch.cuda.synchronize()
    assert P.awq_poll_device_status() == P.AWQ_OK
    assert all(torch.equal(y, (yc, yd)[i % 2]) for i, y in enumerate(out))


def test_drawn_units_after_a_wait_that_ran_out():
    P = lib()
    c = Layer(17, 2, 2, 4224, 4736)
    ref = c.reference()
    c.check(c(), ref)
    for _ in range(3):
        P.awq_debug_set_wait_budget_ns(1)
        try:
            c()
            status = P.awq_poll_device_status()
        finally:
            P.awq_debug_set_wait_budget_ns(0)
        assert status == P.AWQ_ERR_TIMEOUT
        c.check(c(), ref, "after a timeout")
        assert P.awq_poll_device_status() == P.AWQ_OK


@pytest.mark.parametrize("shape", [s for s, _, _ in FORMS if s[4] <= 8192])
def test_forms_in_the_bounds_checked_build(shape):
    torch, P = torch_mod(), lib()
    from weight_only_quantization_w4a16_b200 import build
    rel, dbg = P.load_library(), P.load_library(build.build(debug_bounds=True))
    c = Layer(*shape)
    y = c()
    try:
        P._lib = dbg
        z = c()
        status = P.awq_poll_device_status()
    finally:
        P._lib = rel
    assert status == P.AWQ_OK and torch.equal(y, z)


def test_two_streams_repeat_every_result():
    """A few tokens and many, queued on two streams: each result equals the one before it of the same layer."""
    torch, P = torch_mod(), lib()
    c, d = Layer(4, 16, 4, 512, 384), Layer(32, 8, 2, 512, 640)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        for layer, s in zip((c, d), streams):
            with torch.cuda.stream(s):
                out.append(layer())
    torch.cuda.synchronize()
    assert P.awq_poll_device_status() == P.AWQ_OK
    c.check(out[-2])
    d.check(out[-1])
    assert all(torch.equal(a, b) for a, b in zip(out, out[2:]))
