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
