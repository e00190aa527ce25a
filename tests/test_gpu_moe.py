"""The mixture-of-experts layer on the GPU against the 64-bit oracle, element by element within the
bound that the definition's roundings allow (oracle.block_oracle.moe), and within 1.5 2^-11 in
relative Frobenius norm: two independent roundings to fp16 (of h and of y), each of at most 2^-11
relative per element and about 0.4 of that in the mean square.
"""
import numpy as np
import pytest

from oracle import awq_oracle as O
from oracle import block_oracle as B
from gpu_util import dev, host, lib, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch_mod().cuda.is_available():
        pytest.skip("no CUDA device")
    lib()


def experts(rng, E, N, K):
    """E quantized layers: (packed arrays stacked, dequantized weights)."""
    packed, plain = [], []
    for _ in range(E):
        q, S, z = O.quantize_groups((rng.standard_normal((N, K)) * 0.05).astype(np.float16))
        qw, sc, zb = O.pack(q, S, z)
        packed.append((qw.view(np.int32), sc, zb))
        plain.append(O.dequantize(q, S, z).astype(np.float64))
    return tuple(np.stack(v) for v in zip(*packed)), np.stack(plain)


class Case:
    def __init__(self, T, E, top, K, I, renorm=True, hscale=False, seed=0):
        rng = np.random.default_rng([T, E, top, K, I, seed])
        self.x = rng.standard_normal((T, K)).astype(np.float16)
        self.router = (rng.standard_normal((E, K)) * 0.05).astype(np.float16)
        self.gu, self.gu_w = experts(rng, E, 2 * I, K)
        self.dn, self.dn_w = experts(rng, E, K, I)
        self.hs = np.exp(rng.uniform(-2, 2, (E, I))).astype(np.float32) if hscale else None
        self.top, self.renorm, self.I = top, renorm, I

    def layer(self):
        P = lib()
        return P.AWQMoE(dev(self.router), [dev(v) for v in self.gu], [dev(v) for v in self.dn], self.I, self.top,
                        self.renorm, None if self.hs is None else dev(self.hs))

    def reference(self, x=None):
        return B.moe(self.x if x is None else x, self.router, self.gu_w, self.dn_w, self.top, self.renorm, self.hs)

    def check(self, y, x=None, what=""):
        ref, bound, gap = self.reference(x)
        assert gap > 1e-4, "the oracle's choice of experts is too close to call for this test"
        y = host(y).astype(np.float64)
        bad = ~(np.abs(y - ref) <= bound)
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}"
        rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
        assert rel <= 1.5 * 2.0 ** -11, f"{what}: relative Frobenius error {rel:.2e}"


# (T, E, top, K, I): one token to the most, one group to many, odd group counts, one expert, all experts
SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 512, 1024), (1, 4, 4, 384, 640), (2, 16, 3, 1152, 128), (3, 64, 6, 256, 128),
          (5, 60, 4, 640, 384), (8, 8, 2, 2048, 512), (9, 8, 2, 512, 768), (16, 12, 3, 1152, 640), (17, 5, 5, 256, 256),
          (19, 12, 3, 1152, 640), (31, 3, 1, 384, 1408), (32, 8, 2, 1024, 512), (32, 1, 1, 128, 384),
          (32, 128, 8, 256, 128), (1, 512, 16, 128, 128), (32, 40, 16, 128, 128)]


@pytest.mark.parametrize("T,E,top,K,I", SHAPES)
@pytest.mark.parametrize("renorm,hscale", [(True, False), (False, True)])
def test_layer(T, E, top, K, I, renorm, hscale):
    c = Case(T, E, top, K, I, renorm, hscale)
    y = c.layer()(dev(c.x))
    c.check(y, what=f"T={T} E={E} top={top} K={K} I={I}")
    P = lib()
    assert P.awq_poll_device_status() == P.AWQ_OK


def test_all_tokens_choose_one_expert_and_repeat_bitwise():
    torch = torch_mod()
    c = Case(32, 6, 2, 512, 640)
    c.x = np.abs(c.x)
    c.router[2] = 0.05                       # every token's largest logit
    c.router[4] = 0.03
    layer = c.layer()
    y = layer(dev(c.x))
    assert set(B.route(c.x, c.router, 2, True)[0].reshape(-1)) == {2, 4}
    c.check(y)
    assert all(torch.equal(y, layer(dev(c.x))) for _ in range(3))


def test_ties_go_to_the_lowest_index():
    c = Case(7, 16, 3, 256, 128)
    c.router[:] = c.router[3]                # equal logits everywhere
    y = host(c.layer()(dev(c.x))).astype(np.float64)
    ref, bound, _ = c.reference()            # the oracle's stable order chooses experts 0, 1, 2
    assert (B.route(c.x, c.router, 3, True)[0] == [0, 1, 2]).all()
    assert (np.abs(y - ref) <= bound).all()


def test_non_finite_values_stay_with_their_tokens():
    c = Case(9, 8, 2, 384, 256)
    clean = host(c.layer()(dev(c.x)))
    x = c.x.copy()
    x[4, 17] = np.nan
    x[6, 300] = np.inf
    y = host(c.layer()(dev(x)))
    rest = [t for t in range(9) if t not in (4, 6)]
    assert np.array_equal(y[rest], clean[rest])
    assert np.isnan(y[4]).all() and not np.isfinite(y[6]).any()
    # an expert whose scales overflowed reaches only the tokens that chose it
    ids, _, gap = B.route(c.x, c.router, 2, True)
    assert gap > 1e-4
    bad = int(ids[0, 0])
    for arrays in (c.gu, c.dn):
        arrays[1][bad][:] = np.inf
    y = host(c.layer()(dev(c.x)))
    hit = (ids == bad).any(1)
    assert hit.any() and not hit.all()
    assert np.array_equal(y[~hit], clean[~hit]) and not np.isfinite(y[hit]).any()


def test_captured_calls_share_a_workspace_and_replay():
    torch, P = torch_mod(), lib()
    c, d = Case(5, 16, 4, 512, 384, False), Case(5, 8, 2, 256, 640)
    lc, ld = c.layer(), d.layer()
    need = max(P.load_library().awq_moe_workspace_bytes(5, 16, 512, 384, 4),
               P.load_library().awq_moe_workspace_bytes(5, 8, 256, 640, 2))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    xc, xd = dev(c.x), dev(d.x)
    lc(xc, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for layer, x in ((lc, xc), (ld, xd)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = layer(x, workspace=ws)
        graphs.append((g, y))
    for seed in range(3):
        for case, x, (g, y) in ((c, xc, graphs[0]), (d, xd, graphs[1])):
            v = np.random.default_rng([seed, 77]).standard_normal(case.x.shape).astype(np.float16)
            x.copy_(dev(v))
            g.replay()
            case.check(y, v, "replay")
    assert P.awq_poll_device_status() == P.AWQ_OK


def test_two_streams_at_once():
    torch = torch_mod()
    c, d = Case(4, 16, 4, 512, 384), Case(32, 8, 2, 512, 640)
    work = [(c, c.layer(), dev(c.x), torch.cuda.Stream()), (d, d.layer(), dev(d.x), torch.cuda.Stream())]
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        for case, layer, x, s in work:
            with torch.cuda.stream(s):
                out.append((case, layer(x)))
    torch.cuda.synchronize()
    assert lib().awq_poll_device_status() == lib().AWQ_OK
    for case, y in out[-4:]:
        case.check(y, what="two streams")
    for (_, a), (_, b) in zip(out[::2], out[2::2]):
        assert torch.equal(a, b)


def test_calls_back_to_back_with_early_launching_neighbours():
    """Calls queued without a wait between them, next to kernels that launch their successors early: the
    experts kernel's grid-wide barrier completes every time (the status word records a wait that ran out)."""
    torch, P = torch_mod(), lib()
    c, d = Case(1, 8, 2, 1024, 1024), Case(24, 16, 2, 512, 1024)
    lc, ld = c.layer(), d.layer()
    xc, xd = dev(c.x), dev(d.x)
    ones = torch.ones(1024, device="cuda")
    torch.cuda.synchronize()
    assert P.awq_poll_device_status() == P.AWQ_OK
    out = []
    for i in range(40):
        a = P.awq_scale_activations(xc, ones)
        out.append((lc(a), ld(xd)))
        if i % 4 == 0:
            lc(a)
    assert P.awq_poll_device_status() == P.AWQ_OK
    c.check(out[-1][0])
    d.check(out[-1][1])
    assert all(torch.equal(a, out[0][0]) and torch.equal(b, out[0][1]) for a, b in out)


def test_from_float_and_a_whole_block():
    """norm -> int8 layer -> norm with gate -> experts -> norm, each step against the oracle on the
    step's own inputs as the GPU computed them."""
    P = lib()
    rng = np.random.default_rng(11)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    T, K, I, E, top = 6, 512, 384, 8, 2
    calib = n(64, K).astype(np.float16)
    calib[:, 5] *= 20
    W = (n(K, K) * 0.05).astype(np.float16)
    router = (n(E, K) * 0.05).astype(np.float16)
    Wgu, Wdn = (n(E, 2 * I, K) * 0.05).astype(np.float16), (n(E, K, I) * 0.05).astype(np.float16)
    hs = np.exp(rng.uniform(-1, 1, (E, I))).astype(np.float32)
    w, post = (1 + 0.1 * n(K)).astype(np.float16), (1 + 0.1 * n(K)).astype(np.float16)
    gate = n(1, K).astype(np.float16)
    attn = P.AWQInt8Linear.from_float(dev(W), dev(calib))
    moe = P.AWQMoE.from_float(dev(router), dev(Wgu), dev(Wdn), top, dev(calib), h_scale=dev(hs))
    r = dev(n(T, K).astype(np.float16))
    y0 = dev(n(T, K).astype(np.float16))
    h1, x1 = P.awq_residual_norm(y0, r, dev(w))
    a = attn(x1)
    h2, x2 = P.awq_residual_norm(a, h1, dev(w), post_weight=dev(post), gate=dev(gate), alpha=0.5, s=moe.s)
    m = moe(x2, scaled=True)
    h3, x3 = P.awq_residual_norm(m, h2, dev(w))
    assert P.awq_poll_device_status() == P.AWQ_OK

    s = host(attn.s)
    xq, sx = B.quantize_rows(B.scaled_rows(host(x1), s))
    ref = B.w8a8(xq, sx, *B.quantize_rows(B.scaled_rows(W, s, False)))
    assert (np.abs(host(a) - ref) <= (2.0 ** -11 + 2.0 ** -22) * np.abs(ref) + 2.0 ** -25).all()
    deq = lambda V, f: O.dequantize(*O.quantize_groups(O.fold_weights(V, f))).astype(np.float64)  # noqa: E731
    sm = host(moe.s)
    folded = (router.astype(np.float32) * sm).astype(np.float16)
    ref, bound, gap = B.moe(host(x2), folded, np.stack([deq(v, sm) for v in Wgu]),
                            np.stack([deq(v, hs[e]) for e, v in enumerate(Wdn)]), top, True, hs)
    assert gap > 1e-4 and (np.abs(host(m) - ref) <= bound).all()
    # x2 already carries 1/s: scaling inside the layer gives the same
    _, plain = P.awq_residual_norm(a, h1, dev(w), post_weight=dev(post), gate=dev(gate), alpha=0.5)
    close = host(moe(plain)).astype(np.float64)
    assert np.linalg.norm(close - ref) <= 4e-3 * np.linalg.norm(ref)


def test_bounds_checked_build_agrees():
    torch, P = torch_mod(), lib()
    from weight_only_quantization_w4a16_b200 import build
    rel, dbg = P.load_library(), P.load_library(build.build(debug_bounds=True))
    for shape in ((1, 8, 2, 1152, 640), (9, 60, 4, 256, 384), (32, 5, 2, 512, 128)):
        c = Case(*shape)
        layer, x = c.layer(), dev(c.x)
        y = layer(x)
        try:
            P._lib = dbg
            z = layer(x)
            status = P.awq_poll_device_status()
        finally:
            P._lib = rel
        assert status == P.AWQ_OK and torch.equal(y, z)


def test_wait_budget_runs_out_then_recovers():
    """With a budget of 1 ns the waits give up, the kernels clean up and return; the next calls are right."""
    P = lib()
    c = Case(3, 8, 2, 2048, 1024)
    layer, x = c.layer(), dev(c.x)
    rng = np.random.default_rng(0)
    wq, xq = (rng.integers(-127, 128, (n, 4096)).astype(np.int8) for n in (2048, 600))
    ones = lambda n: dev(np.full(n, 1e-3, np.float32))  # noqa: E731
    wd, xd = dev(wq), dev(xq)
    for call in (lambda: layer(x), lambda: P.awq_w8a8_linear(xd, ones(600), wd, ones(2048)),
                 lambda: P.awq_w8a8_linear(xd[:4].contiguous(), ones(4), wd, ones(2048))):
        call()
        assert P.awq_poll_device_status() == P.AWQ_OK
        P.awq_debug_set_wait_budget_ns(1)
        try:
            call()
            status = P.awq_poll_device_status()
        finally:
            P.awq_debug_set_wait_budget_ns(0)
        assert status == P.AWQ_ERR_TIMEOUT
        assert P.awq_poll_device_status() == P.AWQ_OK
    c.check(layer(x), what="after a timeout")
    ref = B.w8a8(xq, np.full(600, 1e-3, np.float32), wq, np.full(2048, 1e-3, np.float32))
    y = host(P.awq_w8a8_linear(xd, ones(600), wd, ones(2048)))
    assert (np.abs(y - ref) <= (2.0 ** -11 + 2.0 ** -22) * np.abs(ref) + 2.0 ** -25).all()


def test_experts_past_32_bit_offsets():
    """512 experts whose packed gate/up layers take more than 4 GB: the first and the last are reached."""
    torch, P = torch_mod(), lib()
    E, K, I = 512, 2048, 4224
    rng = np.random.default_rng(3)
    stacks = []
    for N, Kin in ((2 * I, K), (K, I)):
        qb, sb, zb = P._packed_sizes_host(N, Kin)
        stacks.append((torch.zeros((E, qb // 4), dtype=torch.int32, device="cuda"),
                       torch.zeros((E, sb // 2), dtype=torch.float16, device="cuda"),
                       torch.zeros((E, zb), dtype=torch.uint8, device="cuda")))
    assert stacks[0][0][: E - 1].numel() * 4 > 2 ** 32
    gu_w, dn_w = {}, {}
    for e in (0, E - 1):
        for stack, (N, Kin), keep in ((stacks[0], (2 * I, K), gu_w), (stacks[1], (K, I), dn_w)):
            q, S, z = O.quantize_groups((rng.standard_normal((N, Kin)) * 0.03).astype(np.float16))
            for t, v in zip(stack, O.pack(q, S, z)):
                t[e] = dev(v.view(np.int32) if v.dtype == np.uint32 else v)
            keep[e] = O.dequantize(q, S, z).astype(np.float64)
    x = np.abs(rng.standard_normal((2, K))).astype(np.float16)
    x[1] = -x[1]
    router = np.zeros((E, K), np.float16)
    router[0], router[E - 1] = 0.01, -0.01          # token 0 chooses the first, token 1 the last
    y = P.awq_moe_w4a16(dev(x), dev(router), stacks[0], stacks[1], I, 1)
    assert P.awq_poll_device_status() == P.AWQ_OK
    for t, e in ((0, 0), (1, E - 1)):
        ref, bound, _ = B.moe(x[t:t + 1], router[[e]], gu_w[e][None], dn_w[e][None], 1, True)
        assert (np.abs(host(y)[t] - ref[0]) <= bound[0]).all()


def test_refusals_on_the_device():
    torch, P = torch_mod(), lib()
    c = Case(4, 8, 2, 256, 128)
    layer = c.layer()
    x = dev(c.x)
    with pytest.raises(ValueError, match="contiguous"):
        layer(torch.zeros((256, 4), dtype=torch.float16, device="cuda").t())
    with pytest.raises(TypeError, match="float16"):
        layer(x.float())
    with pytest.raises(ValueError, match="tokens"):
        layer(torch.zeros((33, 256), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        layer(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        layer(x.cpu())


def test_nan_logits_rank_below_every_number():
    for renorm in (True, False):
        c = Case(6, 40, 3, 256, 128, renorm)
        c.x = np.abs(c.x)
        c.router[5] = -0.05                  # far below the other logits: chosen by no token
        last = host(c.layer()(dev(c.x)))
        c.router[5] = np.nan
        y = host(c.layer()(dev(c.x)))
        if renorm:                           # the sum is over the chosen experts
            assert np.array_equal(y, last) and np.isfinite(y).all()
        else:
            assert np.isnan(y).all()
