"""The row quantizers, the 8-bit product, the residual norm and the experts in the bounds-checking build:
ragged cases of every form, no index check fires and every output equals the normal build's bit for bit."""
import pytest

from gpu_util import lib, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def both():
    if not torch_mod().cuda.is_available():
        pytest.skip("no CUDA device")
    P = lib()
    from weight_only_quantization_w4a16_b200 import build
    rel, dbg = P.load_library(), P.load_library(build.build(debug_bounds=True))

    def run(fn):
        torch = torch_mod()
        a = fn()
        try:
            P._lib = dbg
            b = fn()
            assert P.awq_poll_device_status() == P.AWQ_OK, "a bounds check fired"
        finally:
            P._lib = rel
        for x, y in zip(a, b):
            # bits, so that NaN equals itself
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    return P, run


def rand(seed, *shape):
    torch = torch_mod()
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (7, 8208), (5, 16400), (3, 32784), (601, 1040), (600, 2064), (601, 4112)])
@pytest.mark.parametrize("scaled", [False, True])
def test_row_quantizers(both, rows, K, scaled):
    P, run = both
    x = rand(1, rows, K).half()
    s = rand(2, K).abs() + 0.1 if scaled else None
    run(lambda: P.awq_quantize_tokens(x, s))
    run(lambda: P.awq_quantize_channels(x, s))


# every token tile, weight rows per tile, K split, odd and even N (on 148 SMs)
@pytest.mark.parametrize("M,N,K", [
    (1, 130, 528), (1, 25, 528), (19, 25, 16), (19, 130, 1040), (19, 38001, 80), (41, 25, 16), (41, 38001, 144), (41, 25, 1040),
    (70, 5001, 4112), (70, 2305, 8208), (199, 5001, 1040), (199, 2305, 4112), (333, 5000, 1040), (1025, 3001, 272)])
def test_product(both, M, N, K):
    torch = torch_mod()
    P, run = both
    codes = lambda seed, *shape: (rand(seed, *shape) * 50).clamp(-128, 127).to(torch.int8)  # noqa: E731
    xq, wq = codes(3, M, K), codes(4, N, K)
    sx, sw = rand(5, M).abs() * 1e-3, rand(6, N).abs() * 1e-3
    run(lambda: (P.awq_w8a8_linear(xq, sx, wq, sw),))


@pytest.mark.parametrize("M,K", [(1, 8), (5, 264), (3, 12296), (2, 32768), (600, 1032), (601, 4104), (593, 20488), (2400, 4104)])
@pytest.mark.parametrize("post,gate_rows,scaled", [(False, 0, False), (True, 1, True), (True, -1, False)])
def test_residual_norm(both, M, K, post, gate_rows, scaled):
    P, run = both
    y, r, w = rand(7, M, K).half(), rand(8, M, K).half(), rand(9, K).half()
    gate = None if gate_rows == 0 else rand(10, M if gate_rows < 0 else gate_rows, K).half()
    run(lambda: P.awq_residual_norm(y, r, w, post_weight=w if post else None, gate=gate, alpha=0.5,
                                    s=rand(11, K).abs() + 0.1 if scaled else None))


@pytest.mark.parametrize("T,E,top,K,I", [(1, 4, 2, 128, 128), (13, 6, 3, 640, 1408), (32, 40, 16, 128, 256), (5, 3, 3, 4480, 384)])
def test_experts(both, T, E, top, K, I):
    torch = torch_mod()
    P, run = both
    stack = lambda layers: tuple(torch.stack(t) for t in zip(*layers))  # noqa: E731
    gu = stack([P.awq_quantize_g128((rand(20 + e, 2 * I, K) * 0.05).half()) for e in range(E)])
    dn = stack([P.awq_quantize_g128((rand(70 + e, K, I) * 0.05).half()) for e in range(E)])
    layer = P.AWQMoE((rand(12, E, K) * 0.05).half(), gu, dn, I, top)
    x = rand(13, T, K).half()
    run(lambda: (layer(x),))
