"""The 8-bit integer linear layer on the GPU against the 64-bit oracle.

The quantizers are compared bit for bit. The product differs from the 64-bit value by the roundings
of float(sum), sx * sw and their product (2^-24 each) and of the fp16 output (2^-11, 2^-25 below the
normal range).
"""
import numpy as np
import pytest

from oracle import block_oracle as B
from gpu_util import dev, host, lib, torch_mod

pytestmark = pytest.mark.gpu
REL, ABS = 2.0 ** -11 + 2.0 ** -22, 2.0 ** -25


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch_mod().cuda.is_available():
        pytest.skip("no CUDA device")
    lib()


def check_y(y, ref, what=""):
    y = host(y).astype(np.float64)
    bad = ~(np.abs(y - ref) <= REL * np.abs(ref) + ABS)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the rounding bound, first at {np.argwhere(bad)[0]}"


def same_bits(got, ref, what=""):
    a, b = np.asarray(got), np.asarray(ref)
    if a.dtype == np.float32:
        assert np.array_equal(np.isnan(a), np.isnan(b)), what
        a, b = np.nan_to_num(a), np.nan_to_num(b)
    assert np.array_equal(a, b), f"{what}: {(a != b).sum()} of {a.size} differ"


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 4096), (5, 4112), (7, 11008), (3, 28672), (2, 32784), (1, 131056)])
@pytest.mark.parametrize("scaled", [False, True])
def test_row_quantizers_bit_exact(M, K, scaled):
    P = lib()
    rng = np.random.default_rng(M * K)
    x = (rng.standard_normal((M, K)) * np.exp(rng.uniform(-6, 6, (M, 1)))).astype(np.float16)
    # multiples of the row maximum with quotients on and next to the half steps
    x[0, : K // 2] = (np.abs(x[0]).max() * rng.integers(-254, 255, K // 2) / 254).astype(np.float16)
    s = np.exp(rng.uniform(-3, 3, K)).astype(np.float32) if scaled else None
    sd = dev(s) if scaled else None
    for fn, divide in ((P.awq_quantize_tokens, True), (P.awq_quantize_channels, False)):
        q, step = fn(dev(x), sd)
        qr, sr = B.quantize_rows(B.scaled_rows(x, s, divide))
        same_bits(host(step), sr, "steps")
        same_bits(host(q), qr, "codes")


def test_row_quantizer_over_every_fp16_value():
    """All finite fp16 values as numerators of 64 different steps (subnormal to near the largest)."""
    P = lib()
    every = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    tops = np.linspace(1, 0x7BFF, 64).astype(np.uint16)
    x = np.zeros((64, 31744), np.float16)
    for i, t in enumerate(tops):
        row = np.where(np.arange(31744) <= t, every, -every[t])
        x[i] = np.where(np.arange(31744) % 2, row, -row)
    q, step = P.awq_quantize_tokens(dev(x))
    qr, sr = B.quantize_rows(x)
    same_bits(host(step), sr, "steps")
    same_bits(host(q), qr, "codes")


def test_rows_of_zeros_infinities_and_nans():
    P = lib()
    x = np.ones((6, 64), np.float16)
    x[1] = 0
    x[2, 5] = np.inf
    x[3, 7] = np.nan
    x[4, 3], x[4, 60] = -np.inf, np.nan
    x[5] = -0.0
    q, step = P.awq_quantize_tokens(dev(x))
    qr, sr = B.quantize_rows(x)
    same_bits(host(step), sr, "steps")
    same_bits(host(q), qr, "codes")
    w = np.random.default_rng(0).integers(-127, 128, (9, 64)).astype(np.int8)
    y = host(P.awq_w8a8_linear(q, step, dev(w), dev(np.full(9, 0.01, np.float32))))
    assert np.isnan(y[[2, 3, 4]]).all() and np.isfinite(y[[0, 1, 5]]).all() and (y[[1, 5]] == 0).all()


SHAPES = [(1, 1, 16), (1, 4096, 4096), (2, 77, 144), (16, 200, 4112), (17, 129, 400), (31, 12288, 512), (33, 513, 1040),
          (64, 1000, 2064), (65, 300, 128), (100, 4096, 4096), (129, 257, 656), (300, 5001, 272), (333, 640, 4112),
          (1, 40000, 256), (8, 28672, 1024), (512, 4096, 1024), (1500, 2000, 528), (2, 8, 28672), (4100, 136, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    P = lib()
    rng = np.random.default_rng([M, N, K])
    xq = rng.integers(-127, 128, (M, K)).astype(np.int8)
    wq = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sx = rng.uniform(0.5, 2, M).astype(np.float32) * 1e-2
    sw = rng.uniform(0.5, 2, N).astype(np.float32) * 1e-3
    y = P.awq_w8a8_linear(dev(xq), dev(sx), dev(wq), dev(sw))
    check_y(y, B.w8a8(xq, sx, wq, sw), f"M={M} N={N} K={K}")
    assert P.awq_poll_device_status() == P.AWQ_OK


@pytest.mark.parametrize("M", [1, 40, 200])
def test_largest_sum(M):
    """All codes -128 at the largest K: the sum is 2^31 - 2^18 and the int32 accumulator holds it."""
    P = lib()
    K, N = P.INT8_MAX_K, 24
    xq, wq = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    wq[1::2] = 127
    sx, sw = np.full(M, 2.0 ** -12, np.float32), np.full(N, 2.0 ** -12, np.float32)
    check_y(P.awq_w8a8_linear(dev(xq), dev(sx), dev(wq), dev(sw)), B.w8a8(xq, sx, wq, sw))


@pytest.mark.parametrize("M", [1, 24, 200])
def test_layer_from_float(M):
    """The whole path: statistic, fold, per-channel codes, per-token codes, product; and its error
    against the unquantized layer: rounding errors uniform over a step have variance step^2 / 12, so
    the squared error is expected at sum_mn (sx_m^2 |w'_n|^2 + sw_n^2 |x'_m|^2) / 12; at most twice that."""
    import workloads
    P = lib()
    x, W = workloads.random_case(7, M, 384, 1024)
    layer = P.AWQInt8Linear.from_float(dev(W), dev(x))
    y = layer(dev(x))
    s = host(layer.s)
    wf, xf = B.scaled_rows(W, s, False), B.scaled_rows(x, s, True)
    wq, sw = B.quantize_rows(wf)
    same_bits(host(layer.wq), wq, "weight codes")
    xq, sx = B.quantize_rows(xf)
    check_y(y, B.w8a8(xq, sx, wq, sw), "layer")
    plain = x.astype(np.float64) @ W.astype(np.float64).T
    sq = lambda v: (np.asarray(v, np.float64) ** 2).sum(-1)  # noqa: E731
    expected = (sq(sx) * sq(wf).sum() + sq(sw) * sq(xf).sum()) / 12
    assert sq((host(y) - plain).reshape(-1)) <= 2 * expected


@pytest.mark.parametrize("M", [1, 20, 150])
def test_captured_and_replayed_on_another_stream(M):
    torch, P = torch_mod(), lib()
    rng = np.random.default_rng(M)
    W = (rng.standard_normal((640, 1040)) * 0.02).astype(np.float16)
    layer = P.AWQInt8Linear.from_float(dev(W))
    x = torch.zeros((M, 1040), dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = layer(x)
        z = layer(x)
    for seed in range(3):
        v = np.random.default_rng([M, seed]).standard_normal((M, 1040)).astype(np.float16)
        x.copy_(dev(v))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        xq, sx = B.quantize_rows(v)
        ref = B.w8a8(xq, sx, *B.quantize_rows(W))
        check_y(y, ref, "replay")
        assert torch.equal(y, z)


def test_weights_quantized_right_before_the_product():
    """The product may start reading wq early; a quantizer call just before it must still be seen."""
    torch, P = torch_mod(), lib()
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 2048)).astype(np.float16)
    xq, sx = B.quantize_rows(x)
    xqd, sxd = dev(xq), dev(sx)
    out = (torch.empty((2048, 2048), dtype=torch.int8, device="cuda"), torch.empty(2048, device="cuda"))
    Ws = [(rng.standard_normal((2048, 2048)) * 0.02).astype(np.float16) for _ in range(3)]
    Wd = [dev(W) for W in Ws]
    ys = []
    for W in Wd:
        P.awq_quantize_channels(W, out=out)
        ys.append(P.awq_w8a8_linear(xqd, sxd, *out))
    for W, y in zip(Ws, ys):
        check_y(y, B.w8a8(xq, sx, *B.quantize_rows(W)))


def test_outputs_and_codes_past_2_31_elements():
    torch, P = torch_mod(), lib()
    M, N, K = 65600, 32768, 48
    rng = np.random.default_rng(9)
    wq = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sw = rng.uniform(0.5, 2, N).astype(np.float32) * 1e-3
    x = torch.randn((M, K), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).half()
    y = P.awq_w8a8_forward(x, dev(wq), dev(sw))
    assert y.numel() > 2 ** 31
    rows = [0, 1, 777, 65535, 65536, M - 1]
    xq, sx = B.quantize_rows(host(x[rows]))
    check_y(y[rows], B.w8a8(xq, sx, wq, sw))
    del y
    W = torch.zeros((M, N), dtype=torch.float16, device="cuda")
    tail = rng.standard_normal((3, N)).astype(np.float16)
    W[-3:] = dev(tail)
    q, step = P.awq_quantize_channels(W)
    qr, sr = B.quantize_rows(tail)
    same_bits(host(step[-3:]), sr)
    same_bits(host(q[-3:]), qr)
    assert not step[:-3].any() and not q[:-3].any()


def test_refusals_on_the_device():
    torch, P = torch_mod(), lib()
    layer = P.AWQInt8Linear.from_float(torch.zeros((32, 64), dtype=torch.float16, device="cuda"))
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    assert layer(x).shape == (4, 32) and P.awq_w8a8_forward(x, layer.wq, layer.sw).shape == (4, 32)
    for bad, error in ((x.t().contiguous().t(), ValueError), (x[:, :32], ValueError), (x[:0], ValueError), (x.float(), TypeError),
                       (x.cpu(), ValueError), (x[0], ValueError), (x.cpu().numpy(), TypeError)):
        with pytest.raises(error):
            layer(bad)
    with pytest.raises(ValueError, match="workspace"):
        layer(x, workspace=torch.empty(16, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        layer(x, y=torch.empty((4, 31), dtype=torch.float16, device="cuda"))


def test_two_streams_at_once():
    torch, P = torch_mod(), lib()
    rng = np.random.default_rng(21)
    work = []
    for M, N, K in ((1, 4096, 2048), (300, 1000, 528)):
        W, x = (rng.standard_normal((n, K)).astype(np.float16) for n in (N, M))
        work.append((P.AWQInt8Linear.from_float(dev(W)), dev(x), torch.cuda.Stream(), B.w8a8(*B.quantize_rows(x), *B.quantize_rows(W))))
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        for layer, x, s, ref in work:
            with torch.cuda.stream(s):
                out.append((layer(x), ref))
    torch.cuda.synchronize()
    for y, ref in out[-4:]:
        check_y(y, ref)
    assert all(torch.equal(a[0], b[0]) for a, b in zip(out[::2], out[2::2]))
    assert P.awq_poll_device_status() == P.AWQ_OK


# On 148 SMs these take the remaining combinations of token tile, weight rows per tile and K split: 16 to 64
# columns with tiles of 256 rows, 1 to 8 CTAs a tile, and 128 and 256 columns with K split 2 and 4 ways
FORMS = [(1, 130, 528), (1, 25, 528), (19, 25, 16), (19, 130, 1040), (19, 38001, 80), (19, 25, 1040), (41, 25, 16),
         (41, 38001, 144), (41, 25, 528), (41, 25, 1040), (70, 5001, 4112), (70, 2305, 8208), (199, 5001, 14352),
         (199, 2305, 14352)]


@pytest.mark.parametrize("M,N,K", FORMS)
def test_product_forms(M, N, K):
    test_product(M, N, K)


def test_two_streams_repeat_every_result():
    """One token and a prompt, queued on two streams: each result equals the one before it of the same layer."""
    torch, P = torch_mod(), lib()
    rng = np.random.default_rng(22)
    work = []
    for M, N, K in ((1, 4096, 2048), (300, 1000, 528)):
        W, x = (rng.standard_normal((n, K)).astype(np.float16) for n in (N, M))
        work.append((P.AWQInt8Linear.from_float(dev(W)), dev(x), torch.cuda.Stream(), B.w8a8(*B.quantize_rows(x), *B.quantize_rows(W))))
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        for layer, x, s, _ in work:
            with torch.cuda.stream(s):
                out.append(layer(x))
    torch.cuda.synchronize()
    assert P.awq_poll_device_status() == P.AWQ_OK
    for y, (_, _, _, ref) in zip(out[-2:], work):
        check_y(y, ref)
    assert all(torch.equal(a, b) for a, b in zip(out, out[2:]))


@pytest.mark.parametrize("side", ["tokens", "channels"])
def test_most_tokens_and_channels(side):
    """2^31 - 128 rows of one operand: a tile of 256 rows ends just below 2^31."""
    torch, P = torch_mod(), lib()
    top, K, few = 2 ** 31 - 128, 16, 300
    rng = np.random.default_rng(31)
    tail, one = (rng.integers(-127, 128, (n, K)).astype(np.int8) for n in (few, 1))
    step, unit = rng.uniform(0.5, 2, few).astype(np.float32) * 1e-3, np.full(1, 0.5, np.float32)
    big = torch.zeros((top, K), dtype=torch.int8, device="cuda")
    steps = torch.ones(top, device="cuda")
    big[-few:], steps[-few:] = dev(tail), dev(step)
    y = P.awq_w8a8_linear(*((big, steps, dev(one), dev(unit)) if side == "tokens" else (dev(one), dev(unit), big, steps)))
    assert P.awq_poll_device_status() == P.AWQ_OK
    y = y.view(-1)
    check_y(y[-few:], B.w8a8(tail, step, one, unit).reshape(-1))
    assert not y[:-few].any()
    del big, steps, y
    torch.cuda.empty_cache()
