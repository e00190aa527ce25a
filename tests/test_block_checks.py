"""Argument checks of the 8-bit linear layer and the residual norm, on the CPU (no device call is made)."""
import ctypes

import pytest
import torch

import weight_only_quantization_w4a16_b200 as P

V = ctypes.c_void_p
A, MIS = 0x10000, 0x10008    # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def lib():
    from weight_only_quantization_w4a16_b200 import build as B
    B.build()
    return P.load_library()


def test_row_quantizers_refuse_before_any_device_call(lib):
    for fn in (lib.awq_quantize_tokens, lib.awq_quantize_channels):
        assert fn(None, None, 1, 16, V(A), V(A), None) == 1
        assert fn(V(A), None, 1, 16, None, V(A), None) == 1
        assert fn(V(A), None, 1, 16, V(A), None, None) == 1
        for rows, K in ((0, 16), (-1, 16), (1, 0), (1, 8), (1, 24), (1, 131072), (1, -16)):
            assert fn(V(A), None, rows, K, V(A), V(A), None) == 1
        assert fn(V(MIS), None, 1, 16, V(A), V(A), None) == 3
        assert fn(V(A), V(MIS), 1, 16, V(A), V(A), None) == 3
        assert fn(V(A), None, 1, 16, V(MIS), V(A), None) == 3
        assert fn(V(A), None, 1, 16, V(A), V(A + 2), None) == 3


def test_w8a8_refuses_before_any_device_call(lib):
    fn = lib.awq_w8a8_linear
    for i in range(5):
        args = [V(A)] * 5
        args[i] = None
        assert fn(*args, 1, 1, 16, None) == 1
    for M, N, K in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24), (1, 1, 131072), (2147483647, 1, 16), (1, 2147483647, 16)):
        assert fn(*[V(A)] * 5, M, N, K, None) == 1
    for i in (0, 2, 4):
        args = [V(A)] * 5
        args[i] = V(MIS)
        assert fn(*args, 1, 1, 16, None) == 3
    assert fn(V(A), V(A + 2), V(A), V(A), V(A), 1, 1, 16, None) == 3


def test_w8a8_forward_refuses_before_any_device_call(lib):
    need = lib.awq_w8a8_workspace_bytes(3, 48)
    assert need == 256 + 12 and lib.awq_w8a8_workspace_bytes(1, 24) == 0 and lib.awq_w8a8_workspace_bytes(0, 16) == 0

    def call(x=A, s=A, wq=A, sw=A, y=A, M=3, N=5, K=48, ws=A, n=need):
        p = lambda v: None if v is None else V(v)  # noqa: E731
        return lib.awq_w8a8_forward(p(x), p(s), p(wq), p(sw), p(y), M, N, K, p(ws), n, None)

    for bad in (dict(x=None), dict(wq=None), dict(sw=None), dict(y=None), dict(ws=None), dict(n=need - 1), dict(M=0), dict(N=0),
                dict(K=40), dict(K=131072, n=1 << 30)):
        assert call(**bad) == 1, bad
    for bad in (dict(x=MIS), dict(s=MIS), dict(wq=MIS), dict(y=MIS), dict(ws=MIS), dict(sw=A + 2)):
        assert call(**bad) == 3, bad
    with pytest.raises(ValueError, match="columns"):
        P.validate_w8a8_forward(half(3, 32), torch.zeros((5, 16), dtype=torch.int8), torch.ones(5), None, None, require_cuda=False)
    with pytest.raises(ValueError, match="K=32"):
        P.validate_w8a8_forward(half(3, 32), torch.zeros((5, 32), dtype=torch.int8), torch.ones(5), torch.ones(16), None,
                                require_cuda=False)
    with pytest.raises(ValueError, match="shape"):
        P.validate_w8a8_forward(half(3, 32), torch.zeros((5, 32), dtype=torch.int8), torch.ones(5), None, half(3, 4),
                                require_cuda=False)


def _norm(lib, y=A, r=A, g=A, per=1, pw=A, w=A, s=A, alpha=1.0, eps=1e-6, M=1, K=8, h=A, x=A):
    p = lambda v: None if v is None else V(v)  # noqa: E731
    return lib.awq_residual_norm(p(y), p(r), p(g), per, p(pw), p(w), p(s), alpha, eps, M, K, p(h), p(x), None)


def test_residual_norm_refuses_before_any_device_call(lib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(y=None), dict(w=None), dict(x=None), dict(M=0), dict(K=0), dict(K=12), dict(K=32776), dict(per=0),
                dict(alpha=nan), dict(alpha=inf), dict(eps=nan), dict(eps=-1e-9), dict(eps=inf)):
        assert _norm(lib, **bad) == 1, bad
    for name in ("y", "r", "g", "pw", "w", "s", "h", "x"):
        assert _norm(lib, **{name: MIS}) == 3, name


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_binding_checks_of_the_row_quantizers():
    ok = dict(require_cuda=False)
    P.validate_quantize_rows(half(3, 32), torch.ones(32), torch.zeros((3, 32), dtype=torch.int8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="multiple of 16"):
        P.validate_quantize_rows(half(3, 24), None, torch.zeros((3, 24), dtype=torch.int8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="at least one row"):
        P.validate_quantize_rows(half(0, 32), None, torch.zeros((0, 32), dtype=torch.int8), torch.ones(0), **ok)
    with pytest.raises(ValueError, match="K=32"):
        P.validate_quantize_rows(half(3, 32), torch.ones(31), torch.zeros((3, 32), dtype=torch.int8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="shape"):
        P.validate_quantize_rows(half(3, 32), None, torch.zeros((2, 32), dtype=torch.int8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="3 elements"):
        P.validate_quantize_rows(half(3, 32), None, torch.zeros((3, 32), dtype=torch.int8), torch.ones(4), **ok)
    with pytest.raises(TypeError, match="int8"):
        P.validate_quantize_rows(half(3, 32), None, torch.zeros((3, 32), dtype=torch.uint8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="contiguous"):
        P.validate_quantize_rows(half(32, 3).t(), None, torch.zeros((3, 32), dtype=torch.int8), torch.ones(3), **ok)
    with pytest.raises(ValueError, match="CUDA"):
        P.awq_quantize_tokens(half(3, 32))


def test_binding_checks_of_the_product():
    xq, wq = torch.zeros((3, 32), dtype=torch.int8), torch.zeros((5, 32), dtype=torch.int8)
    P.validate_w8a8(xq, torch.ones(3), wq, torch.ones(5), half(3, 5), require_cuda=False)
    for bad, match in (((xq, torch.ones(4), wq, torch.ones(5), half(3, 5)), "sx"),
                       ((xq, torch.ones(3), wq, torch.ones(4), half(3, 5)), "sw"),
                       ((xq, torch.ones(3), wq, torch.ones(5), half(5, 3)), "shape"),
                       ((xq, torch.ones(3), torch.zeros((5, 16), dtype=torch.int8), torch.ones(5), half(3, 5)), "columns")):
        with pytest.raises(ValueError, match=match):
            P.validate_w8a8(*bad, require_cuda=False)


def test_binding_checks_of_the_norm():
    def check(y=half(6, 16), residual=half(6, 16), weight=half(16), post=half(16), gate=half(2, 16), alpha=1.0, eps=1e-6,
              s=torch.ones(16), h=half(6, 16), x=half(6, 16)):
        P.validate_residual_norm(y, residual, weight, post, gate, alpha, eps, s, h, x, require_cuda=False)

    check()
    check(residual=None, post=None, gate=None, s=None, h=None)
    for bad, match in ((dict(gate=half(4, 16)), "divides"), (dict(gate=half(2, 8)), "divides"), (dict(weight=half(8)), "weight"),
                       (dict(post=half(8)), "post_weight"), (dict(residual=half(5, 16)), "residual"), (dict(x=half(6, 8)), "x must"),
                       (dict(s=torch.ones(8)), "K=16"), (dict(alpha=float("nan")), "finite"), (dict(eps=-1.0), "negative"),
                       (dict(y=half(6, 12)), "multiple of 8"), (dict(y=half(0, 16)), "row")):
        with pytest.raises(ValueError, match=match):
            check(**bad)
    with pytest.raises(TypeError):
        check(weight=None)


# ---------------------------------------------------------------------------- mixture of experts
def _moe(lib, ptr=None, value=None, T=1, E=8, K=256, I=128, top=2, ws=None):
    """One call with pointer argument `ptr` (by position) replaced; the first nine may be checked."""
    p = [V(A)] * 8 + [None]
    if ptr is not None and ptr < 9:
        p[ptr] = value
    y, w = (value if ptr == 9 else V(A)), (value if ptr == 10 else V(A))
    need = lib.awq_moe_workspace_bytes(T, E, K, I, top)
    return lib.awq_moe_w4a16(*p, T, E, K, I, top, 1, y, w, need if ws is None else ws, None)


def test_moe_refuses_before_any_device_call(lib):
    need = lib.awq_moe_workspace_bytes(1, 8, 256, 128, 2)
    assert need > 0
    for i in list(range(8)) + [9, 10]:
        assert _moe(lib, i, None) == 1, i
        assert _moe(lib, i, V(MIS)) == 3, i
    assert _moe(lib, 8, V(MIS)) == 3
    assert _moe(lib, ws=need - 1) == 1
    for bad in (dict(T=0), dict(T=33), dict(E=0), dict(E=513), dict(E=1), dict(top=0), dict(top=17), dict(top=9), dict(K=0),
                dict(K=192), dict(I=0), dict(I=64), dict(I=-128), dict(I=1 << 30, K=1 << 20)):
        sizes = {**dict(T=1, E=8, K=256, I=128, top=2), **bad}
        assert lib.awq_moe_workspace_bytes(sizes["T"], sizes["E"], sizes["K"], sizes["I"], sizes["top"]) == 0, bad
        assert _moe(lib, ws=1 << 40, **bad) == 1, bad


def _stack(E, N, K, dtype=torch.int32):
    qb, sb, zb = P._packed_sizes_host(N, K)
    return (torch.zeros((E, qb // 4), dtype=dtype), torch.zeros((E, sb // 2), dtype=torch.float16),
            torch.zeros((E, zb), dtype=torch.uint8))


def test_binding_checks_of_the_experts():
    def check(router=half(8, 256), gate_up=_stack(8, 256, 256), down=_stack(8, 256, 128), I=128, top=2, hs=None):
        return P._validate_moe_weights(router, gate_up, down, I, top, hs, require_cuda=False)

    assert check() == (8, 256) and check(hs=torch.ones(8, 128)) == (8, 256)
    for bad, match in ((dict(top=0), "top_k"), (dict(top=9), "top_k"), (dict(router=half(4, 256)), "shape"),
                       (dict(gate_up=_stack(8, 128, 256)), "gate_up"), (dict(down=_stack(7, 256, 128)), "down"),
                       (dict(gate_up=_stack(8, 256, 256)[:2]), "gate_up"), (dict(I=64), "multiples of 128"),
                       (dict(router=half(8, 200)), "multiples of 128"), (dict(hs=torch.ones(8, 127)), "h_scale"),
                       (dict(router=half(513, 256)), "experts")):
        with pytest.raises(ValueError, match=match):
            check(**bad)
    with pytest.raises(TypeError, match="int32"):
        check(gate_up=_stack(8, 256, 256, torch.int64))
    P._validate_moe_tokens(half(32, 256), half(32, 256), 8, 256, require_cuda=False)
    for x, y, match in ((half(33, 256), None, "tokens"), (half(0, 256), None, "tokens"), (half(3, 128), None, "K=256"),
                        (half(3, 256), half(2, 256), "shape")):
        with pytest.raises(ValueError, match=match):
            P._validate_moe_tokens(x, y, 8, 256, require_cuda=False)


def test_expert_layer_on_another_device_is_refused():
    layer = object.__new__(P.AWQMoE)         # a layer whose weights are not on the current device
    layer.router = half(8, 256)
    with pytest.raises((TypeError, ValueError, RuntimeError), match="router"):
        layer(half(3, 256))


def test_w8a8_refuses_more_outputs_than_its_tiles_can_count(lib):
    """M N is at most 2^40, and both sizes are taken up to 2^31 - 128."""
    top = 2 ** 31 - 128
    assert lib.awq_w8a8_linear(*[V(A)] * 5, top, top, 16, None) == 1
    assert lib.awq_w8a8_linear(*[V(A)] * 5, 2 ** 20 + 1, 2 ** 20, 16, None) == 1
    assert lib.awq_w8a8_linear(*[V(A)] * 5, top + 1, 1, 16, None) == 1
    assert lib.awq_w8a8_linear(*[V(A)] * 5, 1, top + 1, 16, None) == 1
    # with the sizes in range the next check answers
    for M, N in ((top, 1), (1, top), (2 ** 20, 2 ** 20)):
        assert lib.awq_w8a8_linear(V(MIS), *[V(A)] * 4, M, N, 16, None) == 3


def test_norm_outputs_in_place_and_other_overlaps():
    """An output may be y or the residual themselves; any other overlap is refused."""
    flat = half(200)
    y, r, w, g = half(6, 16), half(6, 16), half(16), half(6, 16)

    def check(h, x, y=y, residual=r, gate=None, s=None, post=None):
        P.validate_residual_norm(y, residual, w, post, gate, 1.0, 1e-6, s, h, x, require_cuda=False)

    for h, x in ((r, y), (y, r), (r, half(6, 16)), (half(6, 16), y), (None, r), (None, y)):
        check(h, x)
    a, b = flat[:96].view(6, 16), flat[16:112].view(6, 16)
    for h, x, kw in ((b, half(6, 16), dict(residual=a)), (half(6, 16), b, dict(y=a)), (y, y, {}), (a, b, {}), (g, y, dict(gate=g)),
                     (r, g, dict(gate=g)), (r, half(6, 16), dict(residual=None, gate=r)), (a, y, dict(post=a[0])),
                     (a, y, dict(s=a[:2].reshape(-1).view(torch.float32)))):
        with pytest.raises(ValueError, match="overlap"):
            check(h, x, **kw)


def test_norm_refuses_an_alpha_that_overflows_the_sum_of_squares(lib):
    assert _norm(lib, alpha=1.0e15) == 1 and _norm(lib, alpha=-16777218.0) == 1
    assert _norm(lib, alpha=-16777216.0, y=MIS) == 3           # in range: the next check answers
    for alpha in (1.0e15, -16777218.0):
        with pytest.raises(ValueError, match="alpha"):
            P.validate_residual_norm(half(6, 16), None, half(16), None, None, alpha, 1e-6, None, None, None, require_cuda=False)
