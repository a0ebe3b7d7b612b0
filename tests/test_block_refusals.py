"""Refusals of the operators around the routed experts: the C ABI's host checks (every device
pointer NULL, so nothing can be launched) and the Python wrappers' checks (no GPU needed)."""

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -8


@pytest.fixture(scope="module")
def lib():
    from w4a16_int4_mixture_gb300 import _binding, _build
    _build.build()
    return _binding.load()


def _route(lib, type=0, T=4, E=64, ld=64, k=8, scoring=1, n_group=1, topk_group=1, group_top=2,
           scale=1.0):
    return lib.chord_moe_route(None, type, T, E, ld, k, scoring, None, n_group, topk_group,
                               group_top, 1, scale, None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(scoring=2), INVALID),
    (dict(T=-1), INVALID), (dict(E=0, ld=0), INVALID), (dict(k=0), INVALID), (dict(ld=63), INVALID),
    (dict(k=33, E=1024, ld=1024), UNSUPPORTED), (dict(E=1025, ld=1025), UNSUPPORTED),
    (dict(n_group=64, topk_group=64), UNSUPPORTED), (dict(n_group=3, topk_group=1), INVALID),
    (dict(n_group=8, topk_group=9), INVALID), (dict(n_group=8, topk_group=0), INVALID),
    (dict(k=9, n_group=8, topk_group=1), INVALID), (dict(group_top=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=0), OK), (dict(), INVALID),
])
def test_route(lib, kw, status):
    assert _route(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(type=7), INVALID), (dict(k=65), INVALID), (dict(E=2000, ld=2000), UNSUPPORTED),
    (dict(ld=1), INVALID), (dict(scale=float("inf")), INVALID), (dict(T=0), OK), (dict(), INVALID),
])
def test_route_backward(lib, kw, status):
    a = dict(type=0, T=4, E=64, ld=64, k=8, scoring=0, renorm=1, scale=1.0)
    a.update(kw)
    assert lib.chord_moe_route_backward(None, None, a["type"], a["T"], a["E"], a["ld"], a["k"],
                                        a["scoring"], a["renorm"], a["scale"], None, None, None,
                                        None) == status


@pytest.mark.parametrize("fn,width", [("chord_int8_quantize", 1), ("chord_int8_silu_mul_quantize", 2)])
def test_quantize(lib, fn, width):
    f = getattr(lib, fn)
    assert f(None, 0, 4, 40, 40 * width, None, 48, None, None) == INVALID  # NULL pointers
    assert f(None, 5, 4, 40, 40 * width, None, 48, None, None) == INVALID
    assert f(None, 0, 4, 40, 40 * width - 1, None, 48, None, None) == INVALID
    assert f(None, 0, 4, 40, 40 * width, None, 40, None, None) == INVALID  # rows off 16 bytes
    assert f(None, 0, 4, 40, 40 * width, None, 32, None, None) == INVALID
    assert f(None, 0, 4, 1 << 17, 1 << 18, None, 1 << 17, None, None) == UNSUPPORTED
    assert f(None, 0, 0, 40, 40 * width, None, 48, None, None) == OK


def _matmul(lib, ld_a=64, ld_w=64, T=4, N=8, K=64, res=None, type=0, ld_out=8, ws=0, flags=0):
    return lib.chord_int8_matmul(None, ld_a, None, None, ld_w, None, T, N, K, res, 0, None, type,
                                 ld_out, None, ws, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ld_a=63), INVALID), (dict(ld_a=72), INVALID), (dict(ld_w=56), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(T=-1), INVALID), (dict(type=9), INVALID), (dict(ld_out=7), INVALID),
    (dict(flags=2), INVALID), (dict(K=1 << 17, ld_a=1 << 17, ld_w=1 << 17), UNSUPPORTED),
    (dict(T=0), OK), (dict(), INVALID),
])
def test_matmul(lib, kw, status):
    assert _matmul(lib, **kw) == status


def test_linear_and_mlp(lib):
    def linear(T=4, N=8, K=64, ld_x=64, ld_w=64, ld_out=8, flags=0, type=0):
        return lib.chord_int8_linear(None, type, ld_x, None, ld_w, None, T, N, K, None, 0, None,
                                     ld_out, None, 0, flags, None)

    def mlp(T=4, H=64, I=32, ld_x=64, ld13=64, ld2=32, ld_out=64, flags=0, type=1):
        return lib.chord_int8_mlp(None, type, ld_x, None, ld13, None, None, ld2, None, T, H, I, None,
                                  0, None, ld_out, None, 0, flags, None)

    assert linear(ld_x=63) == linear(ld_w=65) == linear(ld_out=7) == linear(flags=1 << 10) == INVALID
    assert linear(type=4) == linear() == INVALID
    assert linear(T=0) == OK
    assert mlp(ld13=60) == mlp(ld2=33) == mlp(ld_out=63) == mlp(I=0) == mlp(type=-1) == mlp() == INVALID
    assert mlp(H=1 << 17, ld_x=1 << 17, ld13=1 << 17, ld_out=1 << 17) == UNSUPPORTED
    assert mlp(T=0) == OK


def test_workspace_size(lib):
    f = lib.chord_int8_workspace_size
    assert f(-1, 64, 0) == f(4, 0, 0) == f(4, 1 << 17, 0) == f(4, 64, -1) == 0
    assert f(0, 64, 0) >= 256
    assert f(5, 65, 0) >= 256 + 5 * 80 + 5 * 4
    assert f(5, 64, 33) >= 256 + 5 * 64 + 5 * 2 * 33 * 4 + 5 * 48


def test_wrappers_refuse_host_tensors_and_wrong_types():
    import w4a16_int4_mixture_gb300 as chord

    with pytest.raises(ValueError, match="CUDA"):
        chord.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        chord.moe_route(torch.zeros(2, 8, dtype=torch.float64), 2)
    with pytest.raises(TypeError):
        chord.int8_quantize(torch.zeros(2, 8, dtype=torch.int32))
    with pytest.raises(TypeError):
        chord.int8_matmul(torch.zeros(2, 16), torch.zeros(2), torch.zeros(3, 16), torch.zeros(3))
    with pytest.raises(TypeError):
        chord.int8_mlp(None, None, None, None, None)


def test_quantize_and_rows_refuse_what_is_no_matrix_of_their_type():
    import w4a16_int4_mixture_gb300 as chord

    with pytest.raises(TypeError):
        chord.int8_quantize(None)
    with pytest.raises(TypeError, match="int8"):
        chord.int8_rows(torch.zeros(2, 5))
    with pytest.raises(ValueError, match="2 dims"):
        chord.int8_rows(torch.zeros(5, dtype=torch.int8))
    rows = chord.int8_rows(torch.arange(10, dtype=torch.int8).view(2, 5))
    assert rows.stride() == (16, 1) and rows.tolist() == [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]
