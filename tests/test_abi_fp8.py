"""Host-side checks of the fp8 linear calls and the query/key norm: each call below fails
them (or has nothing to do), so nothing is launched and no pointer is followed."""
import ctypes
import math
import os
import random

import pytest

import w8a8_rotation_quantized_b200 as h3q

INV, UNS, OK = h3q.H3Q_ERR_INVALID_ARG, h3q.H3Q_ERR_UNSUPPORTED, h3q.H3Q_OK
FAKE = 0x10000  # never followed


@pytest.mark.parametrize("name", ["h3q_fp8_quantize", "h3q_fp8_prepare_weight"])
def test_quantizers_reject(name):
    f = getattr(h3q.lib, name)
    ok = [FAKE, 0, 4, 512, FAKE, FAKE, None]
    for i, bad, want in [(0, None, INV), (0, FAKE + 8, INV), (1, 2, INV), (2, -1, INV), (3, 0, INV), (3, 24, INV),
                         (3, -16, INV), (4, None, INV), (4, FAKE + 4, INV), (5, None, INV), (5, FAKE + 8, INV),
                         (2, 2**31 - 1, UNS), (3, 2**31, UNS)]:
        args = list(ok)
        args[i] = bad
        assert f(*args) == want, (i, bad)
    assert f(None, 1, 0, 512, None, None, None) == OK


def test_weight_with_too_many_blocks_is_unsupported():
    assert h3q.lib.h3q_fp8_prepare_weight(FAKE, 1, 2**30, 2**30, FAKE, FAKE, None) == UNS


def _linear_args():
    return [FAKE, FAKE, 4, 512, FAKE, FAKE, 512, None, 0, FAKE, None]


@pytest.mark.parametrize("i,bad,want", [
    (0, None, INV), (1, None, INV), (4, None, INV), (5, None, INV), (9, None, INV),
    (0, FAKE + 8, INV), (1, FAKE + 4, INV), (4, FAKE + 1, INV), (5, FAKE + 8, INV), (7, FAKE + 2, INV), (9, FAKE + 8, INV),
    (2, -1, INV), (3, 8, INV), (3, 520, INV), (6, 0, INV), (6, 12, INV), (8, 2, INV),
    (2, 2**31 - 100, UNS), (6, 2**31 - 8, UNS),
])
def test_linear_rejects(i, bad, want):
    args = _linear_args()
    args[i] = bad
    assert h3q.lib.h3q_linear_fp8(*args) == want


def test_linear_swiglu_needs_whole_blocks():
    args = _linear_args()
    args[8], args[6] = h3q.H3Q_EPI_SWIGLU, 384
    assert h3q.lib.h3q_linear_fp8(*args) == INV
    f = h3q.lib.h3q_linear_fp8_swiglu_quant
    ok = [FAKE, FAKE, 4, 512, FAKE, FAKE, 512, None, FAKE, FAKE, None]
    for i, bad in [(6, 384), (6, 0), (8, None), (9, None), (8, FAKE + 8), (9, FAKE + 8), (3, 40), (2, -5), (0, None)]:
        args = list(ok)
        args[i] = bad
        assert f(*args) == INV, (i, bad)


def test_linear_without_rows_is_a_noop():
    assert h3q.lib.h3q_linear_fp8(None, None, 0, 512, None, None, 256, None, 0, None, None) == OK
    assert h3q.lib.h3q_linear_fp8_swiglu_quant(None, None, 0, 512, None, None, 256, None, None, None, None) == OK


#         q     k     S  Hq Hk D   ldq  ldk  wq    wk    eps   cos   sin   P  rot il pos   qo    ko    ldqo ldko
QK_OK = [FAKE, FAKE, 9, 4, 2, 64, 256, 128, None, None, 1e-6, FAKE, FAKE, 9, 64, 0, None, FAKE, FAKE, 256, 128, None]


@pytest.mark.parametrize("i,bad,want", [
    (0, None, INV), (1, None, INV), (17, None, INV), (18, None, INV), (0, FAKE + 8, INV), (18, FAKE + 2, INV),
    (2, -1, INV), (3, 0, INV), (4, -1, INV), (5, 0, INV), (5, 24, INV), (5, 72, INV), (6, 248, INV), (6, 260, INV),
    (7, 120, INV), (7, 132, INV), (19, 255, INV), (20, 100, INV), (8, FAKE + 4, INV), (9, FAKE + 4, INV),
    (10, -1.0, INV), (10, float("nan"), INV), (10, float("inf"), INV), (11, None, INV), (12, None, INV),
    (11, FAKE + 4, INV), (13, 8, INV), (13, 0, INV), (14, 80, INV), (14, 8, INV), (14, -16, INV), (16, FAKE + 2, INV),
    (2, 2**31, UNS), (3, 65537, UNS), (13, 2**31, UNS),
])
def test_qk_norm_rope_rejects(i, bad, want):
    args = list(QK_OK)
    args[i] = bad
    if i == 5 and bad == 72:
        args[14] = 0
    if i == 3 and bad > 4:
        args[6] = args[19] = bad * 64
    assert h3q.lib.h3q_qk_norm_rope(*args) == want


def test_qk_norm_rope_large_heads_and_empty():
    args = list(QK_OK)
    args[5], args[6], args[7], args[19], args[20] = 272, 2176, 2176, 2176, 2176
    assert h3q.lib.h3q_qk_norm_rope(*args) == UNS
    args = list(QK_OK)
    args[2] = 0
    for i in (0, 1, 11, 12, 17, 18):
        args[i] = None
    assert h3q.lib.h3q_qk_norm_rope(*args) == OK


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    c = torch.zeros((4, 256), dtype=torch.float8_e4m3fn)
    s = torch.zeros((2, 4))
    for call in (lambda: h3q.h3q_fp8_quantize(x, c, s), lambda: h3q.h3q_fp8_prepare_weight(x, c, s),
                 lambda: h3q.h3q_linear_fp8(c, s, c, s, x), lambda: h3q.h3q_linear_fp8_swiglu_quant(c, s, c, s, c, s),
                 lambda: h3q.h3q_qk_norm_rope(x, x, 2, 2, 128, s, s, x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="must be torch.float8_e4m3fn"):
        h3q.h3q_linear_fp8(x, s, c, s, x)
    with pytest.raises(ValueError, match="is required"):
        h3q.h3q_fp8_quantize(None, c, s)


def test_signatures_match_the_header():
    for name, n in [("h3q_fp8_quantize", 7), ("h3q_linear_fp8", 11), ("h3q_linear_fp8_swiglu_quant", 11),
                    ("h3q_qk_norm_rope", 22)]:
        text = open(h3q.HEADER).read().split(name + "(", 1)[1].split(");", 1)[0]
        assert text.count(",") + 1 == n == len(getattr(h3q.lib, name).argtypes)
        assert isinstance(getattr(h3q.lib, name), ctypes._CFuncPtr)


def test_plan_rejects():
    plan = (ctypes.c_int32 * 5)()
    ok = [4, 512, 512, 0, 148, plan]
    for i, bad in [(0, 0), (1, 8), (1, 520), (2, 0), (2, 12), (3, 2), (4, 1), (5, None)]:
        args = list(ok)
        args[i] = bad
        assert h3q.lib.h3q_test_fp8_plan(*args) == INV, (i, bad)
    assert h3q.lib.h3q_test_fp8_plan(4, 512, 384, h3q.H3Q_EPI_SWIGLU, 148, plan) == INV
    for i, bad in [(0, 2**31), (1, 2**40), (2, 2**60)]:
        args = list(ok)
        args[i] = bad
        assert h3q.lib.h3q_test_fp8_plan(*args) == UNS, (i, bad)
    assert h3q.lib.h3q_test_fp8_plan(*ok) == OK


def _sizes(epilogue, n=30000):
    """M, K, N spread over what the products take, small and large."""
    rng = random.Random(epilogue)
    step = 256 if epilogue else 8

    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    for _ in range(n):
        yield spread(1, 4000), 16 * spread(1, 900), step * spread(1, 38000 // step)


@pytest.mark.parametrize("epilogue", [h3q.H3Q_EPI_NONE, h3q.H3Q_EPI_SWIGLU])
def test_every_variant_of_the_products_is_tested(epilogue):
    """The GPU tests' lists hold a size for each kernel and split that the rule on sizes picks."""
    pytest.importorskip("torch")
    from test_gpu_fp8 import LINEAR_VARIANTS, SWIGLU_VARIANTS
    listed = SWIGLU_VARIANTS if epilogue else LINEAR_VARIANTS
    for M, K, N, tile, splits in listed:
        assert h3q.h3q_test_fp8_plan(M, K, 2 * N if epilogue else N, epilogue)[:2] == (tile, splits), (M, K, N)
    picked = {h3q.h3q_test_fp8_plan(M, K, N, epilogue)[:2] for M, K, N in _sizes(epilogue)}
    assert picked <= {v[3:] for v in listed}
    assert {v[3] for v in listed} == {0, 16, 32, 48, 64, 96, 128}


@pytest.mark.parametrize("epilogue", [h3q.H3Q_EPI_NONE, h3q.H3Q_EPI_SWIGLU])
def test_no_product_waits_for_tensor_memory(epilogue):
    """Blocks that fit an SM together (228 KB of shared memory, 1 KB of it kept for each block) hold
    at most its 512 columns, whatever their kernels: each asks for the share of the shared memory
    that its columns are of all columns."""
    for M, K, N in _sizes(epilogue):
        _, _, _, smem, columns = h3q.h3q_test_fp8_plan(M, K, N, epilogue)
        assert columns * 228 * 1024 <= 512 * (smem + 1024) and smem <= 227 * 1024, (M, K, N, smem, columns)


def test_stalled_product_rejects():
    f = h3q.lib.h3q_test_stalled_linear_fp8
    ok = [FAKE, FAKE, 4, 512, FAKE, FAKE, 512, 0, FAKE, 1000, None]
    for i, bad in [(0, None), (2, -1), (3, 8), (4, None), (6, 12), (7, 2), (8, None), (8, FAKE + 8), (9, 10**10 + 1)]:
        args = list(ok)
        args[i] = bad
        assert f(*args) == INV, (i, bad)
    args = list(ok)
    args[6], args[7] = 384, h3q.H3Q_EPI_SWIGLU
    assert f(*args) == INV


@pytest.mark.parametrize("name", ["fp8.cuh", "qk_norm_rope.cuh"])
def test_dependent_launches_read_no_memory_as_constant(name):
    """These kernels may be resident while the calls before them still write, so they may not read
    through the path for data that stays constant during a kernel."""
    text = open(os.path.join(os.path.dirname(h3q.__file__), "csrc", name)).read()
    assert "grid_dependency_wait();" in text and "__ldg" not in text and "ld.global.nc" not in text
