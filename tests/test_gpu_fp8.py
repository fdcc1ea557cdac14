"""The fp8 block-scaled linear layer on the GPU against its definition in 64 bits.

* Quantizers: bit-exact (every fp32 step of the definition is one rounding).
* Products: the tensor cores add a block's 128 products in fp32 in an order of their own,
  each of at most 128 additions off by at most one unit 2^-23 of the sum of magnitudes mag;
  the scale product, its multiply-add per block and the few additions that join a split K
  axis by 2^-24 each. So |acc - ref| <= e = (128 2^-23 + (KB + 18) 2^-24) mag, and the
  bf16 result is off by half a step, 2^-8 of its value, more.
* SwiGLU: |silu'| <= 1.1, so h is off by 1.1 e_g |u| + |silu(g)| e_u + 1.1 e_g e_u, and by
  2^-17 |h| for the exponential and the reciprocal (|g| < 64 there); below, silu is under 2^-80.
* Quantized h: a code stands for h within half a step, 2^-4 of the value or 2^-10 of the
  scale, and the scale is the row block's largest |h| / 448 within that largest value's error.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def h3q():
    import w8a8_rotation_quantized_b200 as m
    return m


def _blocks(n):
    return -(-n // 128)


def _rne_e4m3(v):
    """fp64 numpy -> nearest e4m3 value, ties to even, at most 448 in size."""
    a = np.abs(v)
    e = np.floor(np.log2(np.where((a > 0) & np.isfinite(a), a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def _scale(a):
    a = np.asarray(a, np.float32)
    with np.errstate(all="ignore"):
        s = np.where(a == 0, np.float32(0), np.maximum(a / np.float32(448), np.float32(2.0 ** -126))).astype(np.float32)
        inv = np.where(a == 0, np.float32(0), np.float32(1) / s).astype(np.float32)
    return s, inv


def _quantize_ref(x, rows):
    """fp32 numpy [M, K] -> code values, scales [ceil(M / rows), KB] for blocks of rows x 128."""
    M, K = x.shape
    p = np.pad(x, ((0, -M % rows), (0, -K % 128)))
    b = p.reshape(-1, rows, _blocks(K), 128)
    s, inv = _scale(np.abs(b).max(axis=(1, 3)))
    with np.errstate(all="ignore"):
        t = (b * inv[:, None, :, None]).astype(np.float32)
    codes = _rne_e4m3(t.astype(np.float64)).reshape(p.shape)[:M, :K]
    return codes, s


def _quantize(h3q, x):
    M, K = x.shape
    xq = torch.zeros(M, K, dtype=E4, device=x.device)
    sx = torch.full((_blocks(K), M), -1.0, device=x.device)
    h3q.h3q_fp8_quantize(x, xq, sx)
    return xq, sx


def _prepare(h3q, w):
    N, K = w.shape
    wq = torch.zeros(N, K, dtype=E4, device=w.device)
    sw = torch.full((_blocks(N), _blocks(K)), -1.0, device=w.device)
    h3q.h3q_fp8_prepare_weight(w, wq, sw)
    return wq, sw


def _input(M, K, seed, dev, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 100)]] *= 50
    x *= 2.0 ** torch.randint(-12, 12, (M, 1), generator=g).float()
    if M > 1:
        x[M // 2] = 0
    x[0, : min(K, 128)] = 0
    return x.to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 5376), (3, 128), (130, 144), (257, 1360), (64, 2064), (1000, 256)])
def test_quantize_is_bit_exact(h3q, cuda_device, M, K, dtype):
    x = _input(M, K, M + K, cuda_device, dtype)
    xq, sx = _quantize(h3q, x)
    codes, s = _quantize_ref(x.float().cpu().numpy(), 1)
    assert np.array_equal(sx.cpu().numpy(), s.T)
    assert np.array_equal(xq.float().cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (136, 5376), (300, 1360), (1, 144)])
def test_prepare_weight_is_bit_exact(h3q, cuda_device, N, K, dtype):
    w = _input(N, K, N + K, cuda_device, dtype)
    wq, sw = _prepare(h3q, w)
    codes, s = _quantize_ref(w.float().cpu().numpy(), 128)
    assert np.array_equal(sw.cpu().numpy(), s)
    assert np.array_equal(wq.float().cpu().numpy(), codes)


def test_quantize_extremes(h3q, cuda_device):
    """The smallest and largest finite inputs, and what a NaN or an infinity reaches."""
    x = torch.zeros(6, 256, dtype=torch.float32)
    x[0, 3], x[0, 4] = 2.0 ** -149, -(2.0 ** -140)  # the scale stops at 2^-126: codes 0 or tiny
    x[1] = torch.linspace(-3.4e38, 3.4e38, 256)  # the step overflows: infinities and NaN, equal in both
    x[2, 5] = float("nan")
    x[2, 6:200] = 1.0
    x[3, 130] = float("inf")
    x[3, :128] = 2.0
    x[4, 7] = -0.0
    x[5] = 2.0 ** -120
    d = x.to(cuda_device)
    xq, sx = _quantize(h3q, d)
    v, s = xq.float().cpu().numpy(), sx.cpu().numpy().T
    codes, want = _quantize_ref(x.numpy()[[0, 1, 4, 5]], 1)
    assert np.array_equal(s[[0, 1, 4, 5]], want, equal_nan=True)
    assert np.array_equal(v[[0, 1, 4, 5]], codes, equal_nan=True)
    assert np.isnan(s[2, 0]) and np.isnan(v[2, :128]).all()
    assert np.array_equal(v[2, 128:200], np.full(72, 448.0)) and s[2, 1] == np.float32(1) / np.float32(448)
    assert np.isinf(s[3, 1]) and np.isnan(v[3, 130]) and not np.isnan(np.delete(v[3], 130)).any()
    assert s[3, 0] == np.float32(2) / np.float32(448)
    top = torch.linspace(-1, 1, 256)[None] * 3.4e38
    xq, sx = _quantize(h3q, top.to(cuda_device))
    codes, want = _quantize_ref(top.numpy(), 1)
    assert np.isfinite(want).all() and np.array_equal(sx.cpu().numpy().T, want)
    assert np.array_equal(xq.float().cpu().numpy(), codes)


def _product_ref(xq, sx, wq, sw, bias):
    """fp64 v [M, N] (bias added) and the sum of magnitudes of the products."""
    x, w = xq.double(), wq.double()
    v = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(v)
    cols = sw.double().repeat_interleave(128, dim=0)[: w.shape[0]]
    for b in range(_blocks(x.shape[1])):
        k = slice(128 * b, 128 * b + 128)
        f = sx[b].double()[:, None] * cols[:, b][None, :]
        v += (x[:, k] @ w[:, k].T) * f
        mag += (x[:, k].abs() @ w[:, k].abs().T) * f.abs()
    if bias is not None:
        v += bias.double()
    return v, mag


def _err(v, mag, K):
    return (128 * 2.0 ** -23 + (_blocks(K) + 18) * 2.0 ** -24) * mag + 2.0 ** -24 * v.abs() + 2.0 ** -126


def _swiglu_ref(v, e):
    n = v.shape[1] // 2
    g, u, eg, eu = v[:, :n], v[:, n:], e[:, :n], e[:, n:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -17 * h.abs() + 2.0 ** -80 * u.abs()


def _close(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    r = ((got - want).abs() / bound).max().item()
    assert r <= 1, f"error is {r:.3g} of the bound"


def _operands(h3q, M, K, N, seed, dev, with_bias):
    xq, sx = _quantize(h3q, _input(M, K, seed, dev))
    g = torch.Generator().manual_seed(seed + 1)
    wq, sw = _prepare(h3q, (torch.randn(N, K, generator=g) * 0.02 * 2.0 ** torch.randint(-4, 4, (N, 1), generator=g)).to(dev))
    bias = torch.randn(N, generator=g).bfloat16().to(dev) if with_bias else None
    return xq, sx, wq, sw, bias


SHAPES = [(1, 16, 8), (1, 128, 136), (2, 5376, 264), (3, 144, 1000), (7, 1360, 2056), (15, 512, 128), (16, 4096, 256),
          (17, 272, 40), (31, 2064, 640), (33, 640, 3000), (64, 5376, 392), (65, 896, 1536), (127, 1024, 520),
          (128, 14336, 256), (129, 256, 776), (200, 1920, 2048), (257, 128, 16), (300, 1360, 4352), (520, 2000, 1032),
          (1025, 384, 2568), (4100, 144, 1288)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_within_bound(h3q, cuda_device, M, K, N):
    xq, sx, wq, sw, bias = _operands(h3q, M, K, N, M + N, cuda_device, M % 2 == 1)
    # rows behind the last are the caller's
    y = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device=cuda_device)
    h3q.h3q_linear_fp8(xq, sx, wq, sw, y[:M], bias=bias)
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK
    assert (y[M:] == 7).all()
    v, mag = _product_ref(xq, sx, wq, sw, bias)
    e = _err(v, mag, K)
    _close(y[:M], v, e + 2.0 ** -8 * (v.abs() + e))


SWIGLU_SHAPES = [(1, 16, 128), (1, 5376, 640), (4, 144, 128), (16, 1360, 384), (40, 2064, 512), (64, 512, 1152),
                 (100, 5376, 256), (128, 272, 896), (129, 640, 128), (300, 1360, 2176), (700, 256, 1280)]


@pytest.mark.parametrize("M,K,F", SWIGLU_SHAPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_swiglu_within_bound(h3q, cuda_device, M, K, F, with_bias):
    xq, sx, wq, sw, bias = _operands(h3q, M, K, 2 * F, M + F, cuda_device, with_bias)
    y = torch.full((M + 2, F), 7.0, dtype=torch.bfloat16, device=cuda_device)
    h3q.h3q_linear_fp8(xq, sx, wq, sw, y[:M], bias=bias, epilogue=h3q.H3Q_EPI_SWIGLU)
    hq = torch.full((M + 2, F), 3.0, device=cuda_device).to(E4)
    sh = torch.full((F // 128 + 1, M), 5.0, device=cuda_device)
    h3q.h3q_linear_fp8_swiglu_quant(xq, sx, wq, sw, hq[:M], sh[: F // 128], bias=bias)
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK
    assert (y[M:] == 7).all() and (hq[M:].float() == 3).all() and (sh[F // 128 :] == 5).all()
    v, mag = _product_ref(xq, sx, wq, sw, bias)
    h, e = _swiglu_ref(v, _err(v, mag, K))
    _close(y[:M], h, e + 2.0 ** -8 * (h.abs() + e) + 2.0 ** -133)
    top = h.abs().view(M, -1, 128).amax(dim=2).T
    e_top = e.view(M, -1, 128).amax(dim=2).T
    got = sh[: F // 128]
    _close(got, top / 448, e_top / 448 + 2.0 ** -23 * top + 2.0 ** -126)
    back = hq[:M].double() * got.T.double().repeat_interleave(128, dim=1)
    half_step = torch.maximum(2.0 ** -4 * (h.abs() + e), 2.0 ** -10 * got.T.double().repeat_interleave(128, dim=1))
    _close(back, h, e + half_step * (1 + 2.0 ** -20) + 2.0 ** -126)


def _silu_of(h3q, gates, M, dev, up=1.0):
    """silu(g) up of fp32 gates (repeated to M tokens) by the quantized product, as |h| from the scale
    in 64 bits, and by the bf16 one. A one-hot code makes each token's gate its own scale, exactly."""
    F = 1280
    xq, wq = torch.zeros(M, 256, device=dev), torch.zeros(2 * F, 256, device=dev)
    xq[:, 0] = xq[:, 128] = wq[:F, 0] = wq[F:, 128] = 1
    sx = torch.ones(2, M, device=dev)
    sx[0] = gates.repeat(-(-M // len(gates)))[:M]
    sx[1] = up
    ops = xq.to(E4), sx, wq.to(E4), torch.ones(2 * F // 128, 2, device=dev)
    y, hq, sh = torch.empty(M, F, dtype=torch.bfloat16, device=dev), torch.empty(M, F, dtype=E4, device=dev), torch.empty(F // 128, M, device=dev)
    h3q.h3q_linear_fp8(*ops, y, epilogue=h3q.H3Q_EPI_SWIGLU)
    h3q.h3q_linear_fp8_swiglu_quant(*ops, hq, sh)
    assert torch.equal(sh, sh[:1].expand_as(sh)) or torch.isnan(sh).any()
    return sx[0], y, hq, sh[0].double() * 448


@pytest.mark.parametrize("up", [1.0, 16.0])
@pytest.mark.parametrize("M", [16, 48, 4096])
def test_silu_is_accurate(h3q, cuda_device, M, up):
    """2^x within two units of the last place (4 x 2^-24 of its value), one rounding each for what
    lies past the first product, 1 + e, the Newton step, the last product and the scale: 9 x 2^-24.
    (The scale is at least 2^-126, so it shows no |h| below 448 x 2^-126: 16 silu(-87.3) is above.)"""
    assert h3q.h3q_test_fp8_plan(M, 256, 2560, h3q.H3Q_EPI_SWIGLU)[0] == {16: 16, 48: 48, 4096: 0}[M]
    g = torch.Generator().manual_seed(M)
    parts = [torch.rand(1500, generator=g) * 174.3 - 87.3, torch.randn(1500, generator=g) * 4,
             torch.randn(1000, generator=g) * 2.0 ** torch.randint(-60, 4, (1000,), generator=g).float(),
             torch.tensor([-87.3, -87.0, -64.0, -1.0, -2.0 ** -40, 2.0 ** -40, 1.0, 17.0, 88.0, 89.0, 1e4, 1e37])]
    gates = torch.cat(parts).clamp(min=-87.3)
    gates = gates[torch.randperm(len(gates), generator=g)].to(cuda_device)
    for i in range(0, len(gates), M):
        at, y, hq, got = _silu_of(h3q, gates[i : i + M], M, cuda_device, up)
        v = at.double()
        want = v * torch.sigmoid(v) * up
        shown = want.abs().clamp(min=448 * 2.0 ** -126)
        err = (got - shown).abs() / shown
        assert err.max() <= 9 * 2.0 ** -24, (at[err.argmax()].item(), err.max().item() * 2 ** 24)
        top = want.abs() > 448 * 2.0 ** -126
        assert (hq.float()[top] == 448 * torch.sign(at)[top, None]).all()
        assert ((y.double() - want[:, None]).abs() <= 2.0 ** -8 * (1 + 2.0 ** -15) * want.abs()[:, None]).all()


@pytest.mark.parametrize("M", [16, 4096])
def test_silu_at_its_ends(h3q, cuda_device, M):
    """Gates under -87.3 count as 0, the largest ones as themselves, NaN as NaN."""
    low = torch.tensor([-87.4, -88.0, -88.8, -90.0, -100.0, -104.0, -127.5, -1e3, -1e10, -1e38, -3.4e38], device=cuda_device)
    _, y, _, got = _silu_of(h3q, low, M, cuda_device)
    assert (got <= 2.0 ** -119).all() and (y.abs() <= 2.0 ** -119).all()
    high = torch.tensor([88.8, 127.5, 1e3, 1e10, 1e38, 3.38e38], device=cuda_device)
    at, y, hq, got = _silu_of(h3q, high, M, cuda_device)
    assert torch.equal(y[:, 0], at.bfloat16()) and (hq.float() == 448).all()
    assert ((got - at.double()).abs() <= 2.0 ** -23 * at.double()).all()
    _, y, hq, got = _silu_of(h3q, torch.tensor([float("nan")], device=cuda_device), M, cuda_device)
    assert torch.isnan(y).all() and torch.isnan(hq.float()).all() and torch.isnan(got).all()


# the K axis split over two to eight CTAs, token tiles of every size, and several output
# tiles for each SM pair with an odd number of K blocks
LONG_SHAPES = [(1, 14336, 1024), (9, 14336, 1000), (30, 14336, 1024), (60, 14336, 1016), (100, 14336, 1024),
               (256, 14336, 1024), (512, 14336, 520), (1, 5376, 5376), (20, 5376, 5376), (70, 5376, 5376),
               (192, 5376, 2688), (40, 784, 5000), (5000, 400, 3000), (6000, 1040, 4104), (2100, 2064, 5384)]


@pytest.mark.parametrize("M,K,N", LONG_SHAPES)
def test_linear_over_split_and_many_tiles(h3q, cuda_device, M, K, N):
    test_linear_within_bound(h3q, cuda_device, M, K, N)


@pytest.mark.parametrize("M,K,F", [(1, 14336, 128), (10, 14336, 640), (32, 5376, 2176), (33, 14336, 512), (128, 14336, 384),
                                   (3000, 656, 2560), (3001, 1040, 2688)])
def test_swiglu_over_split_and_many_tiles(h3q, cuda_device, M, K, F):
    test_swiglu_within_bound(h3q, cuda_device, M, K, F, M % 2 == 0)


# Every kernel that the rule on sizes picks (M, K, columns of the output, tokens of a tile or 0 for
# the large kernel, CTAs along K), at odd numbers of tokens and K that is no whole number of blocks;
# test_abi_fp8.py holds the lists against the rule.
LINEAR_VARIANTS = [
    (13, 144, 136, 16, 1), (3, 400, 264, 16, 2), (16, 784, 136, 16, 3), (1, 1040, 1000, 16, 4), (5, 2064, 136, 16, 6),
    (9, 5200, 392, 16, 8), (17, 16, 264, 32, 1), (31, 400, 136, 32, 2), (19, 784, 264, 32, 3), (32, 1040, 136, 32, 4),
    (23, 2064, 264, 32, 6), (29, 5200, 136, 32, 8), (33, 144, 136, 48, 1), (47, 400, 264, 48, 2), (35, 784, 136, 48, 3),
    (48, 1040, 264, 48, 4), (41, 2064, 136, 48, 6), (45, 5200, 264, 48, 8), (49, 16, 136, 64, 1), (63, 400, 264, 64, 2),
    (101, 656, 136, 64, 3), (64, 912, 264, 64, 4), (57, 1440, 136, 64, 6), (50, 4016, 264, 64, 8), (65, 144, 8440, 96, 1),
    (782, 400, 640, 96, 2), (516, 656, 632, 96, 3), (643, 912, 384, 96, 4), (323, 1440, 504, 96, 6), (337, 4000, 376, 96, 8),
    (969, 656, 888, 128, 2), (778, 1040, 632, 128, 3), (971, 912, 504, 128, 4), (485, 3600, 376, 128, 6),
    (391, 4048, 376, 128, 8), (51, 16, 16640, 0, 1), (1500, 272, 2056, 0, 1)]
SWIGLU_VARIANTS = [
    (13, 144, 128, 16, 1), (3, 400, 256, 16, 2), (16, 784, 128, 16, 3), (1, 1040, 256, 16, 4), (5, 2064, 128, 16, 6),
    (9, 5200, 128, 16, 8), (17, 16, 256, 32, 1), (31, 400, 128, 32, 2), (19, 784, 256, 32, 3), (32, 1040, 128, 32, 4),
    (23, 2064, 128, 32, 6), (29, 5200, 256, 32, 8), (33, 144, 128, 48, 1), (47, 400, 256, 48, 2), (35, 784, 128, 48, 3),
    (48, 1040, 256, 48, 4), (41, 2064, 128, 48, 6), (45, 5200, 128, 48, 8), (49, 16, 9600, 64, 1), (651, 672, 512, 64, 2),
    (101, 656, 256, 64, 3), (64, 912, 128, 64, 4), (57, 1424, 128, 64, 6), (50, 3984, 128, 64, 8), (275, 128, 4864, 96, 1),
    (65, 16, 9600, 96, 1), (897, 3264, 640, 96, 2), (975, 1840, 384, 96, 3), (897, 1296, 384, 96, 4), (583, 5152, 256, 96, 6),
    (517, 4016, 256, 96, 8), (1173, 7232, 512, 128, 3), (1013, 5632, 512, 128, 4), (489, 14032, 384, 128, 8),
    (49, 16, 128, 0, 1), (700, 256, 1280, 0, 1)]


@pytest.mark.parametrize("M,K,N,tile,splits", LINEAR_VARIANTS)
def test_linear_in_every_variant(h3q, cuda_device, M, K, N, tile, splits):
    test_linear_within_bound(h3q, cuda_device, M, K, N)


@pytest.mark.parametrize("M,K,F,tile,splits", SWIGLU_VARIANTS)
def test_swiglu_in_every_variant(h3q, cuda_device, M, K, F, tile, splits):
    test_swiglu_within_bound(h3q, cuda_device, M, K, F, M % 2 == 0)


def test_scales_of_any_value_are_applied(h3q, cuda_device):
    """Negative, zero, huge and tiny scales, all codes: the product is what the operands say."""
    M, K, N = 70, 400, 264
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(0, 256, (M + N, K), generator=g, dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0  # the two NaN codes
    codes = codes.to(cuda_device).view(E4)
    xq, wq = codes[:M].contiguous(), codes[M:].contiguous()
    sx = torch.randn(4, M, generator=g).to(cuda_device) * 2.0 ** torch.randint(-40, 40, (4, 1), generator=g).to(cuda_device)
    sx[1, 5] = 0
    sw = torch.randn(3, 4, generator=g).to(cuda_device)
    sw[2, 0] = 0
    y = torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)
    h3q.h3q_linear_fp8(xq, sx, wq, sw, y)
    v, mag = _product_ref(xq, sx, wq, sw, None)
    e = _err(v, mag, K)
    _close(y, v, e + 2.0 ** -8 * (v.abs() + e))


@pytest.mark.parametrize("M", [5, 300])
def test_nan_and_infinity_stay_in_their_rows(h3q, cuda_device, M):
    K, N = 512, 512
    x = _input(M, K, 3, cuda_device)
    clean = torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)
    wq, sw = _prepare(h3q, torch.randn(N, K, generator=torch.Generator().manual_seed(1)).to(cuda_device))
    h3q.h3q_linear_fp8(*_quantize(h3q, x), wq, sw, clean)
    x[1, 300], x[M - 1, 7] = float("nan"), float("inf")
    y = torch.empty_like(clean)
    h3q.h3q_linear_fp8(*_quantize(h3q, x), wq, sw, y)
    assert torch.isnan(y[1]).all() and torch.isnan(y[M - 1]).all()
    keep = [i for i in range(M) if i not in (1, M - 1)]
    assert torch.equal(y[keep], clean[keep])
    hq, sh = torch.empty(M, N // 2, dtype=E4, device=cuda_device), torch.empty(2, M, device=cuda_device)
    h3q.h3q_linear_fp8_swiglu_quant(*_quantize(h3q, x), wq, sw, hq, sh)
    assert torch.isnan(hq[1].float()).all() and torch.isnan(sh[:, M - 1]).all()
    assert not torch.isnan(hq[keep].float()).any() and not torch.isnan(sh[:, keep]).any()


@pytest.mark.parametrize("M,K,N", [(4, 5376, 512), (100, 2048, 768), (600, 1360, 1024)])
def test_same_call_gives_the_same_bits(h3q, cuda_device, M, K, N):
    xq, sx, wq, sw, bias = _operands(h3q, M, K, N, 9, cuda_device, True)
    y = [torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device) for _ in range(6)]
    for t in y:
        h3q.h3q_linear_fp8(xq, sx, wq, sw, t, bias=bias)
    assert all(torch.equal(t, y[0]) for t in y)


def test_rows_do_not_depend_on_each_other(h3q, cuda_device):
    """A row's result with its own batch size differs only by the order of the fp32 sums."""
    K, N = 1360, 1032
    xq, sx, wq, sw, bias = _operands(h3q, 400, K, N, 2, cuda_device, True)
    v, mag = _product_ref(xq, sx, wq, sw, bias)
    e = _err(v, mag, K)
    for rows in (1, 20, 90, 400):
        y = torch.empty(rows, N, dtype=torch.bfloat16, device=cuda_device)
        h3q.h3q_linear_fp8(xq[:rows].contiguous(), sx[:, :rows].contiguous(), wq, sw, y, bias=bias)
        _close(y, v[:rows], (e + 2.0 ** -8 * (v.abs() + e))[:rows])


def test_two_streams_at_once(h3q, cuda_device):
    sets = [_operands(h3q, M, 2048, 1024, M, cuda_device, False) for M in (8, 90, 700)]
    want = [torch.empty(s[0].shape[0], 1024, dtype=torch.bfloat16, device=cuda_device) for s in sets]
    for s, t in zip(sets, want):
        h3q.h3q_linear_fp8(*s[:4], t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[torch.empty_like(t) for t in want] for _ in streams]
    for _ in range(5):
        for st, outs in zip(streams, got):
            for s, t in zip(sets, outs):
                h3q.h3q_linear_fp8(*s[:4], t, stream=st)
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("M", [1, 24, 300])
def test_ffn_captured_and_replayed(h3q, cuda_device, M):
    """quantize -> gate/up with quantized SwiGLU -> down, eager and as a replayed graph with new
    inputs; and against the 64-bit product of the operands that each step was given."""
    K, F = 1360, 640
    dev = cuda_device
    wq, sw = _prepare(h3q, torch.randn(2 * F, K, generator=torch.Generator().manual_seed(1)).to(dev) * 0.02)
    dq, sd = _prepare(h3q, torch.randn(K, F, generator=torch.Generator().manual_seed(2)).to(dev) * 0.02)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    xq, sx = torch.empty(M, K, dtype=E4, device=dev), torch.empty(_blocks(K), M, device=dev)
    hq, sh = torch.empty(M, F, dtype=E4, device=dev), torch.empty(F // 128, M, device=dev)
    y = torch.empty(M, K, dtype=torch.bfloat16, device=dev)

    def ffn():
        h3q.h3q_fp8_quantize(x, xq, sx)
        h3q.h3q_linear_fp8_swiglu_quant(xq, sx, wq, sw, hq, sh)
        h3q.h3q_linear_fp8(hq, sh, dq, sd, y)

    x.copy_(_input(M, K, 1, dev))
    ffn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn()
    for seed in (2, 3):
        x.copy_(_input(M, K, seed, dev))
        ffn()
        eager = [t.clone() for t in (xq.view(torch.uint8), sx, hq.view(torch.uint8), sh, y)]
        for t in (xq, hq):
            t.view(torch.uint8).zero_()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((xq.view(torch.uint8), sx, hq.view(torch.uint8), sh, y), eager):
            assert torch.equal(a, b)
        v, mag = _product_ref(hq, sh, dq, sd, None)
        e = _err(v, mag, F)
        _close(y, v, e + 2.0 ** -8 * (v.abs() + e))
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK


def test_buffers_reused_without_a_pause(h3q, cuda_device):
    """Each call may start while the one before it ends: operands that are overwritten by the next
    step of a chain, call after call, still give what each step gives by itself."""
    M, K, N = 40, 1360, 1280
    wq, sw = _prepare(h3q, torch.randn(N, K, generator=torch.Generator().manual_seed(1)).to(cuda_device) * 0.02)
    xs = [_input(M, K, 10 + i, cuda_device) for i in range(30)]
    want = []
    for x in xs:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)
        h3q.h3q_linear_fp8(*_quantize(h3q, x), wq, sw, y)
        torch.cuda.synchronize()
        want.append(y)
    xq, sx = _quantize(h3q, xs[0])
    y = torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)
    got = []
    for x in xs:
        h3q.h3q_fp8_quantize(x, xq, sx)
        h3q.h3q_linear_fp8(xq, sx, wq, sw, y)
        got.append(y.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_replayed_at_once(h3q, cuda_device):
    streams, graphs, sets = [torch.cuda.Stream() for _ in range(2)], [], []
    for M, st in zip((6, 400), streams):
        ops = _operands(h3q, M, 2064, 1024, M, cuda_device, False)[:4]
        got = [torch.empty(M, 512, dtype=E4, device=cuda_device), torch.empty(4, M, device=cuda_device)]
        want = [torch.empty_like(t) for t in got]
        h3q.h3q_linear_fp8_swiglu_quant(*ops, *want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(4):
                h3q.h3q_linear_fp8_swiglu_quant(*ops, *got)
        graphs.append(graph)
        sets.append((ops, got, want))
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want in sets:
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


def test_large_products_back_to_back(h3q, cuda_device):
    """Launch upon launch of CTA pairs, of one K block and of numbers that leave every place of the
    operand ring last, so that blocks start where others have just left: each product as by itself,
    and no wait ran out."""
    M, N = 1500, 2056
    sets = [_operands(h3q, M, K, N, K, cuda_device, False)[:4] for K in (16, 144, 272, 400, 512, 656, 1040)]
    want, got = ([torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device) for _ in sets] for _ in range(2))
    for s, t in zip(sets, want):
        h3q.h3q_linear_fp8(*s, t)
        torch.cuda.synchronize()
        v, mag = _product_ref(*s, None)
        e = _err(v, mag, s[0].shape[1])
        _close(t, v, e + 2.0 ** -8 * (v.abs() + e))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            for s, t in zip(sets, got):
                h3q.h3q_linear_fp8(*s, t)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK


@pytest.mark.parametrize("limit_ns", [0, 3_000_000])
@pytest.mark.parametrize("M,K,N,epilogue", [(1, 16, 136, 0), (9, 5200, 392, 0), (128, 1040, 8440, 0), (23, 2064, 256, 1),
                                            (489, 14032, 768, 1), (1500, 272, 2056, 0), (700, 1360, 2560, 1)])
def test_waits_that_run_out(h3q, cuda_device, M, K, N, epilogue, limit_ns):
    """Operands that never count as complete: each kernel gives up, waits for its own copies however
    short the limit is, and says so; the same operands give the same result as ever afterwards."""
    ops = _operands(h3q, M, K, N, 6, cuda_device, False)[:4]
    want, y = (torch.zeros(M, N // 2 if epilogue else N, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    h3q.h3q_linear_fp8(*ops, want, epilogue=epilogue)
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK
    h3q.h3q_test_stalled_linear_fp8(*ops, y, limit_ns, epilogue=epilogue)
    h3q.h3q_linear_fp8(*ops, y, epilogue=epilogue)  # at once, behind the call that gave up
    assert h3q.h3q_get_device_status() == h3q.H3Q_ERR_TIMEOUT
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK  # cleared
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 40, 700])
@pytest.mark.parametrize("captured", [False, True])
def test_operands_from_another_stream(h3q, cuda_device, M, captured):
    """A call behind a join of two streams waits for both, eager and in a graph: one operand comes from
    the call before it in its stream, the other late from a side stream, whose call in turn follows the
    main stream's."""
    K, N, F, dev = 1360, 1032, 640, cuda_device
    wq, sw = _prepare(h3q, torch.randn(N, K, generator=torch.Generator().manual_seed(1)).to(dev) * 0.02)
    gq, sg = _prepare(h3q, torch.randn(2 * F, K, generator=torch.Generator().manual_seed(2)).to(dev) * 0.02)
    x, late = (torch.empty(M, K, dtype=torch.bfloat16, device=dev) for _ in range(2))
    bias = torch.empty(N, dtype=torch.bfloat16, device=dev)
    xq, sx = _quantize(h3q, x.zero_())
    hq, sh = torch.empty(M, F, dtype=E4, device=dev), torch.empty(F // 128, M, device=dev)
    y, z = torch.empty(M, N, dtype=torch.bfloat16, device=dev), torch.empty(M, F, dtype=torch.bfloat16, device=dev)
    lq, sl = torch.empty_like(xq), torch.empty_like(sx)
    side = torch.cuda.Stream()

    def step():
        h3q.h3q_fp8_quantize(x, xq, sx)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)
            late.add_(x)
            bias.copy_(x[0, :N])
            h3q.h3q_fp8_quantize(late, lq, sl)
        h3q.h3q_linear_fp8_swiglu_quant(xq, sx, gq, sg, hq, sh)
        torch.cuda.current_stream().wait_stream(side)
        h3q.h3q_linear_fp8(lq, sl, wq, sw, y, bias=bias)
        h3q.h3q_linear_fp8(xq, sx, gq, sg, z, epilogue=h3q.H3Q_EPI_SWIGLU)

    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    for seed in range(5):
        x.copy_(_input(M, K, seed, dev))
        late.copy_(_input(M, K, seed + 10, dev))
        both = late + x
        torch.cuda.synchronize()
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        for t, got in ((x, (xq, sx)), (both, (lq, sl))):
            want = _quantize(h3q, t)
            torch.cuda.synchronize()
            assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
        want = [torch.empty_like(t) for t in (hq, sh, y, z)]
        h3q.h3q_linear_fp8_swiglu_quant(xq, sx, gq, sg, want[0], want[1])
        torch.cuda.synchronize()
        h3q.h3q_linear_fp8(lq, sl, wq, sw, want[2], bias=x[0, :N].contiguous())
        torch.cuda.synchronize()
        h3q.h3q_linear_fp8(xq, sx, gq, sg, want[3], epilogue=h3q.H3Q_EPI_SWIGLU)
        torch.cuda.synchronize()
        for t, w in zip((hq, sh, y, z), want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK


def test_every_variant_on_four_streams_at_once(h3q, cuda_device):
    """Clusters of all kernels share the SMs, their shared and their tensor memory: each call's result
    is the one it has alone, and no wait runs out."""
    calls = []
    for M, K, N, _, _ in LINEAR_VARIANTS:
        ops = _operands(h3q, M, K, N, M + N, cuda_device, False)[:4]
        calls.append((h3q.h3q_linear_fp8, ops, [torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)]))
    for M, K, F, _, _ in SWIGLU_VARIANTS:
        ops = _operands(h3q, M, K, 2 * F, M + F, cuda_device, False)[:4]
        calls.append((h3q.h3q_linear_fp8_swiglu_quant, ops, [torch.empty(M, F, dtype=E4, device=cuda_device),
                                                             torch.empty(F // 128, M, device=cuda_device)]))
    want = []
    for f, ops, out in calls:
        f(*ops, *out)
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[[torch.empty_like(t) for t in out] for _, _, out in calls] for _ in streams]
    torch.cuda.synchronize()
    for turn in range(3):
        for i in range(len(calls)):
            for j, st in enumerate(streams):  # each stream begins elsewhere
                at = (i + j * len(calls) // 4 + turn) % len(calls)
                f, ops, _ = calls[at]
                f(*ops, *got[j][at], stream=st)
    torch.cuda.synchronize()
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK
    for outs in got:
        for a, b in zip(outs, want):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def _some(n):
    """Rows at both ends, and at and past element 2^31 of rows of 14336."""
    return torch.cat([torch.arange(0, 3), torch.arange(149795, 149799), torch.arange(n - 3, n)])


@pytest.mark.parametrize("weight", [False, True])
def test_quantizers_past_32_bits(h3q, cuda_device, weight):
    M, K = 150001, 14336
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=cuda_device)
    rows = _some(M)
    x[rows.to(cuda_device)] = _input(len(rows), K, 5, cuda_device)
    codes, s = (_prepare if weight else _quantize)(h3q, x)
    if weight:  # whole bands of 128 rows
        for f in (rows // 128 * 128).unique().tolist():
            c, sc = _quantize_ref(x[f : f + 128].float().cpu().numpy(), 128)
            assert np.array_equal(s[f // 128].cpu().numpy(), sc[0])
            assert np.array_equal(codes[f : f + 128].float().cpu().numpy(), c)
    else:
        c, sc = _quantize_ref(x[rows.to(cuda_device)].float().cpu().numpy(), 1)
        assert np.array_equal(s[:, rows.to(cuda_device)].cpu().numpy(), sc.T)
        assert np.array_equal(codes[rows.to(cuda_device)].float().cpu().numpy(), c)


@pytest.mark.parametrize("M,N", [(150001, 14344), (40, 53700008)])
def test_linear_past_32_bits(h3q, cuda_device, M, N):
    K = 16
    w = torch.randn(99991, K, generator=torch.Generator().manual_seed(4)).to(cuda_device)
    wq, sw = _prepare(h3q, w.repeat(-(-N // 99991), 1)[:N])
    xq, sx = _quantize(h3q, _input(M, K, 3, cuda_device))
    y = torch.empty(M, N, dtype=torch.bfloat16, device=cuda_device)
    h3q.h3q_linear_fp8(xq, sx, wq, sw, y)
    rows = (_some(M) if M > 1000 else torch.arange(36, 40)).to(cuda_device)
    for lo in (0, N // 2 // 128 * 128, (N - 4000) // 128 * 128):
        hi = min(lo + 4096, N)
        v, mag = _product_ref(xq[rows], sx[:, rows].contiguous(), wq[lo:hi], sw[lo // 128 : -(-hi // 128)], None)
        e = _err(v, mag, K)
        _close(y[rows, lo:hi], v, e + 2.0 ** -8 * (v.abs() + e))


def test_swiglu_quant_past_32_bits(h3q, cuda_device):
    M, K, F = 150001, 16, 14336
    xq, sx, wq, sw, _ = _operands(h3q, M, K, 2 * F, 3, cuda_device, False)
    hq, sh = torch.empty(M, F, dtype=E4, device=cuda_device), torch.empty(F // 128, M, device=cuda_device)
    h3q.h3q_linear_fp8_swiglu_quant(xq, sx, wq, sw, hq, sh)
    rows = _some(M).to(cuda_device)
    v, mag = _product_ref(xq[rows], sx[:, rows].contiguous(), wq, sw, None)
    h, e = _swiglu_ref(v, _err(v, mag, K))
    s = sh[:, rows].T.double().repeat_interleave(128, dim=1)
    half_step = torch.maximum(2.0 ** -4 * (h.abs() + e), 2.0 ** -10 * s)
    _close(hq[rows].double() * s, h, e + half_step * (1 + 2.0 ** -20) + 2.0 ** -126)


def test_binding_refuses_wrong_shapes(h3q, cuda_device):
    xq, sx, wq, sw, bias = _operands(h3q, 5, 272, 264, 1, cuda_device, True)
    y = torch.empty(5, 264, dtype=torch.bfloat16, device=cuda_device)
    for args, kw in [((xq, sx.T.contiguous(), wq, sw, y), {}), ((xq, sx, wq[:, :256].contiguous(), sw, y), {}),
                     ((xq, sx, wq, sw[:2], y), {}), ((xq, sx, wq, sw, y[:, :200]), {}), ((xq, sx, wq, sw, y[:4]), {}),
                     ((xq, sx, wq, sw, y), {"bias": bias[:100]}), ((xq, sx, wq, sw, y.float()), {}),
                     ((xq, sx, wq.t().contiguous().t(), sw, y), {})]:
        with pytest.raises(ValueError):
            h3q.h3q_linear_fp8(*args, **kw)
    with pytest.raises(h3q.H3QError):  # 264 rows are not two halves of whole blocks
        h3q.h3q_linear_fp8(xq, sx, wq, sw, y[:, :132].contiguous(), epilogue=h3q.H3Q_EPI_SWIGLU)
    with pytest.raises(ValueError):
        h3q.h3q_fp8_quantize(y, xq, sx)
    empty = torch.empty(0, 272, dtype=E4, device=cuda_device)
    h3q.h3q_linear_fp8(empty, torch.empty(3, 0, device=cuda_device), wq, sw, y[:0])
