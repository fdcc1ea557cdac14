"""RMS norm of queries and keys with the rotation of positions, against 64 bits, and the block
path that it belongs to (fp8 QKV projection -> norm and rotation -> int8 attention -> fp8 output
projection).

Tolerance: the fp32 steps (a sum of at most 256 squares, a division, a root, a reciprocal, two
products and the rotation's two) are off by less than 64 x 2^-24 of the magnitudes they add,
the one rounding to bf16 by 2^-8 of the result.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h3q():
    import w8a8_rotation_quantized_b200 as m
    return m


def _tables(P, rot, dev):
    angle = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return angle.cos().float().to(dev), angle.sin().float().to(dev)


def _ref(x, H, D, w, cos, sin, rot, inter, pos, eps):
    """(values, sum of magnitudes) [S, H, D] in fp64."""
    S = x.shape[0]
    n = x[:, : H * D].double().reshape(S, H, D)
    n = n / torch.sqrt((n * n).mean(dim=2, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    out, mag = n.clone(), n.abs()
    if rot:
        at = torch.arange(S, device=x.device) if pos is None else pos.long()
        c, s = cos.double()[at][:, None, :], sin.double()[at][:, None, :]
        i = torch.arange(rot // 2, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        a, b = n[..., ia], n[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out.reshape(S, H * D), mag.reshape(S, H * D)


def _close(got, ref):
    want, mag = ref
    got = got.double()
    assert torch.isfinite(got).all()
    err = (got - want).abs() - (2.0 ** -8 * (want.abs() + 2.0 ** -18 * mag) + 2.0 ** -18 * mag + 2.0 ** -133)
    assert (err <= 0).all(), f"{err.max().item():.3g} over the bound"


CASES = [  # S, Hq, Hk, D, rot
    (1, 42, 42, 128, 128), (1, 1, 0, 16, 16), (5, 3, 1, 32, 16), (7, 8, 2, 64, 64), (33, 5, 5, 80, 48), (130, 6, 2, 96, 96),
    (64, 2, 1, 112, 0), (257, 16, 2, 64, 32), (40, 4, 4, 256, 256), (19, 7, 3, 192, 64), (1001, 3, 3, 128, 128),
    (3, 2, 1, 48, 32), (9, 2, 2, 240, 240), (2, 130, 1, 128, 64), (2500, 1, 1, 128, 128),
]


@pytest.mark.parametrize("S,Hq,Hk,D,rot", CASES)
@pytest.mark.parametrize("inter,with_pos,weighted", [(False, False, True), (True, True, True), (False, True, False),
                                                     (True, False, False)])
def test_matches_64_bits(h3q, cuda_device, S, Hq, Hk, D, rot, inter, with_pos, weighted):
    dev = cuda_device
    g = torch.Generator().manual_seed(S + D)
    x = torch.randn(S, (Hq + 2 * Hk) * D + 8, generator=g)
    x *= 2.0 ** torch.randint(-8, 8, (S, 1), generator=g)
    x[S // 2] = 0  # a token of zeros: normalised by eps alone
    x = x.bfloat16().to(dev)
    q, k = x[:, : Hq * D], x[:, Hq * D : (Hq + Hk) * D]
    wq = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(dev) if weighted else None
    wk = torch.randn(D, generator=g).bfloat16().to(dev) if weighted else None
    P = 3 * S + 11
    cos, sin = _tables(P, rot, dev) if rot else (None, None)
    pos = torch.randint(P, (S,), generator=g, dtype=torch.int32).to(dev) if with_pos else None
    # outputs are slices of wider rows: the columns beside them stay
    qo = torch.full((S, Hq * D + 16), 5.0, dtype=torch.bfloat16, device=dev)
    ko = torch.full((S, Hk * D + 24), 5.0, dtype=torch.bfloat16, device=dev)
    h3q.h3q_qk_norm_rope(q, k if Hk else None, Hq, Hk, D, cos, sin, qo[:, 8:], ko[:, 16:] if Hk else None, q_weight=wq,
                         k_weight=wk, positions=pos, eps=1e-5, interleaved=inter)
    _close(qo[:, 8 : 8 + Hq * D], _ref(q, Hq, D, wq, cos, sin, rot, inter, pos, 1e-5))
    assert (qo[:, :8] == 5).all() and (qo[:, 8 + Hq * D :] == 5).all()
    if Hk:
        _close(ko[:, 16 : 16 + Hk * D], _ref(k, Hk, D, wk, cos, sin, rot, inter, pos, 1e-5))
        assert (ko[:, :16] == 5).all() and (ko[:, 16 + Hk * D :] == 5).all()


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_gives_the_same_bits(h3q, cuda_device, inter):
    S, H, D = 300, 6, 128
    x = torch.randn(S, 3 * H * D, generator=torch.Generator().manual_seed(1)).bfloat16().to(cuda_device)
    cos, sin = _tables(S, D, cuda_device)
    q, k, v = x.split(H * D, dim=1)
    qo, ko, v0 = torch.empty(S, H * D, dtype=x.dtype, device=x.device), torch.empty(S, H * D, dtype=x.dtype, device=x.device), v.clone()
    h3q.h3q_qk_norm_rope(q, k, H, H, D, cos, sin, qo, ko, interleaved=inter)
    h3q.h3q_qk_norm_rope(q, k, H, H, D, cos, sin, q, k, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, v0)


def test_positions_outside_the_table_leave_nan(h3q, cuda_device):
    S, H, D, rot, P = 12, 3, 64, 32, 10
    x = torch.randn(S, H * D, generator=torch.Generator().manual_seed(1)).bfloat16().to(cuda_device)
    cos, sin = _tables(P, rot, cuda_device)
    pos = torch.tensor([0, 9, 10, -1, 2**31 - 1, -(2**31), 5, 5, 5, 0, 1, 9], dtype=torch.int32, device=cuda_device)
    good = ((pos >= 0) & (pos < P)).cpu()
    for inter in (False, True):
        out = torch.empty_like(x)
        h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None, positions=pos, interleaved=inter)
        o = out.view(S, H, D)
        assert torch.isnan(o[~good][:, :, :rot]).all()
        want, mag = _ref(x, H, D, None, cos, sin, rot, inter, pos.clamp(0, P - 1), 1e-6)
        _close(out[good], (want[good], mag[good]))
        rest = want.view(S, H, D)[~good][:, :, rot:]
        assert ((o[~good][:, :, rot:].double() - rest).abs() <= 2.0 ** -7 * rest.abs() + 2.0 ** -133).all()


def test_nan_and_infinity_stay_in_their_heads(h3q, cuda_device):
    S, H, D = 6, 4, 128
    x = torch.randn(S, H * D, generator=torch.Generator().manual_seed(1)).bfloat16().to(cuda_device)
    cos, sin = _tables(S, D, cuda_device)
    clean, out = torch.empty_like(x), torch.empty_like(x)
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, clean, None)
    x[2, D + 5], x[4, 3] = float("nan"), float("inf")
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None)
    assert torch.isnan(out.view(S, H, D)[2, 1]).all() and torch.isnan(out.view(S, H, D)[4, 0, 3])
    keep = torch.ones(S, H, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(out.view(S, H, D)[keep], clean.view(S, H, D)[keep])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_infinity_past_the_rotated_part(h3q, cuda_device, inter, weighted):
    """Past the rotated elements nothing meets another element: an infinity makes the mean infinite,
    so its own element NaN and every other one 0, and an infinite weight reaches its own element."""
    S, H, D, rot = 5, 3, 80, 32
    g = torch.Generator().manual_seed(2)
    x = torch.randn(S, H * D, generator=g).bfloat16().to(cuda_device)
    w = torch.rand(D, generator=g).add(0.5).bfloat16().to(cuda_device)
    cos, sin = _tables(S, rot, cuda_device)
    at = [(0, 0, rot, "inf"), (1, 2, D - 1, "-inf"), (3, 1, 48, "inf"), (4, 0, 33, "-inf")]
    for t, h, i, v in at:
        x[t, h * D + i] = float(v)
    out = torch.empty_like(x)
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None, q_weight=w if weighted else None, interleaved=inter)
    o = out.view(S, H, D)
    for t, h, i, _ in at:
        assert torch.isnan(o[t, h, i])
        assert (torch.cat([o[t, h, :i], o[t, h, i + 1 :]]) == 0).all(), (t, h, i)
    w[50] = float("inf")
    x[:] = torch.randn(S, H * D, generator=g).bfloat16().to(cuda_device)
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None, q_weight=w, interleaved=inter)
    o = out.view(S, H, D)
    assert torch.equal(o[:, :, 50], x.view(S, H, D)[:, :, 50] * float("inf"))
    assert torch.isfinite(torch.cat([o[:, :, :50], o[:, :, 51:]], dim=2)).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (80, 32), (128, 128), (256, 128)])
def test_large_elements_and_weights(h3q, cuda_device, inter, D, rot):
    """Elements are divided by the root before a weight can carry them past the largest fp32: where
    the squares' sum overflows (to a divided element of 0) and where it does not."""
    S, H = 7, 3
    g = torch.Generator().manual_seed(D)
    x = torch.randn(S, H * D, generator=g).bfloat16().to(cuda_device)
    cos, sin = _tables(S, rot, cuda_device)
    x.view(S, H, D)[2, 1] = 3.3e38 * torch.sign(x.view(S, H, D)[2, 1])
    x.view(S, H, D)[4, 0, D - 1] = -3.3e38
    x.view(S, H, D)[5, 2, 3] = 1.5e19
    w = (4 + torch.rand(D, generator=g)).bfloat16().to(cuda_device)
    out = torch.empty_like(x)
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None, q_weight=w, interleaved=inter)
    o = out.view(S, H, D)
    assert (o[2, 1] == 0).all() and (o[4, 0] == 0).all()
    keep = torch.ones(S, H, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = False
    for big in (1.0, 2.0 ** 100):
        w = (w.float() * big).bfloat16()
        h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None, q_weight=w, interleaved=inter)
        want, mag = (t.view(S, H, D)[keep] for t in _ref(x, H, D, w, cos, sin, rot, inter, None, 1e-6))
        _close(o[keep], (want, mag))


def test_strides_past_32_bits(h3q, cuda_device):
    """Row offsets beyond 2^32 elements: the last row of a [5, 2^30 + 64] view."""
    ld, S, H, D = 2**30 + 64, 5, 2, 64
    big = torch.empty(S * ld, dtype=torch.bfloat16, device=cuda_device).view(S, ld)
    x = torch.randn(S, H * D, generator=torch.Generator().manual_seed(1)).bfloat16().to(cuda_device)
    big[:, : H * D] = x
    cos, sin = _tables(S, D, cuda_device)
    out = torch.empty_like(x)
    h3q.h3q_qk_norm_rope(big[:, : H * D], None, H, 0, D, cos, sin, big[:, 1024 : 1024 + H * D], None)
    h3q.h3q_qk_norm_rope(x, None, H, 0, D, cos, sin, out, None)
    assert torch.equal(big[:, 1024 : 1024 + H * D], out)


@pytest.mark.parametrize("S", [1, 700])
def test_operands_rewritten_by_the_calls_before(h3q, cuda_device, S):
    """Tables, positions, norm weights and a product's bias are written anew, call after call, while
    the dependents behind may be resident already: each call reads what was written before it."""
    from test_gpu_fp8 import E4, _prepare, _quantize
    H, D, K, rounds = 4, 64, 272, 12
    dev = cuda_device
    g = torch.Generator().manual_seed(S)
    wq, sw = _prepare(h3q, torch.randn(2 * H * D, K, generator=g).to(dev))
    xs = torch.randn(rounds, S, K, generator=g).bfloat16().to(dev)
    tables = torch.rand(rounds, 2, 50, D // 2, generator=g).to(dev)
    weights = torch.randn(rounds, D, generator=g).bfloat16().to(dev)
    biases = torch.randn(rounds, 2 * H * D, generator=g).bfloat16().to(dev)
    at = torch.randint(50, (rounds, S), generator=g, dtype=torch.int32).to(dev)
    table, weight, bias, pos = (torch.empty_like(t[0]) for t in (tables, weights, biases, at))
    xq, sx = _quantize(h3q, xs[0])
    y = torch.empty(S, 2 * H * D, dtype=torch.bfloat16, device=dev)

    def run(wait):
        got = []
        for i in range(rounds):
            for to, of in ((table, tables), (weight, weights), (bias, biases), (pos, at)):
                to.copy_(of[i])
            for call in (lambda: h3q.h3q_fp8_quantize(xs[i], xq, sx), lambda: h3q.h3q_linear_fp8(xq, sx, wq, sw, y, bias=bias),
                         lambda: h3q.h3q_qk_norm_rope(y[:, : H * D], y[:, H * D :], H, H, D, table[0], table[1], y[:, : H * D],
                                                      y[:, H * D :], q_weight=weight, k_weight=weight, positions=pos)):
                if wait:
                    torch.cuda.synchronize()
                call()
            got.append(y.clone())
        torch.cuda.synchronize()
        return got

    assert all(torch.equal(a, b) for a, b in zip(run(False), run(True)))


def test_binding_refuses(h3q, cuda_device):
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=cuda_device)
    cos, sin = _tables(4, 64, cuda_device)
    out = torch.empty_like(x)
    ok = dict(q=x, k=None, Hq=4, Hk=0, D=64, cos=cos, sin=sin, q_out=out, k_out=None)
    for change in [dict(Hq=5), dict(q=x.float()), dict(q_out=out[:3]), dict(cos=cos[:, :16]), dict(cos=None),
                   dict(positions=torch.zeros(4, dtype=torch.int64, device=cuda_device)), dict(Hk=1),
                   dict(q_weight=torch.ones(32, dtype=torch.bfloat16, device=cuda_device)), dict(q=x.t())]:
        with pytest.raises(ValueError):
            h3q.h3q_qk_norm_rope(**{**ok, **change})
    for change in [dict(q=x[:, 4:].expand(4, 252), D=48), dict(cos=cos[:3].contiguous(), sin=sin[:3].contiguous()),
                   dict(eps=-1.0), dict(q_out=x[:1].expand(4, 256))]:
        with pytest.raises(h3q.H3QError):
            h3q.h3q_qk_norm_rope(**{**ok, **change})
    h3q.h3q_qk_norm_rope(x[:0], None, 4, 0, 64, cos, sin, out[:0], None)


@pytest.mark.parametrize("S", [8, 264])
def test_block_path(h3q, cuda_device, S):
    """quantize -> QKV projection -> norm and rotation in place -> int8 attention -> quantize ->
    output projection, eager and replayed: each step against 64 bits on the operands it was given."""
    from test_gpu_fp8 import E4, _blocks, _close as close, _err, _input, _prepare, _product_ref
    import oracle
    import synth
    dev, K, H, D = cuda_device, 272, 2, 128
    g = torch.Generator().manual_seed(S)
    wq, sw = _prepare(h3q, torch.randn(3 * H * D, K, generator=g).to(dev) * 0.02)
    oq, so = _prepare(h3q, torch.randn(K, H * D, generator=g).to(dev) * 0.02)
    bias = torch.randn(3 * H * D, generator=g).bfloat16().to(dev)
    nq = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().to(dev)
    cos, sin = _tables(S, D, dev)
    x = torch.empty(S, K, dtype=torch.bfloat16, device=dev)
    xq, sx = torch.empty(S, K, dtype=E4, device=dev), torch.empty(_blocks(K), S, device=dev)
    qkv, raw = (torch.empty(S, 3 * H * D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    att, y = torch.empty(S, H * D, dtype=torch.bfloat16, device=dev), torch.empty(S, K, dtype=torch.bfloat16, device=dev)
    aq, sa = torch.empty(S, H * D, dtype=E4, device=dev), torch.empty(H * D // 128, S, device=dev)
    ws = torch.empty(h3q.h3q_attention_workspace_size(S, H), dtype=torch.uint8, device=dev)

    def block():
        h3q.h3q_fp8_quantize(x, xq, sx)
        h3q.h3q_linear_fp8(xq, sx, wq, sw, qkv, bias=bias)
        raw.copy_(qkv)
        q, k, v = qkv.split(H * D, dim=1)
        h3q.h3q_qk_norm_rope(q, k, H, H, D, cos, sin, q, k, q_weight=nq, k_weight=nq)
        h3q.h3q_attention_int8(q, k, v, H, att, ws)
        h3q.h3q_fp8_quantize(att, aq, sa)
        h3q.h3q_linear_fp8(aq, sa, oq, so, y)

    x.copy_(_input(S, K, 1, dev))
    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    x.copy_(_input(S, K, 2, dev))
    block()
    eager = y.clone()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert h3q.h3q_get_device_status() == h3q.H3Q_OK
    assert torch.equal(y, eager)
    v, mag = _product_ref(xq, sx, wq, sw, bias)
    e = _err(v, mag, K)
    close(raw, v, e + 2.0 ** -8 * (v.abs() + e))
    for i in range(2):
        cols = slice(i * H * D, (i + 1) * H * D)
        _close(qkv[:, cols], _ref(raw[:, cols], H, D, nq, cos, sin, D, False, None, 1e-6))
    assert torch.equal(qkv[:, 2 * H * D :], raw[:, 2 * H * D :])
    bits = qkv.view(torch.int16).cpu().numpy().view(np.uint16)
    ref, *_ = oracle.attention_int8(bits[:, : H * D], bits[:, H * D : 2 * H * D], bits[:, 2 * H * D :], H)
    vmax = np.abs(synth.bf16_bits_to_fp32(bits[:, 2 * H * D :]).astype(np.float64)).reshape(S, H, D).max(axis=(0, 2))
    bound = 2.0 ** -7 * np.repeat(vmax, D)[None, :] + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(att.float().cpu().numpy() - ref) <= bound)
    v, mag = _product_ref(aq, sa, oq, so, None)
    e = _err(v, mag, H * D)
    close(y, v, e + 2.0 ** -8 * (v.abs() + e))
