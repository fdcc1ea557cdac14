"""Measured cases of the fp8 block-scaled linear layer and the query/key norm with rotation.

Operators, all of one transformer block's path (QKV projection -> norm and rotation of queries and keys -> attention, and the
FFN): `quantize` and `prepare_weight` (e4m3 codes with one fp32 scale per 1 x 128 block of an activation row and per
128 x 128 block of a weight), `linear` (the product of such operands, bf16 out, optional bias and SwiGLU), `swiglu_quant`
(the gate/up product whose SwiGLU output is quantized again, the input of the down projection) and `qk_norm_rope` (RMS norm
of every query and key head and the rotation of positions).

Sizes: hidden 5376, QKV width 16128, FFN width 14336 or 10752, 42 heads of 128, 1 to 16384 tokens, as in this repository's
benchmark, and generic ragged ones.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest normal fp32: the lower bound of a nonzero block's scale


def listed():
    return [
        # one token's activations before a projection: the smallest call, all latency
        dict(name="quantize_1tok", op="quantize", M=1, K=5376, dtype="bf16"),
        # the block input of a full sequence, the FFN benchmark's token count
        dict(name="quantize_16384tok", op="quantize", M=16384, K=5376, dtype="bf16"),
        # weights of the QKV projection, prepared once at load from fp32
        dict(name="weight_qkv", op="prepare_weight", M=16128, K=5376, dtype="f32"),
        # attention-output projection of a single token: bound by reading the weight
        dict(name="linear_out_1tok", op="linear", M=1, K=5376, N=5376, bias=True, swiglu=False),
        # FFN input of a few tokens: the whole gate/up weight is read for 40 rows
        dict(name="linear_swiglu_40tok", op="linear", M=40, K=5376, N=28672, bias=False, swiglu=True),
        # QKV projection of the 4096-token benchmark case
        dict(name="linear_qkv_4096tok", op="linear", M=4096, K=5376, N=16128, bias=True, swiglu=False),
        # down projection of the 16384-token FFN
        dict(name="linear_down_16384tok", op="linear", M=16384, K=14336, N=5376, bias=False, swiglu=False),
        # a ragged batch through a small FFN: last K block of 80, last row tile of 44
        dict(name="swiglu_quant_300tok", op="swiglu_quant", M=300, K=1360, F=2176, bias=True),
        # gate/up projection of the 16384-token FFN: the largest call
        dict(name="swiglu_quant_16384tok", op="swiglu_quant", M=16384, K=5376, F=14336, bias=False),
        # one token's 42 query and key heads
        dict(name="qk_1tok", op="qk", S=1, Hq=42, Hk=42, D=128, rot=128, inter=False, pos=True, weight=True),
        # shared key heads, part of the head rotated in neighbouring pairs, positions of a packed batch, odd token count
        dict(name="qk_shared_777tok", op="qk", S=777, Hq=16, Hk=2, D=64, rot=32, inter=True, pos=True, weight=True),
        # the attention benchmark's sequence, q and k as column slices of the QKV output
        dict(name="qk_16384tok", op="qk", S=16384, Hq=42, Hk=42, D=128, rot=128, inter=False, pos=False, weight=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "prepare_weight", "linear", "linear", "linear", "swiglu_quant", "swiglu_quant", "qk", "qk"])
    if op in ("quantize", "prepare_weight"):
        K = 16 * _log(rng, 8, 896)
        return dict(op=op, M=_log(rng, 1, 16384), K=K, dtype=rng.choice(["bf16", "f32"]))
    if op == "qk":
        D = 16 * rng.randint(2, 16)
        Hq = rng.randint(1, 42)
        Hk = rng.choice([d for d in range(1, Hq + 1) if Hq % d == 0])
        return dict(op=op, S=_log(rng, 1, 12000), Hq=Hq, Hk=Hk, D=D, rot=16 * rng.randint(1, D // 16),
                    inter=rng.random() < 0.5, pos=rng.random() < 0.5, weight=rng.random() < 0.8)
    while True:
        M, K = _log(rng, 1, 16384), 16 * _log(rng, 8, 896)
        if op == "linear":
            swiglu = rng.random() < 0.3
            N = 256 * _log(rng, 1, 112) if swiglu else 8 * _log(rng, 16, 2016)
            if M * K * N <= 4e11:
                return dict(op=op, M=M, K=K, N=N, bias=rng.random() < 0.5, swiglu=swiglu)
        else:
            F = 128 * _log(rng, 1, 112)
            if M * K * 2 * F <= 4e11:
                return dict(op=op, M=M, K=K, F=F, bias=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activation(g, M, K):
    """N(0, 1) with 1% of the channels 50 times larger, as the benchmark's activations."""
    x = torch.randn(M, K, generator=g, device="cuda")
    channels = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
    x[:, channels] *= 50.0
    return x


def _weight(g, N, K):
    return torch.randn(N, K, generator=g, device="cuda") * 0.02


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dev = "cuda"
    s = dict(case)
    if op in ("quantize", "prepare_weight"):
        M, K = case["M"], case["K"]
        x = _activation(g, M, K) if op == "quantize" else _weight(g, M, K)
        s["x"] = x.bfloat16() if case["dtype"] == "bf16" else x
        s["codes"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=dev)
        kb = -(-K // 128)
        s["scales"] = torch.empty((kb, M) if op == "quantize" else (-(-M // 128), kb), device=dev)
    elif op in ("linear", "swiglu_quant"):
        M, K = case["M"], case["K"]
        N = case["N"] if op == "linear" else 2 * case["F"]
        s["xq"], s["sx"] = _plain_quantize(_activation(g, M, K).bfloat16().float())
        s["wq"], s["sw"] = _plain_prepare_weight(_weight(g, N, K))
        s["b"] = (torch.randn(N, generator=g, device=dev) * 0.01).bfloat16() if case["bias"] else None
        if op == "linear":
            s["y"] = torch.empty(M, N // 2 if case["swiglu"] else N, dtype=torch.bfloat16, device=dev)
        else:
            s["hq"] = torch.empty(M, N // 2, dtype=torch.float8_e4m3fn, device=dev)
            s["sh"] = torch.empty(-(-N // 256), M, device=dev)
    else:
        S, Hq, Hk, D, rot = (case[k] for k in ("S", "Hq", "Hk", "D", "rot"))
        # q, k and v side by side, as the QKV projection leaves them
        qkv = torch.randn(S, (Hq + 2 * Hk) * D, generator=g, device=dev).bfloat16()
        s["q"], s["k"] = qkv[:, : Hq * D], qkv[:, Hq * D : (Hq + Hk) * D]
        s["wq"] = s["wk"] = None
        if case["weight"]:
            s["wq"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).bfloat16()
            s["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).bfloat16()
        P = max(2 * S, 4096) if case["pos"] else S
        angle = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["p"] = torch.randint(P, (S,), generator=g, device=dev, dtype=torch.int32) if case["pos"] else None
        s["qo"] = torch.empty(S, Hq * D, dtype=torch.bfloat16, device=dev)
        s["ko"] = torch.empty(S, Hk * D, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- plain forms
def _scale_of(amax):
    # a tensor divisor: torch divides by a Python number through its reciprocal, which is another value
    s = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=TINY)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _codes_of(x, s):
    inv = torch.where(s == 0, torch.zeros_like(s), torch.ones_like(s) / s)
    return (x * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_quantize(x):
    """fp32 [M, K] -> codes [M, K], scales [ceil(K / 128), M]: one scale per 128 elements of a row."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128)).view(M, -1, 128)
    s = _scale_of(x.abs().amax(dim=2))
    return _codes_of(x, s[:, :, None]).view(M, -1)[:, :K].contiguous(), s.t().contiguous()


def _plain_prepare_weight(w):
    """fp32 [N, K] -> codes [N, K], scales [ceil(N / 128), ceil(K / 128)]: one scale per 128 x 128 block."""
    N, K = w.shape
    w = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128)).view(-(-N // 128), 128, -(-K // 128), 128)
    s = _scale_of(w.abs().amax(dim=(1, 3)))
    codes = _codes_of(w, s[:, None, :, None])
    return codes.view(-(-N // 128) * 128, -1)[:N, :K].contiguous(), s


def _plain_product(s):
    K = s["xq"].shape[1]
    N = s["wq"].shape[0]
    x = s["xq"].float() * s["sx"].t().repeat_interleave(128, dim=1)[:, :K]
    w = s["wq"].float() * s["sw"].repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]
    v = x @ w.t()
    return v if s["b"] is None else v + s["b"].float()


def _plain_swiglu(v):
    gate, up = v.chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_norm_rope(x, H, weight, cos, sin, case):
    S, D, rot = x.shape[0], case["D"], case["rot"]
    x = x.float().view(S, H, D)
    n = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + 1e-6)
    if weight is not None:
        n = n * weight.float()
    if case["inter"]:
        a, b = n[..., 0:rot:2], n[..., 1:rot:2]
    else:
        a, b = n[..., : rot // 2], n[..., rot // 2 : rot]
    c, d = cos[:, None, :], sin[:, None, :]
    ra, rb = a * c - b * d, b * c + a * d
    turned = torch.stack((ra, rb), dim=3).flatten(2) if case["inter"] else torch.cat((ra, rb), dim=2)
    return torch.cat((turned, n[..., rot:]), dim=2).reshape(S, H * D).bfloat16()


def run(s):
    op = s["op"]
    if own:
        import w8a8_rotation_quantized_b200 as h3q

        if op == "quantize":
            h3q.h3q_fp8_quantize(s["x"], s["codes"], s["scales"])
            return s["codes"], s["scales"]
        if op == "prepare_weight":
            h3q.h3q_fp8_prepare_weight(s["x"], s["codes"], s["scales"])
            return s["codes"], s["scales"]
        if op == "linear":
            epilogue = h3q.H3Q_EPI_SWIGLU if s["swiglu"] else h3q.H3Q_EPI_NONE
            h3q.h3q_linear_fp8(s["xq"], s["sx"], s["wq"], s["sw"], s["y"], bias=s["b"], epilogue=epilogue)
            return s["y"]
        if op == "swiglu_quant":
            h3q.h3q_linear_fp8_swiglu_quant(s["xq"], s["sx"], s["wq"], s["sw"], s["hq"], s["sh"], bias=s["b"])
            return s["hq"], s["sh"]
        h3q.h3q_qk_norm_rope(s["q"], s["k"], s["Hq"], s["Hk"], s["D"], s["cos"], s["sin"], s["qo"], s["ko"],
                             q_weight=s["wq"], k_weight=s["wk"], positions=s["p"], eps=1e-6, interleaved=s["inter"])
        return s["qo"], s["ko"]
    if op == "quantize":
        return _plain_quantize(s["x"].float())
    if op == "prepare_weight":
        return _plain_prepare_weight(s["x"].float())
    if op == "linear":
        v = _plain_product(s)
        return (_plain_swiglu(v) if s["swiglu"] else v).bfloat16()
    if op == "swiglu_quant":
        return _plain_quantize(_plain_swiglu(_plain_product(s)))
    cos, sin = (s["cos"], s["sin"]) if s["p"] is None else (s["cos"][s["p"]], s["sin"][s["p"]])
    return (_plain_norm_rope(s["q"], s["Hq"], s["wq"], cos, sin, s), _plain_norm_rope(s["k"], s["Hk"], s["wk"], cos, sin, s))


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("quantize", "prepare_weight"):
        M, K = case["M"], case["K"]
        kb = -(-K // 128)
        scales = M * kb if op == "quantize" else -(-M // 128) * kb
        return {"bytes": M * K * (3 if case["dtype"] == "bf16" else 5) + 4 * scales, "flops": 3 * M * K}
    if op in ("linear", "swiglu_quant"):
        M, K = case["M"], case["K"]
        N = case["N"] if op == "linear" else 2 * case["F"]
        kb = -(-K // 128)
        read = M * K + N * K + 4 * kb * (M + -(-N // 128)) + (2 * N if case["bias"] else 0)
        if op == "linear":
            written = 2 * M * (N // 2 if case["swiglu"] else N)
        else:
            written = M * case["F"] + 4 * M * (case["F"] // 128)
        return {"bytes": read + written, "flops": 2 * M * N * K}
    S, heads, D, rot = case["S"], case["Hq"] + case["Hk"], case["D"], case["rot"]
    return {"bytes": 4 * S * heads * D + 4 * S * rot + (4 * S if case["pos"] else 0), "flops": 8 * S * heads * D}


# ---------------------------------------------------------------- definitions in 64 bits
def _e4m3(v):
    """The e4m3 value nearest to each fp64 value (ties to even), at most 448 in size."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _blocks(x, rows):
    """Values of [M, K] in blocks of `rows` x 128: a list of (row slice, column slice, view)."""
    return [(i, j, x[i : i + rows, j : j + 128]) for i in range(0, x.shape[0], rows) for j in range(0, x.shape[1], 128)]


def _exact_rows(x):
    """1 x 128 blocks of an fp64 matrix: code values and scales by the definition (the scale that divides is an fp32 number)."""
    codes, scales = torch.empty_like(x), torch.empty(-(-x.shape[1] // 128), x.shape[0], dtype=torch.float64, device=x.device)
    for _, j, v in _blocks(x, x.shape[0]):
        s = v.abs().max(dim=1).values / E4M3_MAX
        scales[j // 128] = s
        t = s.float().double()[:, None]
        codes[:, j : j + 128] = _e4m3(torch.where(t > 0, v / torch.where(t > 0, t, 1.0), 0.0))
    return codes, scales


def _exact_product(s):
    xq, wq = s["xq"].double(), s["wq"].double()
    M, N = xq.shape[0], wq.shape[0]
    block = torch.arange(N, device=xq.device) // 128
    v = torch.zeros(M, N, dtype=torch.float64, device=xq.device)
    for i, j, part in _blocks(xq, M):
        v += (part @ wq[:, j : j + 128].T) * s["sx"][j // 128].double()[:, None] * s["sw"][:, j // 128].double()[block][None, :]
    return v if s["b"] is None else v + s["b"].double()


def _exact_heads(x, H, weight, s):
    S, D, rot = s["S"], s["D"], s["rot"]
    out = x.double().reshape(S, H, D).clone()
    out /= out.pow(2).sum(-1, keepdim=True).div(D).add(1e-6).sqrt()
    if weight is not None:
        out *= weight.double()
    row = torch.arange(S, device=x.device) if s["p"] is None else s["p"].long()
    turn = torch.complex(s["cos"][row].double(), s["sin"][row].double())[:, None, :]
    first = torch.arange(rot // 2, device=x.device) * (2 if s["inter"] else 1)
    second = first + (1 if s["inter"] else rot // 2)
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out.reshape(S, H * D)


def exact(case, seed):
    op = case["op"]
    if op in ("linear", "swiglu_quant") and work(case)["flops"] > 2e14:
        return None  # minutes in 64 bits
    s = prepare(case, seed)
    if op == "quantize":
        return _exact_rows(s["x"].double())
    if op == "prepare_weight":
        x = s["x"].double()
        codes, scales = torch.empty_like(x), torch.empty_like(s["scales"], dtype=torch.float64)
        for i in range(0, x.shape[0], 128):
            band = x[i : i + 128]
            top = torch.nn.functional.pad(band.abs().max(dim=0).values, (0, -x.shape[1] % 128)).view(-1, 128)
            scales[i // 128] = top.max(dim=1).values / E4M3_MAX
            t = scales[i // 128].float().double().repeat_interleave(128)[: x.shape[1]]
            codes[i : i + 128] = _e4m3(band / t)
        return codes, scales
    if op == "qk":
        return _exact_heads(s["q"], s["Hq"], s["wq"], s), _exact_heads(s["k"], s["Hk"], s["wk"], s)
    v = _exact_product(s)
    if op == "linear" and not case["swiglu"]:
        return v
    n = v.shape[1] // 2
    h = v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]
    return h if op == "linear" else _exact_rows(h)
