"""Cases of the 4-bit MLP operators: MXFP4 quantization and product with its gradient, the gated activation between an
MLP's products, and a whole mixture-of-experts MLP with NVFP4 experts for a few tokens.

With `own` false, run() computes an operator in plain torch operations in 32 bits; with `own` true it calls the library.
A case's "op" is one of

  quantize  X [n, k] -> MXFP4 (E2M1 codes, one power of two per 32) -> the values that it stands for, in X's type
  gemm      Y = Q(X) Q(W)^T, W MXFP4 [m, k]; X [n, k] in bf16 or fp32 (quantized within the call) or MXFP4 already
  gemm_dx   dX = dY Q(W), dY bf16 [n, m]
  swiglu    X [n, 2h] = [gate | up] -> silu(gate) * up; with "grad" the gradient of X
  moe       out[t] = sum_s w[t, s] D_e (silu(G_e x_t) * (U_e x_t)) over the token's experts e, chosen from its logits
            (also returned: ids and weights), or with "given" from ids and weights that the caller has; NVFP4 experts
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token's hidden state on its way into a quantized product, and back
        {"name": "quantize_one_token", "op": "quantize", "n": 1, "k": 4096, "dtype": "bf16"},
        # the weights of the repository's 70B-class down projection
        {"name": "quantize_weights", "op": "quantize", "n": 8192, "k": 28672, "dtype": "f32"},
        # one new token through an attention projection
        {"name": "gemm_one_token", "op": "gemm", "n": 1, "m": 4096, "k": 4096, "input": "bf16", "dtype": "bf16"},
        # a decode batch, an odd number of sequences, through the MLP pair's down projection
        {"name": "gemm_decode", "op": "gemm", "n": 53, "m": 4096, "k": 14336, "input": "bf16", "dtype": "bf16"},
        # a prefill chunk through the MLP pair's gate+up projection
        {"name": "gemm_prefill", "op": "gemm", "n": 8192, "m": 28672, "k": 4096, "input": "bf16", "dtype": "bf16"},
        # odd sizes: ragged outputs, k not a multiple of 64, activations quantized before, fp32 results
        {"name": "gemm_ragged", "op": "gemm", "n": 1537, "m": 1003, "k": 1056, "input": "mxfp4", "dtype": "f32"},
        # tuning earlier layers through a frozen projection, an odd number of tokens
        {"name": "dx_train", "op": "gemm_dx", "n": 8195, "m": 4096, "k": 4096, "dtype": "bf16"},
        # the same on a few short sequences and a ragged layer
        {"name": "dx_ragged", "op": "gemm_dx", "n": 333, "m": 1004, "k": 1056, "dtype": "f32"},
        # a prefill chunk's rows between the experts' products: 16384 tokens x 8
        {"name": "swiglu_prefill", "op": "swiglu", "n": 131072, "h": 1024, "dtype": "bf16", "grad": False},
        # training: forward's gradient at an odd row count and width
        {"name": "swiglu_train", "op": "swiglu", "n": 5003, "h": 2060, "dtype": "f32", "grad": True},
        # one new token through the repository's 256-expert layer
        {"name": "moe_one_token", "op": "moe", "T": 1, "E": 256, "K": 8, "d": 4096, "h": 1024, "dtype": "bf16", "renorm": True, "given": False},
        # a decode batch of an odd number of sequences: most experts see a token or two
        {"name": "moe_decode", "op": "moe", "T": 37, "E": 256, "K": 8, "d": 4096, "h": 1024, "dtype": "bf16", "renorm": True, "given": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gemm", "gemm_dx", "swiglu", "moe", "moe", "moe"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "quantize":
        while True:
            n, k = _log(rng, 1, 65536), 32 * _log(rng, 1, 896)
            if n * k <= 8192 * 28672:
                return {"op": op, "n": n, "k": k, "dtype": dtype}
    if op == "swiglu":
        while True:
            n, h = _log(rng, 1, 131072), _log(rng, 16, 14336)
            if rng.random() < 0.7:
                h = max(8, h // 8 * 8)
            if n * h <= 131072 * 1024:
                return {"op": op, "n": n, "h": h, "dtype": dtype, "grad": rng.random() < 0.5}
    if op == "moe":
        while True:
            E = rng.choice([8, 16, 24, 60, 64, 128, 160, 256])
            T, K, d, h = _log(rng, 1, 64), rng.randint(1, 8), 16 * _log(rng, 8, 448), 16 * _log(rng, 4, 256)
            if E * d * h <= 256 * 4096 * 1024:
                return {"op": op, "T": T, "E": E, "K": K, "d": d, "h": h, "dtype": dtype, "renorm": rng.random() < 0.5,
                        "given": rng.random() < 0.3}
    most = 8192 * 28672 * 4096 if op == "gemm" else 8195 * 4096 * 4096
    while True:
        n, m, k = _log(rng, 1, 16384), _log(rng, 16, 28672), 32 * _log(rng, 4, 896)
        if rng.random() < 0.7:
            m = max(64, m // 64 * 64)
        if n * m * k <= most and m * k <= 8192 * 28672:
            case = {"op": op, "n": n, "m": m, "k": k, "dtype": dtype}
            if op == "gemm":
                case["input"] = rng.choice(["bf16", "f32", "mxfp4"])
            return case


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ---- inputs -------------------------------------------------------------------

def _activations(n, k, gen):
    """Gaussian with log-normal channel sizes, a few channels of them large."""
    channel = torch.exp(0.5 * torch.randn(k, generator=gen, device=DEV))
    channel = torch.where(torch.rand(k, generator=gen, device=DEV) < 0.005, channel * 20, channel)
    return torch.randn(n, k, generator=gen, device=DEV) * channel


def _mxfp4(x):
    """(codes uint8 [n, k/2], scales uint8 [n, k/32]) of fp32 x."""
    n, k = x.shape
    b = x.reshape(n, k // 32, 32)
    e = _block_exponent(b)
    q = _round_e2m1(torch.ldexp(b.abs(), -e))
    index = torch.where(q < 2, 2 * q, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    index = (index | torch.where(b < 0, 8, 0).to(torch.uint8)).reshape(n, k // 2, 2)
    return index[..., 0] | (index[..., 1] << 4), (e[..., 0] + 127).to(torch.uint8)


def _mxfp4_weights(m, k, gen):
    codes = torch.empty(m, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(m, k // 32, dtype=torch.uint8, device=DEV)
    for a in range(0, m, 4096):
        w = torch.randn(min(4096, m - a), k, generator=gen, device=DEV) * 0.02
        codes[a:a + 4096], scales[a:a + 4096] = _mxfp4(w)
    return codes, scales


def _popularity(E):
    """Experts' popularity falls as rank^-1.1, as in the repository's calibration workload."""
    q = np.arange(1, E + 1, dtype=np.float64) ** -1.1
    return q / q.sum()


def _router_logits(T, E, gen):
    """Logits whose top K are K experts drawn by popularity without replacement, the ranks dealt to the experts by the seed."""
    order = torch.randperm(E, generator=gen, device=DEV)
    bias = torch.from_numpy(np.log(_popularity(E))).to(DEV, torch.float32)[order]
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return bias - torch.log(-torch.log(u))


def _nvfp4_experts(E, m, k, size, gen):
    """Quantized experts of the shape of Gaussian layers: E2M1 codes as Gaussian weights take them under a block's largest
    magnitude (a table of 256 quantiles), block scales in E4M3's upper range, one fp32 scale per expert."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    z = torch.erfinv((torch.arange(256) + 0.5) / 128 - 1) * math.sqrt(2) * 2.9   # 6 is at about 2.1 standard deviations
    index = (z.abs()[:, None] - grid).abs().argmin(1)
    table = torch.where((z < 0) & (index > 0), index + 8, index).to(torch.uint8).to(DEV)
    codes = torch.empty(E, m, k // 2, dtype=torch.uint8, device=DEV)
    for e in range(E):
        u = torch.randint(0, 256, (2, m, k // 2), generator=gen, device=DEV, dtype=torch.uint8).int()
        codes[e] = table[u[0]] | (table[u[1]] << 4)
    scales = torch.randint(0x66, 0x7F, (E, m, k // 16), generator=gen, device=DEV, dtype=torch.uint8)
    g = (torch.rand(E, generator=gen, device=DEV) + 0.5) * (size / 2688)
    return codes, scales, g


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        if case["dtype"] == "f32":   # weights
            s["X"] = torch.randn(case["n"], case["k"], generator=gen, device=DEV) * 0.02
        else:
            s["X"] = _activations(case["n"], case["k"], gen).to(torch.bfloat16)
    elif op == "gemm":
        s["W"] = _mxfp4_weights(case["m"], case["k"], gen)
        X = _activations(case["n"], case["k"], gen)
        s["X"] = _mxfp4(X) if case["input"] == "mxfp4" else (X.to(_type(case["input"])), None)
    elif op == "gemm_dx":
        s["W"] = _mxfp4_weights(case["m"], case["k"], gen)
        s["dY"] = torch.randn(case["n"], case["m"], generator=gen, device=DEV).to(torch.bfloat16)
    elif op == "swiglu":
        s["X"] = (torch.randn(case["n"], 2 * case["h"], generator=gen, device=DEV) * 2).to(_type(case["dtype"]))
        if case["grad"]:
            s["dout"] = torch.randn(case["n"], case["h"], generator=gen, device=DEV).to(_type(case["dtype"]))
    else:
        T, E, K, d, h = (case[x] for x in ("T", "E", "K", "d", "h"))
        s["gate_up"] = _nvfp4_experts(E, 2 * h, d, 4 / math.sqrt(d), gen)   # outputs of about unit size
        s["down"] = _nvfp4_experts(E, d, h, 4 / math.sqrt(h), gen)
        s["X"] = torch.randn(T, d, generator=gen, device=DEV).to(torch.bfloat16)
        s["logits"] = _router_logits(T, E, gen)
        if case["given"]:
            s["ids"] = torch.topk(s["logits"], K, dim=1).indices.to(torch.int32)
            s["weights"] = torch.softmax(torch.randn(T, K, generator=gen, device=DEV), 1)
    return s


# ---- the library's calls --------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import post_nvfp4_weight_amd as nvq
    case = s["case"]
    op = case["op"]
    dtype = _type(case["dtype"])
    if op == "quantize":
        codes, scales = nvq.mxfp4_quantize(s["X"])
        return nvq.mxfp4_dequantize(codes, scales, out_dtype=dtype)
    if op == "gemm":
        return nvq.mxfp4_gemm(s["X"][0], *s["W"], x_scales=s["X"][1], out_dtype=dtype)
    if op == "gemm_dx":
        return nvq.mxfp4_gemm_dx(s["dY"], *s["W"], out_dtype=dtype)
    if op == "swiglu":
        return nvq.swiglu_backward(s["dout"], s["X"]) if case["grad"] else nvq.swiglu(s["X"])
    if case["given"]:
        return nvq.nvfp4_moe_mlp(s["X"], s["gate_up"], s["down"], ids=s["ids"], weights=s["weights"], out_dtype=dtype)[0]
    return nvq.nvfp4_moe_mlp(s["X"], s["gate_up"], s["down"], logits=s["logits"], top_k=case["K"], renorm=case["renorm"], out_dtype=dtype)


# ---- the plain forms --------------------------------------------------------------

def _block_exponent(b):
    """floor(log2(largest magnitude)) - 2 of each block, within E8M0's range; int32 [..., 1]."""
    a = b.abs().amax(-1, keepdim=True)
    return torch.where(a > 0, torch.frexp(a).exponent - 3, -127).clamp(-127, 127).to(torch.int32)


def _round_e2m1(y):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code; y >= 0."""
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return torch.clamp(torch.round(y / step) * step, max=6.0)


def _plain_quantize(X):
    x = X.float()
    b = x.reshape(x.shape[0], -1, 32)
    e = _block_exponent(b)
    q = torch.ldexp(_round_e2m1(torch.ldexp(b.abs(), -e)), e)
    return torch.where(b < 0, -q, q).reshape(x.shape)


def _plain_values(codes, scales):
    """MXFP4 to fp32."""
    n, kh = codes.shape
    pair = _pairs()
    v = pair[codes.int()].reshape(n, kh // 16, 32)
    return torch.ldexp(v, scales.int()[:, :, None] - 127).reshape(n, 2 * kh)


def _pairs():
    """[256, 2]: a byte's two E2M1 values, low nibble first."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    return torch.stack((e2m1.repeat(16), e2m1.repeat_interleave(16)), 1)


def _plain_expert(t, e):
    """Expert e's NVFP4 matrix in fp32."""
    codes, scales, g = t[0][e], t[1][e], t[2][e]
    m, kh = codes.shape
    return (_pairs()[codes.int()].reshape(m, kh // 8, 16) * scales.view(torch.float8_e4m3fn).float()[:, :, None] * g).reshape(m, 2 * kh)


def _plain_topk(logits, K, renorm):
    value, ids = (v[:, :K] for v in torch.sort(logits, dim=1, descending=True, stable=True))   # equal logits: the lower index first
    ex = torch.exp(value - value[:, :1])
    total = ex if renorm else torch.exp(logits - value[:, :1])
    return ids.to(torch.int32), ex / total.sum(1, keepdim=True)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    dtype = _type(case["dtype"])
    if op == "quantize":
        return _plain_quantize(s["X"]).to(dtype)
    if op == "gemm":
        X = _plain_quantize(s["X"][0]) if s["X"][1] is None else _plain_values(*s["X"])
        return (X @ _plain_values(*s["W"]).t()).to(dtype)
    if op == "gemm_dx":
        return (s["dY"].float() @ _plain_values(*s["W"])).to(dtype)
    if op == "swiglu":
        gate, up = s["X"].float().chunk(2, 1)
        sig = 1 / (1 + torch.exp(-gate))
        if not case["grad"]:
            return (gate * sig * up).to(dtype)
        dout = s["dout"].float()
        return torch.cat((dout * up * sig * (1 + gate * (1 - sig)), dout * gate * sig), 1).to(dtype)
    if case["given"]:
        ids, w = s["ids"], s["weights"]
    else:
        ids, w = _plain_topk(s["logits"], case["K"], case["renorm"])
    X = s["X"].float()
    out = torch.zeros(case["T"], case["d"], device=DEV)
    for e in torch.unique(ids).tolist():   # each expert in use has its own tokens
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (X[t] @ _plain_expert(s["gate_up"], e).t()).chunk(2, 1)
        act = gate / (1 + torch.exp(-gate)) * up
        out.index_add_(0, t, w[t, slot][:, None] * (act @ _plain_expert(s["down"], e).t()))
    out = out.to(dtype)
    return out if case["given"] else (out, ids, w)


# ---- the definition in 64 bits ------------------------------------------------------

def _exact_e2m1(c):
    """Signed values of 4-bit codes, from sign, exponent and mantissa."""
    ex, man = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.exp2(ex - 1) * (1 + 0.5 * man))
    return torch.where(c >= 8, -mag, mag)


def _exact_nibbles(codes):
    return torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).int()


def _exact_mxfp4(codes, scales):
    return _exact_e2m1(_exact_nibbles(codes)) * torch.repeat_interleave(torch.exp2(scales.double() - 127), 32, dim=1)


def _exact_quantize(X):
    """Each value to the grid point on whose side of the midpoints it lies, under 2^(exponent of the largest - 2)."""
    out = torch.empty(X.shape, dtype=torch.float64, device=DEV)
    rows = max(1, (1 << 25) // X.shape[1])
    for a in range(0, X.shape[0], rows):
        x = X[a:a + rows].double()
        mag = x.abs()
        top = mag.reshape(x.shape[0], -1, 32).max(2).values
        e = torch.floor(torch.log2(top))
        e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))   # where log2 rounded across
        scale = torch.exp2(torch.where(top > 0, e - 2, -127.0).clamp(-127, 127))
        mag = mag / torch.repeat_interleave(scale, 32, dim=1)
        q = torch.zeros_like(mag)
        lower = 0.0
        for mid, upper, even in ((0.25, 0.5, False), (0.75, 1.0, True), (1.25, 1.5, False), (1.75, 2.0, True), (2.5, 3.0, False),
                                 (3.5, 4.0, True), (5.0, 6.0, False)):
            q += (upper - lower) * ((mag >= mid) if even else (mag > mid))
            lower = upper
        out[a:a + rows] = torch.sign(x) * q * torch.repeat_interleave(scale, 32, dim=1)
    return out


def _exact_expert(t, e):
    c = _exact_e2m1(_exact_nibbles(t[0][e]))
    b = t[1][e].int()
    be, bm = (b >> 3).double(), (b & 7).double()
    scale = torch.where(be == 0, bm / 512, torch.exp2(be - 7) * (1 + bm / 8))
    return c * torch.repeat_interleave(scale, 16, dim=1) * t[2][e].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["X"])
    if op == "gemm":
        X = _exact_quantize(s["X"][0]) if s["X"][1] is None else _exact_mxfp4(*s["X"])
        return torch.matmul(X, _exact_mxfp4(*s["W"]).t())
    if op == "gemm_dx":
        return torch.matmul(s["dY"].double(), _exact_mxfp4(*s["W"]))
    if op == "swiglu":
        h = case["h"]
        X = s["X"].double()
        gate, up = X[:, :h], X[:, h:]
        silu = gate * torch.sigmoid(gate)
        if not case["grad"]:
            return silu * up
        dout = s["dout"].double()
        return torch.cat((dout * up * (torch.sigmoid(gate) + silu * torch.sigmoid(-gate)), dout * silu), 1)
    T, K = case["T"], case["K"]
    if case["given"]:
        ids, w = s["ids"].cpu().numpy(), s["weights"].double().cpu().numpy()
    else:
        l = s["logits"].double().cpu().numpy()
        ids = np.argsort(-l, axis=1, kind="stable")[:, :K]
        w = np.exp(np.take_along_axis(l, ids, 1) - l.max(1, keepdims=True))
        w /= (w if case["renorm"] else np.exp(l - l.max(1, keepdims=True))).sum(1, keepdims=True)
    out = torch.zeros(T, case["d"], dtype=torch.float64, device=DEV)
    X = s["X"].double()
    for e in np.unique(ids):
        G, D = _exact_expert(s["gate_up"], int(e)), _exact_expert(s["down"], int(e))
        for t in np.flatnonzero((ids == e).any(1)):
            both = torch.mv(G, X[t])
            gate, up = both[:case["h"]], both[case["h"]:]
            out[t] += float(w[t][ids[t] == e].sum()) * torch.mv(D, gate * torch.sigmoid(gate) * up)
    return out if case["given"] else [out, None, torch.from_numpy(w)]


# ---- what a pass cannot do without ------------------------------------------------------

def _active(T, E, K):
    """Expected number of experts that T tokens use: a token takes expert e with probability 1 - exp(-c popularity), c such
    that these add up to K."""
    if K >= E:
        return float(E)
    q = _popularity(E)
    lo, hi = 0.0, 1e9
    for _ in range(200):
        c = 0.5 * (lo + hi)
        lo, hi = (c, hi) if (1 - np.exp(-c * q)).sum() < K else (lo, c)
    return float((1 - np.exp(-lo * q * T)).sum())


def work(case):
    """Bytes: each input read once and each output written once; an expert's weights only if a token takes it (the expected
    number of such experts).  A quantize pass writes its codes and scales and reads them back."""
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "quantize":
        return {"bytes": case["n"] * case["k"] * (2 * size + 2 * 17 / 32), "flops": 0}
    if op == "swiglu":
        return {"bytes": case["n"] * case["h"] * size * (5 if case["grad"] else 3), "flops": case["n"] * case["h"] * (12 if case["grad"] else 5)}
    if op == "moe":
        T, E, K, d, h = (case[x] for x in ("T", "E", "K", "d", "h"))
        n = _active(T, E, K) * (3 * h * d * 9 / 16 + 8) + T * d * (2 + size) + T * K * 8
        return {"bytes": n + (0 if case["given"] else T * E * 4), "flops": 6 * T * K * d * h}
    n, m, k = case["n"], case["m"], case["k"]
    if op == "gemm_dx":
        return {"bytes": m * k * 17 / 32 + n * m * 2 + n * k * size, "flops": 2 * n * m * k}
    x = {"bf16": 2, "f32": 4, "mxfp4": 17 / 32}[case["input"]]
    return {"bytes": m * k * 17 / 32 + n * k * x + n * m * size, "flops": 2 * n * m * k}
