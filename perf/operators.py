"""Cases of the mixture-of-experts operators: the router's top-k choice, tokens sorted by expert, the experts' products with
NVFP4 weights, and the weighted sum of a token's experts, with their gradients.

With `own` false, run() computes an operator in plain torch operations in 32 bits; with `own` true it calls the library.
A case's "op" is one of

  route    logits [T, E] -> ids [T, K], weights [T, K]; with "grad" also the gradient of the logits
  sort     ids [T, K] -> token of each sorted row, group offsets [E + 1], row of each (token, slot)
  product  Y[r] = X[token of r] W_e^T for the rows r of expert e, W_e NVFP4 [m, k]; with "grad" dX[r] = dY[r] W_e
  combine  out[t] = sum_s weights[t, s] Y[row of (t, s)]; with "grad" the gradients of Y and of the weights
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one new token of one sequence: the router of a 256-expert layer, fp32 logits
        {"name": "route_one_token", "op": "route", "T": 1, "E": 256, "K": 8, "dtype": "f32", "renorm": True, "masked": False, "grad": False},
        # a large prefill chunk, bf16 logits (many equal values), some experts masked off and padded tokens with none left
        {"name": "route_prefill", "op": "route", "T": 65536, "E": 256, "K": 8, "dtype": "bf16", "renorm": True, "masked": True, "grad": False},
        # a router's training step on an odd token count, weights not renormalized: forward and gradient
        {"name": "route_train", "op": "route", "T": 16411, "E": 128, "K": 6, "dtype": "f32", "renorm": False, "masked": False, "grad": True},
        # a decode batch: 37 sequences, one token each
        {"name": "sort_decode", "op": "sort", "T": 37, "E": 256, "K": 8},
        # calibration: every token of the repository's 256-expert layer, ahead of its grouped Hessians
        {"name": "sort_calibration", "op": "sort", "T": 262144, "E": 256, "K": 8},
        # one new token through the gate+up products (2048 x 4096 each) of its 8 experts
        {"name": "product_one_token", "op": "product", "T": 1, "E": 256, "K": 8, "m": 2048, "k": 4096, "dtype": "bf16", "grad": False},
        # a decode batch of 64 sequences: most experts see a token or two
        {"name": "product_decode", "op": "product", "T": 64, "E": 256, "K": 8, "m": 2048, "k": 4096, "dtype": "bf16", "grad": False},
        # a prefill chunk of many sequences: hundreds of rows per expert, very uneven
        {"name": "product_prefill", "op": "product", "T": 16384, "E": 256, "K": 8, "m": 2048, "k": 4096, "dtype": "bf16", "grad": False},
        # a smaller layer with odd sizes: ragged output channels, k not a multiple of 32, fp32 results
        {"name": "product_ragged", "op": "product", "T": 1537, "E": 24, "K": 3, "m": 1003, "k": 1040, "dtype": "f32", "grad": False},
        # tuning the router or earlier layers against frozen experts: the gradient through the products
        {"name": "product_train", "op": "product", "T": 4099, "E": 64, "K": 6, "m": 2048, "k": 2048, "dtype": "bf16", "grad": True},
        # a prefill chunk's results brought back to the tokens
        {"name": "combine_prefill", "op": "combine", "T": 16384, "K": 8, "d": 4096, "dtype": "bf16", "grad": False},
        # the same in training, an odd row length
        {"name": "combine_train", "op": "combine", "T": 5003, "K": 6, "d": 2056, "dtype": "f32", "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "sort", "product", "product", "product", "combine", "combine"])
    E = rng.choice([8, 16, 24, 60, 64, 128, 160, 256])
    K = rng.randint(1, 8)
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "K": K, "dtype": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.5,
                "masked": rng.random() < 0.3, "grad": rng.random() < 0.5}
    if op == "sort":
        return {"op": op, "T": _log(rng, 1, 262144), "E": E, "K": K}
    if op == "combine":
        T = _log(rng, 1, 16384)
        d = _log(rng, 64, 7168) if rng.random() < 0.3 else 8 * _log(rng, 8, 896)
        return {"op": op, "T": T, "K": K, "d": d, "dtype": rng.choice(["f32", "bf16"]), "grad": rng.random() < 0.5}
    most = 2 * 131072 * 2048 * 4096
    while True:
        T, m, k = _log(rng, 1, 16384), _log(rng, 64, 4096), 16 * _log(rng, 16, 448)
        if rng.random() < 0.7:
            m = max(64, m // 64 * 64)
        if E * m * k <= 256 * 2048 * 4096 and 2 * T * K * m * k <= most:
            return {"op": op, "T": T, "E": E, "K": K, "m": m, "k": k, "dtype": rng.choice(["f32", "bf16"]), "grad": rng.random() < 0.4}


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _popularity(E):
    """Experts' popularity falls as rank^-1.1, as in the repository's calibration workload."""
    q = np.arange(1, E + 1, dtype=np.float64) ** -1.1
    return q / q.sum()


def _expert_bias(E, gen):
    """log popularity, the ranks dealt to the experts by the seed."""
    order = torch.randperm(E, generator=gen, device=DEV)
    return torch.from_numpy(np.log(_popularity(E))).to(DEV, torch.float32)[order]


def _route_ids(T, E, K, gen):
    """K distinct experts of each token, drawn by popularity without replacement; int32 [T, K]."""
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return torch.topk(_expert_bias(E, gen) - torch.log(-torch.log(u)), K, dim=1).indices.to(torch.int32)


def _sorted(ids, E):
    """(token of each sorted row, group offsets, row of each slot), in plain torch."""
    T, K = ids.shape
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * K, device=ids.device)
    off = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    off[1:] = torch.cumsum(torch.bincount(flat, minlength=E)[:E], 0)
    return (order // K).to(torch.int32), off, pos.reshape(T, K).to(torch.int32)


def _nvfp4_experts(E, m, k, gen):
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
    g = (torch.rand(E, generator=gen, device=DEV) + 0.5) * (0.09 / 2688)
    return codes, scales, g


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    T, K = case["T"], case["K"]
    s = {"case": case}
    if case["op"] == "route":
        E = case["E"]
        logits = torch.randn(T, E, generator=gen, device=DEV) * 1.5 + 0.5 * _expert_bias(E, gen)
        if case["masked"]:
            logits.masked_fill_(torch.rand(T, E, generator=gen, device=DEV) < 0.1, float("-inf"))
            logits.masked_fill_(torch.rand(T, 1, generator=gen, device=DEV) < 0.05, float("-inf"))   # padded tokens
        s["logits"] = logits.to(_type(case))
        if case["grad"]:
            s["dweights"] = torch.randn(T, K, generator=gen, device=DEV)
    elif case["op"] == "sort":
        s["ids"] = _route_ids(T, case["E"], K, gen)
    elif case["op"] == "product":
        E, m, k = case["E"], case["m"], case["k"]
        s["codes"], s["scales"], s["g"] = _nvfp4_experts(E, m, k, gen)
        s["tok_idx"], s["grp_off"], _ = _sorted(_route_ids(T, E, K, gen), E)
        if case["grad"]:
            s["dY"] = torch.randn(T * K, m, generator=gen, device=DEV).to(torch.bfloat16)
        else:
            channel = torch.exp(0.5 * torch.randn(k, generator=gen, device=DEV))
            s["X"] = (torch.randn(T, k, generator=gen, device=DEV) * channel).to(torch.bfloat16)
    else:
        d = case["d"]
        E = 64
        _, _, s["pos"] = _sorted(_route_ids(T, E, K, gen), E)
        s["Y"] = torch.randn(T * K, d, generator=gen, device=DEV).to(_type(case))
        s["weights"] = torch.softmax(torch.randn(T, K, generator=gen, device=DEV), 1)
        if case["grad"]:
            s["dout"] = torch.randn(T, d, generator=gen, device=DEV).to(_type(case))
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import post_nvfp4_weight_amd as nvq
    case = s["case"]
    if case["op"] == "route":
        ids, weights = nvq.moe_topk(s["logits"], case["K"], renorm=case["renorm"])
        if not case["grad"]:
            return ids, weights
        return ids, weights, nvq.moe_topk_backward(s["logits"], ids, weights, s["dweights"], renorm=case["renorm"])
    if case["op"] == "sort":
        return nvq.moe_sort(s["ids"], case["E"])
    if case["op"] == "product":
        if case["grad"]:
            return nvq.nvfp4_gemm_grouped_dx(s["dY"], s["codes"], s["scales"], s["g"], s["grp_off"], out_dtype=_type(case))
        return nvq.nvfp4_gemm_grouped(s["X"], s["codes"], s["scales"], s["g"], s["grp_off"], tok_idx=s["tok_idx"], out_dtype=_type(case))
    if case["grad"]:
        return nvq.moe_combine_backward(s["dout"], s["Y"], s["pos"], s["weights"])
    return nvq.moe_combine(s["Y"], s["pos"], s["weights"], out_dtype=_type(case))


def _run_plain(s):
    case = s["case"]
    if case["op"] == "route":
        return _plain_route(s["logits"], case["K"], case["renorm"], s.get("dweights"))
    if case["op"] == "sort":
        return _sorted(s["ids"], case["E"])
    if case["op"] == "product":
        return _plain_product(s)
    Y, pos, w = s["Y"].float(), s["pos"].long(), s["weights"]
    if case["grad"]:
        dout = s["dout"].float()
        dY = torch.empty_like(Y)
        dY[pos.reshape(-1)] = (w[:, :, None] * dout[:, None, :]).reshape(-1, dout.shape[1])
        return dY.to(s["Y"].dtype), (dout[:, None, :] * Y[pos]).sum(2)
    return (w[:, :, None] * Y[pos]).sum(1).to(_type(case))


def _plain_route(logits, K, renorm, dweights):
    l = logits.float()
    E = l.shape[1]
    value, ids = (v[:, :K] for v in torch.sort(l, dim=1, descending=True, stable=True))   # equal logits: the lower index first
    taken = value > float("-inf")
    top = torch.where(taken[:, :1], value[:, :1], 0.0)
    ex = torch.exp(value - top)
    every = torch.exp(l - top)
    total = (ex if renorm else every).sum(1, keepdim=True).clamp(min=1e-30)   # a row with no expert left: 0 / 1e-30
    w = ex / total
    ids = torch.where(taken, ids, -1)
    if dweights is None:
        return ids.to(torch.int32), w
    mean = (dweights * w).sum(1, keepdim=True)
    if renorm:
        dl = torch.zeros_like(l).scatter_add_(1, ids.clamp(min=0).long(), torch.where(taken, w * (dweights - mean), 0.0))
    else:
        dw = torch.zeros(l.shape[0], E, device=l.device).scatter_add_(1, ids.clamp(min=0).long(), torch.where(taken, dweights, 0.0))
        dl = every / total * (dw - mean)
    return ids.to(torch.int32), w, dl.to(logits.dtype)


def _plain_product(s):
    case = s["case"]
    m, k = case["m"], case["k"]
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    pair = torch.stack((e2m1.repeat(16), e2m1.repeat_interleave(16)), 1)   # byte -> its two values, low nibble first
    A = s["dY"] if case["grad"] else s["X"]
    out = torch.empty(case["T"] * case["K"], k if case["grad"] else m, dtype=_type(case), device=DEV)
    off = s["grp_off"].tolist()
    for e in range(case["E"]):   # each expert has its own matrix and its own number of rows
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        W = pair[s["codes"][e].int()].reshape(m, k // 16, 16) * s["scales"][e].view(torch.float8_e4m3fn).float()[:, :, None] * s["g"][e]
        W = W.reshape(m, k)
        out[a:b] = A[a:b].float() @ W if case["grad"] else A[s["tok_idx"][a:b].long()].float() @ W.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        ids = s["ids"].cpu().numpy()
        T, K = ids.shape
        rows = np.lexsort((np.arange(T * K), ids.reshape(-1)))   # slots by expert, then by token and slot
        pos = np.empty(T * K, dtype=np.int32)
        pos[rows] = np.arange(T * K)
        off = np.array([0] + [int((ids <= e).sum()) for e in range(case["E"])], dtype=np.int64)
        return [(rows // K).astype(np.int32), off, pos.reshape(T, K)]
    if op == "route":
        l = s["logits"].double().cpu().numpy()
        ids = np.argsort(-l, axis=1, kind="stable")[:, :case["K"]]
        value = np.take_along_axis(l, ids, 1)
        taken = np.isfinite(value)
        top = np.where(taken[:, :1], value[:, :1], 0.0)
        chosen = np.where(taken, np.exp(value - top), 0.0)
        every = np.where(np.isfinite(l), np.exp(l - top), 0.0)
        total = (chosen if case["renorm"] else every).sum(1, keepdims=True)
        total[total == 0] = 1.0
        w = chosen / total
        if not case["grad"]:
            return [None, w]
        dw = s["dweights"].double().cpu().numpy()
        onehot = np.zeros_like(l)
        np.put_along_axis(onehot, ids, np.where(taken, dw, 0.0), 1)
        p = every / total
        if case["renorm"]:
            inside = np.zeros_like(l)
            np.put_along_axis(inside, ids, taken.astype(np.float64), 1)
            p = p * inside
        return [None, w, p * (onehot - (dw * w).sum(1, keepdims=True))]
    if op == "product":
        m, k = case["m"], case["k"]
        A = (s["dY"] if case["grad"] else s["X"]).double()
        out = torch.zeros(case["T"] * case["K"], k if case["grad"] else m, dtype=torch.float64, device=DEV)
        off = s["grp_off"].cpu().numpy()
        for e in np.flatnonzero(np.diff(off)):
            c = s["codes"][e]
            c = torch.stack((c & 15, c >> 4), 2).reshape(m, k).int()
            ex, man = ((c >> 1) & 3).double(), (c & 1).double()
            mag = torch.where(ex == 0, 0.5 * man, torch.exp2(ex - 1) * (1 + 0.5 * man))
            b = s["scales"][e].int()
            be, bm = (b >> 3).double(), (b & 7).double()
            scale = torch.where(be == 0, bm / 512, torch.exp2(be - 7) * (1 + bm / 8))
            W = torch.where(c >= 8, -mag, mag) * torch.repeat_interleave(scale, 16, dim=1) * s["g"][e].double()
            r = slice(int(off[e]), int(off[e + 1]))
            out[r] = torch.matmul(A[r], W) if case["grad"] else torch.matmul(A[s["tok_idx"][r].long()], W.t())
        return out
    Y, w = s["Y"].double(), s["weights"].double()
    T, K = w.shape
    flat = s["pos"].reshape(-1).long()
    if case["grad"]:
        do = s["dout"].double()
        slot = torch.empty_like(flat)
        slot[flat] = torch.arange(T * K, device=DEV)   # slot of each row
        dY = do[slot // K] * w.reshape(-1)[slot][:, None]
        dw = torch.zeros(T * K, dtype=torch.float64, device=DEV)
        dw[slot] = (do[slot // K] * Y).sum(1)
        return [dY, dw.reshape(T, K)]
    out = torch.zeros(T, Y.shape[1], dtype=torch.float64, device=DEV)
    for j in range(K):
        out += w[:, j, None] * Y[s["pos"][:, j].long()]
    return out


def work(case):
    """Bytes: each input read once and each output written once; an expert's weights only if a token takes it (the expected
    number of such experts)."""
    T, K = case["T"], case["K"]
    rows = T * K
    if case["op"] == "sort":
        return {"bytes": rows * 12 + (case["E"] + 1) * 8, "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "route":
        E = case["E"]
        n = T * E * size + rows * 8
        return {"bytes": n + (rows * 4 + T * E * size if case["grad"] else 0), "flops": T * E * (6 if case["grad"] else 3)}
    if case["op"] == "combine":
        d = case["d"]
        n = rows * d * size + T * d * size + rows * 8
        return {"bytes": n + (rows * d * size + rows * 4 if case["grad"] else 0), "flops": rows * d * (3 if case["grad"] else 2)}
    E, m, k = case["E"], case["m"], case["k"]
    active = float(np.sum(1 - (1 - np.minimum(1.0, K * _popularity(E))) ** T))
    n = active * (m * k * 9 / 16 + 4) + (E + 1) * 8
    n += rows * m * 2 + rows * k * size if case["grad"] else T * k * 2 + rows * 4 + rows * m * size
    return {"bytes": n, "flops": 2 * rows * m * k}
