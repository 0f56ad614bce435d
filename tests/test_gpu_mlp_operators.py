"""The 4-bit products, the gated activation and the few-token expert MLP where their kernels change form or where programs
use them unlike a single call: every tile and split at ragged edges, captured and replayed, on two streams at once, beyond 32-bit offsets.

References in fp64 on the device.  Bounds as in the operators' own tests: a product's instruction takes 64 (16 for the
gradient) k into its accumulator with at most two roundings of 2^-23, and at most 16 + 32 additions join parts of a sum (the
gradient has at most 32 of them more): (k / 32 + 48) 2^-23 sum |x w|, (m / 16 + 48) 2^-23 sum |dy w|; a bf16 result adds 2^-8.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)

POWERS = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [float("nan")], dtype=torch.float64)


@pytest.fixture(scope="module")
def nvq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_nvfp4_weight_amd as m
    return m


def _gen(*seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(hash(tuple(seed)) & 0x7FFFFFFF)
    return g


def _codes(g, n, k, lo=110, hi=140):
    return (torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(lo, hi, (n, k // 32), dtype=torch.uint8, device=DEV, generator=g))


def _values(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    s = POWERS.to(DEV)[scales.long()]
    return GRID.to(DEV)[c] * s.repeat_interleave(32, 1)


def _close(got, x, w, terms):
    """got [n, m] against x [n, k] w [k, m] in fp64."""
    ref = x @ w
    bound = (terms + 48) * 2.0 ** -23 * (x.abs() @ w.abs()) + 1e-37
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs()
    assert bool(((got.double() - ref).abs() <= bound).all())


# Sizes on both sides of the choices of kernel, each with ragged last tiles.
FEW = [(1, 8, 4096), (3, 300, 96), (4, 5000, 288), (7, 130, 544), (8, 77, 2080), (9, 33, 160), (13, 400, 1056), (16, 4100, 512)]
TILES = [(17, 31, 32), (33, 300, 2080), (48, 1003, 544), (64, 33, 8224), (100, 3105, 160), (61, 6200, 1056), (128, 3100, 32),   # shared k
         (700, 1201, 224), (1030, 777, 1056),            # 64 x 64
         (701, 2401, 96), (65, 24600, 288),              # 128 x 64
         (1100, 2801, 352), (129, 12300, 32),            # 128 x 128
         (4003, 3101, 160), (300, 24700, 672)]           # 256 x 256


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xtype", ["mxfp4", "f32", "bf16"])
@pytest.mark.parametrize("n,m,k", FEW + TILES)
def test_gemm_forms(nvq, n, m, k, xtype, dtype):
    g = _gen(n, m, k)
    wc, ws = _codes(g, m, k)
    if xtype == "mxfp4":
        xc, xs = _codes(g, n, k)
        Y = nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs, out_dtype=DTYPES[dtype])
    else:
        X = torch.randn(n, k, device=DEV, generator=g).to(DTYPES[xtype])
        xc, xs = nvq.mxfp4_quantize(X)
        Y = nvq.mxfp4_gemm(X, wc, ws, out_dtype=DTYPES[dtype])
    _close(Y, _values(xc, xs), _values(wc, ws).T, k / 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,k", [(1, 1, 32), (2, 7, 1056), (1, 64, 2080), (2, 65, 4096), (1, 300000, 32), (2, 2055, 1056),          # one or two rows
                                   (1, 4100, 96), (2, 1000, 512), (3, 1000, 512), (64, 2049, 288), (65, 9000, 64), (200, 20000, 32), (512, 12345, 288),   # parts of m
                                   (513, 700, 1056), (130, 264, 32992),                                              # none
                                   (3400, 72, 4128), (3400, 200, 4096), (8900, 136, 4096), (13400, 64, 1024),   # expanded
                                   (3400, 77, 4128)])                                                                # rows that rule it out
def test_gemm_dx_forms(nvq, n, m, k, dtype):
    g = _gen(n, m, k, 1)
    wc, ws = _codes(g, m, k)
    dY = torch.randn(n, m + 8, device=DEV, generator=g).to(torch.bfloat16)
    w = _values(wc, ws)
    for d in (dY[:, :m], dY[:, 3:3 + m], dY[:, :m].contiguous()):     # rows apart; unaligned; as they are
        _close(nvq.mxfp4_gemm_dx(d, wc, ws, out_dtype=DTYPES[dtype]), d.double(), w, m / 16)
    buf = torch.full((n + 2, k + 7), 7.0, dtype=DTYPES[dtype], device=DEV)
    dX = buf[1:n + 1, 3:3 + k]
    nvq.mxfp4_gemm_dx(dY[:, :m], wc, ws, dX=dX)
    _close(dX, dY[:, :m].double(), w, m / 16)
    dX.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_gemm_dx_nan_blocks(nvq):
    """A NaN block makes its 32 columns NaN in every form, nothing else changes."""
    for n, m, k in ((1, 2000, 96), (3, 2000, 96), (600, 128, 64), (3400, 64, 4096)):
        g = _gen(n)
        wc, ws = _codes(g, m, k)
        dY = torch.randn(n, m, device=DEV, generator=g).to(torch.bfloat16)
        clean = nvq.mxfp4_gemm_dx(dY, wc, ws)
        bad = ws.clone()
        bad[m - 1, 1] = 255
        dX = nvq.mxfp4_gemm_dx(dY, wc, bad)
        assert bool(dX[:, 32:64].isnan().all())
        dX[:, 32:64] = clean[:, 32:64]
        assert torch.equal(dX, clean)


def test_gemm_dx_expanded_scales(nvq):
    """Rows that are unit vectors give the weights back, under every scale byte that fp32 holds with the codes' range."""
    n, m, k = 3400, 256, 4096
    g = _gen(11)
    wc, _ = _codes(g, m, k)
    ws = torch.arange(m, dtype=torch.uint8, device=DEV).clamp(max=252)[:, None].repeat(1, k // 32)
    at = torch.arange(n, device=DEV) % m
    dY = torch.zeros(n, m, dtype=torch.bfloat16, device=DEV)
    dY[torch.arange(n, device=DEV), at] = 1
    w = _values(wc, ws)
    for dt in DTYPES.values():
        assert torch.equal(nvq.mxfp4_gemm_dx(dY, wc, ws, out_dtype=dt).double(), w[at])     # (exact in bf16 too)


def test_gemm_dx_single_row_scales(nvq):
    """One row, a unit vector: every scale byte that fp32 holds, and one whose values leave it beside zero codes (no NaN)."""
    m, k = 253, 64
    g = _gen(12)
    wc, _ = _codes(g, m, k)
    ws = torch.arange(m, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 2)
    w = _values(wc, ws)
    for i in (0, 1, 2, 100, 251, 252):
        dY = torch.zeros(1, m, dtype=torch.bfloat16, device=DEV)
        dY[0, i] = 1
        assert torch.equal(nvq.mxfp4_gemm_dx(dY, wc, ws)[0].double(), w[i])
    wc[-1], ws[-1] = 0, 254
    dY = torch.full((2, m), 8.0, dtype=torch.bfloat16, device=DEV)
    dY[:, :-1] = 0
    assert bool((nvq.mxfp4_gemm_dx(dY, wc, ws) == 0).all())


@pytest.mark.parametrize("T,K", [(64, 63), (64, 64), (8, 64)])
def test_most_experts_and_slots(nvq, T, K):
    """The largest lists of experts and slots, against the layer on the grouped products."""
    E, d, h, m = 1024, 32, 32, 16
    g = _gen(T, K)
    gu, dn = _experts(g, E, 2 * h, d), _experts(g, E, m, h)
    X = torch.randn(T, d, device=DEV, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, device=DEV, generator=g)
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=K, out_dtype=torch.float32)
    ids6, w6 = nvq.moe_topk(logits, K)
    assert torch.equal(ids, ids6) and torch.equal(w, w6)
    tok, off, pos = nvq.moe_sort(ids6, E)
    act = nvq.swiglu(nvq.nvfp4_gemm_grouped(X, *gu, off, tok_idx=tok), out_dtype=torch.bfloat16)
    out6 = nvq.moe_combine(nvq.nvfp4_gemm_grouped(act, *dn, off), pos, w6)
    # Each path's activation is off by at most 64 roundings of 2^-23 of |G||x| and of |U||x| (silu's slope is below 1.1, so
    # 2 * 2.2 * 64 * 2^-23 < 2^-14 of their product for both together), the grouped one by 2^-8 of itself as well; the
    # second sums add 2^-16 of |D||act| or less, which the factor 1.05 covers with the bound's own roundings.
    mag = nvq.nvfp4_gemm_grouped(X.abs(), gu[0] & 0x77, *gu[1:], off, tok_idx=tok)
    err = 1.05 * (2.0 ** -8 * act.float().abs() + 2.0 ** -14 * mag[:, :h] * mag[:, h:])
    bound = nvq.moe_combine(nvq.nvfp4_gemm_grouped(err.to(torch.bfloat16), dn[0] & 0x77, *dn[1:], off), pos, w6)
    assert bool(((out - out6).abs() <= 1.05 * bound + 1e-30).all())


# ---- as programs use them -------------------------------------------------------------------
def _experts(g, E, m, k):
    return (torch.randint(0, 256, (E, m, k // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(0x20, 0x60, (E, m, k // 16), dtype=torch.uint8, device=DEV, generator=g),
            torch.rand(E, device=DEV, generator=g) / (32 * k ** 0.5))


def _dense_step(nvq, X, dout, W1, W2):
    """A dense MLP on 4-bit operands forward and back; every form that needs a workspace is among these."""
    xc, xs = nvq.mxfp4_quantize(X)
    hid = nvq.mxfp4_gemm(xc, *W1, x_scales=xs, out_dtype=torch.bfloat16)
    act = nvq.swiglu(hid)
    Y = nvq.mxfp4_gemm(act, *W2)
    dhid = nvq.swiglu_backward(nvq.mxfp4_gemm_dx(dout, *W2, out_dtype=torch.bfloat16), hid)
    return Y, hid, act, nvq.mxfp4_gemm_dx(dhid, *W1)


def _moe_step(nvq, X, logits, gu, dn):
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=3, out_dtype=torch.float32)
    return out, ids, w


def _programs(nvq, seed):
    """(name, function of inputs, fresh inputs) for small and large calls."""
    g = _gen(seed)
    d, h = 256, 1056
    W1, W2 = _codes(g, 2 * h, d, 118, 124), _codes(g, d, h, 118, 124)
    gu, dn = _experts(g, 20, 2 * 64, d), _experts(g, 20, 96, 64)
    wide = _codes(g, 64, 4096, 118, 124)

    def draw(n):
        return lambda: [torch.randn(n, d, device=DEV).to(torch.bfloat16), torch.randn(n, d, device=DEV).to(torch.bfloat16)]

    progs = [(f"dense {n}", lambda X, dout: _dense_step(nvq, X, dout, W1, W2), draw(n)) for n in (1, 2, 40, 600)]
    progs += [(f"experts {T}", lambda X, logits: _moe_step(nvq, X, logits, gu, dn),
               lambda T=T: [torch.randn(T, d, device=DEV).to(torch.bfloat16), torch.randn(T, 20, device=DEV)]) for T in (1, 8, 9, 64)]
    progs += [("expanded", lambda dY: [nvq.mxfp4_gemm_dx(dY, *wide)], lambda: [torch.randn(3400, 64, device=DEV).to(torch.bfloat16)])]
    return progs


def _equal(a, b):
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_same_bits_every_time(nvq):
    for _, run, draw in _programs(nvq, 1):
        ins = draw()
        first = [t.clone() for t in run(*ins)]
        for _ in range(3):
            _equal(run(*ins), first)


def test_captured_and_replayed(nvq):
    """Each program in a graph, replayed on new inputs with eager runs of the same shapes between the replays."""
    torch.manual_seed(3)
    for name, run, draw in _programs(nvq, 2):
        ins = draw()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(*ins)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run(*ins)
        for _ in range(4):
            fresh = draw()
            eager = [t.clone() for t in run(*fresh)]
            run(*draw())
            for a, b in zip(ins, fresh):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            _equal(outs, eager)
        del graph


def test_two_graphs_in_turn(nvq):
    """Two captured calls of one operator, replayed in turn and on two streams: neither uses the other's workspace."""
    torch.manual_seed(4)
    for name, run, draw in _programs(nvq, 3):
        made = []
        for _ in range(2):
            ins = draw()
            run(*ins)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = run(*ins)
            made.append((graph, outs, [t.clone() for t in run(*ins)], ins))   # (a graph reads its inputs where they were)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, *_), s in zip(made, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _ in made:
            _equal(outs, want)
        del made


def test_two_streams_at_once(nvq):
    torch.manual_seed(5)
    for name, run, draw in _programs(nvq, 4):
        ins = [draw(), draw()]
        want = [[t.clone() for t in run(*i)] for i in ins]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            for i, s in zip(ins, streams):
                with torch.cuda.stream(s):
                    got.append(run(*i))
        torch.cuda.synchronize()
        for j, outs in enumerate(got):
            _equal(outs, want[j % 2])


# ---- the largest widths -------------------------------------------------------------------------
def _sparse(g, n, k, dtype=torch.bfloat16):
    """[n, k], zero but for 40 columns, the first and the last ones: small sums wherever they lie."""
    X = torch.zeros(n, k, dtype=dtype, device=DEV)
    at = torch.cat((torch.tensor([0, 1, k - 2, k - 1], device=DEV), torch.randint(0, k, (36,), device=DEV, generator=g))).unique()
    X[:, at] = torch.randn(n, len(at), device=DEV, generator=g).to(dtype)
    return X, at


@pytest.mark.parametrize("n", [1, 7, 40, 150])
def test_widest_products(nvq, n):
    g = _gen(n, 21)
    k, m = 3999968, 9
    wc, ws = _codes(g, m, k)
    X, at = _sparse(g, n, k)
    xc, xs = nvq.mxfp4_quantize(X)
    blocks = (at // 32).unique()
    cols = (blocks[:, None] * 32 + torch.arange(32, device=DEV)).flatten()
    x = torch.cat([_values(xc[:, 16 * b:16 * b + 16], xs[:, b:b + 1]) for b in blocks.tolist()], 1)
    w = torch.cat([_values(wc[:, 16 * b:16 * b + 16], ws[:, b:b + 1]) for b in blocks.tolist()], 1)
    assert int((xc != 0).sum()) == int((xc[:, (cols[::2] // 2)] != 0).sum())
    for Y in (nvq.mxfp4_gemm(X, wc, ws), nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs)):
        _close(Y, x, w.T, len(cols) / 32)                   # (zeros add nothing)
    m, k = 4000000, 32
    wc, ws = _codes(g, m, k)
    xc, xs = _codes(g, n, k)
    Y = nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs, out_dtype=torch.bfloat16)
    for rows in (slice(0, 500), slice(m - 500, m)):
        _close(Y[:, rows], _values(xc, xs), _values(wc[rows], ws[rows]).T, k / 32)
    dY, at = _sparse(g, n, m)
    _close(nvq.mxfp4_gemm_dx(dY, wc, ws), dY[:, at].double(), _values(wc[at], ws[at]), len(at) / 16)
    wc, ws = _codes(g, 16, 3999968)
    dY = torch.randn(n, 16, device=DEV, generator=g).to(torch.bfloat16)
    dX = nvq.mxfp4_gemm_dx(dY, wc, ws, out_dtype=torch.bfloat16)
    _close(dX[:, -640:], dY.double(), _values(wc[:, -320:].contiguous(), ws[:, -20:].contiguous()), 1)


E4M3 = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def _expert_values(layer, e, rows, cols):
    codes, scales, gs = layer
    c = (codes[e][rows][:, cols // 2].long() >> (4 * (cols % 2))) & 15
    return GRID.to(DEV)[c] * E4M3.to(DEV)[scales[e][rows][:, cols // 16].long()] * gs[e].double()


@pytest.mark.parametrize("T", [1, 30])
@pytest.mark.parametrize("d,h,m", [(3999984, 32, 8), (32, 3999984, 8), (32, 32, 4000000)])
def test_widest_expert_mlp(nvq, T, d, h, m):
    """At most 48 terms that are not zero per sum: 64 roundings of 2^-23 cover each, as in the operator's own tests."""
    g = _gen(T, d, h)
    gu, dn = _experts(g, 2, 2 * h, d), _experts(g, 2, m, h)
    keep = torch.arange(h, device=DEV)
    if h > 32:                                             # all but some of the activations zero
        keep = torch.cat((torch.tensor([0, h - 1], device=DEV), torch.randint(0, h, (30,), device=DEV, generator=g))).unique()
        codes = torch.zeros_like(gu[0])
        for part in (keep, keep + h):
            codes[:, part] = gu[0][:, part]
        gu = (codes,) + gu[1:]
    gu, dn = ((c, s, v * k ** 0.5) for (c, s, v), k in ((gu, d), (dn, h)))      # (a term's size, not a long sum's)
    X, at = _sparse(g, T, d) if d > 32 else (torch.randn(T, d, device=DEV, generator=g).to(torch.bfloat16), torch.arange(d, device=DEV))
    logits = torch.randn(T, 2, device=DEV, generator=g)
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=1, out_dtype=torch.float32)
    assert torch.equal(ids[:, 0].long(), logits.argmax(1)) and bool((w == 1).all())
    some = torch.arange(m, device=DEV) if m < 1000 else torch.cat((torch.arange(500, device=DEV), torch.arange(m - 500, m, device=DEV)))
    u = 64 * 2.0 ** -23
    for e in (0, 1):
        mine = ids[:, 0] == e
        x = X[mine][:, at].double()
        gate, up = (x @ _expert_values(gu, e, part, at).T for part in (keep, keep + h))
        eg, eu = (u * (x.abs() @ _expert_values(gu, e, part, at).abs().T) for part in (keep, keep + h))
        silu = gate * torch.sigmoid(gate)
        act = silu * up
        ea = 1.1 * eg * up.abs() + silu.abs() * eu + 1.1 * eg * eu + act.abs() * (2.0 ** -16 + 32 * 2.0 ** -24)
        D = _expert_values(dn, e, some, keep).T
        bound = ea @ D.abs() + 2 * u * ((act.abs() + ea) @ D.abs()) + 1e-30
        assert bool(((out[mine][:, some].double() - act @ D).abs() <= bound).all())
    assert float(out.abs().max()) > 0


# ---- beyond 32-bit offsets ---------------------------------------------------------------------
def test_quantize_and_swiglu_past_32_bits(nvq):
    n, k = 70001, 65536                                    # 4.6e9 values
    X = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    X.fill_(1.5)
    X[-3:] = torch.randn(3, k, device=DEV).to(torch.bfloat16)
    codes, scales = nvq.mxfp4_quantize(X)
    c, s = nvq.mxfp4_quantize(X[-3:].contiguous())
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s)
    back = nvq.mxfp4_dequantize(codes, scales, out_dtype=torch.bfloat16)
    assert torch.equal(back[-3:], nvq.mxfp4_dequantize(c, s, out_dtype=torch.bfloat16)) and bool((back[:5] == 1.5).all())
    del back, codes
    act = nvq.swiglu(X)
    assert torch.equal(act[-3:], nvq.swiglu(X[-3:].contiguous())) and torch.equal(act[-4], act[0])
    dX = nvq.swiglu_backward(act, X)
    assert torch.equal(dX[-3:], nvq.swiglu_backward(act[-3:].contiguous(), X[-3:].contiguous())) and torch.equal(dX[-4], dX[0])


@pytest.mark.parametrize("n", [2, 40, 150])
def test_weights_past_32_bits(nvq, n):
    m, k = 290001, 32768                                   # 4.75e9 bytes of codes
    g = _gen(n, 7)
    wc, ws = _codes(g, m, k)
    xc, xs = _codes(g, n, k)
    Y = nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs)
    at = slice(m - 300, m)
    w = _values(wc[at], ws[at])
    _close(Y[:, at], _values(xc, xs), w.T, k / 32)
    dY = torch.zeros(n, m, dtype=torch.bfloat16, device=DEV)
    dY[:, at] = torch.randn(n, 300, device=DEV, generator=g).to(torch.bfloat16)
    _close(nvq.mxfp4_gemm_dx(dY, wc, ws), dY[:, at].double(), w, m / 16)


def test_outputs_past_32_bits(nvq):
    n, m, k = 70000, 70001, 32                             # 4.9e9 results
    g = _gen(8)
    wc, ws = _codes(g, m, k)
    xc, xs = _codes(g, n, k)
    Y = nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs, out_dtype=torch.bfloat16)
    for rows in (slice(0, 64), slice(n - 64, n)):
        _close(Y[rows], _values(xc[rows], xs[rows]), _values(wc, ws).T, k / 32)
    del Y
    dY = torch.randn(n, 64, device=DEV, generator=g).to(torch.bfloat16)
    wc, ws = _codes(g, 64, 65536)
    dX = nvq.mxfp4_gemm_dx(dY, wc, ws, out_dtype=torch.bfloat16)
    for rows in (slice(0, 64), slice(n - 64, n)):
        _close(dX[rows], dY[rows].double(), _values(wc, ws), 64 / 16)


@pytest.mark.parametrize("T", [2, 20])
def test_experts_past_32_bits(nvq, T):
    """Experts behind 4 GiB of codes give what the same experts give in a small layer."""
    E, d, h, m = 640, 4096, 2048, 4096
    g = _gen(T, 9)
    gu, dn = _experts(g, E, 2 * h, d), _experts(g, E, m, h)
    assert gu[0].numel() > 2 ** 32
    X = torch.randn(T, d, device=DEV, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, 6, (T, 3), dtype=torch.int32, device=DEV, generator=g)
    w = torch.rand(T, 3, device=DEV, generator=g)
    last = [tuple(t[E - 6:].contiguous() for t in x) for x in (gu, dn)]
    small, _, _ = nvq.nvfp4_moe_mlp(X, *last, ids=ids, weights=w, out_dtype=torch.float32)
    large, _, _ = nvq.nvfp4_moe_mlp(X, gu, dn, ids=ids + (E - 6), weights=w, out_dtype=torch.float32)
    # Both are within the operator's bound of the exact layer (a wave's share of the second sum may differ): activations by
    # 2 * 2.2 * (d / 16 + 16) 2^-23 < 2^-12 of |G||x| |U||x| and 2^-16 of themselves, below 1.05 * 2^-12 of that together; second
    # sums by (2 * 3 h / 16 + 48) 2^-23 < 2^-13 of |D||act|.  Twice that for two results.
    tok, off, pos = nvq.moe_sort(ids, 6)
    mag = nvq.nvfp4_gemm_grouped(X.abs(), last[0][0] & 0x77, *last[0][1:], off, tok_idx=tok)
    err = 2 * (1.05 * 2.0 ** -12 + 2.0 ** -13) * 1.02 * mag[:, :h] * mag[:, h:]      # (1.02: the bound's own bf16 and sums)
    bound = nvq.moe_combine(nvq.nvfp4_gemm_grouped(err.to(torch.bfloat16), last[1][0] & 0x77, *last[1][1:], off), pos, w)
    assert bool(small.isfinite().all()) and float(small.abs().max()) > 0
    assert bool(((small - large).abs() <= bound).all())
