"""mxfp4_gemm_dx while memory is busy: its kernel copies weights to LDS steps ahead, so a wait that is too short shows as
results that differ from those of a quiet device.  And the steps of an MLP as graphs that run at once, each tensor named.

Bounds as for the product's other tests: the instruction takes 16 of m into its accumulator with at most two roundings of
2^-23, at most 48 additions join parts of a sum: (m / 16 + 48) 2^-23 sum |dy w|.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
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


def _codes(g, n, k, lo=118, hi=124):
    return (torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(lo, hi, (n, k // 32), dtype=torch.uint8, device=DEV, generator=g))


def _values(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    return GRID.to(DEV)[c] * POWERS.to(DEV)[scales.long()].repeat_interleave(32, 1)


# rows x m x k: parts of m of two and more steps, whole and ragged ones, both tile heights, copied rows (m a multiple of 8) and not.
@pytest.mark.parametrize("n,m,k", [(3, 128, 256), (40, 130, 256), (40, 2112, 256), (64, 2049, 288), (333, 1004, 1056), (600, 2112, 256),
                                   (600, 333, 512), (130, 1000, 4128)])
def test_gradient_while_memory_is_busy(nvq, n, m, k):
    g = _gen(n, m, k)
    W = _codes(g, m, k)
    dY = torch.randn(n, m, device=DEV, generator=g).to(torch.bfloat16)
    quiet = nvq.mxfp4_gemm_dx(dY, *W).clone()
    w = _values(*W)
    bound = (m / 16 + 48) * 2.0 ** -23 * (dY.double().abs() @ w.abs())
    assert bool(((quiet.double() - dY.double() @ w).abs() <= bound).all())
    big = torch.randint(0, 255, (1 << 28,), dtype=torch.uint8, device=DEV, generator=g)
    other = torch.empty_like(big)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            other.copy_(big)
        with torch.cuda.stream(streams[1]):
            got.append(nvq.mxfp4_gemm_dx(dY, *W))
    torch.cuda.synchronize()
    for i, dX in enumerate(got):
        assert torch.equal(dX, quiet), f"call {i}: {int((dX != quiet).sum())} of {dX.numel()} values differ"


@pytest.mark.parametrize("n", [1, 2, 3, 40, 130, 600, 1100])
def test_graphs_of_a_dense_step_at_once(nvq, n):
    """A dense MLP on 4-bit operands, forward and back, in two graphs on two streams: each tensor as run by itself."""
    g = _gen(n, 7)
    d, h = 256, 1056
    W1, W2 = _codes(g, 2 * h, d), _codes(g, d, h)

    def step(X, dout):
        xc, xs = nvq.mxfp4_quantize(X)
        hid = nvq.mxfp4_gemm(xc, *W1, x_scales=xs, out_dtype=torch.bfloat16)
        act = nvq.swiglu(hid)
        Y = nvq.mxfp4_gemm(act, *W2)
        dact = nvq.mxfp4_gemm_dx(dout, *W2, out_dtype=torch.bfloat16)
        dhid = nvq.swiglu_backward(dact, hid)
        return {"hid": hid, "act": act, "Y": Y, "dact": dact, "dhid": dhid, "dX": nvq.mxfp4_gemm_dx(dhid, *W1)}

    made = []
    for _ in range(2):
        ins = [torch.randn(n, d, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2)]
        want = {name: t.clone() for name, t in step(*ins).items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*ins)
        made.append((graph, ins, outs, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(6):
        for (graph, *_), s in zip(made, streams):
            with torch.cuda.stream(s):
                graph.replay()
        if turn % 2:
            torch.cuda.synchronize()
            step(*made[0][1])           # eager work between the replays
            torch.cuda.synchronize()
            for i, (_, _, outs, want) in enumerate(made):
                for name in want:
                    assert torch.equal(outs[name], want[name]), (f"{n} rows, graph {i}, {name}: {int((outs[name] != want[name]).sum())} of "
                                                                 f"{want[name].numel()} values differ, turn {turn}")
