"""The few-token expert MLP's own router against moe_topk: the same ids and the same weights, bit for bit, with each
normalization, each number of elements per lane, and on either side of the tokens from which the router runs by itself."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def nvq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_nvfp4_weight_amd as m
    return m


def _experts(g, E, m, k):
    return (torch.randint(0, 256, (E, m, k // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(0x20, 0x60, (E, m, k // 16), dtype=torch.uint8, device=DEV, generator=g),
            torch.rand(E, device=DEV, generator=g) / (32 * k ** 0.5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [1, 8, 60, 64, 65, 100, 128, 129, 256, 257, 300, 512, 513, 1024])
def test_chosen_as_by_moe_topk(nvq, E, renorm, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    gu, dn = _experts(g, E, 64, 32), _experts(g, E, 16, 32)
    K = min(E, 9)
    logits = (4 * torch.randn(64, E + 3, device=DEV, generator=g)).to(dtype)[:, :E]
    X = torch.randn(64, 32, device=DEV, generator=g).to(torch.bfloat16)
    ids, w = nvq.moe_topk(logits, K, renorm=renorm)
    for T in (1, 7, 8, 9, 64):
        out, i, v = nvq.nvfp4_moe_mlp(X[:T], gu, dn, logits=logits[:T], top_k=K, renorm=renorm)
        assert torch.equal(i, ids[:T]), (T, "ids")
        assert torch.equal(v, w[:T]), (T, "weights", (v - w[:T]).abs().max())
        given, _, _ = nvq.nvfp4_moe_mlp(X[:T], gu, dn, ids=ids[:T].contiguous(), weights=w[:T].contiguous())
        assert torch.equal(out, given), (T, "outputs")
