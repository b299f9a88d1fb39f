"""A token's result in gfr.moe_decode depends on its own row and choice alone: its bits
stay as they are when the other tokens of a batch of the same size choose other
experts, or none."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("t", [False, True])
@pytest.mark.parametrize("T, k, E, H, I, N", [
    (6, 2, 8, 1024, 768, 512), (24, 3, 16, 1024, 3200, 640), (64, 4, 8, 640, 1024, 1344),
    (16, 16, 128, 1088, 64, 192)])
def test_same_bits_whatever_the_others_choose(T, k, E, H, I, N, t):
    print(T, k, E, H, I, N, t, flush=True)
    g = torch.Generator().manual_seed(T + E + H)
    code = lambda *s: torch.randn(*s, generator=g).to(torch.float8_e4m3fn).to(DEV)
    scale = lambda *s: torch.randint(119, 125, s, generator=g, dtype=torch.uint8).to(DEV)
    w13, s13 = (code(E, 2 * I, H), scale(2 * I, H // 64, 2)) if t else (
        code(E, H, 2 * I), scale(H // 64, 2 * I, 2))
    w2, s2 = (code(E, N, I), scale(N, I // 64, 2)) if t else (
        code(E, I, N), scale(I // 64, N, 2))
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    weights = torch.rand(T, k, generator=g).to(DEV)

    def ids():
        return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()

    mine = [0, T // 2, T - 1]
    first = ids()
    outs = []
    for i in range(5):
        these = first if i == 0 else torch.full_like(first, -1) if i == 4 else ids()
        these[mine] = first[mine]
        outs.append(gfr.moe_decode(x, w13, s13, w2, s2, these.to(DEV), weights, transpose_w13=t,
                                   transpose_w2=t, out_dtype=torch.float32)[mine])
    torch.cuda.synchronize()
    for i, out in enumerate(outs[1:]):
        assert torch.equal(out, outs[0]), f"batch {i + 1}: {(out != outs[0]).float().mean():.3f}"
