"""The MXFP4 product where columns end inside what a warp stores at a time, in
every kernel and output type."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n0,k", [(3, 256, 256), (300, 9472, 128), (700, 2304, 384)])
def test_every_remainder_of_the_columns(m, n0, k, dtype):
    """Small whole numbers: the sums are exact in float32, whatever their order.
    (3 rows; 128 x 128 tiles on more and fewer than half of the SMs.)"""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.tensor([0.0, 1, 2, 3, 4, 6], device="cuda")[torch.randint(0, 6, (m, k), generator=g, device="cuda")]
    w = torch.tensor([0.0, 1, -2, 3, -4, 6], device="cuda")[torch.randint(0, 6, (n0 + 17, k), generator=g, device="cuda")]
    a = fc2.mxfp4_quantize(x)
    ref = (mx.values(x) @ mx.values(w).T).to(dtype)
    for n in range(n0, n0 + 18):
        buf = torch.full((m, n + 3), 7.0, dtype=dtype, device="cuda")
        fc2.mxfp4_gemm(a, fc2.mxfp4_quantize(w[:n]), out=buf[:, :n])
        assert torch.equal(buf[:, :n], ref[:, :n]), n
        assert bool((buf[:, n:] == 7).all())
