"""What the Python functions of the MXFP4 operators refuse before any work."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,page,heads,dim", [(4, 16, 0, 64), (0, 16, 2, 64), (4, 0, 2, 64), (4, 16, 2, 0)])
def test_caches_without_room(pages, page, heads, dim):
    cache = fc2.empty_mxfp4_cache(pages, page, heads, dim)
    q = torch.zeros(1, 8, dim, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(1, heads, dim, device="cuda", dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for call in (lambda: fc2.mxfp4_cache_attention(q, cache, table, lens),
                 lambda: fc2.mxfp4_cache_write(cache, kv, kv, torch.zeros(1, dtype=torch.int64, device="cuda")),
                 lambda: fc2.mxfp4_cache_read(cache, table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)):
        with pytest.raises(ValueError, match="kv_heads"):
            call()


def test_gradients():
    """No backward pass: refused where a graph would be cut, fine without one."""
    w = fc2.mxfp4_quantize(torch.randn(64, 128, device="cuda").requires_grad_())  # codes have no gradient
    cache = fc2.empty_mxfp4_cache(1, 16, 1, 64)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.zero_()
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for m in (3, 40):
        x = torch.randn(m, 128, device="cuda", requires_grad=True)
        with pytest.raises(ValueError, match="gradient"):
            fc2.mxfp4_linear(x, w)
        want = fc2.mxfp4_linear(x.detach(), w)
        with torch.no_grad():
            assert torch.equal(fc2.mxfp4_linear(x, w), want)
    q = torch.randn(1, 2, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        fc2.mxfp4_cache_attention(q, cache, table, lens)
    with torch.inference_mode():
        fc2.mxfp4_cache_attention(q, cache, table, lens)
