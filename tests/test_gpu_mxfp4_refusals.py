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


def test_rows_that_nothing_would_fill():
    """Outputs that no sequence or query writes, or that rows share."""
    cache = fc2.empty_mxfp4_cache(1, 16, 1, 64)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.zero_()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), i32(1)
    q = torch.randn(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no query"):
        fc2.mxfp4_cache_attention(q, cache, table[:0], lens[:0], i32(0), 2)
    with pytest.raises(ValueError, match="no query"):
        fc2.mxfp4_cache_attention(q, cache, table, lens, i32(0, 2), 0)
    for out in (q[:1].expand(2, 2, 64), q[:, :1].expand(2, 2, 64)):
        with pytest.raises(ValueError, match="overlap"):
            fc2.mxfp4_cache_attention(q, cache, table, lens, i32(0, 2), 2, out=out)
    with pytest.raises(ValueError, match="without sequences"):
        fc2.mxfp4_cache_read(cache, table[:0], i32(0), 3)
    # nothing to do is no error
    assert fc2.mxfp4_cache_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 2, 64)
    assert fc2.mxfp4_cache_attention(q[:0], cache, table, lens, i32(0, 0), 0).shape == (0, 2, 64)
    assert fc2.mxfp4_cache_read(cache, table[:0], i32(0), 0)[0].shape == (0, 1, 64)
