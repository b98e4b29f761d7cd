"""Attention over the 4-bit cache: the ends of its arguments' ranges, and NaN."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_hidden import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 2 ** 40])
def test_windows_past_every_key_hide_none(window, causal):
    """As without a window, also where there are more queries than keys."""
    for lens, nq, hq in (([5, 40], [9, 12], 2), ([3, 0, 100], [200, 5, 130], 2), ([70], [300], 1)):
        for dim in (64, 128, 256):
            case = Case(lens, nq, hq, 1, dim, seed=dim, causal=causal, window=window)
            case.write()
            out = case.run().clone()
            case.check()
            case.mask["window"] = 0
            assert torch.equal(case.run(), out)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_value_of_a_key_without_weight(dim):
    """0 times NaN: a key that a row sees, however small its weight."""
    for nq, hq in ((1, 4), (1, 16), (2, 8), (70, 2)):
        case = Case([100], [nq], hq, 1, dim, seed=nq)
        case.k[:] = 1.0
        case.q[:] = 3.0
        case.k[10] = -60.0   # scores of 3 * dim ** 0.5 and of -180 * dim ** 0.5
        case.v[10, 0, 40] = math.nan
        case.write()
        out = case.run()
        want = torch.zeros_like(out, dtype=torch.bool)
        want[..., 32:64] = True
        assert torch.equal(torch.isnan(out), want), (nq, hq)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_scale_with_codes(dim):
    """E = 255 is NaN whatever the codes beside it are, in a key too."""
    for nq, hq in ((1, 4), (1, 16), (70, 2)):
        for code in (0x22, 0xAA):  # 1 and -1 throughout
            case = Case([100], [nq], hq, 1, dim, seed=nq)
            case.q[:] = 1.0
            case.write()
            slot = case.slots(0)[10]
            case.cache.k_codes[slot // 16, 0, slot % 16] = code
            case.cache.k_scales[slot // 16, 0, slot % 16, 1] = 255
            assert bool(torch.isnan(case.run()).all()), (nq, hq, code)
            assert bool(torch.isnan(case.lse).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_query_rows_past_the_tensor(dim):
    """Starts that lie outside of the query's rows read and write none there."""
    for n, hq in ((5, 2), (60, 4)):
        case = Case([300, 90], [n, n], hq, 1, dim, seed=n)
        case.write()
        want = case.run().clone()
        rows = 2 * n
        lens = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
        buf = torch.full((rows + 40, hq, dim), 3.0, dtype=case.q.dtype, device="cuda")
        for starts in ((0, n, rows + 30), (0, n, 2 ** 31 - 1), (-7, n, rows), (-2 ** 31, n, 2 ** 30)):
            buf.fill_(3.0)
            fc2.mxfp4_cache_attention(case.q, case.cache, case.table, lens,
                                      torch.tensor(starts, dtype=torch.int32, device="cuda"), n, out=buf[20:20 + rows])
            assert torch.equal(buf[20:20 + rows], want)
            assert bool((buf[:20] == 3).all()) and bool((buf[20 + rows:] == 3).all())
        # a second sequence that ends in front of its start has none
        outs = []
        for starts in ((0, n, 0), (0, n, n)):
            buf.fill_(3.0)
            fc2.mxfp4_cache_attention(case.q, case.cache, case.table, lens,
                                      torch.tensor(starts, dtype=torch.int32, device="cuda"), n, out=buf[20:20 + rows])
            outs.append(buf.clone())
        assert torch.equal(outs[0], outs[1]) and bool((buf[20 + n:] == 3).all())
