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
