"""Attention over the 4-bit cache: what the mask hides from a row does not reach
it, whatever its bytes are.

Outputs are compared with the binary64 definition under the bound of the cache's
tests: half an ulp of the output and 2^-10 of sum p |v| of the row's own keys.
Rows that do see an enlarged key are left out where their own scores or outputs
leave the range in which that bound was derived."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx
from test_gpu_mxfp4_cache import HALF_ULP, cache_values, fill, make_cache, make_table

pytestmark = pytest.mark.gpu


class Case:
    """Sequences of `lens` keys with `nq` queries each at their ends."""

    def __init__(self, lens, nq, hq, hkv, dim, page=16, dtype=torch.bfloat16, seed=0, **mask):
        self.lens, self.nq, self.page, self.mask = lens, nq, page, mask
        self.table, pages = make_table(lens, page, seed)
        self.cache = make_cache(pages, page, hkv, dim, seed + 1)
        self.g = torch.Generator(device="cuda").manual_seed(seed + 2)
        self.k = torch.randn(sum(lens), hkv, dim, generator=self.g, device="cuda")
        self.v = torch.randn(sum(lens), hkv, dim, generator=self.g, device="cuda")
        self.starts = [0]
        for n in nq:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn(self.starts[-1], hq, dim, generator=self.g, device="cuda").to(dtype)

    def positions(self, b):
        return torch.arange(self.lens[b] - self.nq[b], self.lens[b], device="cuda").unsqueeze(1)

    def seen(self, b):
        """[queries, keys] of sequence b."""
        p, j = self.positions(b), torch.arange(self.lens[b], device="cuda")
        s = (j <= p) if self.mask.get("causal", True) else torch.ones_like(j <= p)
        if w := self.mask.get("window", 0):
            s = s & ((j > p - w) | (j < self.mask.get("sinks", 0)))
        return s

    def slots(self, b):
        t = torch.arange(self.lens[b], device="cuda")
        return self.table[b, t // self.page].long() * self.page + t % self.page

    def write(self):
        fill(self.cache, self.table, self.lens, self.page, self.k, self.v)

    def run(self):
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        starts = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = fc2.mxfp4_cache_attention(self.q, self.cache, self.table, lens, starts, max(self.nq), lse=self.lse,
                                             status=status, **self.mask)
        assert int(status) == 0
        return self.out

    def check(self, rows=None):
        """`rows`: the query rows to compare (all)."""
        kc, vc = cache_values(self.cache)
        dim = self.q.shape[2]
        ref, ref_lse, mag = mx.attention(self.q.double(), kc, vc, self.table, self.lens, self.starts, self.page, dim ** -0.5,
                                         **self.mask)
        rows = torch.ones(len(ref), dtype=torch.bool, device="cuda") if rows is None else rows
        out, ref, mag, lse, ref_lse = self.out[rows], ref[rows], mag[rows], self.lse[rows], ref_lse[rows]
        assert len(out) > 0
        assert torch.equal(torch.isnan(out), torch.isnan(ref))
        bound = HALF_ULP[out.dtype] * 1.01 * ref.abs() + 2.0 ** -10 * mag
        bound = bound + (2.0 ** -25 if out.dtype is torch.float16 else 0.0)
        fine = ~torch.isnan(ref)
        worst = float(((out.double() - ref).abs() / bound.clamp(min=1e-300))[fine].max())
        assert worst <= 1.0, worst
        none = ref_lse == -math.inf
        assert torch.equal(lse == -math.inf, none)
        live = ~none & ~torch.isnan(ref_lse)
        assert not bool(live.any()) or float((lse.double() - ref_lse)[live].abs().max()) < 2.0 ** -10


def any_bytes(case, lowest=0):
    """Arbitrary codes and scales (at least `lowest`, NaN among them) in every key
    that no query of its sequence sees: pages that left the window hold other data."""
    c = case.cache
    for b in range(len(case.lens)):
        slots = case.slots(b)[~case.seen(b).any(0)]
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            low = lowest if t is c.k_scales or t is c.v_scales else 0
            t[slots // case.page, :, slots % case.page] = torch.randint(
                low, 256, (len(slots), *t.shape[1:2], t.shape[3]), generator=case.g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(20, 0), (50, 4), (100, 70), (1, 1)])
def test_pages_that_left_the_window(dim, window, sinks):
    for nq, hq in ((1, 8), (1, 16), (3, 4), (100, 4)):
        for lowest in (0, 200):
            case = Case([400, 131, 777], [nq] * 3, hq, 1, dim, seed=window + nq, window=window, sinks=sinks)
            case.write()
            any_bytes(case, lowest)
            case.run()
            case.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_that_left_the_window_without_causality(dim):
    for nq in (1, 6, 150):
        case = Case([500, 260], [nq, nq], 4, 2, dim, seed=nq, causal=False, window=60, sinks=3)
        case.write()
        any_bytes(case, 150)
        case.run()
        case.check()


@pytest.mark.parametrize("mul", [2.0 ** 30, 2.0 ** 60, 2.0 ** 120, 2.0 ** -60])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_later_tokens_leave_earlier_rows_alone(dim, mul):
    """Tokens that only the last queries see have values, then keys, far from the
    other tokens' sizes.  (The rows that see them are compared for the values of
    2^30 and 2^60, whose outputs are in range.)"""
    for lens, nq, hq, late in (([70, 300], [9, 4], 2, 3), ([8, 33], [8, 16], 1, 5), ([600, 90], [120, 90], 4, 40),
                               ([1500], [500], 2, 300)):
        for what in ("values", "keys"):
            case = Case(lens, nq, hq, 1, dim, seed=dim + late)
            at = 0
            first = []
            for b, n in enumerate(lens):
                f = max(n - late, 1)
                x = case.v if what == "values" else case.k
                x[at + f:at + n] *= mul
                first.append(f)
                at += n
            case.write()
            case.run()
            rows = torch.cat([case.positions(b)[:, 0] < first[b] for b in range(len(lens))])
            if bool(rows.any()):
                case.check(rows)
            if what == "values" and mul <= 2.0 ** 60:
                case.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_block_of_a_later_token(dim):
    """The largest finite scale in one block of one token, by its bytes."""
    for lens, nq, hq in (([80], [16], 1), ([300], [12], 1), ([300], [100], 2)):
        for which in ("k_scales", "v_scales"):
            case = Case(lens, nq, hq, 1, dim, seed=dim)
            case.write()
            first = lens[0] - 5
            slot = case.slots(0)[first]
            getattr(case.cache, which)[slot // 16, 0, slot % 16, 1] = 254
            case.run()
            case.check(case.positions(0)[:, 0] < first)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_older_tokens_leave_later_rows_alone(dim):
    """The same at the other end: keys that the window of later rows has passed."""
    for lens, nq, hq, window in (([300], [14], 1, 100), ([300], [7], 2, 130), ([900], [130], 2, 333), ([64], [16], 1, 4)):
        for mul in (2.0 ** 30, 2.0 ** 100):
            for what in ("values", "keys"):
                case = Case(lens, nq, hq, 1, dim, seed=dim + window, window=window)
                first = lens[0] - nq[0] - window + 1  # the oldest key of the first row
                edge = first + nq[0] // 2
                (case.v if what == "values" else case.k)[first:edge] *= mul
                case.write()
                case.run()
                case.check(case.positions(0)[:, 0] - window >= edge - 1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_split_over_workers(dim):
    """Long sequences whose keys many warps or blocks share, large values late."""
    for nq, hq, late in ((4, 4, 2), (80, 2, 50)):
        case = Case([9000], [nq], hq, 1, dim, page=64, seed=nq)
        case.v[9000 - late:] *= 2.0 ** 50
        case.k[9000 - late:, :, :32] *= 2.0 ** 50
        case.write()
        case.run()
        case.check(case.positions(0)[:, 0] < 9000 - late)
