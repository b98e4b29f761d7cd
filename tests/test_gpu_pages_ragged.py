"""Page operations whose lanes and warps have unequal shares of the work, before
and between the barriers of the kernels' cluster."""
import random

import pytest

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_pages import both, extend, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,page,rows,per_row", [(4001, 16, 33, 121), (4001, 16, 257, 31), (9001, 16, 1061, 13),
                                                     (3001, 32, 8193, 2), (2003, 64, 5, 403)])
def test_unequal_rows(pages, page, rows, per_row):
    rng = random.Random(pages + rows)
    host, dev = both(pages, page, rows, per_row)
    room = min(per_row * page // 3, max(2, pages * page // (3 * rows)))
    for step in range(4):
        # one row in five holds something: most lanes have nothing to do, some much
        extend(host, dev, [rng.choice([0, 0, 0, 0, rng.randint(1, room)]) for _ in range(rows)])
        select(host, dev, [rng.choice([b, b, b, -1, rng.randrange(rows)]) for b in range(rows)])
        extend(host, dev, [rng.choice([0, 1]) for _ in range(rows)])
        moves, used = fc2.mxfp4_pages_compact(dev)
        want = host.compact()
        assert moves.tolist() == want[0] and int(used) == want[1]
        host.check(dev)
        select(host, dev, [b if rng.random() < 0.4 else -1 for b in range(rows)])
