"""Drafted tokens over pages of 32 and of 128 rows, and deep caches, against softmax attention in 64 bits."""
import random

import pytest

from approximate_long_context_b200 import binding
from serving import UBF
from test_gpu_tree import DT, Filled, ints, offsets_of, options, random_masks, signed, verify

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ha():
    h = binding.HyperAttention(0)
    yield h
    h.close()


SHAPES = {
    "decode": ([0, 1, 31, 32, 127, 128, 129, 255, 256, 300], [1] * 10, 1),
    "trees": ([0, 64, 127, 128, 500, 1000], [64, 17, 1, 64, 33, 5], 64),
    "loose_bound": ([200, 130], [1, 2], 64),             # max_draft far above the drafts
    "deep": ([9000], [40], 40),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("heads", [(1, 1), (2, 4), (1, 8), (1, 3)], ids=["kv1x1", "kv2x4", "kv1x8", "kv1x3"])
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16_simt"])
def test_tree_over_pages_of_32_and_128(ha, kind, d, page, heads, shape):
    lens, drafts, bound = SHAPES[shape]
    hk, group = heads
    dtype = kind[:4]
    f = Filled(lens, drafts, page=page, hk=hk, d=d, dtype=dtype, seed=d + page + group)
    total = sum(drafts)
    q = torch.randn(total, hk * group, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    masks = random_masks(drafts, random.Random(4), empty=shape == "trees")
    if shape == "trees":
        masks = [m or 1 for m in masks[:64]] + masks[64:]     # the first sequence has no committed rows: no row of it is empty
    options(ha, dtype, kernel="simt" if kind.endswith("simt") else "auto")
    O, lse = torch.full_like(q, 7.0, device="cuda"), torch.full((hk * group, total), 7.0, device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(f.order), ints(offsets_of(drafts)), mask=signed(masks), max_draft=bound,
            layer=f.layer, scale=d ** -0.5, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(f, q, O, lse, lens, drafts, masks, d ** -0.5, UBF if kind == "bf16" else None, dtype == "bf16")
