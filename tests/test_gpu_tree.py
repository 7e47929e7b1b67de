"""Attention of drafted tokens over the paged cache (hyper_attn_tree), the cache's steps (hyper_attn_cache_*), and both in a
run together with the prompt attention, as a server uses them."""
import random

import numpy as np
import pytest

from approximate_long_context_b200 import binding
from serving import UBF, ListCache, attend, check, tolerances

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ha():
    h = binding.HyperAttention(0)
    yield h
    h.close()


def options(ha, dtype, **kw):
    ha.set_options(dtype=dtype, stream=torch.cuda.current_stream().cuda_stream, **kw)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets_of(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def random_masks(drafts, rng, empty=False):
    """Each token sees its ancestors in a random tree and itself; empty: some tokens see nothing of the draft."""
    out = []
    for t in drafts:
        mine = []
        for i in range(t):
            parent = rng.randint(-1, i - 1)
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        if empty:
            mine = [0 if rng.random() < 0.4 else m for m in mine]
        out += mine
    return out


def signed(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


class Filled:
    """A cache whose slots hold lens committed and drafts reserved rows on shuffled pages; every row that is not part of a
    sequence is NaN."""

    def __init__(self, lens, drafts, *, page, hk, d, dtype, seed, layers=2, layer=1, order=None):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        need = [-(-(a + b) // page) for a, b in zip(lens, drafts)]
        pages, most = sum(need) + 5, max(need + [1]) + 2
        shape = (layers, pages, hk, page, d)
        k, v = torch.full(shape, float("nan")), torch.full(shape, float("nan"))
        ids = list(range(pages))
        rng.shuffle(ids)
        slots = len(lens) + 2
        self.order = order or rng.sample(range(slots), len(lens))
        table = np.full((slots, most), -1, np.int32)
        full_lens, held, refs = [0] * slots, [0] * slots, [0] * pages
        self.keys, self.values = [], []
        for i, s in enumerate(self.order):
            n = lens[i] + drafts[i]
            mine, ids = ids[:need[i]], ids[need[i]:]
            table[s, :need[i]] = mine
            full_lens[s], held[s] = lens[i], need[i]
            rows = torch.randn(2, n, hk, d, generator=g)
            for j in range(n):
                k[layer, mine[j // page], :, j % page] = rows[0, j]
                v[layer, mine[j // page], :, j % page] = rows[1, j]
            for p in mine:
                refs[p] = 1
            self.keys.append(rows[0].to(DT[dtype]))
            self.values.append(rows[1].to(DT[dtype]))
        self.layer = layer
        self.cache = binding.PagedCache(k.to(DT[dtype]).cuda(), v.to(DT[dtype]).cuda(), torch.from_numpy(table).cuda(),
                                        ints(full_lens), ints(held), ints(refs))


def verify(f, q, o, lse, lens, drafts, masks, scale, p_bits, out_bf16, skip=()):
    at = offsets_of(drafts)
    for i, (n, t) in enumerate(zip(lens, drafts)):
        if t == 0 or i in skip:
            continue
        a, b = at[i], at[i + 1]
        seen = torch.ones(t, n + t, dtype=torch.bool)
        for r in range(t):
            m = masks[a + r] if masks is not None else (1 << (r + 1)) - 1
            seen[r, n:] = torch.tensor([bool(m >> j & 1) for j in range(t)])
        want = attend(q[a:b], f.keys[i], f.values[i], seen, scale)
        want = (torch.nan_to_num(want[0]),) + want[1:]
        tol = tolerances(*[torch.nan_to_num(x, neginf=0.0) if j == 1 else x for j, x in enumerate(want)], n + t, q.shape[2],
                         p_bits=p_bits, out_bf16=out_bf16)
        check(o[a:b], None if lse is None else lse[:, a:b], want[:2], tol, f"sequence {i}: {n} + {t}")


SHAPES = {
    # committed rows, drafted rows
    "one_token": ([1000], [1]),
    "first_token": ([0], [1]),
    "decode": ([0, 1, 15, 16, 17, 127, 128, 129, 255, 300], [1] * 10),
    "trees": ([0, 3, 64, 100, 127, 128, 500], [64, 1, 17, 33, 2, 64, 5]),
    "idle": ([40, 70, 0, 9], [0, 3, 0, 2]),
    "long": ([5000, 20], [7, 64]),
}
HEADS = [(1, 1), (2, 4), (1, 8), (3, 5)]


@pytest.mark.parametrize("shape", list(SHAPES), ids=list(SHAPES))
@pytest.mark.parametrize("heads", HEADS, ids=[f"kv{a}x{b}" for a, b in HEADS])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16_simt"])
def test_tree_matches_definition(ha, kind, d, page, heads, shape):
    lens, drafts = SHAPES[shape]
    hk, group = heads
    dtype = kind[:4]
    f = Filled(lens, drafts, page=page, hk=hk, d=d, dtype=dtype, seed=d + page + group)
    total = sum(drafts)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(total, hk * group, d, generator=g).to(DT[dtype])
    masks = random_masks(drafts, random.Random(4))
    options(ha, dtype, kernel="simt" if kind.endswith("simt") else "auto")
    O, lse = torch.full_like(q, 7.0, device="cuda"), torch.full((hk * group, total), 7.0, device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(f.order), ints(offsets_of(drafts)), mask=signed(masks), max_draft=max(drafts),
            layer=f.layer, scale=d ** -0.5, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(f, q, O, lse, lens, drafts, masks, d ** -0.5, UBF if kind == "bf16" else None, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group,draft", [(128, 1), (100, 3), (16, 64), (7, 19)])
def test_many_rows_to_one_key_head(ha, dtype, group, draft):
    lens, drafts = [333, 10], [draft, 1]
    f = Filled(lens, drafts, page=32, hk=1, d=64, dtype=dtype, seed=group)
    q = torch.randn(sum(drafts), group, 64, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O, lse = torch.empty_like(q, device="cuda"), torch.empty(group, sum(drafts), device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(f.order), ints(offsets_of(drafts)), max_draft=64, layer=1, scale=0.125, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(f, q, O, lse, lens, drafts, None, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")


@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16_to_fp32"])
@pytest.mark.parametrize("draft", [1, 20])
def test_many_sequences(ha, kind, draft):
    """More sequences than a warp has lanes, some idle, one of them out of range; a slot that two sequences read."""
    rng = random.Random(draft)
    dtype, hk, group, d = kind[:4], 2, 8, 64
    lens = [rng.choice([0, 1, 77, 128, 300, 1000]) for _ in range(110)]
    drafts = [0 if rng.random() < 0.1 else rng.randint(1, draft) for _ in lens]
    drafts[40] = drafts[41] = 1
    f = Filled(lens, drafts, page=16, hk=hk, d=d, dtype=dtype, seed=draft)
    slots = list(f.order)
    slots[40] = slots[41]                       # both read slot 41's rows
    slots[77] = 10 ** 6
    lens[40], f.keys[40], f.values[40] = lens[41], f.keys[41], f.values[41]
    drafts[77] = max(drafts[77], 1)
    total = sum(drafts)
    q = torch.randn(total, hk * group, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    bf = kind == "bf16"
    options(ha, dtype, out_dtype="fp32" if kind.endswith("to_fp32") else None)
    O = torch.full(q.shape, 7.0, dtype=torch.bfloat16 if bf else torch.float32, device="cuda")
    lse = torch.full((hk * group, total), 7.0, device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(slots), ints(offsets_of(drafts)), max_draft=draft, layer=1, scale=0.125, lse=lse)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    verify(f, q, O.cpu(), lse.cpu(), lens, drafts, None, 0.125, UBF if dtype == "bf16" else None, bf, skip=(77,))
    a = offsets_of(drafts)
    assert bool((O[a[77]:a[78]] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group,draft", [(2, 5), (8, 64)])
def test_not_finite_in_a_long_cache(ha, dtype, group, draft):
    """A context cut over many blocks: infinities in a drafted row and in the last, partly masked tile of the context
    reach the tokens that see them and no other."""
    n, d = 6000, 128
    f = Filled([n], [draft], page=64, hk=1, d=d, dtype=dtype, seed=5, order=[0])
    masks = [1 << i for i in range(draft)]      # every token sees itself alone of the draft
    at = n + 3
    cache = f.cache
    cache.v[1, cache.table[0, at // 64].item(), 0, at % 64, 9] = float("inf")
    q = torch.randn(draft, group, d, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O = torch.empty_like(q, device="cuda")
    call = lambda: ha.tree(q.cuda(), cache, O, None, ints([0, draft]), mask=signed(masks), max_draft=draft, layer=1, scale=0.09)  # noqa: E731
    call()
    assert ha.status() == 0, ha.last_error()
    assert bool((O[3, :, 9].float() == float("inf")).all())
    O[3, :, 9] = 0
    assert bool(torch.isfinite(O).all())
    f.values[0][at, 0, 9] = 0
    keep = [i for i in range(draft) if i != 3]
    seen = torch.ones(draft, n + draft, dtype=torch.bool)
    seen[:, n:] = torch.eye(draft, dtype=torch.bool)
    want = attend(q, f.keys[0], f.values[0], seen, 0.09)
    tol = tolerances(*want, n + draft, d, p_bits=UBF if dtype == "bf16" else None, out_bf16=dtype == "bf16")
    check(O.cpu()[keep], None, [want[0][keep], want[1]], [tol[0][keep], tol[1]])
    at = n - 1                                  # the context's last row, in a masked tile: every token sees it
    cache.v[1, cache.table[0, at // 64].item(), 0, at % 64, 11] = float("-inf")
    call()
    assert bool((O[:, :, 11].float() == float("-inf")).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_graphs_on_two_streams(ha, dtype):
    """Two captured decode steps replayed at once on two streams, each with its own workspace."""
    lens, drafts = [700, 3000, 64], [4, 1, 9]
    total = sum(drafts)
    state = []
    for i in range(2):
        s = torch.cuda.Stream()
        f = Filled(lens, drafts, page=32, hk=2, d=64, dtype=dtype, seed=50 + i)
        q = torch.randn(total, 8, 64, generator=torch.Generator().manual_seed(i)).to(DT[dtype])
        Q, at, slots = q.cuda(), ints(offsets_of(drafts)), ints(f.order)
        O = torch.empty_like(Q)
        torch.cuda.synchronize()
        ha.set_options(dtype=dtype, stream=s.cuda_stream)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                ha.tree(Q, f.cache, O, slots, at, max_draft=9, layer=1, scale=0.125)
        state.append((s, f, q, Q, O, g, at, slots))
    options(ha, dtype)
    for r in range(4):
        for _, _, _, _, O, _, _, _ in state:
            O.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, _, _, _, _, g, _, _ in state:
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for _, f, q, _, O, _, _, _ in state:
            verify(f, q, O.cpu(), None, lens, drafts, None, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert ha.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_see_nothing(ha, dtype):
    """Masks that leave drafted tokens of the context, and with an empty context nothing at all: 0 and -inf."""
    lens, drafts = [0, 0, 50], [9, 1, 12]
    f = Filled(lens, drafts, page=16, hk=2, d=128, dtype=dtype, seed=3)
    masks = random_masks(drafts, random.Random(2), empty=True)
    masks[0], masks[9] = 0, 0
    q = torch.randn(22, 4, 128, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O, lse = torch.full_like(q, 7.0, device="cuda"), torch.full((4, 22), 7.0, device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(f.order), ints(offsets_of(drafts)), mask=signed(masks), max_draft=12, layer=1,
            scale=0.1, lse=lse)
    assert ha.status() == 0, ha.last_error()
    assert bool((O[0] == 0).all()) and bool((O[9] == 0).all()) and bool(torch.isneginf(lse[:, 9]).all())
    verify(f, q, O, lse, lens, drafts, masks, 0.1, UBF if dtype == "bf16" else None, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
def test_not_finite_in_masked_drafts(ha, dtype, value, d):
    """A drafted row that is not finite reaches the tokens that see it and no other."""
    lens, drafts = [100], [6]
    f = Filled(lens, drafts, page=16, hk=1, d=d, dtype=dtype, seed=8)
    masks = [1, 2, 5, 9, 16, 33]
    at = 102                         # drafted row 2, seen by token 2 alone
    page, row = f.cache.table[f.order[0]][at // 16], at % 16
    f.cache.v[1, page, 0, row, 7] = value
    q = torch.randn(6, 2, d, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O = torch.empty_like(q, device="cuda")
    call = lambda: ha.tree(q.cuda(), f.cache, O, ints(f.order), ints([0, 6]), mask=signed(masks), max_draft=6, layer=1, scale=0.125)  # noqa: E731
    call()
    assert ha.status() == 0, ha.last_error()
    hit = O[2, :, 7].float()
    assert bool(torch.isnan(hit).all()) if value != value else bool((hit == value).all())
    O[2, :, 7] = 0
    assert bool(torch.isfinite(O).all())
    want = O.clone()
    f.cache.k[1, page, 0, row, 3] = float("nan")
    call()
    assert bool(torch.isnan(O[2]).all())
    O[2], want[2] = 0, 0
    assert torch.equal(O, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fault", ["slot", "negative_slot", "held", "length", "draft", "offsets"])
def test_bad_state_is_left_out(ha, dtype, fault):
    """One sequence with a slot, length or offset out of range: it is left out and reported, the others are right."""
    lens, drafts = [30, 200, 17], [4, 3, 5]
    f = Filled(lens, drafts, page=16, hk=2, d=64, dtype=dtype, seed=6)
    q = torch.randn(12, 4, 64, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O = torch.full_like(q, 5.0, device="cuda")
    slots, at, most = list(f.order), offsets_of(drafts), 5
    if fault == "slot":
        slots[1] = 5
    elif fault == "negative_slot":
        slots[1] = -1
    elif fault == "held":
        f.cache.held[slots[1]] = f.cache.args.max_pages + 1
    elif fault == "length":
        f.cache.lens[slots[1]] = 16 * int(f.cache.held[slots[1]]) - 2
    elif fault == "draft":
        drafts, at, most = [3, 4, 5], [0, 3, 7, 12], 3
    else:
        at = [0, 4, 7, 13]
    ha.tree(q.cuda(), f.cache, O, ints(slots), ints(at), max_draft=most, layer=1, scale=0.125)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    p_bits, bf = UBF if dtype == "bf16" else None, dtype == "bf16"
    if fault == "draft":             # sequences of 4 and 5 rows where 3 were promised
        f.keys[0], f.values[0] = f.keys[0][:33], f.values[0][:33]
        verify(f, q, O, None, lens, drafts, None, 0.125, p_bits, bf, skip=(1, 2))
        assert bool((O[3:] == 5).all())
    elif fault == "offsets":
        verify(f, q, O, None, lens, [4, 3, 0], None, 0.125, p_bits, bf)
        assert bool((O[7:] == 5).all())
    else:
        verify(f, q, O, None, lens, drafts, None, 0.125, p_bits, bf, skip=(1,))
        assert bool((O[4:7] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_are_reported(ha, dtype, bad, d):
    """A page out of range in one sequence: nothing is read there, the call reports it, the other sequences are right."""
    lens, drafts = [30, 200, 17], [4, 3, 5]
    f = Filled(lens, drafts, page=16, hk=2, d=d, dtype=dtype, seed=6)
    f.cache.table[f.order[1], 4] = bad
    q = torch.randn(12, 4, d, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    options(ha, dtype)
    O = torch.full_like(q, 5.0, device="cuda")
    ha.tree(q.cuda(), f.cache, O, ints(f.order), ints(offsets_of(drafts)), max_draft=5, layer=1, scale=0.125)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    verify(f, q, O, None, lens, drafts, None, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16", skip=(1,))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_rows_behind_and_strides(ha, dtype):
    lens, drafts = [70, 3], [5, 1]
    f = Filled(lens, drafts, page=32, hk=2, d=64, dtype=dtype, seed=6, order=[0, 1])
    wide = torch.randn(9, 8, 64 + 16, generator=torch.Generator().manual_seed(2)).to(DT[dtype]).cuda()
    q = wide[:, ::2, :64]
    whole = torch.full((4, 9, 64), 5.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((4, 9), 5.0, device="cuda")
    options(ha, dtype)
    ha.tree(q, f.cache, whole.transpose(0, 1), None, ints([0, 5, 6]), max_draft=5, layer=1, scale=0.125, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(f, q.cpu(), whole.transpose(0, 1), lse, lens, drafts, None, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert bool((whole[:, 6:] == 5).all()) and bool((lse[:, 6:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pages_far_into_the_cache(ha, dtype):
    """Row offsets beyond 2^32 bytes and 2^31 elements."""
    d, hk, page = 128, 8, 256
    pages = (2 ** 31) // (d * hk * page) + 40
    cache = binding.PagedCache.empty(layers=1, pages=pages, kv_heads=hk, page=page, d=d, slots=1, max_pages=2, dtype=dtype)
    g = torch.Generator().manual_seed(4)
    k, v = torch.randn(2, 300, hk, d, generator=g).to(DT[dtype])
    options(ha, dtype)
    cache.refs.fill_(1)
    cache.refs[-3:] = 0
    ha.cache_reserve(cache, ints([0]), ints([300]))
    ha.cache_append(cache, ints([0]), ints([0, 300]), k[None].cuda(), v[None].cuda())
    ha.cache_commit(cache, ints([0]), ints([297]))
    q = torch.randn(3, hk * 2, d, generator=g).to(DT[dtype])
    O = torch.empty_like(q, device="cuda")
    ha.tree(q.cuda(), cache, O, None, ints([0, 3]), max_draft=3, scale=0.1)
    assert ha.status() == 0, ha.last_error()
    assert cache.table[0].tolist() == [pages - 3, pages - 2]
    f = type("F", (), {"keys": [k], "values": [v]})
    verify(f, q, O, None, [297], [3], None, 0.1, UBF if dtype == "bf16" else None, dtype == "bf16")


def test_tree_equal_calls_give_equal_bits(ha):
    lens, drafts = [3000, 17, 900], [9, 64, 1]
    f = Filled(lens, drafts, page=64, hk=4, d=128, dtype="bf16", seed=6)
    q = torch.randn(74, 16, 128).to(torch.bfloat16).cuda()
    options(ha, "bf16")
    outs = [torch.empty_like(q) for _ in range(3)]
    for o in outs:
        ha.tree(q, f.cache, o, ints(f.order), ints(offsets_of(drafts)), layer=1, scale=0.1)
    assert ha.status() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_tree_refusals(ha):
    f = Filled([20], [2], page=16, hk=2, d=64, dtype="bf16", seed=1, order=[0])
    options(ha, "bf16")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 9.0)
    cu = ints([0, 2])

    def refused(code, *args, **kw):
        with pytest.raises(binding.HAError) as e:
            ha.tree(*args, **kw)
        assert e.value.code == code and ha.last_error()

    inv, uns = binding.HA_ERR_INVALID_ARG, binding.HA_ERR_UNSUPPORTED
    for bad in (0, 65, -1):
        refused(inv, q, f.cache, o, None, cu, max_draft=bad)
    for bad in (-1, 2):
        refused(inv, q, f.cache, o, None, cu, layer=bad)
    refused(inv, q, f.cache, o, None, cu, scale=0.0)
    refused(inv, q, f.cache, q, None, cu)
    three = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    refused(inv, three, f.cache, three.clone(), None, cu)
    odd = torch.zeros(2, 4, 2, 24, 64, dtype=torch.bfloat16, device="cuda")
    c = binding.PagedCache(odd, odd.clone(), f.cache.table, f.cache.lens, f.cache.held, ints([0] * 4))
    refused(uns, q, c, o, None, cu)                             # pages of 24 rows
    for bad in ((q.float(), f.cache, o, None, cu), (q, f.cache, o, ints([0, 1]), cu), (q, f.cache, o, None, cu.long())):
        with pytest.raises(ValueError):
            ha.tree(*bad)
    with pytest.raises(ValueError):
        ha.tree(q, f.cache, o, None, cu, mask=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        binding.PagedCache(f.cache.k, f.cache.v[:1], f.cache.table, f.cache.lens, f.cache.held, f.cache.refs)
    args = binding.TreeArgs()
    assert binding.lib().hyper_attn_tree(ha._h, None, args) == inv
    assert binding.lib().hyper_attn_tree(ha._h, f.cache.args, None) == inv
    assert binding.lib().hyper_attn_tree(None, f.cache.args, args) == inv
    torch.cuda.synchronize()
    assert bool((o == 9).all()) and ha.status() == 0


# ---- the cache's steps

def same_state(cache, ref):
    table, lens, held, refs = ref.state()
    assert np.array_equal(cache.lens.cpu().numpy(), lens)
    assert np.array_equal(cache.held.cpu().numpy(), held)
    assert np.array_equal(cache.refs.cpu().numpy(), refs)
    assert np.array_equal(cache.table.cpu().numpy(), table)


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("seed,page,hk,d,pages", [(1, 16, 2, 64, 40), (2, 32, 1, 128, 14), (3, 256, 3, 64, 9), (4, 16, 8, 128, 70)])
def test_cache_steps_random_run(ha, dtype, seed, page, hk, d, pages):
    """A long random run of all steps against plain Python lists, in a pool that runs out now and then."""
    rng = random.Random(seed)
    slots, most, layers = 9, 12, 3
    cache = binding.PagedCache.empty(layers=layers, pages=pages, kv_heads=hk, page=page, d=d, slots=slots, max_pages=most, dtype=dtype)
    options(ha, dtype)
    ref = ListCache(bits(cache.k).copy(), bits(cache.v).copy(), slots, most)
    short = 0
    for step in range(60):
        act = rng.choice(["grow", "grow", "grow", "fork", "free"])
        if act == "free":
            who = rng.sample(range(slots), rng.randint(1, 3))
            ha.cache_free(cache, ints(who))
            ref.free(who)
        elif act == "fork":
            empty = [s for s in range(slots) if not ref.rows[s] and not ref.lens[s]]
            full = [s for s in range(slots) if s not in empty]
            if not empty or not full:
                continue
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(full) for _ in dst]
            ha.cache_fork(cache, ints(src), ints(dst))
            ref.fork(src, dst)
        else:
            who = rng.sample(range(slots), rng.randint(1, slots))
            add = [min(rng.choice([0, 1, 3, 17, page, 2 * page + 1]), most * page - ref.lens[s]) for s in who]
            granted = torch.full((len(who),), -5, dtype=torch.int32, device="cuda")
            ha.cache_reserve(cache, ints(who), ints(add), granted)
            want = ref.reserve(who, add)
            assert granted.tolist() == want
            short += want != add
            at = offsets_of(want)
            new = [torch.randn(layers, at[-1], hk, d, generator=torch.Generator().manual_seed(step + i)).to(DT[dtype]) for i in (0, 99)]
            if at[-1]:
                ha.cache_append(cache, ints(who), ints(at), new[0].cuda(), new[1].cuda())
                ref.append(who, at, bits(new[0]), bits(new[1]))
            if rng.random() < 0.5:
                counts = [rng.randint(0, n) for n in want]
                keep = [sorted(rng.sample(range(n), c)) for n, c in zip(want, counts)]
                wide = max(want + [1])
                ha.cache_commit(cache, ints(who), ints(counts), ints([k + [-9] * (wide - len(k)) for k in keep]).view(len(who), wide))
                ref.commit(who, counts, keep)
            else:
                counts = [rng.randint(0, n) for n in want]
                ha.cache_commit(cache, ints(who), ints(counts))
                ref.commit(who, counts)
        assert ha.status() == 0, ha.last_error()
        same_state(cache, ref)
    assert short or pages > 30
    assert np.array_equal(bits(cache.k), ref.k) and np.array_equal(bits(cache.v), ref.v)


def test_append_strides_and_layers(ha):
    """One layer at a time, from a fused projection's output; a broadcast head."""
    cache = binding.PagedCache.empty(layers=3, pages=8, kv_heads=2, page=16, d=64, slots=2, max_pages=4)
    options(ha, "bf16")
    ha.cache_reserve(cache, ints([1]), ints([20]))
    fused = torch.randn(20, 6 * 64, device="cuda").to(torch.bfloat16)
    k, v = fused[:, 128:256].view(1, 20, 2, 64), fused[:, 256:].view(1, 20, 2, 64)
    ha.cache_append(cache, ints([1]), ints([0, 20]), k, v, layer=2)
    ha.cache_append(cache, ints([1]), ints([0, 20]), k[:, :, :1].expand(1, 20, 2, 64), v[:, :1].expand(1, 20, 2, 64), layer=0)
    assert ha.status() == 0, ha.last_error()
    rows = lambda x, l: x[l][cache.table[1][:2].long()].transpose(1, 2).reshape(32, 2, 64)[:20]  # noqa: E731
    assert torch.equal(rows(cache.k, 2), k[0]) and torch.equal(rows(cache.v, 2), v[0])
    assert torch.equal(rows(cache.k, 0), k[0, :, :1].expand(20, 2, 64)) and torch.equal(rows(cache.v, 0), v[0, :1].expand(20, 2, 64))
    assert bool((cache.k[1] == 0).all())


def test_cache_entries_out_of_range(ha):
    """Bad and repeated entries are left out and reported; the rest of the list is served."""
    options(ha, "bf16")

    def fresh():
        c = binding.PagedCache.empty(layers=1, pages=10, kv_heads=1, page=16, d=64, slots=4, max_pages=3)
        ha.cache_reserve(c, ints([0]), ints([20]))
        ha.cache_commit(c, ints([0]), ints([20]))
        assert ha.status() == 0
        return c

    def bad(n=1):
        assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0

    c = fresh()
    ha.cache_free(c, ints([0, 7, 0, -1]))
    bad()
    assert c.lens.tolist() == [0] * 4 and c.refs.tolist() == [0] * 10
    c = fresh()
    ha.cache_fork(c, ints([0, 0, 0, 9, 0]), ints([1, 1, 9, 2, 0]))      # twice, out of range twice, onto itself
    bad()
    assert c.lens.tolist() == [20, 0, 0, 0]                                # 0 is a destination too: no fork from it
    ha.cache_fork(c, ints([0, 0, 9]), ints([1, 1, 2]))
    bad()
    assert c.lens.tolist() == [20, 20, 0, 0] and c.refs.tolist() == [2, 2] + [0] * 8
    ha.cache_fork(c, ints([0]), ints([1]))                                  # not empty
    bad()
    assert c.refs.tolist() == [2, 2] + [0] * 8
    g = ints([-5] * 5)
    ha.cache_reserve(c, ints([1, 1, 4, 2, 3]), ints([1, 5, 1, -1, 49]), g)  # twice, out of range, negative, beyond the table
    bad()
    assert g.tolist() == [1, 0, 0, 0, 0]
    assert c.table.tolist() == [[0, 1, -1], [0, 2, -1], [-1] * 3, [-1] * 3] and c.refs.tolist() == [2, 1, 1] + [0] * 7
    row = torch.ones(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    ha.cache_append(c, ints([2, 0]), ints([0, 2, 4]), row, row)             # nothing reserved; slot 0 fits in its page
    bad()
    assert c.k.sum().item() == 2 * 64
    ha.cache_append(c, ints([0, 5]), ints([0, 2, 4]), row, row)
    bad()
    ha.cache_append(c, ints([1]), ints([0, 13]), torch.ones(1, 13, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 13, 1, 64, dtype=torch.bfloat16, device="cuda"))
    bad()                                                                   # the 13th row has no page
    for counts, keep in (([13], None), ([-1], None), ([2], [[3, 3]]), ([2], [[5, 4]]), ([2], [[0, 12]]), ([2], [[-1, 2]]), ([3], [[0, 1]])):
        before = c.k.clone()
        ha.cache_commit(c, ints([1]), ints(counts), None if keep is None else ints(keep))
        bad()
        assert c.lens.tolist() == [20, 20, 0, 0] and torch.equal(c.k, before)
    ha.cache_commit(c, ints([1, 1, 8]), ints([3, 4, 1]))
    bad()
    assert c.lens.tolist() == [20, 23, 0, 0]


def test_append_does_not_write_a_shared_page(ha):
    options(ha, "bf16")
    c = binding.PagedCache.empty(layers=1, pages=6, kv_heads=1, page=16, d=64, slots=2, max_pages=3)
    ha.cache_reserve(c, ints([0]), ints([20]))
    ha.cache_commit(c, ints([0]), ints([20]))
    ha.cache_fork(c, ints([0]), ints([1]))
    row = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    ha.cache_append(c, ints([1]), ints([0, 1]), row, row)                   # no reserve since the fork
    assert ha.status() == binding.HA_ERR_INVALID_ARG
    assert c.k.abs().sum().item() == 0
    ha.cache_reserve(c, ints([1]), ints([1]))
    ha.cache_append(c, ints([1]), ints([0, 1]), row, row)
    assert ha.status() == 0 and c.k.sum().item() == 64
    assert c.table.tolist() == [[0, 1, -1], [0, 2, -1]]


def test_append_takes_a_slot_once(ha):
    """The second entry of a slot is left out and reported, at the front and behind more entries than a block has threads."""
    options(ha, "fp32")
    n = 700
    c = binding.PagedCache.empty(layers=1, pages=n, kv_heads=1, page=16, d=64, slots=n, max_pages=1, dtype="fp32")
    ha.cache_reserve(c, ints(list(range(n))), ints([2] * n))
    who = list(range(n))
    who[1], who[n - 1] = 0, 300
    row = torch.arange(1, 2 * n + 1, device="cuda").float()[None, :, None, None].repeat(1, 1, 1, 64)
    ha.cache_append(c, ints(who), ints(list(range(0, 2 * n + 1, 2))), row, row)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    want = torch.arange(1, 2 * n + 1, device="cuda").float().view(n, 2)
    want[[1, n - 1]] = 0
    for x in (c.k, c.v):
        assert torch.equal(x[0, c.table[:, 0].long(), 0, :2, 5], want)


def test_commit_does_not_write_a_shared_page(ha):
    """Slot 1 is forked from slot 0, then slot 0 commits drafted rows of the page that both hold."""
    options(ha, "bf16")
    c = binding.PagedCache.empty(layers=1, pages=6, kv_heads=1, page=16, d=64, slots=2, max_pages=3)
    row = torch.randn(1, 6, 1, 64, device="cuda").to(torch.bfloat16)
    ha.cache_reserve(c, ints([0]), ints([6]))
    ha.cache_append(c, ints([0]), ints([0, 6]), row, row)
    ha.cache_commit(c, ints([0]), ints([2]))
    ha.cache_fork(c, ints([0]), ints([1]))
    ha.cache_commit(c, ints([0]), ints([1]))                                # nothing moves: rows 0..2 of the page
    assert ha.status() == 0 and c.lens.tolist() == [3, 2]
    before = c.k.clone()
    ha.cache_commit(c, ints([1]), ints([1]), ints([[1]]))                   # would write slot 0's row 2
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    assert torch.equal(c.k, before) and c.lens.tolist() == [3, 2]
    ha.cache_commit(c, ints([1]), ints([0]), ints([[1]]))
    assert ha.status() == 0 and c.lens.tolist() == [3, 2] and torch.equal(c.k, before)


def test_empty_lists_and_graph_of_steps(ha):
    """Lists of no entries do nothing; a captured cycle of all steps gives the same state at every replay."""
    side = torch.cuda.Stream()
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    c = binding.PagedCache.empty(layers=2, pages=12, kv_heads=2, page=16, d=64, slots=3, max_pages=4)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    row = torch.randn(2, 21, 2, 64, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    ha.cache_free(c, none)
    ha.cache_fork(c, none, none)
    ha.cache_reserve(c, none, none)
    ha.cache_append(c, none, ints([0]), row[:, :0], row[:, :0])
    ha.cache_commit(c, none, none)
    ha.cache_reserve(c, ints([0]), ints([21]))
    ha.cache_append(c, ints([0]), ints([0, 21]), row, row)
    ha.cache_commit(c, ints([0]), ints([21]))
    assert ha.status() == 0, ha.last_error()
    lists = dict(src=ints([0, 0]), dst=ints([2, 1]), add=ints([3, 14]), at=ints([0, 3, 17]), n=ints([2, 5]),
                 keep=ints([[0, 2, -1, -1, -1], [1, 3, 4, 8, 13]]))
    granted = ints([0, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ha.cache_free(c, lists["dst"])
        ha.cache_fork(c, lists["src"], lists["dst"])
        ha.cache_reserve(c, lists["dst"], lists["add"], granted)
        ha.cache_append(c, lists["dst"], lists["at"], row[:, :17], row[:, :17])
        ha.cache_commit(c, lists["dst"], lists["n"], lists["keep"])
    states = []
    for _ in range(3):
        with torch.cuda.stream(side):
            g.replay()
        assert ha.status() == 0, ha.last_error()
        states.append([x.clone() for x in (c.k, c.v, c.table, c.lens, c.held, c.refs, granted)])
        torch.cuda.synchronize()
    for s in states[1:]:
        assert all(torch.equal(x, y) for x, y in zip(states[0], s))
    assert c.lens.tolist() == [21, 26, 23] and granted.tolist() == [3, 14]
    rows = lambda slot, n: c.k[:, c.table[slot][:-(-n // 16)].long()].transpose(2, 3).flatten(1, 2)[:, :n]  # noqa: E731
    assert torch.equal(rows(2, 23), torch.cat([row, row[:, [0, 2]]], 1))
    assert torch.equal(rows(1, 26), torch.cat([row, row[:, [4, 6, 7, 11, 16]]], 1))
    del g
    options(ha, "bf16")


def test_many_entries(ha):
    """More entries than the planning block has threads: a shared page among them, and a pool that ends in between."""
    n, pages = 1500, 1400
    c = binding.PagedCache.empty(layers=1, pages=pages, kv_heads=1, page=16, d=64, slots=n, max_pages=2)
    options(ha, "bf16")
    ref = ListCache(bits(c.k).copy(), bits(c.v).copy(), n, 2)
    row = torch.randn(1, 5, 1, 64).to(torch.bfloat16)
    ha.cache_reserve(c, ints([7]), ints([5]))
    ha.cache_append(c, ints([7]), ints([0, 5]), row.cuda(), row.cuda())
    ha.cache_commit(c, ints([7]), ints([5]))
    ref.reserve([7], [5])
    ref.append([7], [0, 5], bits(row), bits(row))
    ref.commit([7], [5])
    dst = list(range(100, 1300))
    ha.cache_fork(c, ints([7] * len(dst)), ints(dst))
    ref.fork([7] * len(dst), dst)
    who = list(range(n))[::-1]
    add = [1 + (s % 3) * 8 for s in who]
    granted = torch.zeros(n, dtype=torch.int32, device="cuda")
    ha.cache_reserve(c, ints(who), ints(add), granted)
    assert granted.tolist() == ref.reserve(who, add)
    assert 0 < sum(g == 0 for g in granted.tolist()) < n
    assert ha.status() == 0, ha.last_error()
    same_state(c, ref)
    assert np.array_equal(bits(c.k), ref.k)
    counts = [min(1, g) for g in granted.tolist()]
    ha.cache_commit(c, ints(who), ints(counts))
    ref.commit(who, counts)
    ha.cache_free(c, ints(who[:900]))
    ref.free(who[:900])
    assert ha.status() == 0, ha.last_error()
    same_state(c, ref)


def test_cache_refusals(ha):
    options(ha, "bf16")
    c = binding.PagedCache.empty(layers=2, pages=6, kv_heads=1, page=16, d=64, slots=2, max_pages=3)
    row = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    inv = binding.HA_ERR_INVALID_ARG
    for layer in (-1, 2):
        with pytest.raises(binding.HAError) as e:
            ha.cache_append(c, ints([0]), ints([0, 1]), row, row, layer=layer)
        assert e.value.code == inv
    with pytest.raises(ValueError):
        ha.cache_append(c, ints([0]), ints([0, 1]), row.float(), row)
    with pytest.raises(ValueError):
        ha.cache_append(c, ints([0]), ints([0]), row, row)
    with pytest.raises(ValueError):
        ha.cache_fork(c, ints([0, 1]), ints([1]))
    with pytest.raises(ValueError):
        ha.cache_commit(c, ints([0]), ints([1]), ints([1]))
    ha.set_options(dtype="fp32", stream=torch.cuda.current_stream().cuda_stream)
    with pytest.raises(ValueError):
        ha.cache_free(c, ints([0]))
    options(ha, "bf16")
    L = binding.lib()
    assert L.hyper_attn_cache_free(ha._h, None, None, 1) == inv
    assert L.hyper_attn_cache_free(ha._h, c.args, None, 1) == inv
    assert L.hyper_attn_cache_free(ha._h, c.args, None, -1) == inv
    assert L.hyper_attn_cache_free(ha._h, c.args, None, 0) == 0
    for call, most in ((L.hyper_attn_cache_free, 16384), (L.hyper_attn_cache_append, 65536)):
        more = (most + 1,) if call is L.hyper_attn_cache_free else (None, most + 1, 1, None, None, None, None, 0, 1)
        assert call(ha._h, c.args, None, *more) == inv
    assert L.hyper_attn_cache_reserve(ha._h, c.args, c.lens.data_ptr(), c.lens.data_ptr(), 1, None, None, 0) == inv
    assert L.hyper_attn_cache_commit(ha._h, c.args, c.lens.data_ptr(), c.lens.data_ptr(), c.lens.data_ptr(), 0, 1) == inv
    assert ha.status() == 0


# ---- a run of them together

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_run(ha, dtype):
    """Prefill two packed prompts, fork one, then steps of drafting a tree, attending, keeping one path; every token's output
    is that of causal attention over its own sequence. The steps run as one captured graph, replayed with new inputs."""
    d, hk, group, page = 64, 2, 4, 16
    hq, scale = hk * group, d ** -0.5
    g = torch.Generator().manual_seed(11)
    rows = lambda n, h: torch.randn(n, h, d, generator=g).to(DT[dtype])  # noqa: E731
    p_bits, bf = (UBF if dtype == "bf16" else None), dtype == "bf16"
    side = torch.cuda.Stream()
    ha.set_options(dtype=dtype, stream=side.cuda_stream)
    cache = binding.PagedCache.empty(layers=1, pages=64, kv_heads=hk, page=page, d=d, slots=4, max_pages=20, dtype=dtype)
    lens = [45, 130]
    q, k, v = rows(175, hq), rows(175, hk), rows(175, hk)
    O = torch.empty_like(q, device="cuda")
    Q, K, V, cu, two = q.cuda(), k.cuda(), v.cuda(), ints([0, 45, 175]), ints([0, 2])
    torch.cuda.synchronize()
    ha.prompt(Q, K, V, O, cu, max_len=130, scale=scale)
    ha.cache_reserve(cache, two, ints(lens))
    ha.cache_append(cache, two, cu, K[None], V[None])
    ha.cache_commit(cache, two, ints(lens))
    ha.cache_fork(cache, ints([2]), ints([3]))
    assert ha.status() == 0, ha.last_error()
    keys = {0: k[:45], 2: k[45:], 3: k[45:]}
    values = {0: v[:45], 2: v[45:], 3: v[45:]}
    for a, b in ((0, 45), (45, 175)):
        want = attend(q[a:b], k[a:b], v[a:b], torch.ones(b - a, b - a, dtype=torch.bool).tril(), scale)
        check(O[a:b], None, want[:2], tolerances(*want, b - a, d, p_bits=p_bits, out_bf16=bf), "prompt")
    # drafts: a chain of one, a tree of four, a tree of four (tokens 1 and 2 are siblings, 3 follows 2)
    who, drafts, at = [0, 2, 3], [1, 4, 4], [0, 1, 5, 9]
    tree, keep = [1, 0b0011, 0b0101, 0b1101], [[0, -1, -1], [0, 1, -1], [0, 2, 3]]
    counts = [1, 2, 3]
    masks = signed([1] + tree + tree)
    WHO, ADD, AT, KEEP, COUNTS = ints(who), ints(drafts), ints(at), ints(keep), ints(counts)
    Qd, Kd, Vd = (torch.empty(9, h, d, dtype=DT[dtype], device="cuda") for h in (hq, hk, hk))
    Od, granted = torch.empty_like(Qd), ints([0, 0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ha.cache_reserve(cache, WHO, ADD, granted)
        ha.cache_append(cache, WHO, AT, Kd[None], Vd[None])
        ha.tree(Qd, cache, Od, WHO, AT, mask=masks, max_draft=4, scale=scale)
        ha.cache_commit(cache, WHO, COUNTS, KEEP)
    for step in range(9):
        qd, kd, vd = rows(9, hq), rows(9, hk), rows(9, hk)
        for x, y in ((Qd, qd), (Kd, kd), (Vd, vd)):
            x.copy_(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        assert ha.status() == 0, ha.last_error()
        assert granted.tolist() == drafts
        for i, s in enumerate(who):
            a, b = at[i], at[i + 1]
            n = keys[s].shape[0]
            kk, vv = torch.cat([keys[s], kd[a:b]]), torch.cat([values[s], vd[a:b]])
            seen = torch.ones(b - a, n + b - a, dtype=torch.bool)
            for r in range(b - a):
                seen[r, n:] = torch.tensor([bool(tree[r] >> j & 1) for j in range(b - a)])
            want = attend(qd[a:b], kk, vv, seen, scale)
            check(Od[a:b], None, want[:2], tolerances(*want, n + b - a, d, p_bits=p_bits, out_bf16=bf), f"step {step}, slot {s}")
            kept = [j for j in keep[i] if j >= 0]
            keys[s], values[s] = torch.cat([keys[s], kd[a:b][kept]]), torch.cat([values[s], vd[a:b][kept]])
        assert cache.lens.tolist() == [45 + step + 1, 0, 130 + 2 * (step + 1), 130 + 3 * (step + 1)]
    ha.cache_free(cache, ints([0, 2, 3]))
    assert ha.status() == 0 and cache.refs.abs().sum().item() == 0
    assert cache.table.tolist() == [[-1] * 20] * 4
    del graph


def test_profile_and_launch_counts(ha):
    options(ha, "bf16")
    ha.profile(True)
    ha.profile_read()
    q = torch.randn(50, 2, 64).to(torch.bfloat16).cuda()
    ha.prompt(q, q, q, torch.empty_like(q), ints([0, 50]))
    assert ha.last_launch_count() >= 1
    c = binding.PagedCache.empty(layers=1, pages=6, kv_heads=2, page=16, d=64, slots=2, max_pages=3)
    ha.cache_reserve(c, ints([0]), ints([1]))
    ha.tree(q[:1], c, torch.empty_like(q[:1]), ints([0]), ints([0, 1]), max_draft=1)
    prof = ha.profile_read()
    ha.profile(False)
    assert ha.status() == 0
    for cls in ("prompt", "tree", "cache"):
        assert prof[cls][1] >= 1 and prof[cls][0] > 0, cls
    assert prof["hash"] == (0.0, 0)
