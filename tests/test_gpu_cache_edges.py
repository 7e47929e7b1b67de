"""The cache's steps on lists and tables that are not in order: offsets of an append that are out of range, page numbers and
lengths that a fork must not take over, and what a free does with them."""
import pytest

from approximate_long_context_b200 import binding

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ha():
    h = binding.HyperAttention(0)
    h.set_options(dtype="fp32", stream=torch.cuda.current_stream().cuda_stream)
    yield h
    h.close()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def in_range(at, i, tokens):
    return 0 <= at[i] <= at[i + 1] <= tokens


def spoil(at, how):
    """Offsets of n sequences of three rows each with a fault in them."""
    n, tokens = len(at) - 1, at[-1]
    at, mid = list(at), (len(at) - 1) // 2
    if how == "negative_first":
        at[0] = -5
    elif how == "end_behind_the_rows":
        at[n] = tokens + 4
    elif how == "falls_back":           # one descends; the one in front of it gets longer and shares rows with the one behind
        at[mid] = at[mid + 1] + 2
    elif how == "falls_far_back":
        at[mid + 1] = 1
    elif how == "empty_behind_the_rows":
        at[n - 1] = at[n] = tokens + 9
    elif how == "all_negative":
        at = [x - 100000 for x in at]
    return at


FAULTS = ["negative_first", "end_behind_the_rows", "falls_back", "falls_far_back", "empty_behind_the_rows", "all_negative"]


@pytest.mark.parametrize("layers", [1, 9])
@pytest.mark.parametrize("n", [3, 5, 256, 257, 700, 4097])
@pytest.mark.parametrize("how", FAULTS)
def test_append_offsets_out_of_range(ha, how, n, layers):
    """A sequence whose offsets are not rows of the call is left out as a whole and reported; all others are written as a
    whole, also where they share rows with one another."""
    good = list(range(0, 3 * n + 1, 3))
    tokens, at = good[-1], spoil(good, how)
    c = binding.PagedCache.empty(layers=layers, pages=2 * n, kv_heads=1, page=16, d=64, slots=n, max_pages=2, dtype="fp32")
    ha.cache_reserve(c, ints(list(range(n))), ints([5] * n))
    ha.cache_commit(c, ints(list(range(n))), ints([5] * n))
    ha.cache_reserve(c, ints(list(range(n))), ints([27] * n))
    assert ha.status() == 0, ha.last_error()
    row = torch.arange(1, tokens + 1, device="cuda").float()[None, :, None, None].repeat(layers, 1, 1, 64)
    ha.cache_append(c, ints(list(range(n))), ints(at), row, -row)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    want = torch.zeros(n, 32)
    for i in range(n):
        if not in_range(at, i, tokens):
            continue
        rows = range(at[i], min(at[i + 1], at[i] + 27))     # more rows than the slot has room for: those have no page
        for j, t in enumerate(rows):
            want[i, 5 + j] = t + 1
    pages = c.table.long()
    for x, sign in ((c.k, 1), (c.v, -1)):
        for layer in (0, layers - 1):
            got = x[layer, pages, 0, :, 7].reshape(n, 32).cpu()
            assert torch.equal(got, sign * want)


def test_append_rows_of_no_sequence(ha):
    """Rows in front of the first sequence and behind the last one belong to none: they are left out, and that is no fault."""
    c = binding.PagedCache.empty(layers=1, pages=4, kv_heads=1, page=16, d=64, slots=2, max_pages=2, dtype="fp32")
    ha.cache_reserve(c, ints([0, 1]), ints([8, 8]))
    row = torch.arange(1, 11, device="cuda").float()[None, :, None, None].repeat(1, 1, 1, 64)
    ha.cache_append(c, ints([0, 1]), ints([2, 5, 7]), row, row)
    assert ha.status() == 0, ha.last_error()
    got = c.k[0, c.table[:, 0].long(), 0, :4, 0].cpu()
    assert got.tolist() == [[3, 4, 5, 0], [6, 7, 0, 0]]
    assert c.k.abs().sum().item() == 64 * 25 and c.v.abs().sum().item() == 64 * 25


def one_sequence():
    """Slot 0 with 40 rows on three pages, slot 3 with 20 on two."""
    return binding.PagedCache.empty(layers=1, pages=10, kv_heads=1, page=16, d=64, slots=5, max_pages=4, dtype="fp32")


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10, 2 ** 31 - 1])
@pytest.mark.parametrize("where", [0, 1, 2])
def test_fork_of_a_damaged_row(ha, bad, where):
    """A source whose row of the table has a page out of range is not forked, nor is any of its pages counted again."""
    c = one_sequence()
    ha.cache_reserve(c, ints([0, 3]), ints([40, 20]))
    ha.cache_commit(c, ints([0, 3]), ints([40, 20]))
    assert ha.status() == 0
    c.table[0, where] = bad
    refs = c.refs.tolist()
    ha.cache_fork(c, ints([0, 3]), ints([1, 4]))
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    assert c.table[1].tolist() == [-1] * 4 and c.lens.tolist() == [40, 0, 0, 20, 20] and c.held.tolist() == [3, 0, 0, 2, 2]
    want = list(refs)
    for p in c.table[3, :2].tolist():
        want[p] += 1
    assert c.refs.tolist() == want and c.table[4].tolist() == c.table[3].tolist()


@pytest.mark.parametrize("length", [-1, 49, 2 ** 31 - 15, 2 ** 31 - 1])
def test_fork_of_a_damaged_length(ha, length):
    c = one_sequence()
    ha.cache_reserve(c, ints([0]), ints([40]))
    ha.cache_commit(c, ints([0]), ints([40]))
    assert ha.status() == 0
    c.lens[0] = length
    refs = c.refs.tolist()
    ha.cache_fork(c, ints([0]), ints([1]))
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    assert c.lens.tolist() == [length, 0, 0, 0, 0] and c.held.tolist() == [3, 0, 0, 0, 0] and c.refs.tolist() == refs
    assert c.table[1].tolist() == [-1] * 4


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10, 2 ** 31 - 1])
def test_free_of_a_damaged_row(ha, bad):
    """The slot is emptied and its other pages are released, so that a damaged row does not hold pages for good."""
    c = one_sequence()
    ha.cache_reserve(c, ints([0, 3]), ints([40, 20]))
    ha.cache_commit(c, ints([0, 3]), ints([40, 20]))
    assert ha.status() == 0
    lost = c.table[0, 1].item()
    c.table[0, 1] = bad
    refs = c.refs.tolist()
    for p in c.table[0, [0, 2]].tolist():
        refs[p] -= 1
    ha.cache_free(c, ints([0]))
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    assert c.table[0].tolist() == [-1] * 4 and c.lens.tolist() == [0, 0, 0, 20, 0] and c.held.tolist() == [0, 0, 0, 2, 0]
    assert c.refs.tolist() == refs and refs[lost] == 1
