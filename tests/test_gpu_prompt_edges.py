"""Packed prompts where the work is found in other ways than in a short call: values that are not finite in items of two key heads
and in listed items, offsets that fall back among many, and prompts of thousands of rows."""
import random

import pytest

from approximate_long_context_b200 import binding
from serving import UBF, attend, check, tolerances

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


def offsets_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(total, hq, hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(total, h, d, generator=g).to(DT[dtype]) for h in (hq, hk, hk)]


def verify(q, k, v, o, lse, spans, scale, p_bits, out_bf16):
    for a, b in spans:
        n = b - a
        if n == 0:
            continue
        want = attend(q[a:b], k[a:b], v[a:b], torch.ones(n, n, dtype=torch.bool).tril(), scale)
        tol = tolerances(*want, n, q.shape[2], p_bits=p_bits, out_bf16=out_bf16)
        check(o[a:b], None if lse is None else lse[:, a:b], want[:2], tol, f"rows {a} to {b}")


# sequences, longest, key heads, group: a list with sequences of one and of several tiles, pairs of tiles, two heads at a time
WAYS = {"list": (100, 400, 2, 2), "list_odd_heads": (90, 300, 3, 2), "pairs": (300, 60, 2, 4), "singles": (200, 100, 2, 1),
        "singles_odd_heads": (200, 120, 3, 1)}


def lens_of(seqs, most, seed):
    rng = random.Random(seed)
    return [rng.randint(1, most) for _ in range(seqs)]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("way", list(WAYS))
def test_not_finite_values_among_many(ha, way, d, value, out):
    """In some sequences one value of one key head is not finite: the rows of its head that see it get it in its column, and
    everything else has the bits of the call without it, its neighbours and the other head of an item among them."""
    seqs, most, hk, group = WAYS[way]
    lens = lens_of(seqs, most, seed=seqs + d)
    at = offsets_of(lens)
    total = at[-1]
    q, k, v = make(total, hk * group, hk, d, "bf16", seed=d)
    rng = random.Random(11)
    hits = []
    for i in range(0, seqs, 3):
        hits.append((i, rng.randrange(lens[i]), rng.randrange(hk), rng.randrange(d)))
    for i in range(1, seqs, 9):                                  # two of them in one tile
        hits += [(i, rng.randrange(lens[i]), 0, 3), (i, rng.randrange(lens[i]), hk - 1, d - 1)]
    options(ha, "bf16", out_dtype=out)
    Q, K, V, cu = q.cuda(), k.cuda(), v.cuda(), ints(at)
    clean = torch.empty_like(Q, dtype=DT[out])
    ha.prompt(Q, K, V, clean, cu, max_len=most, scale=0.1)
    assert ha.last_kernel() == "tc" and ha.status() == 0, ha.last_error()
    some = range(0, seqs, max(1, seqs // 25))
    verify(q, k, v, clean.cpu(), None, [(at[i], at[i + 1]) for i in some], 0.1, UBF, out == "bf16")
    seen = torch.zeros(clean.shape, dtype=torch.bool)
    for i, row, h, col in hits:
        V[at[i] + row, h, col] = value
        seen[at[i] + row:at[i + 1], h * group:(h + 1) * group, col] = True
    got = torch.empty_like(clean)
    lse = torch.empty(hk * group, total, device="cuda")
    ha.prompt(Q, K, V, got, cu, max_len=most, scale=0.1, lse=lse)
    assert ha.status() == 0, ha.last_error()
    seen = seen.cuda()
    hit = got[seen].float()
    assert bool(torch.isnan(hit).all()) if value != value else bool((hit == value).all())
    assert torch.equal(got[~seen], clean[~seen]) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("way", ["list", "pairs", "singles", "singles_odd_heads"])
def test_offsets_that_fall_back_among_many(ha, way, dtype):
    """An offset lies behind the next one: the sequence in front of it is longer than promised, its own ends before it begins.
    Both are left out, all others are right."""
    seqs, most, hk, group = WAYS[way]
    lens = lens_of(seqs, most, seed=5)
    k0 = seqs // 2
    lens[k0 - 1] = most
    at = offsets_of(lens)
    total = at[-1]
    q, k, v = make(total, hk * group, hk, 64, dtype, seed=6)
    bad = list(at)
    bad[k0] = at[k0 + 1] + 1
    options(ha, dtype)
    O = torch.full_like(q, 7.0, device="cuda")
    lse = torch.full((hk * group, total), 7.0, device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, ints(bad), max_len=most, scale=0.125, lse=lse)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    o, l = O.cpu(), lse.cpu()
    a, b = at[k0 - 1], at[k0 + 1]
    assert bool((o[a:b] == 7).all()) and bool((l[:, a:b] == 7).all())
    spans = [(at[i], at[i + 1]) for i in range(seqs) if i not in (k0 - 1, k0) and (i % max(1, seqs // 40) == 0 or abs(i - k0) < 4)]
    verify(q, k, v, o, l, spans, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")


LONG = {"one": [5000], "ragged": [2500, 1, 130, 2049, 64, 900], "many": [1500, 300] * 12}


@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16_simt"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", list(LONG))
def test_prompts_of_thousands_of_rows(ha, lens, d, kind):
    lens, dtype = LONG[lens], kind[:4]
    at = offsets_of(lens)
    q, k, v = make(at[-1], 8, 2, d, dtype, seed=d)
    options(ha, dtype, kernel="simt" if kind == "bf16_simt" else "auto")
    O = torch.full_like(q, 7.0, device="cuda")
    lse = torch.full((8, at[-1]), 7.0, device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, ints(at), max_len=max(lens), scale=d ** -0.5, lse=lse)
    assert ha.status() == 0, ha.last_error()
    spans = [(at[i], at[i + 1]) for i in range(len(lens)) if i < 6]
    verify(q, k, v, O.cpu(), lse.cpu(), spans, d ** -0.5, UBF if kind == "bf16" else None, dtype == "bf16")
