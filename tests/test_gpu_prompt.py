"""Attention over packed prompts (hyper_attn_prompt) against softmax attention in 64 bits."""
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


def make(total, hq, hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(total, h, d, generator=g).to(DT[dtype]) for h in (hq, hk, hk)]


def verify(q, k, v, o, lse, lens, scale, p_bits, out_bf16, at=None):
    at = at or offsets_of(lens)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        a, b = at[i], at[i] + n
        want = attend(q[a:b], k[a:b], v[a:b], torch.ones(n, n, dtype=torch.bool).tril(), scale)
        tol = tolerances(*want, n, q.shape[2], p_bits=p_bits, out_bf16=out_bf16)
        check(o[a:b], None if lse is None else lse[:, a:b], want[:2], tol, f"sequence {i} of {n} rows")


LENS = {
    "one": [1],
    "edges": [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129],
    "empty_between": [0, 5, 0, 0, 130, 1, 0],
    "long": [700, 3, 257],
}
HEADS = [(1, 1), (2, 1), (2, 3), (1, 8), (2, 5)]


@pytest.mark.parametrize("lens", list(LENS), ids=list(LENS))
@pytest.mark.parametrize("heads", HEADS, ids=[f"kv{a}x{b}" for a, b in HEADS])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16_simt", "bf16_to_fp32"])
def test_prompt_matches_definition(ha, kind, d, heads, lens):
    dtype = kind[:4]
    hk, group = heads
    lens = LENS[lens]
    total = sum(lens)
    q, k, v = make(total, hk * group, hk, d, dtype, seed=d + total)
    options(ha, dtype, kernel="simt" if kind.endswith("simt") else "auto", out_dtype="fp32" if kind.endswith("to_fp32") else None)
    Q, K, V = q.cuda(), k.cuda(), v.cuda()
    out_bf16 = kind in ("bf16", "bf16_simt")
    O = torch.full(Q.shape, 7.0, dtype=torch.bfloat16 if out_bf16 else torch.float32, device="cuda")
    lse = torch.full((hk * group, total), 7.0, device="cuda")
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    ha.prompt(Q, K, V, O, cu, max_len=max(lens), scale=d ** -0.5, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(q, k, v, O, lse, lens, d ** -0.5, UBF if kind in ("bf16", "bf16_to_fp32") else None, out_bf16)


@pytest.mark.parametrize("d,most", [(64, 128), (64, 15), (128, 64), (128, 33)])
@pytest.mark.parametrize("group", [1, 3, 16, 128])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_a_few_short_prompts(ha, d, most, group, out):
    """Calls of one round of small blocks: strided rows, lengths around 16 and 64, rows behind the last sequence."""
    lens = [n for n in (1, 0, 15, 16, 17, 33, 63, 64, 65, 127, 128) if n <= most]
    if group == 128:
        lens = [1, 0, 17] if most > 16 else [1, 0, 15]
    hk = 2 if group < 16 else 1
    total = sum(lens)
    q, k, v = make(total + 3, hk * group, hk, d, "bf16", seed=d + group)
    k[total:], v[total:] = float("nan"), float("inf")
    wide = torch.randn(total + 3, hk * group, d + 8).to(torch.bfloat16).cuda()
    Q = wide[:, :, :d]
    Q.copy_(q)
    options(ha, "bf16", out_dtype=out)
    whole = torch.full((hk * group, total + 3, d), 7.0, dtype=DT[out], device="cuda")
    O = whole.transpose(0, 1)
    lse = torch.full((hk * group, total + 3), 7.0, device="cuda")
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    ha.prompt(Q, k.cuda(), v.cuda(), O, cu, max_len=max(lens), scale=d ** -0.5, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(q, k, v, O, lse, lens, d ** -0.5, UBF, out == "bf16")
    assert bool((O[total:] == 7).all()) and bool((lse[:, total:] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 7, 15, 16, 40, 62])
def test_not_finite_in_short_prompts(ha, d, value, at):
    n = 63
    q, k, v = make(n, 6, 2, d, "bf16", seed=at)
    clean = v.clone()
    v[at, 1, 5] = value
    options(ha, "bf16")
    O = torch.empty_like(q, device="cuda")
    lse = torch.empty(6, n, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, cu, scale=0.125, lse=lse)
    assert ha.status() == 0, ha.last_error()
    hit = O[at:, 3:, 5].clone()
    assert bool(torch.isnan(hit.float()).all()) if value != value else bool((hit.float() == value).all())
    # elsewhere it is the clean answer
    want = torch.empty_like(O)
    ha.prompt(q.cuda(), k.cuda(), clean.cuda(), want, cu, scale=0.125)
    O[at:, 3:, 5] = want[at:, 3:, 5]
    assert torch.equal(O, want)
    verify(q, k, clean, O, lse, [n], 0.125, UBF, True)
    k[at, 0, 3] = float("nan")
    ha.prompt(q.cuda(), k.cuda(), clean.cuda(), O, cu, scale=0.125)
    assert bool(torch.isnan(O[at:, :3].float()).all())
    O[at:, :3] = want[at:, :3]
    assert torch.equal(O, want)


def random_lens(n, most, seed, empty=0.1):
    import random
    rng = random.Random(seed)
    return [0 if rng.random() < empty else rng.randint(1, most) for _ in range(n)]


MANY = {
    # sequences, longest, key heads, group: all the ways in which a call's work is found and ordered
    "list": (100, 400, 2, 2),
    "list_shared_heads": (90, 300, 3, 7),
    "pairs": (300, 60, 2, 4),
    "singles": (400, 32, 2, 4),
    "singles_odd_heads": (200, 120, 3, 1),
    "singles_even_heads": (200, 100, 2, 1),
    "many_small_blocks": (700, 20, 6, 2),
    "few": (7, 200, 2, 1),
    "no_head_room": (170, 9, 1, 128),
    "thousands": (5000, 3, 1, 2),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", list(MANY), ids=list(MANY))
def test_many_sequences(ha, dtype, case):
    seqs, most, hk, group = MANY[case]
    lens = random_lens(seqs, most, seed=seqs)
    total, d = sum(lens), 64
    q, k, v = make(total, hk * group, hk, d, dtype, seed=7)
    options(ha, dtype)
    O = torch.full_like(q, 7.0, device="cuda")
    lse = torch.full((hk * group, total), 7.0, device="cuda")
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, cu, max_len=most, scale=0.125, lse=lse)
    assert ha.status() == 0, ha.last_error()
    o, l = O.cpu(), lse.cpu()
    step = max(1, seqs // 150)          # all of them, or every so many
    at = offsets_of(lens)
    keep = [i for i in range(seqs) if i % step == 0 or i >= seqs - 3]
    verify(q, k, v, o, l, [lens[i] for i in keep], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16", at=[at[i] for i in keep])
    assert not bool((o == 7).all(2).any()) and not bool((l == 7).any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ["list", "pairs", "singles", "few"])
def test_bad_offsets_among_many(ha, dtype, case):
    """One sequence longer than promised and one offset that falls back, among many: the others are right, those are left."""
    seqs, most, hk, group = MANY[case]
    lens = random_lens(seqs, most, seed=seqs, empty=0.0)
    lens[3] = most + 1
    total = sum(lens)
    at = offsets_of(lens)
    q, k, v = make(total, hk * group, hk, 64, dtype, seed=8)
    options(ha, dtype)
    O = torch.full_like(q, 7.0, device="cuda")
    bad = list(at)
    bad[seqs] = total + 1                # the last sequence ends behind the rows
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, torch.tensor(bad, dtype=torch.int32, device="cuda"), max_len=most, scale=0.125)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    o = O.cpu()
    assert bool((o[at[3]:at[4]] == 7).all()) and bool((o[at[seqs - 1]:] == 7).all())
    good = [i for i in range(0, seqs - 1, max(1, seqs // 40)) if i != 3]
    verify(q, k, v, o, None, [lens[i] for i in good], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16", at=[at[i] for i in good])


def test_two_handles_on_two_streams():
    """Eager calls of two handles that overlap on the device."""
    lens = random_lens(60, 500, seed=3)
    total = sum(lens)
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    handles = [binding.HyperAttention(0) for _ in streams]
    data = [make(total, 4, 2, 128, "bf16", seed=40 + i) for i in range(2)]
    dev = [[x.cuda() for x in d] for d in data]
    outs = [[torch.empty_like(d[0]) for _ in range(4)] for d in dev]
    torch.cuda.synchronize()
    for h, s in zip(handles, streams):
        h.set_options(dtype="bf16", stream=s.cuda_stream)
    for r in range(4):
        for h, d, o in zip(handles, dev, outs):
            h.prompt(*d, o[r], cu, max_len=500, scale=0.1)
    for h, d, o in zip(handles, data, outs):
        assert h.status() == 0, h.last_error()
        for x in o[1:]:
            assert torch.equal(o[0], x)
        verify(*d, o[0], None, lens, 0.1, UBF, True)
        h.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", [16, 100, 128])
def test_many_query_heads_to_one_key_head(ha, dtype, group):
    lens = [37, 1, 140]
    q, k, v = make(sum(lens), group, 1, 64, dtype, seed=group)
    options(ha, dtype)
    O = torch.empty_like(q, device="cuda")
    lse = torch.empty(group, sum(lens), device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda"),
              max_len=140, scale=0.125, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(q, k, v, O, lse, lens, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores(ha, dtype):
    """Scores of a few hundred: the running maximum moves all the time."""
    lens, d = [400], 64
    q, k, v = make(400, 4, 2, d, dtype, seed=5)
    q, k = q * 6, k * 6
    ramp = torch.linspace(0.2, 3.0, 400)[:, None, None].to(k.dtype)
    k = (k.float() * ramp.float()).to(k.dtype)
    options(ha, dtype)
    O, lse = torch.empty_like(q, device="cuda"), torch.empty(4, 400, device="cuda")
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, torch.tensor([0, 400], dtype=torch.int32, device="cuda"), scale=0.3, lse=lse)
    assert ha.status() == 0, ha.last_error()
    verify(q, k, v, O, lse, lens, 0.3, UBF if dtype == "bf16" else None, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides(ha, dtype):
    """q, k, v as parts of one projection's output, o head by head."""
    lens, hk, group, d = [200, 77], 2, 3, 64
    total, hq = sum(lens), hk * group
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(total, (hq + 2 * hk) * d + 24, generator=g).to(DT[dtype]).cuda()
    Q = fused[:, :hq * d].view(total, hq, d)
    K = fused[:, hq * d:(hq + hk) * d].view(total, hk, d)
    V = fused[:, (hq + hk) * d:(hq + 2 * hk) * d].view(total, hk, d)
    whole = torch.full((hq, total + 3, d), 3.0, dtype=DT[dtype], device="cuda")
    O = whole[:, 1:total + 1].transpose(0, 1)
    options(ha, dtype)
    ha.prompt(Q, K, V, O, torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda"), scale=0.1)
    assert ha.status() == 0, ha.last_error()
    verify(Q.cpu(), K.cpu(), V.cpu(), O, None, lens, 0.1, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert bool((whole[:, 0] == 3).all()) and bool((whole[:, total + 1:] == 3).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_behind_the_last_sequence_stay(ha, dtype):
    lens, total = [129, 4], 300
    q, k, v = make(total, 4, 2, 128, dtype, seed=2)
    k[133:], v[133:] = float("nan"), float("nan")
    O = torch.full_like(q, 5.0, device="cuda")
    lse = torch.full((4, total), 5.0, device="cuda")
    options(ha, dtype)
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, torch.tensor([0, 129, 133], dtype=torch.int32, device="cuda"), lse=lse, scale=0.1)
    assert ha.status() == 0, ha.last_error()
    verify(q, k, v, O, lse, lens, 0.1, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert bool((O[133:] == 5).all()) and bool((lse[:, 133:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 1, 40, 127, 128, 199])
def test_not_finite_in_later_rows(ha, dtype, value, at):
    """A value row and a key row that are not finite: the rows in front of them do not notice; the rows that see them do."""
    n, d = 200, 64
    q, k, v = make(n, 2, 1, d, dtype, seed=at)
    q2, k2, v2 = [x.repeat(2, 1, 1) for x in (q, k, v)]     # a second, clean sequence behind it
    v2[at, 0, 5] = value
    options(ha, dtype)
    O = torch.empty_like(q2, device="cuda")
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    ha.prompt(q2.cuda(), k2.cuda(), v2.cuda(), O, cu, scale=0.125)
    assert ha.status() == 0, ha.last_error()
    verify(q[:at], k[:at], v[:at], O[:at], None, [at], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    verify(q, k, v, O[n:], None, [n], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    hit = O[at:n, :, 5].float()
    assert bool(torch.isnan(hit).all()) if value != value else bool((hit == value).all())
    others = torch.cat([O[at:n, :, :5], O[at:n, :, 6:]], 2)
    assert bool(torch.isfinite(others).all())
    k2[at, 0, 3] = float("nan")
    ha.prompt(q2.cuda(), k2.cuda(), v2.cuda(), O, cu, scale=0.125)
    verify(q[:at], k[:at], v[:at], O[:at], None, [at], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    verify(q, k, v, O[n:], None, [n], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert bool(torch.isnan(O[at:n]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad,good", [([0, 50, 40, 90], [(0, 50), (40, 90)]), ([0, 50, 101], [(0, 50)]), ([-3, 50, 90], [(50, 90)]),
                                      ([0, 2 ** 31 - 1, 50, 90], [(50, 90)]), ([0, 10, 95], [(0, 10)])])
def test_bad_offsets_are_left_out(ha, dtype, bad, good):
    """Descending offsets, offsets outside the rows, and a sequence longer than max_len (80)."""
    total = 100
    q, k, v = make(total, 2, 2, 64, dtype, seed=3)
    O = torch.full_like(q, 5.0, device="cuda")
    options(ha, dtype)
    ha.prompt(q.cuda(), k.cuda(), v.cuda(), O, torch.tensor(bad, dtype=torch.int32, device="cuda"), max_len=80, scale=0.125)
    assert ha.status() == binding.HA_ERR_INVALID_ARG
    assert "out of range" in ha.last_error()
    assert ha.status() == 0
    if good == [(0, 50), (40, 90)]:
        # rows 40..49 belong to two sequences
        verify(q, k, v, O, None, [40], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
        return
    touched = torch.zeros(total, dtype=torch.bool)
    for a, b in good:
        verify(q, k, v, O, None, [b - a], 0.125, UBF if dtype == "bf16" else None, dtype == "bf16", at=[a])
        touched[a:b] = True
    assert bool((O.cpu()[~touched] == 5).all())


def test_equal_calls_give_equal_bits(ha):
    lens = [513, 1, 900, 64]
    q, k, v = [x.cuda() for x in make(sum(lens), 8, 2, 128, "bf16", seed=9)]
    options(ha, "bf16")
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in range(3)]
    for o in outs:
        ha.prompt(q, k, v, o, cu, scale=0.1)
    assert ha.status() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_graph_and_side_stream(ha, dtype):
    """Two graphs captured on one handle and replayed on two streams at once, with new inputs each time."""
    lens = [300, 41, 128]
    total = sum(lens)
    cu = torch.tensor(offsets_of(lens), dtype=torch.int32, device="cuda")
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    state = []
    for i, s in enumerate(side):
        q, k, v = [x.cuda() for x in make(total, 4, 2, 64, dtype, seed=20 + i)]
        o = torch.empty_like(q)
        torch.cuda.synchronize()
        ha.set_options(dtype=dtype, stream=s.cuda_stream)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ha.prompt(q, k, v, o, cu, scale=0.125)
        state.append((q, k, v, o, g))
    big = torch.empty(4000, 64, 128, device="cuda", dtype=DT[dtype])   # a larger call on the same handle in between
    ha.set_options(dtype=dtype, stream=torch.cuda.current_stream().cuda_stream)
    ha.prompt(big, big, big, torch.empty_like(big), torch.tensor([0, 4000], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for r in range(3):
        fresh = [make(total, 4, 2, 64, dtype, seed=30 + 2 * r + i) for i in range(2)]
        for i in range(2):
            for x, y in zip(state[i][:3], fresh[i]):
                x.copy_(y)
        torch.cuda.synchronize()
        for i, s in enumerate(side):
            with torch.cuda.stream(s):
                for _ in range(5):
                    state[i][4].replay()
        torch.cuda.synchronize()
        for i in range(2):
            verify(*fresh[i], state[i][3], None, lens, 0.125, UBF if dtype == "bf16" else None, dtype == "bf16")
    assert ha.status() == 0
    options(ha, dtype)


def test_zero_sizes(ha):
    options(ha, "bf16")
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ha.prompt(e, kv, kv, torch.empty_like(e), torch.tensor([0], dtype=torch.int32, device="cuda"))
    ha.prompt(e, kv, kv, torch.empty_like(e), torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"))
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 2.0)
    kv = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    ha.prompt(q, kv, kv, o, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    ha.prompt(q, kv, kv, o, torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert ha.status() == 0
    assert bool((o == 2).all())


def test_refusals(ha):
    options(ha, "bf16")
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 9.0)
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")

    def refused(code, *args, **kw):
        with pytest.raises(binding.HAError) as e:
            ha.prompt(*args, **kw)
        assert e.value.code == code and ha.last_error()

    inv, uns = binding.HA_ERR_INVALID_ARG, binding.HA_ERR_UNSUPPORTED
    three = torch.zeros(8, 3, 64, dtype=torch.bfloat16, device="cuda")
    refused(inv, q, three, three, o, cu)                                           # 4 heads over 3
    for s in (0.0, -1.0, float("inf"), float("nan")):
        refused(inv, q, kv, kv, o, cu, scale=s)
    refused(inv, q, kv, kv, o, cu, max_len=0)
    refused(inv, q, kv, kv, q, cu)                                                 # o is q
    w = torch.zeros(8, 4, 96, dtype=torch.bfloat16, device="cuda")
    refused(uns, w, w, w, torch.zeros_like(w), cu)                                 # d = 96
    room = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    refused(inv, room.as_strided((8, 4, 64), (260, 65, 1)), kv, kv, o, cu)         # strides not of 16 bytes
    refused(inv, q, kv, kv, o.as_strided((8, 4, 64), (64, 64, 1)), cu)             # output rows overlap
    refused(inv, q, kv.expand(8, 2, 64).as_strided((8, 2, 64), (0, 64, 1)), kv, o, cu)   # broadcast rows
    flat = torch.zeros(8 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    refused(inv, flat[1:1 + 2048].view(8, 4, 64), kv, kv, o, cu)                   # not 16-byte aligned
    many = torch.zeros(8, 129, 64, dtype=torch.bfloat16, device="cuda")
    refused(uns, many, kv[:, :1].contiguous(), kv[:, :1].contiguous(), torch.zeros_like(many), cu)
    for bad in ((q.float(), kv, kv, o, cu), (q, kv, kv, o.float(), cu), (q, kv, kv, o, cu.long()), (q, kv, kv[:4], o, cu),
                (q.cpu(), kv, kv, o, cu), (q.transpose(1, 2), kv, kv, o, cu)):
        with pytest.raises(ValueError):
            ha.prompt(*bad)
    with pytest.raises(ValueError):
        ha.prompt(q, kv, kv, o, cu, lse=torch.zeros(8, 4, device="cuda"))
    f = q.float()
    ha.set_options(dtype="fp32", kernel="tc", stream=torch.cuda.current_stream().cuda_stream)
    refused(uns, f, kv.float(), kv.float(), f.clone(), cu)
    options(ha, "bf16")
    a = binding.PromptArgs()
    assert binding.lib().hyper_attn_prompt(ha._h, None) == inv
    assert binding.lib().hyper_attn_prompt(None, a) == inv
    torch.cuda.synchronize()
    assert bool((o == 9).all()) and ha.status() == 0
