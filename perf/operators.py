"""Cases of the exact operators for serving: attention over packed prompts (`prompt`), attention of a tree of drafted
tokens over a paged cache (`tree`), and a cycle of the paged cache's own steps (`branch`): the old branches freed, new
ones forked, their pages reserved (a shared last page is copied), the drafted rows appended and the accepted ones kept.

`run` computes them in plain torch in 32 bits where `own` is false, and by the library's calls where it is true.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one short question to a small model: nothing but latency
        {"name": "prompt_one_short", "op": "prompt", "dtype": "bf16", "seqs": 1, "longest": 77, "spread": 0, "kv_heads": 2,
         "group": 4, "d": 64},
        # a prefill step of a server: prompts of all lengths packed behind one another, grouped heads
        {"name": "prompt_ragged", "op": "prompt", "dtype": "bf16", "seqs": 16, "longest": 2047, "spread": 1, "kv_heads": 8,
         "group": 4, "d": 128},
        # many one-paragraph prompts, as many key heads as query heads
        {"name": "prompt_many_short", "op": "prompt", "dtype": "bf16", "seqs": 256, "longest": 128, "spread": 2,
         "kv_heads": 16, "group": 1, "d": 64},
        # the prefill length of the causal workload, one long document (8 of 32 heads: one GPU's share of four)
        {"name": "prompt_long", "op": "prompt", "dtype": "bf16", "seqs": 1, "longest": 32768, "spread": 0, "kv_heads": 2,
         "group": 4, "d": 128},
        # fp32 evaluation of a small model
        {"name": "prompt_fp32", "op": "prompt", "dtype": "fp32", "seqs": 8, "longest": 1023, "spread": 3, "kv_heads": 4,
         "group": 2, "d": 64},
        # one user, one token at a time: latency
        {"name": "decode_one", "op": "tree", "dtype": "bf16", "seqs": 1, "longest": 1001, "spread": 0, "draft": 1,
         "kv_heads": 2, "group": 4, "d": 64, "page": 16},
        # a server's decode step: 64 users, contexts of all lengths, one token each
        {"name": "decode_batch", "op": "tree", "dtype": "bf16", "seqs": 64, "longest": 16384, "spread": 4, "draft": 1,
         "kv_heads": 8, "group": 4, "d": 128, "page": 64},
        # speculative decoding: 16 users, trees of up to 32 drafted tokens each
        {"name": "tree_batch", "op": "tree", "dtype": "bf16", "seqs": 16, "longest": 8191, "spread": 5, "draft": 32,
         "kv_heads": 8, "group": 4, "d": 128, "page": 16},
        # one user with the long workload's context, a full tree of 64 tokens, eight query heads to a key head
        {"name": "tree_long", "op": "tree", "dtype": "bf16", "seqs": 1, "longest": 131072, "spread": 0, "draft": 64,
         "kv_heads": 4, "group": 8, "d": 128, "page": 128},
        # fp32 evaluation
        {"name": "tree_fp32", "op": "tree", "dtype": "fp32", "seqs": 4, "longest": 2047, "spread": 6, "draft": 5,
         "kv_heads": 4, "group": 2, "d": 64, "page": 32},
        # two continuations of one prompt in a one-layer draft model: latency
        {"name": "branch_few", "op": "branch", "dtype": "bf16", "layers": 1, "sources": 1, "seqs": 2, "longest": 333,
         "spread": 7, "draft": 5, "kv_heads": 2, "d": 64, "page": 16},
        # 64 speculative branches of 8 prompts, all 32 layers
        {"name": "branch_many", "op": "branch", "dtype": "bf16", "layers": 32, "sources": 8, "seqs": 64, "longest": 1000,
         "spread": 8, "draft": 16, "kv_heads": 8, "d": 128, "page": 16},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["prompt", "tree", "branch"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "fp32"]), "d": rng.choice([64, 128]), "spread": rng.randrange(1, 1 << 20)}
    if op == "prompt":
        case.update(seqs=_log(rng, 1, 256), longest=_log(rng, 1, 32768), kv_heads=_log(rng, 1, 16), group=_log(rng, 1, 16))
        most = 2 ** 33 if case["dtype"] == "bf16" else 2 ** 29
        while case["seqs"] * case["kv_heads"] * case["group"] * case["longest"] ** 2 > most:
            case["longest"] = case["longest"] * 2 // 3
            case["seqs"] = max(1, case["seqs"] * 3 // 4)
    elif op == "tree":
        case.update(seqs=_log(rng, 1, 128), longest=_log(rng, 1, 131072), draft=_log(rng, 1, 64), kv_heads=_log(rng, 1, 8),
                    group=_log(rng, 1, 16), page=rng.choice([16, 32, 64, 128]))
        most = 2 ** 30 if case["dtype"] == "bf16" else 2 ** 27
        while (case["seqs"] * case["kv_heads"] * case["longest"] * case["d"] > most
               or case["seqs"] * case["kv_heads"] * case["group"] * case["draft"] * case["longest"] > most):
            case["longest"] = max(1, case["longest"] * 2 // 3)
            case["seqs"] = max(1, case["seqs"] * 3 // 4)
    else:
        case.update(layers=_log(rng, 1, 32), sources=_log(rng, 1, 8), seqs=_log(rng, 1, 64), longest=_log(rng, 1, 1000),
                    draft=_log(rng, 1, 16), kv_heads=_log(rng, 1, 8), page=rng.choice([16, 32, 64, 128]))
    return case


def _lengths(case):
    """The sequences' lengths: all the longest where `spread` is 0, else from 1 to the longest, the first one the longest."""
    n = case["sources"] if case["op"] == "branch" else case["seqs"]
    if not case["spread"]:
        return [case["longest"]] * n
    rng = random.Random(case["spread"])
    return [case["longest"]] + [rng.randint(1, case["longest"]) for _ in range(n - 1)]


def _drafts(case):
    """The drafted tokens of each sequence, from 1 to `draft`, the first one has them all."""
    rng = random.Random(case["spread"] + 1)
    return [case["draft"]] + [rng.randint(1, case["draft"]) for _ in range(case["seqs"] - 1)]


def _kept(case):
    """The rows of each branch's draft that are accepted: ascending, the first one among them."""
    rng = random.Random(case["spread"] + 2)
    return [[0] + sorted(rng.sample(range(1, t), rng.randint(0, t - 1))) for t in _drafts(case)]


def _offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, d = DT[case["dtype"]], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    state = dict(case, lengths=_lengths(case), scale=d ** -0.5)
    if case["op"] == "prompt":
        lens, hk = state["lengths"], case["kv_heads"]
        hq, total = hk * case["group"], sum(lens)
        state.update(q=normal(total, hq, d), k=normal(total, hk, d), v=normal(total, hk, d), cu=_ints(_offsets(lens)),
                     o=torch.empty(total, hq, d, dtype=dtype, device="cuda"), lse=torch.empty(hq, total, device="cuda"),
                     total=total)
        return state
    lens, drafts, page, hk = state["lengths"], _drafts(case), case["page"], case["kv_heads"]
    total = sum(drafts)
    state.update(cu=_ints(_offsets(drafts)), total=total)
    pick = random.Random(seed)
    if case["op"] == "tree":
        hq = hk * case["group"]
        need = [-(-(a + b) // page) for a, b in zip(lens, drafts)]
        pool, slots = sum(need) + 3, len(lens)
        # each token's parent is any earlier one or the context's end; it sees its ancestors and itself
        masks = []
        for t in drafts:
            mine = []
            for i in range(t):
                parent = pick.randint(-1, i - 1)
                mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
            masks += [m - (1 << 64) if m >> 63 else m for m in mine]
        state.update(q=normal(total, hq, d), o=torch.empty(total, hq, d, dtype=dtype, device="cuda"),
                     lse=torch.empty(hq, total, device="cuda"), seqs_at=torch.arange(slots, dtype=torch.int32, device="cuda"),
                     mask=torch.tensor(masks, dtype=torch.int64, device="cuda"), layers=1)
    else:
        need = [-(-a // page) for a in lens]
        # a branch needs at most a copy of its last page and pages for its draft
        pool = sum(need) + case["seqs"] * (2 + -(-case["draft"] // page)) + 3
        slots = len(lens) + case["seqs"]
        kept = _kept(case)
        state.update(src=_ints([pick.randrange(len(lens)) for _ in range(case["seqs"])]),
                     dst=torch.arange(len(lens), slots, dtype=torch.int32, device="cuda"), add=_ints(drafts),
                     granted=torch.zeros(case["seqs"], dtype=torch.int32, device="cuda"),
                     counts=_ints([len(x) for x in kept]),
                     keep=_ints([x + [-1] * (case["draft"] - len(x)) for x in kept]),
                     k_new=normal(case["layers"], total, hk, d), v_new=normal(case["layers"], total, hk, d))
    most = -(-(max(lens) + case["draft"]) // page)
    ids = list(range(pool))
    pick.shuffle(ids)
    at, rows, refs = 0, [], [0] * pool
    for n in need:
        mine = ids[at:at + n]
        at += n
        for p in mine:
            refs[p] = 1
        rows.append(mine + [-1] * (most - n))
    rows += [[-1] * most] * (slots - len(rows))
    state.update(k_pages=normal(state["layers"], pool, hk, page, d), v_pages=normal(state["layers"], pool, hk, page, d),
                 table=_ints(rows), lens=_ints(lens + [0] * (slots - len(lens))),
                 held=_ints(need + [0] * (slots - len(need))), refs=_ints(refs), pool=pool, most=most)
    return state


# ---- the plain forms

def _padded(cu, total, longest):
    """Where each sequence's rows lie, padded to the longest, and where each row lies in that."""
    cu = cu.long()
    at = torch.arange(longest, device=cu.device)
    index = (cu[:-1, None] + at).clamp(max=total - 1)
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return index, seq, row - cu[seq]


def _softmax_product(s, v):
    """softmax(s) v over the last axis in place, and the log of the sum; s is -inf where nothing is seen."""
    top = s.amax(-1, keepdim=True)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    return (s @ v) / total, (top + total.log()).squeeze(-1)


def _prompt(st):
    hk, g, d = st["kv_heads"], st["group"], st["d"]
    longest = max(st["lengths"])
    index, seq, pos = _padded(st["cu"], st["total"], longest)
    b = index.shape[0]
    q = st["q"][index].float().view(b, longest, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * longest, d)
    k = st["k"][index].float().permute(0, 2, 3, 1)
    v = st["v"][index].float().transpose(1, 2)
    s = (q @ k).mul_(st["scale"]).view(b, hk, g, longest, longest)
    at = torch.arange(longest, device=s.device)
    s.masked_fill_(at[None, :] > at[:, None], float("-inf"))
    o, lse = _softmax_product(s.view(b, hk, g * longest, longest), v)
    o = o.view(b, hk * g, longest, d)[seq, :, pos]
    lse = lse.view(b, hk * g, longest)[seq, :, pos]
    return o.to(st["q"].dtype), lse.t().contiguous()


def _tree(st):
    hk, g, d, page, draft = st["kv_heads"], st["group"], st["d"], st["page"], st["draft"]
    index, seq, pos = _padded(st["cu"], st["total"], draft)
    b, n = index.shape[0], st["most"] * page
    table = st["table"][st["seqs_at"].long()].long().clamp(min=0)
    lens, counts = st["lens"][st["seqs_at"].long()].long(), st["cu"].long().diff()
    at = torch.arange(n, device=table.device)
    k = st["k_pages"][0][table].transpose(1, 2).reshape(b, hk, n, d).float()
    v = st["v_pages"][0][table].transpose(1, 2).reshape(b, hk, n, d).float()
    v.masked_fill_((at[None, :] >= (lens + counts)[:, None])[:, None, :, None], 0.0)
    q = st["q"][index].float().view(b, draft, hk, g, d).transpose(1, 2).reshape(b, hk, draft * g, d)
    s = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(b, hk, draft, g, n)
    own_row = at[None, :] - lens[:, None]
    bit = st["mask"][index][:, :, None] >> own_row.clamp(0, 63)[:, None, :] & 1
    inside = (own_row >= 0) & (own_row < counts[:, None])
    seen = (own_row < 0)[:, None, :] | inside[:, None, :] & (bit == 1)
    s.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    o, lse = _softmax_product(s.view(b, hk, draft * g, n), v)
    o = o.view(b, hk, draft, g, d).transpose(1, 2).reshape(b, draft, hk * g, d)[seq, pos]
    lse = lse.view(b, hk, draft, g).transpose(1, 2).reshape(b, draft, hk * g)[seq, pos]
    return o.to(st["q"].dtype), lse.t().contiguous()


def _free(st, slots):
    ids = st["table"][slots].long()
    st["refs"].index_add_(0, ids.clamp(min=0).view(-1), -(ids >= 0).int().view(-1))
    st["table"][slots] = -1
    st["lens"][slots] = 0
    st["held"][slots] = 0


def _fork(st, src, dst):
    held = (st["lens"][src] + st["page"] - 1) // st["page"]
    ids = st["table"][src].masked_fill(torch.arange(st["most"], device=held.device) >= held[:, None], -1)
    st["table"][dst] = ids
    st["lens"][dst] = st["lens"][src]
    st["held"][dst] = held
    ids = ids.long()
    st["refs"].index_add_(0, ids.clamp(min=0).view(-1), (ids >= 0).int().view(-1))


def _reserve(st, slots):
    page, most, add = st["page"], st["most"], st["add"]
    lens, held = st["lens"][slots], st["held"][slots]
    last_at = (lens // page).long().clamp(max=most - 1)
    last = st["table"][slots, last_at].long()
    partial = (lens % page != 0) & (add > 0)
    same = (last[:, None] == last[None, :]) & partial[:, None] & partial[None, :]
    copy = partial & (st["refs"][last.clamp(min=0)] - same.tril(-1).sum(1) > 1)
    new = ((lens + add + page - 1) // page - held).clamp(min=0)
    need = new + copy.int()
    upto = need.cumsum(0)
    fits = (upto <= (st["refs"] == 0).sum()) & (lens + add <= most * page)
    st["granted"].copy_(torch.where(fits, add, torch.zeros_like(add)))
    free = torch.sort((st["refs"] != 0).to(torch.uint8), stable=True).indices
    start = upto - need
    copy, new = copy & fits, torch.where(fits, new, torch.zeros_like(new))
    # the copy of a shared last page: its committed rows
    fresh = torch.where(copy, free[start.clamp(max=free.numel() - 1)], last)
    to, source = fresh.clamp(min=0), last.clamp(min=0)
    rows = (torch.arange(page, device=lens.device) < (lens % page)[:, None]) & copy[:, None]
    rows = rows[None, :, None, :, None]
    st["k_pages"][:, to] = torch.where(rows, st["k_pages"][:, source], st["k_pages"][:, to])
    st["v_pages"][:, to] = torch.where(rows, st["v_pages"][:, source], st["v_pages"][:, to])
    st["table"][slots, last_at] = fresh.int()
    st["refs"].index_add_(0, source, -copy.int())
    st["refs"].index_add_(0, to, copy.int())
    # new pages
    at = torch.arange(2 + st["draft"] // page, device=lens.device)
    inside = at < new[:, None]
    ids = free[(start + copy.int())[:, None].add(at).clamp(max=free.numel() - 1)]
    where = (held[:, None] + at).clamp(max=most - 1).long()
    where = torch.where(inside, where, torch.full_like(where, most))
    wide = torch.cat([st["table"], st["table"][:, :1]], 1)
    wide[slots[:, None], where] = ids.int()
    st["table"].copy_(wide[:, :most])
    st["refs"].index_add_(0, ids.view(-1), inside.int().view(-1))
    st["held"][slots] = held + new


def _append(st, slots):
    _, seq, pos = _padded(st["cu"], st["total"], st["draft"])
    at = st["lens"][slots][seq] + pos
    ids, row = st["table"][slots[seq], at // st["page"]].long(), at % st["page"]
    st["k_pages"][:, ids, :, row] = st["k_new"].transpose(0, 1)
    st["v_pages"][:, ids, :, row] = st["v_new"].transpose(0, 1)


def _commit(st, slots):
    page, counts = st["page"], st["counts"]
    lens, held = st["lens"][slots], st["held"][slots]
    # past a sequence's count its last row is moved once more
    at = torch.minimum(torch.arange(st["draft"], device=lens.device)[None, :], counts[:, None] - 1)
    to = lens[:, None] + at
    source = lens[:, None] + st["keep"].gather(1, at.long())
    pages = st["table"][slots].long()
    a, b = pages.gather(1, (source // page).long()).view(-1), (source % page).view(-1)
    x, y = pages.gather(1, (to // page).long()).view(-1), (to % page).view(-1)
    st["k_pages"][:, x, :, y] = st["k_pages"][:, a, :, b]
    st["v_pages"][:, x, :, y] = st["v_pages"][:, a, :, b]
    after = lens + counts
    keep = (after + page - 1) // page
    out = torch.arange(st["most"], device=lens.device)
    out = (out >= keep[:, None]) & (out < held[:, None])
    st["refs"].index_add_(0, pages.clamp(min=0).view(-1), -out.int().view(-1))
    st["table"][slots] = pages.masked_fill(out, -1).int()
    st["lens"][slots] = after
    st["held"][slots] = keep


# ---- one pass

_handles = {}


def _handle(dtype, device):
    """The program's handle for a type and device, made once; its calls go to the stream that is current."""
    stream = torch._C._cuda_getCurrentRawStream(device)   # torch.cuda.current_stream takes 2 us
    entry = _handles.get((dtype, device))
    if entry is None:
        from approximate_long_context_b200 import binding
        entry = _handles[dtype, device] = [binding.HyperAttention(device), None]
    if entry[1] != stream:
        entry[0].set_options(dtype=dtype, stream=stream)
        entry[1] = stream
    return entry[0]


def _cache(st):
    from approximate_long_context_b200 import binding
    return binding.PagedCache(st["k_pages"], st["v_pages"], st["table"], st["lens"], st["held"], st["refs"])


def run(st):
    op = st["op"]
    if op == "prompt":
        if not own:
            return _prompt(st)
        ha = _handle(st["dtype"], st["q"].get_device())
        ha.prompt(st["q"], st["k"], st["v"], st["o"], st["cu"], max_len=max(st["lengths"]), scale=st["scale"], lse=st["lse"])
        return st["o"], st["lse"]
    if op == "tree":
        if not own:
            return _tree(st)
        ha = _handle(st["dtype"], st["q"].get_device())
        ha.tree(st["q"], _cache(st), st["o"], st["seqs_at"], st["cu"], mask=st["mask"], max_draft=st["draft"],
                scale=st["scale"], lse=st["lse"])
        return st["o"], st["lse"]
    if own:
        cache = _cache(st)
        ha = _handle(st["dtype"], cache.device)
        ha.cache_free(cache, st["dst"])
        ha.cache_fork(cache, st["src"], st["dst"])
        ha.cache_reserve(cache, st["dst"], st["add"], st["granted"])
        ha.cache_append(cache, st["dst"], st["cu"], st["k_new"], st["v_new"])
        ha.cache_commit(cache, st["dst"], st["counts"], keep=st["keep"])
    else:
        src, dst = st["src"].long(), st["dst"].long()
        _free(st, dst)
        _fork(st, src, dst)
        _reserve(st, dst)
        _append(st, dst)
        _commit(st, dst)
    return {n: st[n] for n in ("k_pages", "v_pages", "table", "lens", "held", "refs", "granted")}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    lens, d, hk = _lengths(case), case["d"], case["kv_heads"]
    if case["op"] == "prompt":
        hq, total = hk * case["group"], sum(lens)
        return {"bytes": es * d * total * 2 * (hq + hk) + 4 * hq * total, "flops": sum(2 * d * hq * n * (n + 1) for n in lens)}
    drafts, page = _drafts(case), case["page"]
    if case["op"] == "tree":
        hq, total, rows = hk * case["group"], sum(drafts), sum(lens) + sum(drafts)
        return {"bytes": es * d * 2 * (hk * rows + hq * total) + 4 * hq * total,
                "flops": sum(4 * d * hq * t * (n + 1) for n, t in zip(lens, drafts))}
    # each branch: its rows of the draft in and out, the kept ones that move (at most all), half a page copied
    moved = sum(sum(i != j for i, j in enumerate(k)) for k in _kept(case))
    row = 2 * es * d * hk * case["layers"]
    copied = sum(lens) * case["seqs"] // len(lens) % page if len(lens) > 1 else case["seqs"] * (lens[0] % page)
    return {"bytes": 2 * row * (sum(drafts) + moved + copied), "flops": 0}


# ---- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "branch":
        return _exact_branch(st)
    hk, g, d = case["kv_heads"], case["group"], case["d"]
    out = torch.zeros(st["total"], hk * g, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(hk * g, st["total"], dtype=torch.float64, device="cuda")
    at = st["cu"].tolist()
    masks = st["mask"].tolist() if case["op"] == "tree" else None
    table = st["table"].tolist() if case["op"] == "tree" else None
    for i, n in enumerate(st["lengths"]):
        a, b = at[i], at[i + 1]
        if case["op"] == "prompt":
            keys, values, past = st["k"][a:b].transpose(0, 1), st["v"][a:b].transpose(0, 1), 0
        else:
            ids = torch.tensor([p for p in table[i] if p >= 0], device="cuda")
            keys = st["k_pages"][0, ids].transpose(0, 1).flatten(1, 2)[:, :n + b - a]
            values = st["v_pages"][0, ids].transpose(0, 1).flatten(1, 2)[:, :n + b - a]
            past = n
        step = max(1, 2 ** 28 // keys.shape[1])
        for first in range(a, b, step):
            rows = range(first, min(b, first + step))
            seen = torch.ones(len(rows), keys.shape[1], dtype=torch.bool, device="cuda")
            if case["op"] == "prompt":
                seen = seen.tril(first - a)
            else:
                seen[:, past:] = torch.tensor([[masks[r] >> j & 1 for j in range(b - a)] for r in rows], device="cuda") == 1
            for h in range(hk * g):
                s = st["q"][first:first + len(rows), h].double() @ keys[h // g].double().t() * st["scale"]
                s = s.masked_fill_(~seen, float("-inf"))
                lse[h, first:first + len(rows)] = torch.logsumexp(s, 1)
                out[first:first + len(rows), h] = torch.softmax(s, 1) @ values[h // g].double()
    return out, lse


def _exact_branch(st):
    """The cycle one sequence after another, with lists for the pages."""
    page, k, v = st["page"], st["k_pages"], st["v_pages"]
    table = [[p for p in row if p >= 0] for row in st["table"].tolist()]
    lens, refs, granted = st["lens"].tolist(), st["refs"].tolist(), []
    at, keep = st["cu"].tolist(), _kept(st)

    def take():
        p = refs.index(0)
        refs[p] = 1
        return p

    for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
        table[t], lens[t] = list(table[s]), lens[s]
        for p in table[t]:
            refs[p] += 1
    for t, add in zip(st["dst"].tolist(), st["add"].tolist()):
        rest = lens[t] % page
        if rest and refs[table[t][-1]] > 1:
            old, table[t][-1] = table[t][-1], take()
            refs[old] -= 1
            for x in (k, v):
                x[:, table[t][-1], :, :rest] = x[:, old, :, :rest]
        while len(table[t]) * page < lens[t] + add:
            table[t].append(take())
        granted.append(add)
    for i, t in enumerate(st["dst"].tolist()):
        ids = torch.tensor(table[t], device="cuda")
        for x, rows in ((k, st["k_new"]), (v, st["v_new"])):
            where = torch.arange(lens[t], lens[t] + at[i + 1] - at[i], device="cuda")
            new = rows[:, at[i]:at[i + 1]]
            x[:, ids[where // page], :, where % page] = new.transpose(0, 1)
            kept = where[:len(keep[i])]
            x[:, ids[kept // page], :, kept % page] = new[:, keep[i]].transpose(0, 1)
        lens[t] += len(keep[i])
        while len(table[t]) * page - page >= lens[t]:
            refs[table[t].pop()] -= 1
    held = [len(x) for x in table]
    rows = [x + [-1] * (st["most"] - len(x)) for x in table]
    return {"k_pages": k, "v_pages": v, "table": _ints(rows), "lens": _ints(lens), "held": _ints(held), "refs": _ints(refs),
            "granted": _ints(granted)}
