"""Workloads of the operators that serve drafts and forks from a paged key/value
cache: a tree of drafted tokens and who sees whom in it, appending its tokens,
attention over the cache and the tree, keeping the accepted path, and the
pages themselves (forked, grown, cut, freed, copied before they are written).

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges,
``prepare(case, seed)`` builds what a program holds before the call and
``run(state)`` makes one pass: in elementary torch operations in 32 bits, or,
where ``own`` is true, through the library.  ``exact(case, seed)`` computes the
same outputs in 64 bits and ``work(case)`` counts what a pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one sequence's draft of 8 tokens: latency
        dict(name="tree_tiny", op="tree", B=1, new_lo=8, new_hi=8, ragged=1),
        # large drafts of 256 sequences of unequal size
        dict(name="tree_batch", op="tree", B=256, new_lo=20, new_hi=500, ragged=2),
        # drafts of up to 64 tokens of 64 sequences entering one layer's cache
        # (heads of the grouped-query workload)
        dict(name="append_drafts", op="append", dtype="bf16", B=64, H=32, Hkv=8, DK=128, DV=128, rot=128, page=16,
             new_lo=8, new_hi=64, past_lo=0, past_hi=2047, ragged=3, interleaved=False, norm=True),
        # three sequences, a head width that is no power of two, adjacent pairs
        # of a part of the columns rotated
        dict(name="append_odd", op="append", dtype="f16", B=3, H=12, Hkv=4, DK=80, DV=80, rot=32, page=24,
             new_lo=1, new_hi=40, past_lo=0, past_hi=700, ragged=4, interleaved=True, norm=False),
        # a verification step of 32 sequences: drafts of 8 to 64 tokens behind
        # unequal pasts
        dict(name="verify_batch", op="attention", dtype="bf16", B=32, H=32, Hkv=8, DK=128, DV=128, page=16,
             new_lo=8, new_hi=64, past_lo=64, past_hi=4095, ragged=5),
        # one sequence with a very long cache and a draft of 64 tokens
        dict(name="verify_long", op="attention", dtype="bf16", B=1, H=32, Hkv=8, DK=128, DV=128, page=64,
             new_lo=64, new_hi=64, past_lo=131000, past_hi=131000, ragged=6),
        # trees of hundreds of tokens: the masked part is a large share
        dict(name="verify_wide", op="attention", dtype="f16", B=8, H=16, Hkv=4, DK=64, DV=64, page=32,
             new_lo=100, new_hi=500, past_lo=0, past_hi=3500, ragged=7),
        # one short sequence in 32 bits, a head width of 80: latency
        dict(name="verify_short_f32", op="attention", dtype="f32", B=1, H=8, Hkv=2, DK=80, DV=80, page=24,
             new_lo=7, new_hi=7, past_lo=499, past_hi=499, ragged=8),
        # the accepted paths of 64 sequences in all layers of a model
        dict(name="accept_batch", op="accept", dtype="bf16", B=64, Hkv=8, DK=128, DV=128, page=16, layers=32,
             new_lo=8, new_hi=64, past_lo=0, past_hi=200, ragged=9),
        # five sequences in one layer, 32 bits, odd sizes: latency
        dict(name="accept_odd", op="accept", dtype="f32", B=5, Hkv=2, DK=80, DV=40, page=24, layers=1,
             new_lo=1, new_hi=40, past_lo=0, past_hi=700, ragged=10),
        # between two verification steps of 256 sequences over a large pool of
        # pages: what was kept stays, room for the next draft, some sequences
        # end and others enter
        dict(name="reserve_step", op="reserve", dtype="bf16", B=256, Hkv=1, DK=64, DV=64, page=16, layers=1,
             mode="step", beams=1, past_lo=100, past_hi=6000, grow=64, pages=131072, ragged=11),
        # 16 prompts forked into 8 beams each, in all layers of a model: pages
        # shared, the last one copied for every beam that will write into it
        dict(name="reserve_fork", op="reserve", dtype="bf16", B=128, Hkv=8, DK=128, DV=128, page=64, layers=32,
             mode="fork", beams=8, past_lo=64, past_hi=500, grow=1, pages=0, ragged=12),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "append", "attention", "attention", "attention", "accept", "reserve", "reserve"])
    ragged = rng.randint(0, 1 << 30)
    if op == "tree":
        new = _spread(rng, 1, 500)
        return dict(op=op, B=_spread(rng, 1, 256), new_lo=max(1, new // 4), new_hi=new, ragged=ragged)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    D = rng.choice([64, 80, 96, 128, 128])
    page = rng.choice([16, 16, 24, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, dtype=dtype, Hkv=Hkv, DK=D, DV=D, page=page, ragged=ragged)
    if op == "append":
        most = _spread(rng, 1, 64)
        return dict(c, H=Hkv * rng.choice([1, 2, 3, 4]), rot=rng.choice([D, D, 32]), interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.8, B=_spread(rng, 1, 64), new_lo=max(1, most // 4), new_hi=most, past_lo=0,
                    past_hi=_spread(rng, 1, 2000))
    if op == "attention":
        if dtype == "f32":  # on the CUDA cores: smaller batches
            B, most, past, group = _spread(rng, 1, 6), _spread(rng, 1, 40), _spread(rng, 1, 1000), rng.choice([1, 2])
        elif rng.random() < 0.7:
            B, most, group = _spread(rng, 1, 32), _spread(rng, 1, 64), rng.choice([1, 2, 4, 7] if Hkv <= 4 else [1, 2, 4])
            past = _spread(rng, 1, 100000 if B == 1 else 4000)
        else:
            B, most, past, group = _spread(rng, 1, 4), _spread(rng, 64, 500), _spread(rng, 1, 3000), rng.choice([1, 2, 4])
        return dict(c, H=Hkv * group, B=B, new_lo=max(1, most // 4), new_hi=most, past_lo=past // 8, past_hi=past)
    if op == "accept":
        return dict(c, B=_spread(rng, 1, 64), layers=rng.choice([1, 2, 8, 24]), new_lo=1, new_hi=_spread(rng, 2, 64),
                    past_lo=0, past_hi=_spread(rng, 1, 200))
    mode = rng.choice(["step", "fork", "reorder"])
    beams = 1 if mode == "step" else rng.choice([2, 4, 5, 8])
    return dict(c, B=beams * _spread(rng, 1, 128 // beams), layers=rng.choice([1, 2, 8, 16]), mode=mode, beams=beams,
                past_lo=1, past_hi=_spread(rng, 2, 400), grow=_spread(rng, 1, 64) if mode == "step" else 1,
                pages=0)


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """New tokens and tokens held after them, of each sequence."""
    r = np.random.RandomState(case["ragged"])
    new = r.randint(case["new_lo"], case["new_hi"] + 1, case["B"])
    past = r.randint(case["past_lo"], case["past_hi"] + 1, case["B"]) if "past_lo" in case else 0 * new
    return new, new + past


def _parents(new, r):
    """Drafts: half of the tokens continue the one before, the others any earlier
    one (or, as the first does, the cache's last token: -1)."""
    i = np.concatenate([np.arange(n) for n in new])
    p = np.floor(r.rand(i.size) * (i + 1)).astype(np.int64) - 1
    return np.where(r.rand(i.size) < 0.5, i - 1, p)


def _sight(new, parents):
    """(tokens, 32 words) of truth values: who sees whom, and the words."""
    words = -(-int(max(new)) // 32)
    dense = np.zeros((len(parents), 32 * words), dtype=bool)
    t0 = 0
    for n in new:
        for i in range(n):
            if parents[t0 + i] >= 0:
                dense[t0 + i] = dense[t0 + parents[t0 + i]]
            dense[t0 + i, i] = True
        t0 += n
    bits = np.packbits(dense.reshape(-1, 32), axis=1, bitorder="little").view("<u4").view(np.int32)
    return dense, bits.reshape(len(parents), words)


def _drafts(case):
    """(new, total, who sees whom, the same in bits, the last accepted token or -1)"""
    new, total = _lengths(case)
    r = np.random.RandomState(case["ragged"] + 1)
    dense, bits = _sight(new, _parents(new, r))
    last = np.floor(r.rand(len(new)) * new).astype(np.int64)
    return new, total, dense, bits, np.where(r.rand(len(new)) < 0.1, -1, last)


def _tables(length, rot, device):
    """Cosines and sines of every position, angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return a.cos().float(), a.sin().float()


def _int32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _scenario(case):
    """What a scheduler has decided: (logical pages of each row's entries or -1,
    how many there are, source or None, tokens kept, tokens to have room for)."""
    r = np.random.RandomState(case["ragged"])
    B, page, mode, beams = case["B"], case["page"], case["mode"], case["beams"]
    up = lambda x: -(-x // page)  # noqa: E731
    if mode == "step":
        past = r.randint(case["past_lo"], case["past_hi"] + 1, B)
        held = past + case["grow"]
        kept = past + r.randint(0, case["grow"] + 1, B)
        lens = kept + case["grow"]
        fate = r.rand(B)
        lens = np.where(fate < 0.04, 0, lens)  # ended
        enters = fate > 0.96
        held, kept = np.where(enters, 0, held), np.where(enters, 0, kept)
        shared, source = 0 * held, None
    else:
        groups = B // beams
        first = np.repeat(np.arange(groups) * beams, beams)
        prompt = np.repeat(r.randint(case["past_lo"], case["past_hi"] + 1, groups), beams)
        if mode == "fork":
            held = np.where(np.arange(B) == first, prompt, 0)
            source, kept, shared = first, prompt, 0 * held
        else:
            held = prompt + np.repeat(r.randint(1, 2 * page, groups), beams)
            source, kept = first + r.randint(0, beams, B), held
            shared = np.where(np.arange(B) == first, 0, prompt // page)
        lens = kept + case["grow"]
    need = np.maximum(up(held), up(lens))
    logical = np.full((B, int(need.max()) + 2), -1, dtype=np.int64)
    count = 0
    for b in range(B):
        own_pages = int(up(held[b]) - shared[b])
        if shared[b]:
            logical[b, : shared[b]] = logical[b - b % beams, : shared[b]]
        logical[b, shared[b]: shared[b] + own_pages] = count + np.arange(own_pages)
        count += own_pages
    room = count + int(np.maximum(up(lens) - up(np.minimum(kept, lens)) + 1, 0).sum()) + 3
    return logical, max(room, case["pages"]), source, kept, lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)

    def normal(shape, t):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    if case["op"] == "tree":
        new, _ = _lengths(case)
        s["most"] = int(new.max())
        s["starts"] = _int32(np.concatenate([[0], np.cumsum(new)]))
        s["parents"] = _int32(_parents(new, np.random.RandomState(int(seed) % (1 << 32))))
        return s
    dt, Hkv, DK, DV, page = _DT[case["dtype"]], case["Hkv"], case["DK"], case["DV"], case["page"]
    if case["op"] == "reserve":
        logical, count, source, kept, lens = _scenario(case)
        order = torch.randperm(count, generator=g, device="cuda").cpu().numpy()
        table = np.where(logical >= 0, order[logical], -1)
        s["table"], s["kept"], s["lens"] = _int32(table), _int32(kept), _int32(lens)
        s["refs"] = _int32(np.bincount(table[table >= 0], minlength=count))
        s["source"] = None if source is None else _int32(source)
        s["k_cache"] = normal((case["layers"], count, Hkv, page, DK), dt)
        s["v_cache"] = normal((case["layers"], count, Hkv, page, DV), dt)
        return s
    new, total, _, bits, last = _drafts(case)
    T = s["T"] = int(new.sum())
    s["most_new"], s["most_keys"] = int(new.max()), int(total.max())
    s["starts"], s["lens"], s["seen"] = _int32(np.concatenate([[0], np.cumsum(new)])), _int32(total), _int32(bits)
    need = -(-total // page)
    count = int(need.sum()) + 2
    order = torch.randperm(count, generator=g, device="cuda")
    s["table"] = torch.zeros((case["B"], int(need.max())), dtype=torch.int32, device="cuda")
    live = torch.arange(int(need.max()), device="cuda") < torch.as_tensor(need, device="cuda")[:, None]
    s["table"].masked_scatter_(live, order[: int(need.sum())].to(torch.int32))
    layers = (case["layers"],) if case["op"] == "accept" else ()
    s["k_cache"] = normal((*layers, count, Hkv, page, DK), dt)
    s["v_cache"] = normal((*layers, count, Hkv, page, DV), dt)
    if case["op"] == "accept":
        s["last"] = _int32(last)
    elif case["op"] == "append":
        H = case["H"]
        # one row of the projection holds the token's queries, keys and values
        q, k, v = normal((T, H * DK + Hkv * DK + Hkv * DV), dt).split([H * DK, Hkv * DK, Hkv * DV], dim=-1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (H, DK)), k.unflatten(-1, (Hkv, DK)), v.unflatten(-1, (Hkv, DV))
        s["wq"] = (1 + 0.2 * normal((DK,), torch.float32)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * normal((DK,), torch.float32)).to(dt) if case["norm"] else None
        s["cos"], s["sin"] = _tables(s["most_keys"], case["rot"], "cuda")
    else:
        s["q"] = normal((T, case["H"], DK), dt)
        s["scale"] = DK ** -0.5
    return s


# ------------------------------------------------------------------ plain forms


def _places(s):
    """Of every token: its sequence, its number there, that sequence's past."""
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), new, output_size=s["T"])
    return seq, torch.arange(s["T"], device=lens.device) - starts[seq], (lens - new)[seq]


def _unpacked(seen):
    """(tokens, 32 words) of truth values"""
    bit = torch.arange(32, device=seen.device)
    return ((seen.long()[:, :, None] >> bit) & 1).bool().flatten(1)


def _plain_tree(s):
    starts, n = s["starts"].long(), s["most"]
    B, T = len(starts) - 1, len(s["parents"])
    words = -(-n // 32)
    new = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(B, device=starts.device), new, output_size=T)
    i = torch.arange(T, device=starts.device) - starts[seq]
    # reach[b, i, j]: j is i or one of its ancestors within 1, 2, 4, ... steps
    reach = torch.zeros((B, n, n + 1), device=starts.device)
    reach[seq, i, s["parents"].long()] = 1.0  # (-1: the column behind the last)
    reach = reach[:, :, :n]
    reach[seq, i, i] = 1.0
    for _ in range(n.bit_length()):
        reach = ((reach @ reach) > 0).float()
    sees = torch.nn.functional.pad(reach[seq, i].long(), (0, 32 * words - n)).view(T, words, 32)
    value = (sees << torch.arange(32, device=starts.device)).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def _turn(x, cos, sin, interleaved):
    """Rotates the first 2 * cos.shape[-1] columns of x; cos, sin broadcast."""
    half = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        y[..., 0: 2 * half: 2] = a * cos - b * sin
        y[..., 1: 2 * half: 2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half: 2 * half]
        y[..., :half] = a * cos - b * sin
        y[..., half: 2 * half] = b * cos + a * sin
    return y


def _norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_append(s):
    il, page, dt = s["case"]["interleaved"], s["case"]["page"], s["q"].dtype
    seq, i, past = _places(s)
    sees = _unpacked(s["seen"])
    earlier = torch.arange(sees.shape[1], device=i.device) < i[:, None]
    pos = past + (sees & earlier).sum(-1)  # as far behind the past as it is deep in the tree
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _turn(_norm(s["q"].float(), s["wq"]), cos, sin, il).to(dt)
    k = _turn(_norm(s["k"].float(), s["wk"]), cos, sin, il).to(dt)
    at = past + i
    where = s["table"][seq, at // page].long()
    s["k_cache"][where, :, at % page] = k
    s["v_cache"][where, :, at % page] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    B, H, Hkv, DK, DV, page, N = c["B"], c["H"], c["Hkv"], c["DK"], c["DV"], c["page"], s["most_new"]
    starts, lens = s["starts"].long(), s["lens"].long()
    past = lens - (starts[1:] - starts[:-1])
    i = torch.arange(N, device=lens.device)
    token = (starts[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][token].float().view(B, N, Hkv, H // Hkv, DK).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, DK)
    pages = s["table"].long()
    L = pages.shape[1] * page
    m = torch.arange(L, device=lens.device)
    held = (m < lens[:, None])[:, None, :, None]
    k = s["k_cache"][pages].float().transpose(1, 2).reshape(B, Hkv, L, DK)
    v = s["v_cache"][pages].float().transpose(1, 2).reshape(B, Hkv, L, DV).masked_fill(~held, 0.0)
    sees = _unpacked(s["seen"])[token]
    j = (m - past[:, None]).clamp(0, sees.shape[2] - 1)[:, None].expand(B, N, L)
    sees = sees.gather(2, j) & (m <= past[:, None, None] + i[:, None]) | (m < past[:, None, None])
    sees = sees[:, None, :, None].expand(B, 1, N, H // Hkv, L).reshape(B, 1, -1, L)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~sees, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = ((x @ v) / total).view(B, Hkv, N, H // Hkv, DV).permute(0, 2, 1, 3, 4)
    lse = (top + total.log()).view(B, Hkv, N, H // Hkv).permute(0, 2, 1, 3)
    seq, row, _ = _places(s)
    o = o[seq, row].reshape(s["T"], H, DV).to(s["q"].dtype)
    return o, lse[seq, row].reshape(s["T"], H).t().contiguous()


def _plain_accept(s):
    page = s["case"]["page"]
    starts, lens, last = s["starts"].long(), s["lens"].long(), s["last"].long()
    past = lens - (starts[1:] - starts[:-1])
    row = _unpacked(s["seen"])[(starts[:-1] + last).clamp(min=0)]
    taken = row & (torch.arange(row.shape[1], device=row.device) <= last[:, None])
    b, j = taken.nonzero(as_tuple=True)
    to = past[b] + (taken.cumsum(-1) - 1)[b, j]
    at = past[b] + j
    src, dst = s["table"][b, at // page].long(), s["table"][b, to // page].long()
    s["k_cache"][:, dst, :, to % page] = s["k_cache"][:, src, :, at % page]
    s["v_cache"][:, dst, :, to % page] = s["v_cache"][:, src, :, at % page]
    return (past + taken.sum(-1)).to(torch.int32), s["k_cache"], s["v_cache"]


def _plain_reserve(s):
    page, table, refs = s["case"]["page"], s["table"].long(), s["refs"].long()
    (B, W), pages, dev = table.shape, len(refs), table.device
    row, slot = torch.arange(B, device=dev), torch.arange(W, device=dev)
    source = row if s["source"] is None else s["source"].long()
    lens = s["lens"].long()
    kept = torch.where(source >= 0, torch.minimum(s["kept"].long(), lens), 0)
    first, end = (kept + page - 1) // page, (lens + page - 1) // page
    carried = torch.where(slot < first[:, None], table[source.clamp(min=0)], -1)

    def count(entries):  # how often each page is named (-1: not at all)
        return torch.zeros(pages + 1, dtype=torch.long, device=dev).scatter_add_(
            0, entries.flatten() % (pages + 1), torch.ones_like(entries.flatten()))[:pages]

    # a row that goes on inside a page wants it for itself: the first such row keeps
    # a page that no other row holds, the others get copies
    writes = (kept % page != 0) & (lens > kept)
    mine = carried[row, (kept // page).clamp(max=W - 1)]
    mine = torch.where(writes, mine, -1)
    refs = refs - count(table) + count(carried) - count(mine)
    lowest = torch.full((pages + 1,), B, device=dev).scatter_reduce_(0, mine % (pages + 1), row, "amin")
    keeps = writes & (refs[mine] == 0) & (lowest[mine % (pages + 1)] == row)
    copies = writes & ~keeps
    refs = refs + count(torch.where(keeps, mine, -1))
    fresh = (slot >= (first - copies.long())[:, None]) & (slot < end[:, None])
    rank = fresh.flatten().cumsum(0).view(B, W) - 1
    free = (refs == 0).sum()
    order = torch.argsort((refs != 0).long(), stable=True)  # the free ones, lowest first
    given = torch.where(fresh & (rank < free), order[rank.clamp(0, pages - 1)], -1)
    new = torch.where(fresh, given, carried)
    s["table"].copy_(new)
    s["refs"].copy_(refs + count(given))
    to = new[row, (kept // page).clamp(max=W - 1)]
    b = (copies & (to >= 0)).nonzero().flatten()
    part = (torch.arange(page, device=dev) < (kept % page)[b, None])[:, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, to[b]] = torch.where(part, cache[:, mine[b]], cache[:, to[b]])
    spare = (free - fresh.sum()).to(torch.int32).view(1)
    return s["table"], s["refs"], spare, s["k_cache"], s["v_cache"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        plain = {"tree": _plain_tree, "append": _plain_append, "attention": _plain_attention, "accept": _plain_accept,
                 "reserve": _plain_reserve}
        return plain[op](s)
    from attention_backward_tcgen05_gb300 import binding

    if op == "tree":
        return binding.draft_tree(s["starts"], s["parents"], s["most"])
    if op == "append":
        q = binding.paged_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["starts"], s["lens"],
                                 s["table"], s["k_cache"], s["v_cache"], EPS, s["case"]["interleaved"], seen=s["seen"])
        return q, s["k_cache"], s["v_cache"]
    if op == "attention":
        return binding.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["starts"], s["lens"], s["table"],
                                       scale=s["scale"], seen=s["seen"])
    if op == "accept":
        lens = binding.paged_accept(s["starts"], s["lens"], s["table"], s["seen"], s["last"], s["k_cache"],
                                    s["v_cache"])
        return lens, s["k_cache"], s["v_cache"]
    spare = binding.paged_reserve(s["table"], s["refs"], s["kept"], s["lens"], s["k_cache"], s["v_cache"],
                                  source=s["source"])
    return s["table"], s["refs"], spare, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ 64 bits


def _exact_rows(x, w, cos, sin, interleaved):
    """Rows x in 64 bits, normalised and rotated as complex pairs."""
    x = x.double()
    rot = 2 * cos.shape[-1]
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    by = torch.complex(cos.double(), sin.double())
    a = x[..., :rot]
    if interleaved:
        z = torch.view_as_real(torch.view_as_complex(a.unflatten(-1, (-1, 2)).contiguous()) * by).flatten(-2)
    else:
        z = torch.complex(a[..., : rot // 2].contiguous(), a[..., rot // 2:].contiguous()) * by
        z = torch.cat([z.real, z.imag], -1)
    return torch.cat([z, x[..., rot:]], -1)


def exact(case, seed):
    if case["op"] not in ("append", "attention"):
        return None  # whole numbers, and rows moved as they are
    s = prepare(case, seed)
    new, total, dense, _, _ = _drafts(case)
    page = case["page"]
    table = s["table"].cpu()
    if case["op"] == "append":
        deep = dense.sum(1) - 1
        pos = np.repeat(total - new, new) + deep
        pos = torch.as_tensor(pos, device="cuda")
        cos, sin = s["cos"][pos].unsqueeze(1), s["sin"][pos].unsqueeze(1)
        q = _exact_rows(s["q"], s["wq"], cos, sin, case["interleaved"])
        k = _exact_rows(s["k"], s["wk"], cos, sin, case["interleaved"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        t0 = 0
        for b, (n, t) in enumerate(zip(new.tolist(), total.tolist())):
            p = torch.arange(t - n, t)
            slot = (table[b][p // page].long().cuda(), slice(None), (p % page).cuda())
            kc[slot] = k[t0: t0 + n]
            vc[slot] = s["v"][t0: t0 + n].double()
            t0 += n
        return q, kc, vc
    H, G = case["H"], case["H"] // case["Hkv"]
    o = torch.empty((s["T"], H, case["DV"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((H, s["T"]), dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, t) in enumerate(zip(new.tolist(), total.tolist())):
        at = table[b][: -(-t // page)].long().cuda()
        hidden = torch.zeros((n, t), dtype=torch.bool, device="cuda")
        hidden[:, t - n:] = torch.as_tensor(~dense[t0: t0 + n, :n], device="cuda")
        for hk in range(case["Hkv"]):
            k = s["k_cache"][at, hk].flatten(0, 1)[:t].double()
            v = s["v_cache"][at, hk].flatten(0, 1)[:t].double()
            for h in range(hk * G, hk * G + G):
                x = s["scale"] * (s["q"][t0: t0 + n, h].double() @ k.t())
                x.masked_fill_(hidden, float("-inf"))
                z = torch.logsumexp(x, -1)
                lse[h, t0: t0 + n] = z
                o[t0: t0 + n, h] = torch.exp(x - z[:, None]) @ v
        t0 += n
    return o, lse


# ------------------------------------------------------------------ work


def work(case):
    B = case["B"]
    if case["op"] == "tree":
        new, _ = _lengths(case)
        T = int(new.sum())
        return dict(bytes=4 * (T + B + 1) + 4 * T * -(-int(new.max()) // 32), flops=0)
    e, Hkv, DK, DV, page = _SIZE[case["dtype"]], case["Hkv"], case["DK"], case["DV"], case["page"]
    if case["op"] == "reserve":
        logical, count, source, kept, lens = _scenario(case)
        kept = np.minimum(kept, lens)
        first, end = -(-kept // page), -(-lens // page)
        src = np.arange(B) if source is None else source
        writes = (kept % page != 0) & (lens > kept)
        mine = logical[src, kept // page]
        # copied for every row that goes on inside a page, but the first where no other row holds it
        wanted = np.where(writes, mine, -1)
        held = {int(x): 0 for x in wanted}
        for b in range(B):
            for x in logical[src[b], : first[b]].tolist():
                if x in held:
                    held[x] += 1
        keeps = {int(x): int(np.flatnonzero(wanted == x)[0]) for x in np.unique(wanted)
                 if x >= 0 and held[int(x)] == (wanted == x).sum()}
        copied = [b for b in range(B) if writes[b] and keeps.get(int(mine[b])) != b]
        moved = sum(int(kept[b]) % page for b in copied) * case["layers"] * Hkv * (DK + DV) * e
        entries = int((logical >= 0).sum()) + int(end.sum())  # those there are, and those there will be
        return dict(bytes=2 * moved + 4 * entries + 4 * count + 12 * B, flops=0)
    new, total, dense, bits, last = _drafts(case)
    T = int(new.sum())
    if case["op"] == "accept":
        moved, t0 = 0, 0
        for n, a in zip(new.tolist(), last.tolist()):
            if a >= 0:
                at = np.flatnonzero(dense[t0 + a, : a + 1])
                moved += int((at != np.arange(at.size)).sum())
            t0 += n
        return dict(bytes=2 * moved * case["layers"] * Hkv * (DK + DV) * e + 4 * B * (bits.shape[1] + 4), flops=0)
    H, sight = case["H"], 4 * bits.size
    heads = H * DK + Hkv * DK  # normalised and rotated values of a token
    if case["op"] == "append":
        table = min(T, int(total.max())) * case["rot"] * 4 + 8 * B + 4 * T + sight
        return dict(bytes=2 * T * (heads + Hkv * DV) * e + table, flops=10 * T * heads)
    pairs = int((new * (total - new)).sum()) + int(dense.sum())
    nbytes = int(total.sum()) * Hkv * (DK + DV) * e + T * H * (DK + DV) * e + T * H * 4 + sight
    nbytes += int((-(-total // page)).sum()) * 4
    return dict(bytes=nbytes, flops=2 * pairs * H * (DK + DV))
