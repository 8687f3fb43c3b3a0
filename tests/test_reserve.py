"""The pages of a cache: handed out, shared, copied before they are written and
freed, against a loop over rows; and whole serving steps with drafts and forks
against the attention over plain sequences.
"""
import ctypes
import random
from collections import Counter

import pytest
import torch

from attention_backward_tcgen05_gb300 import binding
from test_drafts import BAD_CACHE, cache_dims, draw_parents, packed, sight, starts_of
from test_norm_rope import DT, half_step, tables
from test_paged import A, gpu  # noqa: F401 (gpu: a fixture)


def call_reserve(dims, table=A, refs=A, source=A, kept=A, lens=A, dtype=1, kc=A, vc=A, ws=A, wsb=1 << 40, spare=A):
    return binding.lib().fab_paged_reserve(table, refs, source, kept, lens, dtype, ctypes.byref(dims), kc, vc, ws, wsb,
                                           spare, None)


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_refused_dims(bad):
    assert call_reserve(cache_dims(**bad)) == binding.FAB_ERR_INVALID
    assert binding.fab_paged_reserve_workspace_bytes(cache_dims(**bad)) == 0


@pytest.mark.parametrize("bad", [dict(table=None), dict(refs=A + 4), dict(refs=None), dict(source=A + 1),
                                 dict(kept=None), dict(lens=A + 2), dict(dtype=-1), dict(kc=None), dict(vc=A + 8),
                                 dict(spare=None), dict(spare=A + 2)], ids=str)
def test_refused_arguments(bad):
    assert call_reserve(cache_dims(), **bad) == binding.FAB_ERR_INVALID


def test_workspace_and_width_refusals():
    need = binding.fab_paged_reserve_workspace_bytes(cache_dims())
    assert need > 0
    for bad in (dict(wsb=need - 1), dict(ws=A + 8), dict(ws=None)):
        assert call_reserve(cache_dims(), **bad) == binding.FAB_ERR_WORKSPACE
    assert call_reserve(cache_dims(DK=264, layers=1)) == binding.FAB_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["table", "refs", "source", "kept", "lens", "ws"])
def test_spare_over_what_the_call_uses_is_refused(name):
    at = {n: A + 4096 * i for i, n in enumerate(("table", "refs", "source", "kept", "lens", "ws"))}
    need = binding.fab_paged_reserve_workspace_bytes(cache_dims())
    assert need <= 4096
    last = dict(table=20, refs=28, source=4, kept=4, lens=4, ws=need - 4)[name]  # bytes to the last element
    for spare in (at[name], at[name] + last):
        assert call_reserve(cache_dims(), wsb=need, spare=spare, **at) == binding.FAB_ERR_INVALID


def test_binding_refuses_what_does_not_fit():
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(5, 2, 16, 64)
    with pytest.raises(ValueError):
        binding.paged_reserve(i32(2, 3), i32(5), i32(2), i32(2), k, k)  # not CUDA tensors
    with pytest.raises(ValueError):
        binding.paged_reserve(i32(2), i32(5), i32(2), i32(2), k, k)  # table not 2-D


# ------------------------------------------------------------------ a loop over rows


def reference(table, pages, page, source, kept, lens):
    """(table, references, pages left or missing, {fresh page: (page, rows) it gets a copy of})"""
    B, W = len(table), len(table[0])
    carried, writes = [], []
    for b in range(B):
        s = b if source is None else source[b]
        keep = min(kept[b], lens[b]) if s >= 0 else 0
        carried.append(list(table[s][: -(-keep // page)]) if keep else [])
        writes.append(keep % page if lens[b] > keep else 0)
    holders = Counter(p for row in carried for p in row)
    writers = {}
    for b in range(B):
        if writes[b]:
            writers.setdefault(carried[b][-1], []).append(b)
    copy = {}
    for p, rows in writers.items():
        if holders[p] == len(rows):
            rows = rows[1:]  # the first keeps it
        for b in rows:
            copy[b] = (carried[b].pop(), writes[b])
    used = {p for row in carried for p in row}
    free = [p for p in range(pages) if p not in used]
    out, copies, given = [], {}, 0
    for b in range(B):
        row = list(carried[b])
        for i in range(len(carried[b]), -(-lens[b] // page)):
            row.append(free[given] if given < len(free) else -1)
            if b in copy and i == len(carried[b]) and row[-1] >= 0:
                copies[row[-1]] = copy[b]
            given += 1
        out.append(row + [-1] * (W - len(row)))
    count = Counter(p for row in out for p in row if p >= 0)
    return out, [count[p] for p in range(pages)], len(free) - given, copies


class Pool:
    def __init__(self, B, W, pages, page, Hkv, DK, DV, dtype, layers, seed, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.pages = page, pages
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        make = lambda D: torch.randn((layers, pages * Hkv * page * D + gap), generator=g).to(DT[dtype]).cuda()[  # noqa: E731
            :, : pages * Hkv * page * D].unflatten(1, (pages, Hkv, page, D))
        self.k, self.v = make(DK), make(DV)

    def call(self, kept, lens, source=None):
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return binding.paged_reserve(self.table, self.refs, i32(kept), i32(lens), self.k, self.v, i32(source))

    def step(self, kept, lens, source=None):
        """A call, all of it compared with the loop over rows."""
        was, k, v = self.table.cpu().tolist(), self.k.cpu(), self.v.cpu()
        table, refs, spare, copies = reference(was, self.pages, self.page, source, kept, lens)
        got = self.call(kept, lens, source)
        assert self.table.cpu().tolist() == table
        assert self.refs.cpu().tolist() == refs
        assert int(got) == spare
        for to, (a, rows) in copies.items():
            k[:, to, :, :rows], v[:, to, :, :rows] = k[:, a, :, :rows], v[:, a, :, :rows]
        assert torch.equal(self.k.cpu(), k) and torch.equal(self.v.cpu(), v)
        return spare


# B, entries of a row, pages, page, Hkv, DK, DV, dtype, layers, gap
POOLS = {
    "bf16": (6, 9, 60, 16, 2, 64, 64, "bf16", 3, 0),
    "f16_gaps": (6, 9, 60, 24, 3, 80, 80, "f16", 2, 8),
    "f32_odd": (7, 9, 64, 5, 1, 7, 3, "f32", 2, 1),
    "bf16_odd_gap": (5, 9, 50, 8, 2, 64, 32, "bf16", 2, 3),
    "bf16_wide_page": (5, 3, 20, 128, 2, 128, 128, "bf16", 1, 0),
    "f32_page_of_one": (5, 40, 300, 1, 1, 4, 4, "f32", 1, 0),
    "bf16_many_rows": (1500, 3, 4600, 16, 1, 8, 8, "bf16", 1, 0),
    "bf16_one_row": (1, 1, 2, 16, 1, 8, 8, "bf16", 1, 0),
    "bf16_three_rows": (3, 2, 5, 16, 1, 8, 8, "bf16", 2, 0),
    "bf16_large_pool": (4, 9, 150001, 4, 1, 8, 8, "bf16", 1, 0),
    "bf16_rows_of_several_shares": (9000, 2, 18001, 2, 1, 8, 8, "bf16", 1, 0),
    "bf16_long_rows": (3, 2600, 9001, 4, 1, 8, 8, "bf16", 1, 0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", POOLS)
def test_drawn_steps(gpu, name):
    B, W, pages, page, Hkv, DK, DV, dtype, layers, gap = POOLS[name]
    x = Pool(B, W, pages, page, Hkv, DK, DV, dtype, layers, 5, gap)
    r = random.Random(sum(map(ord, name)))
    most = W * page
    held = [0] * B  # tokens that each row has room for
    for i in range(14 if B < 100 else 6 if B < 5000 else 4):
        source = None
        if i % 3 == 1:  # forks, ends, and rows that go on
            source = [r.choice([b, b, r.randrange(B), r.randrange(B), -1]) for b in range(B)]
        elif i % 3 == 2:  # all continue one of a few
            few = [r.randrange(B) for _ in range(2)]
            source = [r.choice(few) for _ in range(B)]
        kept, lens = [], []
        for b in range(B):
            s = b if source is None else source[b]
            kept.append(r.choice([held[s], held[s], r.randint(0, held[s]), 0]) if s >= 0 else r.randint(0, most))
            keep = kept[b] if s >= 0 else 0
            lens.append(r.choice([min(most, keep + r.choice([0, 1, 1, r.randint(0, 3 * page)])), keep, 0,
                                  r.randint(0, keep)]))
        x.step(kept, lens, source)
        held = lens
    x.step(held, [0] * B)
    assert (x.refs == 0).all() and (x.table == -1).all()


@pytest.mark.gpu
def test_who_keeps_a_shared_page(gpu):
    x = Pool(5, 4, 12, 16, 2, 64, 64, "bf16", 2, 6)
    x.step([0] * 5, [20, 0, 0, 0, 0])                                # one row, its second page partly filled
    x.step([20, 20, 20, 20, 0], [20, 20, 20, 20, 0], [0, 0, 0, 0, -1])  # forked, nobody writes: all shared
    assert x.refs[x.table[0, 1].long()] == 4
    x.step([20] * 4 + [0], [21, 20, 20, 20, 0])                      # the owner writes, the others still hold it
    x.step([21, 20, 20, 20, 0], [21, 21, 21, 21, 0])                 # the rest all write: the first of them keeps it
    assert (x.refs[x.table[:4, 1].long()] == 1).all() and x.refs[x.table[0, 0].long()] == 4
    x.step([21, 21, 21, 21, 0], [0, 16, 40, 16, 0])                  # freed, cut to a whole page, grown
    x.step([0, 16, 40, 16, 0], [0, 17, 40, 17, 0])                   # behind a whole page: nothing to copy


@pytest.mark.gpu
def test_too_few_pages(gpu):
    x = Pool(3, 6, 7, 16, 2, 64, 64, "bf16", 1, 7)
    assert x.step([0, 0, 0], [40, 0, 0]) == 4
    assert x.step([40, 40, 40], [60, 60, 60], [0, 0, 0]) == -1       # the last row's last entry gets none
    assert x.table[2].tolist().count(-1) == 6 - 3
    assert x.step([60, 60, 0], [60, 60, 0]) == 1                     # of 7: 2 shared, 2 of each row's own


@pytest.mark.gpu
def test_copies_that_get_no_page(gpu):
    x = Pool(6, 4, 5, 16, 2, 64, 64, "bf16", 2, 7)
    x.step([0] * 6, [20, 0, 0, 0, 0, 0])
    assert x.step([20] * 6, [21] * 6, [0] * 6) == -2  # the first row keeps the page, three get copies, two nothing
    assert x.table[:, 1].tolist() == [1, 2, 3, 4, -1, -1] and x.refs.tolist() == [6, 1, 1, 1, 1]
    assert x.step([21, 21, 0, 16, 16, 16], [33, 21, 0, 16, 16, 40]) == -1


# B, entries of a row, pages, page, Hkv, DK, DV, dtype, layers, gap; steps.  Fewer pages than the rows ask for:
# in each, several steps run short, and copies of a page get none
SHORT = {
    "bf16": ((6, 9, 7, 16, 2, 64, 64, "bf16", 3, 0), 14),
    "f32_odd": ((7, 9, 7, 5, 1, 7, 3, "f32", 2, 1), 14),
    "bf16_many_rows": ((1500, 3, 1700, 16, 1, 8, 8, "bf16", 1, 0), 6),
    "bf16_rows_of_several_shares": ((9000, 2, 9200, 2, 1, 8, 8, "bf16", 1, 0), 5),
    "bf16_one_page": ((4, 2, 1, 16, 1, 8, 8, "bf16", 2, 0), 14),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHORT)
def test_drawn_steps_with_too_few_pages(gpu, name):
    (B, W, pages, page, *rest), steps = SHORT[name]
    x = Pool(B, W, pages, page, *rest[:5], 5, rest[5])
    r = random.Random(sum(map(ord, name)))
    held, short = [0] * B, 0  # tokens that each row has pages for
    for i in range(steps):
        source = None if i % 3 == 0 else [r.choice([b, r.randrange(B), r.randrange(min(B, 9))]) for b in range(B)]
        kept = [r.choice([held[s], held[s], r.randint(0, held[s])]) for s in (source or range(B))]
        lens = [min(W * page, k + r.choice([0, 1, 1, r.randint(0, 2 * page)])) for k in kept]
        short += x.step(kept, lens, source) < 0
        held = [min((row + [-1]).index(-1) * page, n) for row, n in zip(x.table.tolist(), lens)]
    assert short >= 2
    x.step(held, [0] * B)
    assert (x.refs == 0).all() and (x.table == -1).all()


@pytest.mark.gpu
def test_a_row_swapped_for_another(gpu):
    x = Pool(4, 5, 40, 8, 1, 16, 16, "f32", 1, 8)
    x.step([0] * 4, [5, 13, 29, 33])
    x.step([33, 29, 13, 5], [34, 30, 14, 6], [3, 2, 1, 0])
    x.step([30, 34, 6, 14], [40, 40, 40, 40], [1, 0, 3, 2])  # (kept: of what the row continued holds)
    x.step([40] * 4, [40] * 4, [0, 0, -1, 3])


@pytest.mark.gpu
def test_what_is_out_of_range_is_reported(gpu):
    def pool():
        x = Pool(3, 4, 20, 16, 1, 16, 16, "f32", 1, 9)
        x.step([0, 0, 0], [40, 20, 0])
        return x

    for kept, lens, source in (([40, 20, 0], [41, 20, 0], [0, 3, -1]), ([40, 20, 0], [41, 20, 0], [0, -2, -1]),
                               ([40, -1, 0], [41, 20, 0], None), ([40, 20, 0], [41, 65, 0], None),
                               ([40, 20, 0], [41, -5, 0], None), ([40, 1 << 30, 0], [41, 20, 0], None),
                               ([40, 33, 0], [41, 40, 0], None), ([40, 20, 10], [41, 20, 20], None)):
        x = pool()
        x.call(kept, lens, source)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        assert x.table[0].tolist()[:3] == [0, 1, 2]  # the row that was right
    for entry in (20, 1 << 30, -1):
        x = pool()
        x.table[1, 0] = entry
        x.call([40, 20, 0], [41, 21, 0])
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        assert x.table[0].tolist()[:3] == [0, 1, 2]
    x = pool()
    x.refs[1] = 0  # held by row 0
    x.call([40, 20, 0], [0, 21, 0])
    assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("W, page", [(4, 16), (300, 4)])
def test_counts_too_low_are_reported(gpu, W, page):
    # a page that a row holds would be handed out, or written by one row while another holds it
    most = 5 * page // 2 if W == 4 else 250 * page - 2

    def pool():
        x = Pool(3, W, 3 * W + 2, page, 1, 16, 16, "f32", 1, 9)
        x.step([0, 0, 0], [most, 20, 0])
        return x, x.table[0].tolist()

    end = (most - 1) // page  # the entry of the last, partly filled page
    for entry in {0, 1, end - 1}:
        x, row = pool()
        x.refs[row[entry]] = 0
        x.call([most, 20, 0], [most, 40, 20])
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID, entry
        x, row = pool()  # handed on: row 2 goes on with what row 0 held
        x.refs[row[entry]] = 0
        x.call([0, 20, most], [0, 40, most], [-1, 1, 0])
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID, entry
    x, row = pool()
    x.step([most, 20, most], [most, 20, most], [0, 1, 0])
    x.refs[row[end]] = 1  # of two
    x.call([most, 20, most], [most + 1, 20, most])
    assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
    x, row = pool()
    x.refs[row[end]] = 0
    x.call([most, 20, 0], [most + 1, 20, 0])
    assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID


@pytest.mark.gpu
def test_a_count_too_low_among_many_rows(gpu):
    B = 9000
    x = Pool(B, 2, 3 * B, 2, 1, 8, 8, "bf16", 1, 9)
    x.step([0] * B, [3] * B)
    for b in (0, 1124, 1125, 5000, B - 1):
        at = int(x.table[b, 0])
        x.refs[at] = 0
        x.call([3] * B, [3] * B)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID, b
        x.refs[at] = 1
        x.call([3] * B, [3] * B)
        assert binding.fab_last_device_error() == binding.FAB_OK, b


@pytest.mark.gpu
def test_counts_above_the_table_hold_pages(gpu):
    # pages that something besides the table holds: never written, handed out or freed
    x = Pool(2, 4, 9, 16, 2, 64, 64, "bf16", 2, 6)
    x.step([0, 0], [40, 0])
    x.refs[1:3] += 1
    was = x.k.clone(), x.v.clone()
    assert int(x.call([40, 0], [41, 17])) == 3
    assert x.table.tolist() == [[0, 1, 3, -1], [4, 5, -1, -1]] and x.refs.tolist() == [1, 2, 1, 1, 1, 1, 0, 0, 0]
    for c, old in zip((x.k, x.v), was):
        assert torch.equal(c[:, :3], old[:, :3]) and torch.equal(c[:, 3, :, :8], old[:, 2, :, :8])
    assert int(x.call([41, 17], [0, 0])) == 7
    assert x.refs.tolist() == [0, 1, 1, 0, 0, 0, 0, 0, 0]


@pytest.mark.gpu
def test_operands_that_do_not_match_are_refused(gpu):
    x = Pool(3, 4, 20, 16, 1, 16, 16, "f32", 2, 9)
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in ((x.table, x.refs[:-1], n, n, x.k, x.v), (x.table, x.refs, n[:2], n, x.k, x.v),
                (x.table, x.refs, n, n.long(), x.k, x.v), (x.table[:, ::2], x.refs, n, n, x.k, x.v),
                (x.table, x.refs, n, n, x.k, x.v.half()), (x.table, x.refs, n, n, x.k[0], x.v),
                (x.table, x.refs, n, n, x.k.cpu(), x.v), (x.table, x.refs, n, n, x.k, x.v, n[:1])):
        with pytest.raises(ValueError):
            binding.paged_reserve(*bad)
    d = x.table, x.refs, None, n, n, x.k, x.v
    spare = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(binding.FabError):
        binding.fab_paged_reserve(*d, None, spare)
    with pytest.raises(ValueError):
        binding.fab_paged_reserve(*d, torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2], spare)


@pytest.mark.gpu
def test_far_offsets(gpu):
    # pages whose first element lies past 2^31 elements of a layer
    Hkv, page, D = 4, 64, 128
    pages = (1 << 31) // (Hkv * page * D) + 12
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[pages - 3, pages - 9], [-1, -1]], dtype=torch.int32, device="cuda")
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")  # all held ...
    refs[-12:] = 0                                              # ... but the last
    refs[table[0].long()] = 1
    k[pages - 9].normal_()
    v[pages - 9].normal_()
    n = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    assert int(binding.paged_reserve(table, refs, n(100, 100), n(101, 101), k, v, n(0, 0))) == 12 - 3
    assert table.tolist() == [[pages - 3, pages - 9], [pages - 3, pages - 12]]
    for c in (k, v):
        assert torch.equal(c[pages - 12, :, :36], c[pages - 9, :, :36]) and (c[pages - 12, :, 36:] == 0).all()


# ------------------------------------------------------------------ together


class Model:
    """Layers whose projections of a token depend on the token alone, so that any
    path's attention can be had from a plain sequence."""

    def __init__(self, dtype, D=64, H=4, Hkv=2, layers=2, tokens=97, P=200):
        g = torch.Generator().manual_seed(11)
        self.dt, self.H, self.Hkv, self.D, self.layers = DT[dtype], H, Hkv, D, layers
        self.rows = torch.randn((layers, tokens, (H + 2 * Hkv) * D), generator=g).to(self.dt).cuda()
        self.w = (1 + 0.2 * torch.randn((2, layers, D), generator=g)).to(self.dt).cuda()
        self.cos, self.sin = (t.cuda() for t in tables(P, D))

    def project(self, layer, tokens):
        H, Hkv, D = self.H, self.Hkv, self.D
        q, k, v = self.rows[layer][tokens].split([H * D, Hkv * D, Hkv * D], -1)
        return q.unflatten(-1, (H, D)), k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D))

    def plain(self, layer, tokens):
        """Keys (Hkv,N,D), values and attention (N,H,D) of a whole sequence."""
        q, k, v = (t[None] for t in self.project(layer, torch.tensor(tokens).cuda()))
        Q, K, V = binding.qk_norm_rope(q, k, v, self.w[0, layer], self.w[1, layer], self.cos, self.sin)
        return K[0], V[0], binding.forward(Q, K, V, None, True)[0][0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_serving_with_drafts_and_forks(gpu, dtype):
    m, B, page, pages, W = Model(dtype), 4, 16, 48, 12
    r = random.Random(12)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    k = torch.zeros((m.layers, pages, m.Hkv, page, m.D), dtype=m.dt, device="cuda")
    v = torch.zeros_like(k)
    past = [[] for _ in range(B)]  # the tokens of each sequence

    def step(tokens, parents, source=None):
        """Drafts appended and attended to; each token's output compared with its path's own sequence."""
        nonlocal past
        if source is not None:
            past = [list(past[s]) if s >= 0 else [] for s in source]
        new, kept = [len(t) for t in tokens], [len(p) for p in past]
        lens = i32([a + n for a, n in zip(kept, new)])
        assert int(binding.paged_reserve(table, refs, i32(kept), lens, k, v,
                                         None if source is None else i32(source))) >= 0
        starts = starts_of(new).cuda()
        seen = binding.draft_tree(starts, i32([p for row in parents for p in row]), max(new))
        at = torch.tensor([t for row in tokens for t in row]).cuda()
        for layer in range(m.layers):
            a, b, c = m.project(layer, at)
            q = binding.paged_append(a, b, c, m.w[0, layer], m.w[1, layer], m.cos, m.sin, starts, lens, table,
                                     k[layer], v[layer], seen=seen)
            o, _ = binding.paged_attention(q, k[layer], v[layer], starts, lens, table, seen=seen)
            t0 = 0
            for s in range(B):
                paths = []
                for i in range(new[s]):
                    paths.append((paths[parents[s][i]] if parents[s][i] >= 0 else []) + [tokens[s][i]])
                    want = m.plain(layer, past[s] + paths[i])[2][-1]
                    # both round weights and result once: two half steps each way of the weighted sum of |v| (below 4)
                    assert (o[t0 + i].double() - want.double()).abs().max() <= 16 * half_step(m.dt) + 1e-5
                t0 += new[s]
        return starts, lens, seen

    def keep(starts, lens, seen, tokens, parents):
        last = [r.randint(-1, len(t) - 1) if t else -1 for t in tokens]
        now = binding.paged_accept(starts, lens, table, seen, i32(last), k, v)
        for s, i in enumerate(last):
            path = []
            while i >= 0:
                path.insert(0, tokens[s][i])
                i = parents[s][i]
            past[s] += path
        assert now.tolist() == [len(p) for p in past]
        for layer in range(m.layers):
            for s in range(B):
                n = torch.arange(len(past[s]))
                if len(n):
                    K, V, _ = m.plain(layer, past[s])
                    where = table.cpu()[s, n // page].long().cuda(), slice(None), (n % page).cuda()
                    assert torch.equal(k[layer][where], K.transpose(0, 1)) and torch.equal(v[layer][where],
                                                                                           V.transpose(0, 1))

    def draft(sizes):
        tokens = [[r.randrange(97) for _ in range(n)] for n in sizes]
        return tokens, [draw_parents(n, r, "mixed") for n in sizes]

    for sizes, source in (((30, 7, 0, 17), None), ((9, 12, 33, 1), [0, 0, 3, 1]), ((6, 1, 5, 8), None),
                          ((10, 4, 4, 3), [2, 2, 2, 0]), ((1, 1, 1, 1), [3, 0, 0, 0]), ((5, 0, 7, 7), [1, -1, 0, 0])):
        tokens, parents = draft(sizes)
        if source is None and not past[0]:
            parents = [draw_parents(n, r, "chain") for n in sizes]  # prompts
        state = step(tokens, parents, source)
        keep(*state, tokens, parents)
    binding.paged_reserve(table, refs, i32([0] * B), i32([0] * B), k, v)
    assert (refs == 0).all() and (table == -1).all()


@pytest.mark.gpu
def test_captured_step_follows_what_it_is_given(gpu):
    # a whole step captured once: tables, trees, lengths and sources change between replays
    m, B, page, pages, W, T = Model("bf16"), 3, 16, 40, 10, 60
    r = random.Random(13)
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, lens, kept, source, last, parents = z(B + 1), z(B), z(B), z(B), z(B), z(T)
    table, refs = z(B, W) - 1, z(pages)
    tokens = torch.zeros(T, dtype=torch.long, device="cuda")
    k = torch.zeros((m.layers, pages, m.Hkv, page, m.D), dtype=m.dt, device="cuda")
    v = torch.zeros_like(k)

    def step():
        spare = binding.paged_reserve(table, refs, kept, lens, k, v, source)
        seen = binding.draft_tree(starts, parents, 40)
        outs = []
        for layer in range(m.layers):
            a, b, c = m.project(layer, tokens)
            q = binding.paged_append(a, b, c, m.w[0, layer], m.w[1, layer], m.cos, m.sin, starts, lens, table,
                                     k[layer], v[layer], seen=seen)
            outs.append(binding.paged_attention(q, k[layer], v[layer], starts, lens, table, seen=seen)[0])
        return outs, binding.paged_accept(starts, lens, table, seen, last, k, v), spare

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, now, spare = step()
    held = [0] * B
    for i in range(6):
        new = [r.randint(0 if i else 1, 20) for _ in range(B)]
        src = [r.choice([b, b, r.randrange(B)]) for b in range(B)]
        par = [p for n in new for p in draw_parents(n, r, "mixed" if i else "chain")]
        live = sum(new)
        keep = [held[s] for s in src]
        starts.copy_(starts_of(new))
        kept.copy_(torch.tensor(keep))
        lens.copy_(torch.tensor([a + n for a, n in zip(keep, new)]))
        source.copy_(torch.tensor(src))
        last.copy_(torch.tensor([r.randint(-1, n - 1) for n in new]))
        parents[:live] = torch.tensor(par, dtype=torch.int32)
        tokens.random_(0, 97)
        before = [t.clone() for t in (table, refs, k, v)]
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in (table, refs, k, v)]
        got = [o[:live].clone() for o in outs], now.clone(), spare.clone()
        for t, b in zip((table, refs, k, v), before):
            t.copy_(b)
        want = step()
        assert all(torch.equal(a, b[:live]) for a, b in zip(got[0], want[0]))
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert all(torch.equal(a, b) for a, b in zip(after, (table, refs, k, v)))
        held = now.tolist()


@pytest.mark.gpu
def test_streams_side_by_side(gpu):
    # the same steps of two pools on two streams at once, and one after the other
    def run(streams):
        out = []
        pools = [Pool(40, 9, 400, 16, 2, 64, 64, "bf16", 3, s) for s in (1, 2)]
        torch.cuda.synchronize()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        plans = [(i32([0] * 40), i32([20 + b for b in range(40)]), None),
                 (i32([20 + b // 2 * 2 for b in range(40)]), i32([60] * 40), i32([b // 2 * 2 for b in range(40)])),
                 (i32([55] * 40), i32([70] * 40), None)]
        torch.cuda.synchronize()
        for kept, lens, source in plans:
            for x, s in zip(pools, streams):
                binding.paged_reserve(x.table, x.refs, kept, lens, x.k, x.v, source, stream=s)
        torch.cuda.synchronize()
        for x in pools:
            out += [x.table, x.refs, x.k, x.v]
        return out

    for a, b in zip(run([None, None]), run([torch.cuda.Stream(), torch.cuda.Stream()])):
        assert torch.equal(a, b)
