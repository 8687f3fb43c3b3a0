"""Trees of drafted tokens over a paged cache: who sees whom, appending,
attention, keeping the accepted path; each against plain loops, and together.

Tolerances of the attention are those of test_paged.py: roundings counted, the
hidden keys left out of the sums.  Masks, lengths and moved rows are exact.
"""
import ctypes
import math
import random

import pytest
import torch

from attention_backward_tcgen05_gb300 import binding
from test_norm_rope import DT, U32, close, half_step, ref_forward, tables
from test_paged import A, Batch, gpu, paged_dims  # noqa: F401 (gpu: a fixture)

# ------------------------------------------------------------------ refusals (CPU)


def cache_dims(**kw):
    d = dict(B=2, T=4, words=1, Hkv=2, DK=64, DV=64, page=16, pages=8, max_pages=3, layers=3, ldk=16384, ldv=16384)
    d.update(kw)
    return binding.fab_cache_dims(*[d[n] for n, _ in binding.fab_cache_dims._fields_])


def call_tree(starts=A, parents=A, B=2, T=4, words=1, seen=A):
    return binding.lib().fab_draft_tree(starts, parents, B, T, words, seen, None)


def call_append(dims, seen=A, words=1, q=A, kc=A):
    return binding.lib().fab_paged_append_tree(q, A, A, A, A, A, A, 1e-6, 0, A, A, A, seen, words, 1,
                                               ctypes.byref(dims), A, kc, A, None)


def call_attention(dims, seen=A, words=1, q=A, scale=1.0, ws=A, wsb=1 << 40):
    return binding.lib().fab_paged_attention_tree(q, A, A, A, A, A, seen, words, scale, 1, ctypes.byref(dims), ws, wsb,
                                                  A, A, None)


def call_accept(dims, starts=A, lens=A, table=A, seen=A, last=A, dtype=1, kc=A, vc=A, out=A):
    return binding.lib().fab_paged_accept(starts, lens, table, seen, last, dtype, ctypes.byref(dims), kc, vc, out, None)


@pytest.mark.parametrize("bad", [dict(starts=None), dict(starts=A + 2), dict(parents=None), dict(parents=A + 1),
                                 dict(B=0), dict(B=1 << 31), dict(T=-1), dict(T=1 << 31), dict(words=0),
                                 dict(words=-3), dict(words=1 << 40), dict(seen=None), dict(seen=A + 4)], ids=str)
def test_tree_refuses(bad):
    assert call_tree(**bad) == binding.FAB_ERR_INVALID


def test_tree_width_and_nothing_to_do():
    assert call_tree(words=binding.DRAFT_MAX_WORDS + 1) == binding.FAB_ERR_UNSUPPORTED
    assert call_tree(T=0, parents=None, seen=None) == binding.FAB_OK


@pytest.mark.parametrize("seen, words", [(A, 1), (A - 48, 1), (A + 8192 - 16, 1), (A + 8192 + 16, 1), (A + 8192 + 64, 1),
                                         (A + 8192, 2), (A + 8192 - 144, 2), (A + 8192 + 64, 2)])
def test_tree_refuses_rows_over_what_it_reads(seen, words):
    # 20 tokens of two sequences; rows of one word may take the place of the parents
    assert call_tree(starts=A, parents=A + 8192, B=2, T=20, words=words, seen=seen) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(seen=None), dict(seen=A + 8), dict(words=0), dict(words=-1),
                                 dict(words=1 << 40), dict(q=None)], ids=str)
def test_append_and_attention_refuse(bad):
    assert call_append(paged_dims(), **bad) == binding.FAB_ERR_INVALID
    assert call_attention(paged_dims(), **bad) == binding.FAB_ERR_INVALID


def test_other_refusals_are_those_of_the_plain_calls():
    assert call_append(paged_dims(H=3)) == binding.FAB_ERR_INVALID
    assert call_append(paged_dims(), kc=A + 8) == binding.FAB_ERR_INVALID
    assert call_attention(paged_dims(), scale=float("nan")) == binding.FAB_ERR_INVALID
    assert call_attention(paged_dims(max_pages=3000), ws=None, wsb=0) == binding.FAB_ERR_WORKSPACE
    assert call_attention(paged_dims(DK=264)) == binding.FAB_ERR_UNSUPPORTED
    assert call_attention(paged_dims(T=0), seen=None, q=None) == binding.FAB_OK
    assert call_append(paged_dims(T=0), seen=None, q=None) == binding.FAB_OK
    lib = binding.lib()
    assert lib.fab_paged_append_tree(A, A, A, A, A, A, A, 1e-6, 0, A, A, A, A, 1, 1, None, A, A, A, None) == 1
    assert lib.fab_paged_attention_tree(A, A, A, A, A, A, A, 1, 1.0, 1, None, A, 1 << 40, A, A, None) == 1


BAD_CACHE = [dict(B=0), dict(Hkv=0), dict(DK=0), dict(DV=-1), dict(page=0), dict(pages=0), dict(max_pages=0),
             dict(layers=0), dict(ldk=16383), dict(ldv=16383), dict(ldk=1 << 40), dict(pages=1 << 31),
             dict(B=1 << 30, max_pages=2), dict(layers=1 << 24), dict(pages=1 << 30, page=1 << 20)]


@pytest.mark.parametrize("bad", BAD_CACHE + [dict(T=-1), dict(T=1 << 31), dict(words=0)], ids=str)
def test_accept_refuses_dims(bad):
    assert call_accept(cache_dims(**bad)) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(starts=None), dict(lens=A + 2), dict(table=None), dict(seen=A + 4),
                                 dict(last=None), dict(dtype=3), dict(kc=A + 8), dict(vc=None), dict(out=None)],
                         ids=str)
def test_accept_refuses_arguments(bad):
    assert call_accept(cache_dims(), **bad) == binding.FAB_ERR_INVALID


def test_accept_refuses_widths():
    assert call_accept(cache_dims(DK=264, layers=1)) == binding.FAB_ERR_UNSUPPORTED


AT = dict(starts=A, lens=A + 4096, table=A + 8192, seen=A + 12288, last=A + 16384)
LAST = dict(starts=8, lens=4, table=20, seen=12, last=4)  # bytes to the last element (cache_dims' sizes)


@pytest.mark.parametrize("step", ["first", "last", "before"])
@pytest.mark.parametrize("name", AT)
def test_accept_refuses_lengths_over_what_it_reads(name, step):
    # lens_out has two elements
    out = AT[name] + {"first": 0, "last": LAST[name], "before": -4}[step]
    assert call_accept(cache_dims(), out=out, **AT) == binding.FAB_ERR_INVALID


def test_binding_refuses_what_does_not_fit():
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(5, 2, 16, 64)
    for call in (lambda: binding.draft_tree(i32(3), i32(4), 4),           # not CUDA tensors
                 lambda: binding.draft_tree(i32(3, 1), i32(4), 4),        # not 1-D
                 lambda: binding.draft_tree(i32(3), i32(4), 0),           # no words
                 lambda: binding.draft_tree(i32(3), i32(4), 32 * 512 + 1),
                 lambda: binding.paged_accept(i32(3), i32(2), i32(2, 3), i32(4, 1), i32(2), k, k),
                 lambda: binding.paged_attention(torch.zeros(3, 2, 64), k, k, i32(2), i32(1), i32(1, 2), causal=False,
                                                 seen=i32(3, 1))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ who sees whom


def draw_parents(n, r, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    if kind == "recent":  # siblings close by: long paths through every block
        return [max(-1, i - r.randint(1, 3)) for i in range(n)]
    return [r.randint(-1, i - 1) if r.random() < 0.5 else i - 1 for i in range(n)]


def sight(new, parents):
    """Truth values (T, most tokens): who sees whom."""
    dense = torch.zeros(sum(new), max(max(new), 1), dtype=torch.bool)
    t0 = 0
    for n in new:
        for i in range(n):
            if parents[t0 + i] >= 0:
                dense[t0 + i] = dense[t0 + parents[t0 + i]]
            dense[t0 + i, i] = True
        t0 += n
    return dense


def packed(dense, words):
    wide = torch.nn.functional.pad(dense, (0, 32 * words - dense.shape[1])).view(len(dense), words, 32)
    value = (wide.long() << torch.arange(32)).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def starts_of(new):
    return torch.tensor([0] + new).cumsum(0).to(torch.int32)


TREES = {"one": [1], "tiny": [8], "blocks": [31, 32, 33, 64, 65, 0, 1, 96], "long": [2000], "words_of_four": [97, 128],
         "words_of_eight": [250, 3], "many": [i % 40 for i in range(700)], "longest": [16384], "nine_words": [270, 288]}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mixed", "chain", "star", "recent"])
@pytest.mark.parametrize("name", TREES)
def test_tree(gpu, name, kind):
    new, r = TREES[name], random.Random(len(name))
    parents = [p for n in new for p in draw_parents(n, r, kind)]
    got = binding.draft_tree(starts_of(new).cuda(), torch.tensor(parents, dtype=torch.int32).cuda(), max(new))
    assert torch.equal(got.cpu(), packed(sight(new, parents), -(-max(new) // 32)))


@pytest.mark.gpu
def test_tree_leaves_padding_and_takes_wider_rows(gpu):
    new = [5, 40]
    parents = [p for n in new for p in draw_parents(n, random.Random(1), "mixed")]
    seen = torch.full((60, 7), 99, dtype=torch.int32, device="cuda")
    pad = torch.tensor(parents + [-77] * 15, dtype=torch.int32).cuda()
    binding.fab_draft_tree(starts_of(new).cuda(), pad, seen)
    assert (seen[45:] == 99).all() and torch.equal(seen[:45].cpu(), packed(sight(new, parents), 7))
    none = binding.draft_tree(torch.zeros(4, dtype=torch.int32).cuda(), pad[:0], 5)
    assert none.shape == (0, 1)


@pytest.mark.gpu
def test_rows_of_one_word_take_the_parents_place(gpu):
    new = [i % 33 for i in range(500)]
    parents = [p for n in new for p in draw_parents(n, random.Random(n), "mixed")]
    both = torch.tensor(parents, dtype=torch.int32).cuda()
    binding.fab_draft_tree(starts_of(new).cuda(), both, both.view(-1, 1))
    assert torch.equal(both.cpu().view(-1, 1), packed(sight(new, parents), 1))


@pytest.mark.gpu
def test_tree_reports_what_is_out_of_range(gpu):
    new, parents = [6, 40], [p for n in (6, 40) for p in draw_parents(n, random.Random(2), "mixed")]
    for at, p in ((3, 3), (3, 5), (8, -2), (20, 1 << 30), (0, 0)):
        bad = list(parents)
        bad[at] = p
        got = binding.draft_tree(starts_of(new).cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), 40)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        bad[at] = -1
        assert torch.equal(got.cpu(), packed(sight(new, bad), 2))
    wide = torch.tensor(parents, dtype=torch.int32).cuda()
    binding.draft_tree(starts_of(new).cuda(), wide, 20)  # rows too narrow for the second sequence
    assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
    for starts in ([0, 50, 46], [-3, 6, 46], [0, 6, 1000]):
        binding.draft_tree(torch.tensor(starts, dtype=torch.int32).cuda(), wide, 60)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID


# ------------------------------------------------------------------ attention


def check_tree(x, dense, o, lse, scale):
    """Every live token's row against softmax over what it sees, in 64 bits."""
    o, lse, u, t0 = o.double().cpu(), lse.double().cpu(), half_step(x.dt), 0
    for b, (n, h) in enumerate(zip(x.new, x.held)):
        G = x.H // x.Hkv
        for hq in range(x.H if n else 0):
            K, V, Q = x.rows(x.k, b, h, hq // G), x.rows(x.v, b, h, hq // G), x.q[t0: t0 + n, hq].double()
            hidden = torch.zeros(n, h, dtype=torch.bool)
            for i in range(n):
                for j in range(n):  # new token j is key h - n + j
                    if h - n + j >= 0 and (j > i or not dense[t0 + i, j]):
                        hidden[i, h - n + j] = True
            xs = (scale * Q @ K.t()).masked_fill(hidden, float("-inf"))
            size = (abs(scale) * Q.abs() @ K.abs().t()).masked_fill(hidden, 0.0)
            empty = hidden.all(-1)
            got, z = o[t0: t0 + n, hq], lse[hq, t0: t0 + n]
            assert (got[empty] == 0).all() and (z[empty] == float("inf")).all(), (b, hq)
            if empty.all():
                continue
            xs, size, got, z = xs[~empty], size[~empty], got[~empty], z[~empty]
            p, want = xs.softmax(-1), torch.logsumexp(xs, -1)
            d = (x.DK + 16) * U32 * size.amax(-1) + 8 * U32 * xs.masked_fill(xs.isinf(), 0).abs().amax(-1)
            add = (h + 16) * U32
            W = p @ V
            room = ((u if x.dt != torch.float32 else 0.0) + 2 * d + add)[:, None] * (p @ V.abs()) * 1.01
            room = room + u * (W.abs() + room) + torch.finfo(x.dt).smallest_normal * torch.finfo(x.dt).eps
            worst = ((got - W).abs() / room).max().item()
            assert math.isfinite(worst) and worst <= 1, (b, hq, worst)
            off = ((z - want).abs() / (d + add + 8 * U32 * (1 + want.abs()))).max().item()
            assert math.isfinite(off) and off <= 1, (b, hq, "lse", off)
        t0 += n


def drafted(x, seed, kind="mixed"):
    r = random.Random(seed)
    dense = sight(x.new, [p for n in x.new for p in draw_parents(n, r, kind)])
    words = -(-max(max(x.new), 1) // 32)
    seen = packed(torch.nn.functional.pad(dense, (0, 0, 0, x.T - len(dense))), words)
    return dense, seen.cuda()


# name: new, held, H, Hkv, DK, DV, page, dtype
TREE_ATTENTION = {
    "bf16_drafts": ([8, 33, 64, 1], [208, 400, 700, 129], 8, 2, 128, 128, 16, "bf16"),
    "f16_drafts_d64": ([16, 20, 3], [300, 20, 67], 4, 4, 64, 64, 64, "f16"),
    "bf16_past_ends_in_a_word": ([40, 40, 40], [40 + 127, 40 + 128, 40 + 129], 8, 2, 128, 128, 32, "bf16"),
    "bf16_tree_over_tiles": ([300], [410], 2, 2, 128, 128, 256, "bf16"),
    "f16_tree_over_tiles_d64": ([257, 140], [600, 200], 4, 1, 64, 64, 16, "f16"),
    "bf16_no_past": ([5, 70], [5, 70], 4, 2, 128, 128, 16, "bf16"),
    "bf16_fewer_keys_than_tokens": ([40, 3, 2], [25, 1, 0], 4, 2, 128, 128, 16, "bf16"),
    "f32_fewer_keys_than_tokens": ([40, 3, 2], [25, 1, 0], 4, 2, 64, 64, 16, "f32"),
    "bf16_mixed_with_none": ([10, 0, 1, 200], [60, 30, 700, 300], 6, 2, 128, 128, 48, "bf16"),
    "f16_group_of_three": ([50, 90], [350, 90], 9, 3, 64, 64, 32, "f16"),
    "bf16_group_past_a_tile": ([9], [150], 160, 1, 64, 64, 16, "bf16"),
    "bf16_d80": ([40, 1], [240, 137], 4, 2, 80, 80, 16, "bf16"),
    "bf16_page_of_5": ([10, 37], [57, 131], 4, 2, 128, 128, 5, "bf16"),
    "bf16_d256": ([36, 1], [140, 137], 4, 2, 256, 256, 32, "bf16"),
    "f32_drafts": ([40, 1, 100], [240, 33, 163], 6, 2, 80, 80, 24, "f32"),
    "f32_one": ([1], [1], 2, 1, 64, 64, 16, "f32"),
    "f32_wide": ([33], [70], 2, 1, 256, 200, 16, "f32"),
    "f32_odd_widths": ([5, 37], [70, 37], 2, 1, 3, 5, 7, "f32"),
    "f16_odd_widths": ([36, 1], [70, 77], 4, 2, 37, 21, 16, "f16"),
    "bf16_long_split": ([24], [5000], 4, 1, 128, 128, 64, "bf16"),
    "f32_long_split": ([6], [3000], 4, 1, 64, 64, 64, "f32"),
    "bf16_many_sequences": ([(3 * i) % 7 for i in range(300)], [(7 * i) % 150 + 7 for i in range(300)], 4, 2, 64, 64,
                            16, "bf16"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 5000], ids=["as_is", "wide_table"])  # whole units, work cut over the SMs
@pytest.mark.parametrize("name", TREE_ATTENTION)
def test_tree_attention(gpu, name, room):
    new, held, *rest = TREE_ATTENTION[name]
    x = Batch(new, held, *rest, seed=sum(map(ord, name)))
    x.table = torch.nn.functional.pad(x.table, (0, room // x.page), value=-7)
    dense, seen = drafted(x, 3)
    scale = rest[2] ** -0.5
    o, lse = binding.paged_attention(*x.cuda(), scale=scale, seen=seen)
    check_tree(x, dense, o, lse, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_a_chain_is_the_causal_call(gpu, dtype):
    x = Batch([70, 1, 130, 0, 33], [70, 400, 300, 90, 1000], 8, 2, 64, 64, 32, dtype, seed=4)
    _, seen = drafted(x, 0, "chain")
    for got, want in zip(binding.paged_attention(*x.cuda(), scale=0.1, seen=seen),
                         binding.paged_attention(*x.cuda(), True, 0.1)):
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_masks_that_no_tree_gives(gpu, scale):
    # bits are taken as they are: rows that see nothing, not even themselves, and
    # bits of later tokens, which do not count
    for dtype, D in (("bf16", 128), ("f16", 64), ("f32", 48)):
        x = Batch([30, 45, 3], [30, 300, 3], 4, 2, D, D, 16, dtype, seed=5)
        g = torch.Generator().manual_seed(6)
        dense = torch.rand((x.T, 45), generator=g) < 0.3
        dense[2:7] = False
        dense[-3:] = False
        o, lse = binding.paged_attention(*x.cuda(), scale=scale, seen=packed(dense, 2).cuda())
        check_tree(x, dense, o, lse, scale)
        assert (o[2:7] == 0).all() and (o[-3:] == 0).all() and (lse[:, -3:] == float("inf")).all()


@pytest.mark.gpu
def test_keys_that_are_not_seen_may_be_anything_but_values_finite(gpu):
    # a key of another branch that is NaN or infinite scores nothing
    for dtype in ("bf16", "f32"):
        for junk in (float("nan"), float("inf"), -float("inf")):
            x = Batch([6], [140], 2, 1, 64, 64, 16, dtype, seed=9)
            dense = sight([6], [-1, 0, 0, 1, 2, 3])  # two branches: 1 3 5 and 2 4
            seen = packed(dense, 1).cuda()
            want, wl = binding.paged_attention(*x.cuda(), scale=0.125, seen=seen)
            for j in (2, 4):
                x.k[int(x.table[0, (134 + j) // 16]), :, (134 + j) % 16] = junk
            o, lse = binding.paged_attention(*x.cuda(), scale=0.125, seen=seen)
            keep = [0, 1, 3, 5]
            assert torch.equal(o[keep], want[keep]) and torch.equal(lse[:, keep], wl[:, keep])


@pytest.mark.gpu
def test_padding_tokens_are_left_alone(gpu):
    for dtype in ("bf16", "f32"):
        x = Batch([5, 1], [60, 133], 4, 2, 64, 64, 16, dtype, seed=10, spare=40)
        dense, seen = drafted(x, 1)
        seen[6:] = -1
        q, k, v, starts, lens, table = x.cuda()
        o = torch.full((x.T, 4, 64), 3.0, dtype=x.dt, device="cuda")
        lse = torch.full((4, x.T), 3.0, device="cuda")
        binding.fab_paged_attention_tree(q, k, v, starts, lens, table, seen, 0.125,
                                         binding.alloc_paged(q, k, v, table), o, lse)
        assert (o[6:] == 3).all() and (lse[:, 6:] == 3).all()
        check_tree(x, dense, o, lse, 0.125)
        row = torch.randn(x.T, 4, 64, device="cuda").to(x.dt)
        qo = torch.full((x.T, 4, 64), 3.0, dtype=x.dt, device="cuda")
        binding.fab_paged_append_tree(row, row[:, :2].contiguous(), row[:, 2:].contiguous(), None, None, None, None,
                                      1e-6, False, starts, lens, table, seen, qo, k, v)
        assert (qo[6:] == 3).all() and torch.equal(qo[:6], row[:6])


@pytest.mark.gpu
def test_rows_too_narrow_are_reported(gpu):
    for dtype in ("bf16", "f32"):
        x = Batch([40, 2], [60, 133], 4, 2, 64, 64, 16, dtype, seed=11)
        dense, seen = drafted(x, 1)
        q, k, v, starts, lens, table = x.cuda()
        narrow = seen[:, :1].contiguous()
        o, lse = binding.paged_attention(q, k, v, starts, lens, table, scale=0.125, seen=narrow)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        want, wl = binding.paged_attention(q, k, v, starts, lens, table, scale=0.125, seen=seen)
        assert torch.equal(o[40:], want[40:]) and torch.equal(lse[:, 40:], wl[:, 40:])
        binding.paged_append(q, q[:, :2].contiguous(), q[:, 2:].contiguous(), None, None, None, None, starts, lens,
                             table, k, v, seen=narrow)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID


@pytest.mark.gpu
def test_operands_that_do_not_match_are_refused(gpu):
    x = Batch([2], [20], 4, 2, 64, 64, 16, "bf16", seed=10)
    d = x.cuda()
    good = torch.ones(2, 1, dtype=torch.int32, device="cuda")
    for bad in (good.long(), good[:1], good.view(-1), good.cpu(), torch.ones(2, 4, dtype=torch.int32).cuda()[:, ::2],
                torch.ones(2, 0, dtype=torch.int32).cuda()):
        with pytest.raises(ValueError):
            binding.paged_attention(*d, seen=bad)
        with pytest.raises(ValueError):
            binding.paged_append(d[0], d[0][:, :2], d[0][:, 2:], None, None, None, None, d[3], d[4], d[5], d[1], d[2],
                                 seen=bad)
    off = torch.ones(9, dtype=torch.int32, device="cuda")[1:3].view(2, 1)  # not at 16 bytes
    with pytest.raises(binding.FabError):
        binding.paged_attention(*d, seen=off)
    with pytest.raises(ValueError):
        binding.paged_attention(*d, causal=False, seen=good)


@pytest.mark.gpu
def test_drawn_trees(gpu):
    r = random.Random(78)
    for i in range(30):
        dtype = r.choice(["bf16", "f16", "f32"])
        Hkv, G = r.choice([1, 2, 3]), r.choice([1, 2, 3, 4, 6, 8])
        DK = r.choice([64, 128, 128, 64, 80, 24])
        DV = DK if r.random() < 0.7 else r.choice([64, 128, 32])
        page, B = r.choice([8, 16, 24, 32, 64, 128, 20]), r.randint(1, 5)
        new = [r.choice([0, 1, 7, r.randint(1, 64), r.randint(1, 150)]) for _ in range(B)]
        if sum(new) == 0:
            new[0] = 1
        held = [n + r.choice([0, 1, r.randint(0, 100), r.randint(0, 700)]) for n in new]
        x = Batch(new, held, Hkv * G, Hkv, DK, DV, page, dtype, seed=i, std=r.choice([0.3, 1.0, 2.0]))
        if i % 2:
            x.table = torch.nn.functional.pad(x.table, (0, 5000 // page), value=-7)
        dense, seen = drafted(x, i, r.choice(["mixed", "star", "recent"]))
        o, lse = binding.paged_attention(*x.cuda(), seen=seen)
        check_tree(x, dense, o, lse, DK ** -0.5)


# ------------------------------------------------------------------ appending

# name: new, held, H, Hkv, DK, DV, page, dtype, rot, interleaved, norm
APPEND = {
    "bf16_drafts": ([8, 33, 64, 1], [25, 33, 128, 70], 8, 2, 128, 128, 16, "bf16", 128, False, True),
    "f16_no_norm": ([30, 0, 1, 57], [30, 5, 9, 200], 4, 4, 64, 64, 64, "f16", 64, False, False),
    "bf16_pairs_part": ([30, 3], [33, 77], 4, 2, 80, 64, 24, "bf16", 32, True, True),
    "f32_no_rot": ([3, 11], [13, 11], 4, 2, 64, 64, 16, "f32", 0, False, True),
    "f32_odd": ([3, 41], [13, 41], 4, 2, 7, 5, 3, "f32", 6, False, True),
    "bf16_many_sequences": ([(7 * i) % 3 if i % 50 else 0 for i in range(1500)],
                            [(7 * i) % 3 + i % 9 + 1 for i in range(1500)], 2, 1, 16, 16, 8, "bf16", 16, False, True),
    "f32_many_sequences_odd": ([(5 * i) % 4 for i in range(1100)], [(5 * i) % 4 + i % 9 for i in range(1100)], 2, 1, 7, 5,
                               8, "f32", 4, False, True),
    "f16_forty_sequences": ([(7 * i) % 5 for i in range(40)], [(7 * i) % 5 + i for i in range(40)], 4, 2, 64, 64, 16,
                            "f16", 64, False, True),
    "bf16_wide_tree": ([300, 1, 100], [900, 4, 600], 8, 2, 128, 128, 32, "bf16", 128, False, True),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", APPEND)
def test_append(gpu, name):
    new, held, H, Hkv, DK, DV, page, dtype, rot, il, norm = APPEND[name]
    x = Batch(new, held, H, Hkv, DK, DV, page, dtype, seed=3)
    dense, seen = drafted(x, 5)
    row = torch.randn((x.T, H * DK + Hkv * (DK + DV)), generator=x.g).to(x.dt)
    split = lambda t: [a.unflatten(-1, (h, d)) for a, h, d in  # noqa: E731
                       zip(t.split([H * DK, Hkv * DK, Hkv * DV], -1), (H, Hkv, Hkv), (DK, DK, DV))]
    weight = lambda: (1 + 0.3 * torch.randn((DK,), generator=x.g)).to(x.dt) if norm else None  # noqa: E731
    wq, wk = weight(), weight()
    cos, sin = tables(max(held), rot)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    kc, vc = x.k.cuda(), x.v.cuda()
    got = binding.paged_append(*split(row.cuda()), dev(wq), dev(wk), dev(cos) if rot else None,
                               dev(sin) if rot else None, x.starts.cuda(), x.lens.cuda(), x.table.cuda(), kc, vc, 1e-6,
                               il, seen=seen)
    q, k, v = split(row)
    at = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)])
    number = torch.cat([torch.arange(n) for n in new])
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
    pos = at - number + dense.sum(1) - 1  # one place behind its last ancestor
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    if not rot:
        c = s = torch.zeros((x.T, 1, 0), dtype=torch.float64)
    want, bound = ref_forward(q, wq, c, s, il, 1e-6)
    close(got, want, bound, x.dt, "q")
    where = x.table[seq, at // page].long()
    want, bound = ref_forward(k, wk, c, s, il, 1e-6)
    close(kc.cpu()[where, :, at % page], want, bound, x.dt, "k")
    assert torch.equal(vc.cpu()[where, :, at % page], v)
    touched = torch.zeros(x.pages, page, dtype=torch.bool)
    touched[where, at % page] = True
    for cache, was in ((kc, x.k), (vc, x.v)):
        same = cache.cpu().transpose(1, 2)[~touched]
        assert torch.equal(same.nan_to_num(9), was.transpose(1, 2)[~touched].nan_to_num(9))


@pytest.mark.gpu
def test_sight_past_32_bits(gpu):
    # 2^31 words and more of `seen`: chains of 512 tokens, which are the plain calls
    B, n, page, D = 8200, 512, 64, 8
    assert B * n * n > 1 << 31
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    parents = torch.arange(B * n, dtype=torch.int32, device="cuda") % n - 1
    seen = binding.draft_tree(starts, parents, n * 32)
    assert seen.shape == (B * n, n)
    bits = (1 << (torch.arange(n, device="cuda") % 32 + 1)) - 1  # of the word that a token's own bit is in
    own = torch.arange(n, device="cuda") // 32
    last = seen[-n:].long() & 0xffffffff
    assert torch.equal(last[torch.arange(n), own], bits) and (last.sum(1) == bits + own * 0xffffffff).all()
    cos, sin = (t.cuda() for t in tables(n, D))
    for dtype in ("bf16", "f32"):
        q, k, v = (torch.randn(B * n, 1, D, device="cuda").to(DT[dtype]) for _ in range(3))
        out = []
        for sight_of in (None, seen):
            kc = torch.zeros(B * n // page, 1, page, D, dtype=DT[dtype], device="cuda")
            vc = torch.zeros_like(kc)
            x = binding.paged_append(q, k, v, None, None, cos, sin, starts, lens, table, kc, vc, seen=sight_of)
            out.append((x, kc, vc, *binding.paged_attention(x, kc, vc, starts, lens, table, seen=sight_of)))
        for a, b in zip(*out):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ the accepted path


def accepted(x, k, v, dense, last):
    """(lengths, keys, values) with the paths moved row by row; k, v (layers, ...)."""
    k, v, lens, t0 = k.clone(), v.clone(), list(x.held), 0
    for b, (n, h) in enumerate(zip(x.new, x.held)):
        if n:
            path = [j for j in range(last[b] + 1) if dense[t0 + last[b], j]] if last[b] >= 0 else []
            for i, j in enumerate(path):
                a, z = h - n + j, h - n + i
                for c in (k, v):
                    c[:, int(x.table[b, z // x.page]), :, z % x.page] = c[:, int(x.table[b, a // x.page]), :, a % x.page]
            lens[b] = h - n + len(path)
        t0 += n
    return torch.tensor(lens, dtype=torch.int32), k, v


def layered(x, layers, gap):
    """Caches of `layers` layers, `gap` elements between them."""
    out = []
    for c in (x.k, x.v):
        flat = torch.randn((layers, c.numel() + gap), generator=x.g).to(x.dt)
        out.append(flat.cuda()[:, : c.numel()].unflatten(1, c.shape))
    return out


# name: new, held, Hkv, DK, DV, page, dtype, layers, gap, kind
ACCEPT = {
    "bf16": ([8, 33, 64, 1, 0, 20], [40, 33, 164, 70, 9, 50], 2, 128, 128, 16, "bf16", 4, 0, "mixed"),
    "f16_gaps": ([30, 7], [31, 77], 3, 64, 64, 64, "f16", 3, 8, "mixed"),
    "bf16_odd_gaps": ([30, 7], [31, 77], 3, 64, 64, 64, "bf16", 3, 5, "recent"),
    "f32_two_widths": ([40, 7], [131, 77], 2, 80, 40, 24, "f32", 1, 0, "recent"),
    "f32_odd_widths": ([40, 7], [131, 77], 2, 7, 5, 3, "f32", 2, 0, "recent"),
    "bf16_odd_widths": ([40, 7], [131, 77], 2, 33, 21, 5, "bf16", 2, 1, "mixed"),
    "bf16_long_paths": ([700, 300], [900, 301], 2, 64, 64, 32, "bf16", 2, 0, "recent"),
    "f32_wide_long": ([200], [331], 1, 256, 256, 16, "f32", 2, 0, "recent"),
    "f16_chain": ([100, 5], [100, 9], 2, 64, 64, 16, "f16", 2, 0, "chain"),
    "bf16_star": ([40, 5], [60, 9], 2, 64, 64, 16, "bf16", 9, 0, "star"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["end", "any", "none"])
@pytest.mark.parametrize("name", ACCEPT)
def test_accept(gpu, name, which):
    new, held, Hkv, DK, DV, page, dtype, layers, gap, kind = ACCEPT[name]
    x = Batch(new, held, Hkv, Hkv, DK, DV, page, dtype, seed=7)
    dense, seen = drafted(x, 8, kind)
    r = random.Random(9)
    last = [-1 if which == "none" else n - 1 if which == "end" else r.randint(-1, n - 1) for n in new]
    k, v = layered(x, layers, gap)
    want, wk, wv = accepted(x, k.cpu(), v.cpu(), dense, last)
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), x.table.cuda(), seen,
                               torch.tensor(last, dtype=torch.int32).cuda(), k, v)
    assert torch.equal(got.cpu(), want) and torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)


@pytest.mark.gpu
def test_accept_takes_bits_as_they_are(gpu):
    # rows of `seen` that no tree gives: what is kept is what the last token sees, up to itself
    x = Batch([40, 70, 5], [45, 133, 5], 2, 2, 64, 64, 16, "bf16", seed=7)
    dense = torch.rand((x.T, 70), generator=x.g) < 0.5
    dense[39], dense[114] = True, False
    last = [39, 69, 4]
    k, v = layered(x, 2, 0)
    want, wk, wv = accepted(x, k.cpu(), v.cpu(), dense, last)
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), x.table.cuda(), packed(dense, 3).cuda(),
                               torch.tensor(last, dtype=torch.int32).cuda(), k, v)
    assert want.tolist()[::2] == [45, 0]
    assert torch.equal(got.cpu(), want) and torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)


@pytest.mark.gpu
def test_accept_without_new_tokens(gpu):
    x = Batch([0, 0], [20, 0], 2, 2, 64, 64, 16, "bf16", seed=7)
    k, v = layered(x, 2, 0)
    was = k.clone(), v.clone()
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), x.table.cuda(),
                               torch.empty((0, 1), dtype=torch.int32).cuda(),
                               torch.tensor([5, -9], dtype=torch.int32).cuda(), k, v)  # (last is not read)
    assert got.tolist() == [20, 0] and torch.equal(k, was[0]) and torch.equal(v, was[1])


@pytest.mark.gpu
def test_accept_of_many_sequences(gpu):
    # more than the threads of a block, most of them with nothing to move
    new = [(7 * i) % 5 if i % 3 else 0 for i in range(700)]
    held = [n + (3 * i) % 20 for i, n in enumerate(new)]
    x = Batch(new, held, 1, 1, 8, 16, 8, "f16", seed=7)
    dense, seen = drafted(x, 8, "recent")
    r = random.Random(9)
    last = [r.randint(-1, n - 1) for n in new]
    k, v = layered(x, 1, 0)
    want, wk, wv = accepted(x, k.cpu(), v.cpu(), dense, last)
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), x.table.cuda(), seen,
                               torch.tensor(last, dtype=torch.int32).cuda(), k[0], v[0])
    assert torch.equal(got.cpu(), want) and torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)


@pytest.mark.gpu
def test_accept_of_one_layer_and_far_offsets(gpu):
    # 4-D caches whose pages lie past 2^31 elements
    Hkv, D, page = 4, 128, 64
    pages = (1 << 31) // (Hkv * page * D) + 20
    x = Batch([30, 64], [50, 150], Hkv, Hkv, D, D, page, "bf16", seed=13, extra=0)
    assert x.pages <= 20
    dense, seen = drafted(x, 14)
    k = torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-x.pages:], v[-x.pages:] = x.k.nan_to_num(1).cuda(), x.v.nan_to_num(2).cuda()
    far = torch.where(x.table >= 0, x.table + pages - x.pages, x.table)
    want, wk, wv = accepted(x, x.k.nan_to_num(1)[None], x.v.nan_to_num(2)[None], dense, [29, 60])
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), far.cuda(), seen,
                               torch.tensor([29, 60], dtype=torch.int32).cuda(), k, v)
    assert torch.equal(got.cpu(), want)
    assert torch.equal(k[-x.pages:].cpu(), wk[0]) and torch.equal(v[-x.pages:].cpu(), wv[0])


@pytest.mark.gpu
def test_layers_far_apart(gpu):
    # layers 2^31 elements from each other, keys and values between one another's
    x = Batch([30, 64], [50, 150], 2, 2, 64, 64, 16, "bf16", seed=13)
    dense, seen = drafted(x, 14)
    n, far = x.k.numel(), 1 << 31
    flat = torch.empty(far + 2 * n, dtype=torch.bfloat16, device="cuda")
    k, v = (flat[at:].as_strided((2, *x.k.shape), (far, *x.k.stride())) for at in (0, n))
    k.normal_()
    v.normal_()
    want, wk, wv = accepted(x, k.cpu(), v.cpu(), dense, [29, 60])
    got = binding.paged_accept(x.starts.cuda(), x.lens.cuda(), x.table.cuda(), seen,
                               torch.tensor([29, 60], dtype=torch.int32).cuda(), k, v)
    assert torch.equal(got.cpu(), want) and torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)
    table = torch.tensor([[0, 1], [-1, -1]], dtype=torch.int32, device="cuda")
    refs = torch.zeros(x.pages, dtype=torch.int32, device="cuda")
    refs[:2] = 1
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    binding.paged_reserve(table, refs, i32(20, 20), i32(21, 21), k, v, i32(0, 0))
    assert table.tolist() == [[0, 1], [0, 2]]
    for c in (k, v):
        assert torch.equal(c[:, 2, :, :4], c[:, 1, :, :4])


@pytest.mark.gpu
def test_accept_reports_what_is_out_of_range(gpu):
    x = Batch([8, 33], [40, 60], 2, 2, 64, 64, 16, "bf16", seed=7)
    dense, seen = drafted(x, 8, "recent")
    last = torch.tensor([7, 32], dtype=torch.int32).cuda()
    starts, lens, table = x.starts.cuda(), x.lens.cuda(), x.table.cuda()

    def alter(t, at, value):
        t = t.clone()
        t.view(-1)[at] = value
        return t

    for bad in ((starts, lens, table, seen, alter(last, 1, 33)), (starts, lens, table, seen, alter(last, 1, -2)),
                (starts, lens, table, seen[:, :1].contiguous(), last), (starts, alter(lens, 1, 32), table, seen, last),
                (starts, alter(lens, 1, 16 * table.shape[1] + 1), table, seen, last),
                (starts, lens, alter(table, table.shape[1] + 3, -1), seen, last),
                (starts, lens, alter(table, table.shape[1] + 3, 1 << 30), seen, last),
                (alter(starts, 2, 1000), lens, table, seen, last), (alter(starts, 2, 3), lens, table, seen, last)):
        k, v = layered(x, 2, 0)
        want, wk, wv = accepted(x, k.cpu(), v.cpu(), dense, [7, 32])
        got = binding.paged_accept(*bad, k, v)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        assert int(got[0]) == int(want[0])
        own = x.table[0, :3].long()  # the other sequence's pages
        assert torch.equal(k.cpu()[:, own], wk[:, own]) and torch.equal(v.cpu()[:, own], wv[:, own])


@pytest.mark.gpu
def test_accept_refuses_what_does_not_match(gpu):
    x = Batch([8, 33], [40, 60], 2, 2, 64, 64, 16, "bf16", seed=7)
    _, seen = drafted(x, 8)
    last = torch.tensor([7, 32], dtype=torch.int32).cuda()
    starts, lens, table = x.starts.cuda(), x.lens.cuda(), x.table.cuda()
    k, v = layered(x, 2, 0)
    for bad in ((starts, lens, table, seen, last, k, v[:1]), (starts, lens, table, seen, last, k, v[0]),
                (starts, lens, table, seen, last[:1], k, v), (starts, lens, table, seen, last.long(), k, v),
                (starts, lens, table, seen, last, k.half(), v), (starts[:2], lens, table, seen, last, k, v),
                (starts, lens, table, seen, last, k[:1].expand(2, -1, -1, -1, -1), v),
                (starts, lens, table, seen, last, k.transpose(1, 2), v), (starts, lens, table, seen, last, k, v.cpu())):
        with pytest.raises(ValueError):
            binding.paged_accept(*bad)
    with pytest.raises(ValueError):
        binding.fab_paged_accept(starts, lens, table, seen, last, k, v, lens)


@pytest.mark.gpu
def test_lengths_over_what_accept_reads_are_refused(gpu):
    x = Batch([8, 33], [40, 60], 2, 2, 64, 64, 16, "bf16", seed=7)
    _, seen = drafted(x, 8)
    last = torch.tensor([7, 32], dtype=torch.int32).cuda()
    starts, lens, table = x.starts.cuda(), x.lens.cuda(), x.table.cuda()
    k, v = layered(x, 2, 0)
    for out in (starts[:2], starts[1:], lens, last, table.view(-1)[:2], table.view(-1)[-2:], seen.view(-1)[:2],
                seen.view(-1)[-2:]):
        with pytest.raises(ValueError):
            binding.fab_paged_accept(starts, lens, table, seen, last, k, v, out)


@pytest.mark.gpu
def test_a_step_without_drafts(gpu):
    x = Batch([0, 0], [20, 0], 2, 2, 64, 64, 16, "bf16", seed=7)
    starts, lens, table = x.starts.cuda(), x.lens.cuda(), x.table.cuda()
    parents = torch.empty(0, dtype=torch.int32, device="cuda")
    seen = binding.draft_tree(starts, parents, 0)
    assert seen.shape == (0, 1) and seen.dtype == torch.int32
    k, v = layered(x, 2, 0)
    none = torch.empty((0, 2, 64), dtype=x.dt, device="cuda")
    q = binding.paged_append(none, none, none, None, None, None, None, starts, lens, table, k[0], v[0], seen=seen)
    o, lse = binding.paged_attention(q, k[0], v[0], starts, lens, table, seen=seen)
    assert q.shape == o.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert binding.paged_accept(starts, lens, table, seen, lens, k, v).tolist() == [20, 0]
    for most in (-1, -32, -33):
        with pytest.raises(ValueError):
            binding.draft_tree(starts, parents, most)


# ------------------------------------------------------------------ streams, graphs, repeats


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_a_step_on_another_stream(gpu, dtype, handle):
    # every call is told the stream, on which what it reads is written milliseconds later
    x = Batch([30, 45, 3], [130, 300, 3], 4, 2, 64, 64, 16, dtype, seed=5)
    parents = [p for n in x.new for p in draw_parents(n, random.Random(4), "recent")]
    last = torch.tensor([29, 44, -1], dtype=torch.int32).cuda()
    q, k, v = torch.randn(x.T, 8, 64, generator=x.g).to(x.dt).cuda().split([4, 2, 2], 1)
    cos, sin = (t.cuda() for t in tables(310, 64))
    given = torch.tensor(parents, dtype=torch.int32).cuda(), x.starts.cuda(), x.lens.cuda(), x.table.cuda()
    kept = torch.tensor([100, 255, 0], dtype=torch.int32).cuda()

    def step(stream, kc, vc, refs, parents, starts, lens, table):
        spare = binding.paged_reserve(table, refs, kept, lens, kc, vc, stream=stream)
        seen = binding.draft_tree(starts, parents, 45, stream=stream)
        qo = binding.paged_append(q, k, v, None, None, cos, sin, starts, lens, table, kc, vc, stream=stream, seen=seen)
        o, lse = binding.paged_attention(qo, kc, vc, starts, lens, table, stream=stream, seen=seen)
        now = binding.paged_accept(starts, lens, table, seen, last, kc, vc, stream=stream)
        return spare, seen, qo, o, lse, now, kc, vc, table, refs

    def state():
        refs = torch.bincount(x.table[x.table >= 0].long(), minlength=x.pages).int().cuda()
        return x.k.nan_to_num(1).cuda(), x.v.nan_to_num(1).cuda(), refs

    want = step(None, *state(), *(t.clone() for t in given))
    side, late, own = torch.cuda.Stream(), [torch.zeros_like(t) for t in given], state()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = torch.randn(6000, 6000, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-3
        for t, g in zip(late, given):
            t.copy_(g)
    got = step(side.cuda_stream if handle else side, *own, *late)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_calls_captured_behind_forks_joins_and_copies(gpu):
    # each call behind something that is no kernel of the library: a copy, another stream's work, a join
    x = Batch([30, 45, 3], [130, 300, 3], 4, 2, 64, 64, 16, "bf16", seed=5)
    parents = [p for n in x.new for p in draw_parents(n, random.Random(4), "recent")]
    given = (torch.tensor(parents, dtype=torch.int32).cuda(), x.starts.cuda(), x.k.nan_to_num(1).cuda(),
             x.v.nan_to_num(1).cuda(), torch.randn(1, 300, 8, 64, generator=x.g).to(x.dt).cuda(), x.table.cuda(),
             torch.bincount(x.table[x.table >= 0].long(), minlength=x.pages).int().cuda())
    lens, last, kept = x.lens.cuda(), torch.tensor([29, 44, -1]).int().cuda(), torch.tensor([100, 250, 0]).int().cuda()
    cos, sin = (t.cuda() for t in tables(310, 64))
    used = [torch.zeros_like(t) for t in given]
    side = torch.cuda.Stream()

    def step():
        main, (par, starts, k, v, rows, table, refs) = torch.cuda.current_stream(), used
        side.wait_stream(main)
        with torch.cuda.stream(side):
            par.copy_(given[0])
            starts.copy_(given[1])
            seen = binding.draft_tree(starts, par, 45)
        for t, g in zip(used[2:], given[2:]):
            t.copy_(g)
        outs = binding.qk_norm_rope(rows[:, :, :4], rows[:, :, 4:6], rows[:, :, 6:], None, None, cos, sin)
        main.wait_stream(side)
        now = binding.paged_accept(starts, lens, table, seen, last, k, v)
        moved = k.clone(), v.clone()
        spare = binding.paged_reserve(table, refs, kept, lens, k, v)
        return [seen, now, spare, table.clone(), refs.clone(), *moved, *outs]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(5):
        for t in (*got, *used):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_the_same_call_gives_the_same_bits(gpu, dtype):
    x = Batch([64, 8, 33, 1, 200], [4000, 900, 33, 700, 1500], 8, 2, 128, 128, 16, dtype, seed=5)
    _, seen = drafted(x, 6)
    q, k, v, starts, lens, table = x.cuda()
    ws = binding.alloc_paged(q, k, v, table)
    want = binding.paged_attention(q, k, v, starts, lens, table, seen=seen)
    for i in range(25):
        ws.fill_(i * 10 + 1)  # (what it holds before does not matter)
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        binding.fab_paged_attention_tree(q, k, v, starts, lens, table, seen, 128 ** -0.5, ws, o, lse)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
