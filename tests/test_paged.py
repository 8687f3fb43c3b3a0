"""Appending to a paged key/value cache and attention over it, against plain
loops in 64 bits.

Tolerances count roundings (u = half a step of the type, 2^-24 for f32).  A
score is off by at most d = (DK + 16) 2^-24 of the sum of |products| that it
adds up; that moves a weight by the factor e^d.  Weights are rounded to the
type for their product (16-bit types), sums of L weights add L + 16 roundings
of f32, and the result is rounded once.
"""
import ctypes
import math
import random
import sys
import threading

import pytest
import torch

from attention_backward_tcgen05_gb300 import binding
from test_norm_rope import DT, U32, close, half_step, ref_forward, tables

# ------------------------------------------------------------------ refusals (CPU)

A = 1 << 20  # an address that is never read


def paged_dims(**kw):
    d = dict(B=2, T=4, H=4, Hkv=2, DK=64, DV=64, page=16, pages=8, max_pages=3, rot=64, P=48, ldq=512, ldk=512, ldv=512)
    d.update(kw)
    return binding.fab_paged_dims(*[d[n] for n, _ in binding.fab_paged_dims._fields_])


def call_append(dims, q=A, k=A, v=A, wq=A, wk=A, cos=A, sin=A, eps=1e-6, starts=A, lens=A, table=A, dtype=1, qo=A,
                kc=A, vc=A):
    return binding.lib().fab_paged_append(q, k, v, wq, wk, cos, sin, eps, 0, starts, lens, table, dtype,
                                          ctypes.byref(dims), qo, kc, vc, None)


def call_attention(dims, q=A, kc=A, vc=A, starts=A, lens=A, table=A, scale=1.0, dtype=1, ws=A, wsb=1 << 40, o=A, lse=A):
    return binding.lib().fab_paged_attention(q, kc, vc, starts, lens, table, 1, scale, dtype, ctypes.byref(dims), ws,
                                             wsb, o, lse, None)


BAD_DIMS = [dict(B=0), dict(T=-1), dict(H=3), dict(Hkv=0), dict(DK=0), dict(DV=-8), dict(page=0), dict(pages=0),
            dict(max_pages=0), dict(T=1 << 31), dict(pages=1 << 31), dict(pages=1 << 30, page=1 << 20),
            dict(B=1 << 30, max_pages=1 << 30), dict(T=1, H=1 << 31, DK=8, DV=8, rot=8, ldq=1 << 35)]


@pytest.mark.parametrize("bad", BAD_DIMS, ids=str)
def test_refused_dims(bad):
    assert call_append(paged_dims(**bad)) == binding.FAB_ERR_INVALID
    assert call_attention(paged_dims(**bad)) == binding.FAB_ERR_INVALID
    assert binding.fab_paged_attention_workspace_bytes(paged_dims(**bad), binding.FAB_BF16) == 0


@pytest.mark.parametrize("bad", [dict(rot=3), dict(rot=66), dict(P=0), dict(ldq=255), dict(ldk=127), dict(ldv=0)],
                         ids=str)
def test_append_refuses_dims(bad):
    assert call_append(paged_dims(**bad)) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=A + 1), dict(v=None), dict(cos=None), dict(sin=A + 1),
                                 dict(eps=-1.0), dict(starts=None), dict(lens=A + 2), dict(table=None), dict(dtype=3),
                                 dict(qo=None), dict(kc=A + 8), dict(vc=None), dict(wk=A + 1)], ids=str)
def test_append_refuses_arguments(bad):
    assert call_append(paged_dims(), **bad) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=A + 2), dict(kc=None), dict(vc=A + 8), dict(starts=A + 1),
                                 dict(lens=None), dict(table=A + 2), dict(dtype=9), dict(o=None), dict(lse=A + 4),
                                 dict(scale=float("nan")), dict(scale=float("inf"))], ids=str)
def test_attention_refuses_arguments(bad):
    assert call_attention(paged_dims(), **bad) == binding.FAB_ERR_INVALID


def test_workspace_and_width_refusals():
    long = paged_dims(max_pages=3000)
    need = binding.fab_paged_attention_workspace_bytes(long, binding.FAB_BF16)
    assert need > 0 and binding.fab_paged_attention_workspace_bytes(long, 4) == 0
    assert call_attention(long, wsb=need - 1) == binding.FAB_ERR_WORKSPACE
    assert call_attention(long, ws=A + 4) == binding.FAB_ERR_WORKSPACE
    assert call_attention(long, ws=None, wsb=0) == binding.FAB_ERR_WORKSPACE
    wide = paged_dims(DK=264, ldq=4096, ldk=4096)
    assert call_append(wide) == binding.FAB_ERR_UNSUPPORTED
    assert call_attention(wide) == binding.FAB_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [(1 << 31) - 256, (1 << 31) - 1])
def test_tokens_that_the_kernels_cannot_number_are_refused(T):
    # a unit's tiles end up to 255 tokens behind its last one, and 32 bits have to hold their numbers
    dims = paged_dims(T=T, H=1, Hkv=1, DK=8, DV=8, rot=8)
    assert call_append(dims) == binding.FAB_ERR_INVALID
    assert call_attention(dims) == binding.FAB_ERR_INVALID
    assert binding.fab_paged_attention_workspace_bytes(dims, binding.FAB_BF16) == 0
    dims.T = (1 << 31) - 257
    assert binding.fab_paged_attention_workspace_bytes(dims, binding.FAB_BF16) > 0


def test_no_tokens_is_nothing_to_do():
    assert call_append(paged_dims(T=0), q=None, k=None, v=None, qo=None) == binding.FAB_OK
    assert call_attention(paged_dims(T=0), q=None, o=None, lse=None) == binding.FAB_OK


def test_binding_refuses_what_does_not_fit():
    q = torch.zeros(3, 4, 64)
    k, v = torch.zeros(5, 2, 16, 64), torch.zeros(5, 2, 16, 64)
    starts, lens = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for args in ((q, k, v, starts, lens, table),        # not CUDA tensors
                 (q[0], k, v, starts, lens, table),     # not 3-D
                 (q, k[0], v, starts, lens, table),     # not 4-D
                 (q, k, v, starts, lens, table[0])):    # not 2-D
        with pytest.raises(ValueError):
            binding.paged_attention(*args)
        with pytest.raises(ValueError):
            binding.paged_append(args[0], q[:, :2], q[:, :2], None, None, None, None, *args[3:], args[1], args[2])


@pytest.mark.parametrize("workspace", [torch.empty(64, dtype=torch.uint8)[::2], torch.empty(1).expand(1 << 20),
                                       torch.empty(8, 8)[:, :4]], ids=["strided", "expanded", "columns"])
def test_binding_refuses_a_workspace_with_gaps(workspace):
    # as many elements as are asked for, but not the bytes behind its address (device -1: the CPU's)
    with pytest.raises(ValueError):
        binding._bytes(workspace, -1)
    assert binding._bytes(workspace.contiguous(), -1) == workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------ a paged batch


class Batch:
    """Caches with shuffled pages, their unused rows full of NaN, and the
    sequences' lengths: `new` tokens each, `held` tokens after them."""

    def __init__(self, new, held, H, Hkv, DK, DV, page, dtype, seed, spare=0, extra=2, std=1.0):
        self.new, self.held, self.H, self.Hkv, self.DK, self.DV, self.page = new, held, H, Hkv, DK, DV, page
        self.dt, self.T = DT[dtype], sum(new) + spare
        g = self.g = torch.Generator().manual_seed(seed)
        need = [-(-h // page) for h in held]
        self.pages = sum(need) + extra
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(max(need), 1) + 1
        self.table = torch.full((len(new), width), -7, dtype=torch.int32)  # entries that no token needs are never read
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        self.starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        self.lens = torch.tensor(held, dtype=torch.int32)
        self.k = torch.full((self.pages, Hkv, page, DK), float("nan"), dtype=self.dt)
        self.v = torch.full((self.pages, Hkv, page, DV), float("nan"), dtype=self.dt)
        for b, h in enumerate(held):
            for m in range(h):
                at = (int(self.table[b, m // page]), slice(None), m % page)
                self.k[at] = (torch.randn((Hkv, DK), generator=g) * std).to(self.dt)
                self.v[at] = torch.randn((Hkv, DV), generator=g).to(self.dt)
        self.q = (torch.randn((self.T, H, DK), generator=g) * std).to(self.dt)

    def cuda(self):
        return [t.cuda() for t in (self.q, self.k, self.v, self.starts, self.lens, self.table)]

    def rows(self, cache, b, count, hk):
        """The first `count` rows of sequence b's head hk, 64 bits."""
        m = torch.arange(count)
        return cache[self.table[b, m // self.page].long(), hk, m % self.page].double()

    def check(self, o, lse, causal, scale):
        """Every live token's row against softmax in 64 bits."""
        o, lse = o.double().cpu(), lse.double().cpu()
        u = half_step(self.dt)
        t0 = 0
        for b, (n, h) in enumerate(zip(self.new, self.held)):
            G = self.H // self.Hkv
            for hq in range(self.H if n else 0):
                K, V = self.rows(self.k, b, h, hq // G), self.rows(self.v, b, h, hq // G)
                Q = self.q[t0: t0 + n, hq].double()
                x = scale * Q @ K.t()
                size = abs(scale) * Q.abs() @ K.abs().t()
                last = torch.arange(h - n, h) if causal else torch.full((n,), h - 1)
                hidden = torch.arange(h) > last[:, None]
                x = x.masked_fill(hidden, float("-inf"))
                size = size.masked_fill(hidden, 0.0)
                empty = last < 0
                got, z = o[t0: t0 + n, hq], lse[hq, t0: t0 + n]
                assert (got[empty] == 0).all() and (z[empty] == float("inf")).all()
                if empty.all():
                    continue
                x, size, got, z = x[~empty], size[~empty], got[~empty], z[~empty]
                p, want = x.softmax(-1), torch.logsumexp(x, -1)
                d = (self.DK + 16) * U32 * size.amax(-1) + 8 * U32 * x.masked_fill(x.isinf(), 0).abs().amax(-1)
                add = (h + 16) * U32
                weight = (u if self.dt != torch.float32 else 0.0) + 2 * d + add
                W = p @ V
                room = weight[:, None] * (p @ V.abs()) * 1.01
                room = room + u * (W.abs() + room) + torch.finfo(self.dt).smallest_normal * torch.finfo(self.dt).eps
                worst = ((got - W).abs() / room).max().item()
                assert math.isfinite(worst) and worst <= 1, (b, hq, worst)
                off = ((z - want).abs() / (d + add + 8 * U32 * (1 + want.abs()))).max().item()
                assert math.isfinite(off) and off <= 1, (b, hq, "lse", off)
            t0 += n


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()
    yield
    assert binding.fab_last_device_error() == binding.FAB_OK


# name: new, held, H, Hkv, DK, DV, page, dtype
ATTENTION = {
    "bf16_decode": ([1, 1, 1, 1], [1, 17, 128, 700], 8, 2, 128, 128, 16, "bf16"),
    "bf16_decode_one_head": ([1, 1], [129, 255], 1, 1, 128, 128, 128, "bf16"),
    "f16_decode_d64": ([1, 1, 1], [300, 5, 64], 4, 4, 64, 64, 64, "f16"),
    "bf16_chunks": ([70, 1, 130, 0, 33], [70, 400, 300, 90, 1000], 8, 2, 128, 128, 32, "bf16"),
    "f16_chunks_d64": ([5, 257, 64], [600, 257, 65], 4, 1, 64, 64, 16, "f16"),
    "bf16_chunk_one_group": ([300], [700], 2, 2, 128, 128, 256, "bf16"),
    "f16_group_of_three": ([50, 90], [350, 90], 9, 3, 64, 64, 32, "f16"),
    "bf16_group_of_seven": ([1, 40], [333, 140], 7, 1, 128, 128, 16, "bf16"),
    "bf16_group_of_five_long": ([200], [900], 10, 2, 64, 64, 64, "bf16"),
    "bf16_all_heads_one_key_head": ([1, 3], [250, 90], 64, 1, 64, 64, 16, "bf16"),
    "bf16_group_past_a_tile": ([2], [150], 160, 1, 64, 64, 16, "bf16"),
    "bf16_page_of_eight": ([9, 1], [200, 130], 4, 2, 128, 128, 8, "bf16"),
    "f16_page_of_24": ([30, 1], [200, 130], 4, 2, 64, 64, 24, "f16"),
    "bf16_page_of_48": ([30, 1], [300, 131], 4, 2, 128, 128, 48, "bf16"),
    "bf16_page_of_5": ([10, 1], [57, 131], 4, 2, 128, 128, 5, "bf16"),
    "f16_page_of_one": ([3, 1], [19, 40], 2, 1, 64, 64, 1, "f16"),
    "bf16_d80": ([40, 1], [240, 137], 4, 2, 80, 80, 16, "bf16"),
    "f16_d96_v64": ([20, 1], [240, 137], 4, 2, 96, 64, 16, "f16"),
    "bf16_d40_v128": ([20, 1], [140, 137], 4, 4, 40, 128, 32, "bf16"),
    "bf16_d8": ([20, 1], [140, 137], 2, 2, 8, 8, 32, "bf16"),
    "bf16_d256": ([6, 1], [140, 137], 4, 2, 256, 256, 32, "bf16"),
    "f16_odd_widths": ([6, 1], [40, 77], 4, 2, 37, 21, 16, "f16"),
    "f32_decode": ([1, 1, 1], [1, 77, 600], 8, 2, 64, 64, 16, "f32"),
    "f32_chunks": ([40, 1, 100], [240, 33, 100], 6, 2, 80, 80, 24, "f32"),
    "f32_wide": ([5], [70], 2, 1, 256, 200, 16, "f32"),
    "f32_odd_widths": ([5, 17], [70, 17], 2, 1, 3, 5, 7, "f32"),
    "bf16_fewer_keys_than_tokens": ([40, 3, 2], [25, 1, 0], 4, 2, 128, 128, 16, "bf16"),
    "f32_fewer_keys_than_tokens": ([40, 3, 2], [25, 1, 0], 4, 2, 64, 64, 16, "f32"),
    "bf16_many_sequences": ([1] * 200 + [0] * 100 + [2] * 100, [(7 * i) % 150 + 2 for i in range(400)], 4, 2, 64, 64,
                            16, "bf16"),
    "bf16_long_split": ([1], [9000], 4, 1, 128, 128, 64, "bf16"),
    "f16_long_split_chunk": ([70], [5000], 2, 1, 64, 64, 128, "f16"),
    "f32_long_split": ([2], [3000], 4, 1, 64, 64, 64, "f32"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name", ATTENTION)
def test_attention(gpu, name, causal):
    new, held, *rest = ATTENTION[name]
    x = Batch(new, held, *rest, seed=sum(map(ord, name)))
    scale = rest[2] ** -0.5
    o, lse = binding.paged_attention(*x.cuda(), causal, scale)
    x.check(o, lse, causal, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name", ATTENTION)
def test_attention_with_a_wide_table(gpu, name, causal):
    # room for 5000 keys a sequence: the work of short calls is then cut over the
    # SMs too, and joined
    new, held, *rest = ATTENTION[name]
    x = Batch(new, held, *rest, seed=1 + sum(map(ord, name)))
    x.table = torch.nn.functional.pad(x.table, (0, 5000 // x.page), value=-7)
    scale = rest[2] ** -0.5
    o, lse = binding.paged_attention(*x.cuda(), causal, scale)
    x.check(o, lse, causal, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_attention_scales(gpu, scale):
    # zero, negative and large scales; the last makes scores of some tens
    for dtype, D in (("bf16", 128), ("f16", 64), ("f32", 48)):
        x = Batch([30, 1], [170, 260], 4, 2, D, D, 16, dtype, seed=5)
        o, lse = binding.paged_attention(*x.cuda(), True, scale)
        x.check(o, lse, True, scale)


@pytest.mark.gpu
def test_attention_of_growing_scores(gpu):
    # every key's score is far above the ones before: the running maximum moves at each tile
    for dtype in ("bf16", "f16", "f32"):
        x = Batch([3, 1], [900, 500], 4, 2, 64, 64, 32, dtype, seed=6)
        for b, h in enumerate(x.held):
            for m in range(h):
                x.k[int(x.table[b, m // 32]), :, m % 32] = 0.05 * m / 8
        x.q.fill_(1.0)
        o, lse = binding.paged_attention(*x.cuda(), True, 0.125)
        x.check(o, lse, True, 0.125)


@pytest.mark.gpu
def test_scores_of_minus_infinity(gpu):
    # a key row of -inf scores -inf everywhere: its weight is 0, and a token
    # that sees no other key is empty
    for dtype in ("bf16", "f32"):
        x = Batch([2, 2], [200, 2], 2, 1, 64, 64, 16, dtype, seed=8)
        x.q.abs_()
        for m in range(150):
            x.k[int(x.table[0, m // 16]), :, m % 16] = float("-inf")
        for m in range(2):
            x.k[int(x.table[1, 0]), :, m] = float("-inf")
        o, lse = binding.paged_attention(*x.cuda(), True, 0.125)
        assert (o[2:] == 0).all() and (lse[:, 2:] == float("inf")).all()
        y = Batch([2], [50], 2, 1, 64, 64, 16, dtype, seed=8)  # the 50 keys that count, in a cache of their own
        keep = torch.arange(150, 200)
        src = (x.table[0, keep // 16].long(), slice(None), keep % 16)
        dst = (y.table[0, (keep - 150) // 16].long(), slice(None), (keep - 150) % 16)
        y.k[dst], y.v[dst], y.q = x.k[src], x.v[src], x.q[:2]
        y.check(o[:2], lse[:, :2], True, 0.125)


@pytest.mark.gpu
def test_nan_stays_in_its_row(gpu):
    for dtype in ("bf16", "f32"):
        x = Batch([3, 1], [130, 40], 2, 1, 64, 64, 16, dtype, seed=9)
        x.q[1, 0, 5] = float("nan")
        o, lse = binding.paged_attention(*x.cuda(), True, 0.125)
        assert o[1, 0].isnan().all() and lse[0, 1].isnan()
        ok = torch.ones(4, 2, dtype=torch.bool)
        ok[1, 0] = False
        assert o.cpu()[ok].isfinite().all() and lse.t().cpu()[ok].isfinite().all()
        # the key of the last position is seen by the last token alone
        x = Batch([3, 1], [130, 40], 2, 1, 64, 64, 16, dtype, seed=9)
        x.k[int(x.table[0, 129 // 16]), :, 129 % 16] = float("nan")
        x.v[int(x.table[0, 129 // 16]), :, 129 % 16] = float("nan")
        o, lse = binding.paged_attention(*x.cuda(), True, 0.125)
        assert o[2].isnan().all()
        assert lse[:, :2].isfinite().all() and lse[:, 3].isfinite().all() and o[3].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_calls_need_no_workspace(gpu, dtype):
    x = Batch([1, 2], [100, 60], 8, 2, 64, 64, 16, dtype, seed=31)
    d = x.cuda()
    assert binding.alloc_paged(d[0], d[1], d[2], d[5]).numel() == 0
    o, lse = torch.empty_like(d[0]), torch.empty((8, 3), dtype=torch.float32, device="cuda")
    binding.fab_paged_attention(*d, True, 0.125, None, o, lse)
    x.check(o, lse, True, 0.125)
    x.table = torch.nn.functional.pad(x.table, (0, 300), value=-7)
    d = x.cuda()
    with pytest.raises(binding.FabError):
        binding.fab_paged_attention(*d, True, 0.125, None, o, lse)
    binding.fab_paged_attention(*d, True, 0.125, binding.alloc_paged(d[0], d[1], d[2], d[5]), o, lse)
    x.check(o, lse, True, 0.125)


@pytest.mark.gpu
def test_padding_tokens_are_left_alone(gpu):
    for dtype in ("bf16", "f32"):
        x = Batch([5, 1], [60, 133], 4, 2, 64, 64, 16, dtype, seed=10, spare=40)
        q, k, v, starts, lens, table = x.cuda()
        o = torch.full((x.T, 4, 64), 3.0, dtype=x.dt, device="cuda")
        lse = torch.full((4, x.T), 3.0, device="cuda")
        ws = binding.alloc_paged(q, k, v, table)
        binding.fab_paged_attention(q, k, v, starts, lens, table, True, 0.125, ws, o, lse)
        assert (o[6:] == 3).all() and (lse[:, 6:] == 3).all()
        x.check(o, lse, True, 0.125)
        o2 = torch.empty_like(o)  # without the log-sum-exp
        binding.fab_paged_attention(q, k, v, starts, lens, table, True, 0.125, ws, o2, None)
        assert torch.equal(o2[:6], o[:6])
        before = k.clone(), v.clone()
        row = torch.randn(x.T, 4 * 64 + 2 * 2 * 64, device="cuda").to(x.dt)
        a, b, c = row.split([256, 128, 128], -1)
        qo = torch.full((x.T, 4, 64), 3.0, dtype=x.dt, device="cuda")
        binding.fab_paged_append(a.unflatten(-1, (4, 64)), b.unflatten(-1, (2, 64)), c.unflatten(-1, (2, 64)), None,
                                 None, None, None, 1e-6, False, starts, lens, table, qo, k, v)
        assert (qo[6:] == 3).all() and torch.equal(qo[:6].flatten(1), a[:6])
        changed = (k.isnan() != before[0].isnan()) | ((k != before[0]) & ~k.isnan())
        assert changed.any(-1).sum() <= 6 * 2


@pytest.mark.gpu
def test_no_tokens(gpu):
    # T = 0 through the binding, and sequences none of which has a new token
    x = Batch([2], [20], 4, 2, 64, 64, 16, "bf16", seed=10)
    q, k, v, starts, lens, table = x.cuda()
    before = k.clone()
    for n in (0, 2):
        qn = q[:n]
        starts.zero_()
        o, lse = binding.paged_attention(qn, k, v, starts, lens, table, True, 0.125)
        assert o.shape == (n, 4, 64) and lse.shape == (4, n)
        binding.paged_append(qn, qn[:, :2], qn[:, :2], None, None, None, None, starts, lens, table, k, v)
    assert torch.equal(k.nan_to_num(9), before.nan_to_num(9))


@pytest.mark.gpu
def test_operands_that_do_not_match_are_refused(gpu):
    x = Batch([2], [20], 4, 2, 64, 64, 16, "bf16", seed=10)
    q, k, v, starts, lens, table = x.cuda()
    for bad in ((q.half(), k, v, starts, lens, table), (q.transpose(0, 1), k, v, starts, lens, table),
                (q, k, v.half(), starts, lens, table), (q, k, v[:-1], starts, lens, table),
                (q, k.transpose(1, 2), v, starts, lens, table), (q, k, v, starts.long(), lens, table),
                (q, k, v, starts[:1], lens, table), (q, k, v, starts, lens, table[:, ::2]),
                (q[:, :3], k, v, starts, lens, table), (q, k, v, starts, lens.cpu(), table),
                (q[..., :32].contiguous(), k, v, starts, lens, table)):
        with pytest.raises((ValueError, binding.FabError)):
            binding.paged_attention(*bad)


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 5000], ids=["as_is", "wide_table"])  # whole units, work cut over the SMs
def test_graphs_side_by_side(gpu, room):
    # two captured steps, each with the workspace that its capture allocated, replayed on two streams at once
    x = [Batch([1, 9], [900, 350], 8, 2, 128, 128, 16, "bf16", seed=s) for s in (20, 21)]
    for b in x:
        b.table = torch.nn.functional.pad(b.table, (0, room // b.page), value=-7)
    dev = [b.cuda() for b in x]
    want = [binding.paged_attention(*d, True, 0.1) for d in dev]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.paged_attention(*d, True, 0.1))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in x]
    for _ in range(20):
        for o, lse in outs:
            o.fill_(float("nan"))
            lse.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.gpu
def test_bad_pages_are_reported(gpu):
    for dtype in ("bf16", "f32"):
        for bad in (-1, 1 << 30, None):
            x = Batch([5, 1], [60, 133], 4, 2, 64, 64, 16, dtype, seed=11)
            if bad is None:
                x.lens[1] = 16 * x.table.shape[1] + 1  # one token more than its row of the table can hold
                x.table[1] = 0
            else:
                x.table[1, 2] = x.pages if bad > 0 else bad
            q, k, v, starts, lens, table = x.cuda()
            o, lse = binding.paged_attention(q, k, v, starts, lens, table, True, 0.125)
            assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
            good = Batch([5, 1], [60, 133], 4, 2, 64, 64, 16, dtype, seed=11)
            want, wlse = binding.paged_attention(*good.cuda(), True, 0.125)
            assert torch.equal(o[:5], want[:5]) and torch.equal(lse[:, :5], wlse[:, :5])


@pytest.mark.gpu
@pytest.mark.parametrize("starts", [[0, 4, 2, 6], [0, 3, 9, 6], [-2, 3, 5, 6], [2, 3, 5, 6], [0, 3, 5, 100]], ids=str)
def test_bad_starts_are_reported(gpu, starts):
    for dtype in ("bf16", "f32"):
        x = Batch([2, 2, 2], [60, 133, 20], 4, 2, 64, 64, 16, dtype, seed=11)
        x.starts = torch.tensor(starts, dtype=torch.int32)
        x.table[x.table < 0] = 0
        q, k, v, st, lens, table = x.cuda()
        binding.paged_attention(q, k, v, st, lens, table, True, 0.125)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
        binding.paged_append(q, q[:, :2], q[:, :2], None, None, None, None, st, lens, table, k, v)
        assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID


# name: new, held, H, Hkv, DK, DV, page, dtype, rot, interleaved, norm
APPEND = {
    "bf16_decode": ([1, 1, 1, 1], [1, 17, 128, 70], 8, 2, 128, 128, 16, "bf16", 128, False, True),
    "f16_chunks": ([30, 0, 1, 57], [30, 5, 9, 200], 4, 4, 64, 64, 64, "f16", 64, False, False),
    "bf16_pairs_part": ([30, 3], [33, 77], 4, 2, 80, 64, 24, "bf16", 32, True, True),
    "f32_no_rot": ([3, 11], [13, 11], 4, 2, 64, 64, 16, "f32", 0, False, True),
    "f32_odd": ([3, 11], [13, 11], 4, 2, 7, 5, 3, "f32", 6, False, True),
    "f16_odd_pairs": ([3, 11], [13, 30], 3, 1, 50, 33, 5, "f16", 22, True, False),
    "bf16_long": ([700, 1, 600], [900, 4, 600], 8, 2, 128, 128, 32, "bf16", 128, False, True),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", APPEND)
def test_append(gpu, name):
    new, held, H, Hkv, DK, DV, page, dtype, rot, il, norm = APPEND[name]
    x = Batch(new, [0] * len(new), H, Hkv, DK, DV, page, dtype, seed=3, extra=sum(-(-h // page) for h in held) + 2)
    order = torch.randperm(x.pages, generator=x.g).to(torch.int32)
    width = max(-(-h // page) for h in held)
    x.table, i = torch.full((len(new), width), -3, dtype=torch.int32), 0
    for b, h in enumerate(held):
        c = -(-h // page)
        x.table[b, :c] = order[i: i + c]
        i += c
    x.lens = torch.tensor(held, dtype=torch.int32)
    row = torch.randn((x.T, H * DK + Hkv * (DK + DV)), generator=x.g).to(x.dt)
    q, k, v = row.split([H * DK, Hkv * DK, Hkv * DV], -1)
    q, k, v = q.unflatten(-1, (H, DK)), k.unflatten(-1, (Hkv, DK)), v.unflatten(-1, (Hkv, DV))
    weight = lambda: (1 + 0.3 * torch.randn((DK,), generator=x.g)).to(x.dt) if norm else None
    wq, wk = weight(), weight()
    cos, sin = tables(max(held), rot)
    dev = lambda t: None if t is None else t.cuda()
    rows = row.cuda()
    dq, dk, dv = rows.split([H * DK, Hkv * DK, Hkv * DV], -1)
    kc, vc = x.k.cuda(), x.v.cuda()
    got = binding.paged_append(dq.unflatten(-1, (H, DK)), dk.unflatten(-1, (Hkv, DK)), dv.unflatten(-1, (Hkv, DV)),
                               dev(wq), dev(wk), dev(cos) if rot else None, dev(sin) if rot else None,
                               x.starts.cuda(), x.lens.cuda(), x.table.cuda(), kc, vc, 1e-6, il)
    pos = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)])
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    if not rot:
        c = s = torch.zeros((x.T, 1, 0), dtype=torch.float64)
    want, bound = ref_forward(q, wq, c, s, il, 1e-6)
    close(got, want, bound, x.dt, "q")
    where = x.table[seq, pos // page].long()
    want, bound = ref_forward(k, wk, c, s, il, 1e-6)
    close(kc.cpu()[where, :, pos % page], want, bound, x.dt, "k")
    assert torch.equal(vc.cpu()[where, :, pos % page], v)
    touched = torch.zeros(x.pages, page, dtype=torch.bool)
    touched[where, pos % page] = True
    for cache in (kc, vc):  # every other row is the NaN that it was
        assert cache.cpu().transpose(1, 2)[~touched].isnan().all()


@pytest.mark.gpu
def test_served_as_trained(gpu):
    # a prompt in two chunks and then tokens one by one, appended and attended
    # to in a paged cache, equal the causal forward over the whole sequence
    H, Hkv, D, N, page = 8, 2, 64, 150, 16
    g = torch.Generator().manual_seed(12)
    for dtype in ("bf16", "f16", "f32"):
        dt = DT[dtype]
        row = torch.randn((1, N, (H + 2 * Hkv) * D), generator=g).to(dt).cuda()
        q, k, v = row.split([H * D, Hkv * D, Hkv * D], -1)
        q, k, v = q.unflatten(-1, (H, D)), k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D))
        wq, wk = ((1 + 0.2 * torch.randn((D,), generator=g)).to(dt).cuda() for _ in range(2))
        cos, sin = (t.cuda() for t in tables(N, D))
        Q, K, V = binding.qk_norm_rope(q, k, v, wq, wk, cos, sin)
        o, lse = binding.forward(Q, K, V, None, True, 0.125)
        kc = torch.full((12, Hkv, page, D), float("nan"), dtype=dt, device="cuda")
        vc = kc.clone()
        table = torch.randperm(12, generator=g)[:10].to(torch.int32).view(1, 10).cuda()
        done = 0
        for n in [70, 65] + [1] * 15:
            starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            lens = torch.tensor([done + n], dtype=torch.int32, device="cuda")
            part = slice(done, done + n)
            qn = binding.paged_append(q[0, part], k[0, part], v[0, part], wq, wk, cos, sin, starts, lens, table, kc, vc)
            assert torch.equal(qn, Q[0, :, part].transpose(0, 1))
            on, ln = binding.paged_attention(qn, kc, vc, starts, lens, table, True, 0.125)
            # both round weights and result once: two half steps each way of the weighted sum of |v| (below 4)
            assert (on.double() - o[0, part].double()).abs().max() <= 16 * half_step(dt) + 1e-5
            assert (ln - lse[0, :, part]).abs().max() <= 4 * half_step(dt) + 1e-5
            done += n


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 5000], ids=["as_is", "wide_table"])  # whole units, work cut over the SMs
def test_captured_step_follows_lengths(gpu, room):
    # a captured decoding step replayed with longer sequences and other pages
    H, Hkv, D, page, B = 8, 2, 128, 16, 3
    g = torch.Generator().manual_seed(13)
    kc = torch.randn((60, Hkv, page, D), generator=g).to(torch.bfloat16).cuda()
    vc = torch.randn((60, Hkv, page, D), generator=g).to(torch.bfloat16).cuda()
    cos, sin = (t.cuda() for t in tables(300, D))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    row = torch.randn((B, (H + 2 * Hkv) * D), generator=g).to(torch.bfloat16).cuda()
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    table = torch.randperm(60, generator=g).to(torch.int32).view(B, 20)
    table = torch.nn.functional.pad(table, (0, room // page), value=-7).cuda()

    def step():
        q, k, v = row.split([H * D, Hkv * D, Hkv * D], -1)
        q = binding.paged_append(q.unflatten(-1, (H, D)), k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D)), w, w,
                                 cos, sin, starts, lens, table, kc, vc)
        return binding.paged_attention(q, kc, vc, starts, lens, table, True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for now in ([5, 250, 16], [300, 1, 129], [17, 17, 0]):
        lens.copy_(torch.tensor(now))
        starts.copy_(torch.tensor([0, 1, 2, 2 if now[2] == 0 else 3]))
        row.normal_()
        graph.replay()
        live = int(starts[-1])
        a, b = o[:live].clone(), lse[:, :live].clone()
        want, wl = step()
        assert torch.equal(a, want[:live]) and torch.equal(b, wl[:, :live])


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 5000], ids=["as_is", "wide_table"])  # whole units, work cut over the SMs
def test_captured_behind_a_fork_and_a_copy(gpu, room):
    # the call's operands come from another branch of the graph and from a copy
    # right before it; what follows reads its result at once
    x = Batch([1, 9, 70], [900, 350, 200], 8, 2, 128, 128, 16, "bf16", seed=22)
    x.table = torch.nn.functional.pad(x.table, (0, room // x.page), value=-7)
    q, k, v, starts, lens, table = x.cuda()
    want, wl = binding.paged_attention(q, k, v, starts, lens, table, True, 0.1)
    qs, ks = torch.zeros_like(q), torch.zeros_like(k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            ks.copy_(k)
        qs.add_(q)
        main.wait_stream(side)
        qs.copy_(q)
        o, lse = binding.paged_attention(qs, ks, v, starts, lens, table, True, 0.1)
        twice = o + o
        qs.zero_()
        ks.zero_()
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(twice, want + want)


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 5000], ids=["as_is", "wide_table"])  # whole units, work cut over the SMs
def test_two_streams_with_workspaces_of_their_own(gpu, room):
    x = [Batch([1, 9], [900, 350], 8, 2, 128, 128, 16, "bf16", seed=s) for s in (20, 21)]
    for b in x:
        b.table = torch.nn.functional.pad(b.table, (0, room // b.page), value=-7)
    dev = [b.cuda() for b in x]
    want = [binding.paged_attention(*d, True, 0.1) for d in dev]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in x]
    for _ in range(20):
        got = [binding.paged_attention(*d, True, 0.1, stream=s) for d, s in zip(dev, side)]
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 80), ("f32", 128)])
def test_offsets_past_32_bits(gpu, dtype, D):
    # pages whose first element lies past 2^31 elements of the cache
    Hkv, page = 4, 64
    pages = (1 << 31) // (Hkv * page * D) + 40
    dt = DT[dtype]
    k = torch.empty((pages, Hkv, page, D), dtype=dt, device="cuda")
    v = torch.empty_like(k)
    x = Batch([1, 20], [900, 300], 8, Hkv, D, D, page, dtype, seed=30, extra=0)
    assert x.pages < 40
    k[pages - x.pages:], v[pages - x.pages:] = x.k.cuda(), x.v.cuda()
    far = torch.where(x.table >= 0, x.table + (pages - x.pages), x.table).cuda()
    q, _, _, starts, lens, _ = x.cuda()
    o, lse = binding.paged_attention(q, k, v, starts, lens, far, True, 0.1)
    x.check(o, lse, True, 0.1)
    row = torch.randn(21, Hkv, D, device="cuda").to(dt)
    binding.paged_append(q, row, row, None, None, None, None, starts, lens, far, k, v)
    at = torch.tensor([899] + list(range(280, 300)))
    seq = torch.tensor([0] + [1] * 20)
    where = far.cpu()[seq, at // page].long().cuda()
    assert torch.equal(k[where, :, (at % page).cuda()], row)


@pytest.mark.gpu
def test_drawn_batches(gpu):
    r = random.Random(77)
    for i in range(40):
        dtype = r.choice(["bf16", "f16", "f32"])
        Hkv, G = r.choice([1, 2, 3]), r.choice([1, 2, 3, 4, 6, 8])
        DK = r.choice([64, 128, 128, 64, 80, 96, 24])
        DV = DK if r.random() < 0.7 else r.choice([64, 128, 32])
        page, causal = r.choice([8, 16, 24, 32, 64, 128, 256, 20]), r.random() < 0.7
        B = r.randint(1, 6)
        new = [r.choice([0, 1, 1, 2, r.randint(1, 150)]) for _ in range(B)]
        held = [n + r.choice([0, 0, 1, r.randint(0, 100), r.randint(0, 700)]) for n in new]
        if sum(new) == 0:
            new[0], held[0] = 1, 1 + held[0]
        x = Batch(new, held, Hkv * G, Hkv, DK, DV, page, dtype, seed=i, std=r.choice([0.3, 1.0, 2.0]))
        if i % 2:
            x.table = torch.nn.functional.pad(x.table, (0, 5000 // page), value=-7)
        o, lse = binding.paged_attention(*x.cuda(), causal, DK ** -0.5)
        x.check(o, lse, causal, DK ** -0.5)


@pytest.mark.gpu
def test_threads_of_several_widths(gpu):
    # widths whose calls on the CUDA cores share a kernel and need different amounts of shared memory,
    # from threads of their own: in the C entry points, where they run at the same time
    x = [Batch([1], [20], 1, 1, D, D, 16, "f32", seed=D) for D in (32, 64, 96, 128) for _ in range(2)]
    dev, refused, out = [b.cuda() for b in x], [0] * len(x), []
    streams = [torch.cuda.Stream() for _ in x]
    for b in x:
        out.append((torch.empty(b.q.shape, device="cuda"), torch.empty((1, 1), device="cuda")))
    torch.cuda.synchronize()

    def calls(i):
        b, (q, k, v, starts, lens, table), (o, lse) = x[i], dev[i], out[i]
        dims = binding.fab_paged_dims(1, 1, 1, 1, b.DK, b.DV, b.page, b.pages, table.shape[1])
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), starts.data_ptr(), lens.data_ptr(), table.data_ptr(), 1, 0.1,
                binding.FAB_F32, ctypes.byref(dims), None, 0, o.data_ptr(), lse.data_ptr(), streams[i].cuda_stream)
        call = binding.lib().fab_paged_attention
        for _ in range(3000):
            refused[i] += call(*args) != binding.FAB_OK

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(x))]
    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    torch.cuda.synchronize()
    assert refused == [0] * len(x)
    for b, (o, lse) in zip(x, out):
        b.check(o, lse, True, 0.1)


@pytest.mark.gpu
def test_workspaces_with_gaps_are_refused(gpu):
    x = Batch([1, 2], [100, 60], 8, 2, 64, 64, 16, "bf16", seed=31)
    x.table = torch.nn.functional.pad(x.table, (0, 300), value=-7)
    d = x.cuda()
    o, lse = torch.empty_like(d[0]), torch.empty((8, 3), dtype=torch.float32, device="cuda")
    ws = binding.alloc_paged(d[0], d[1], d[2], d[5])
    gaps = torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2]
    for bad in (gaps, torch.empty(1, dtype=torch.uint8, device="cuda").expand(ws.numel()), ws.cpu()):
        with pytest.raises(ValueError):
            binding.fab_paged_attention(*d, True, 0.125, bad, o, lse)
        g = torch.zeros(1, 4, 2, 64, device="cuda")
        w = torch.ones(64, device="cuda")
        with pytest.raises(ValueError):
            rows = g.transpose(1, 2).contiguous()
            binding.fab_qk_norm_rope_backward(rows, rows, None, g, g, w, w, None, None, None, 1e-6, False, bad, g, g,
                                              None, w, w)
    binding.fab_paged_attention(*d, True, 0.125, ws, o, lse)
    x.check(o, lse, True, 0.125)
