"""Query/key norms with rotation and their gradient where the kernels step and
loop: rows that are not there beside rows that are, heads a CTA walks over,
items behind one another, heads by the million.  Against the formulas in 64
bits, computed on the GPU.

Tolerances as in test_norm_rope.py; a weight's gradient adds `depth` values one
after another at most, each addition within half a step of what it adds up.
"""
import math

import pytest
import torch

from attention_backward_tcgen05_gb300 import binding
from test_norm_rope import DT, U32, gpu, half_step, ref_backward, ref_forward, tables  # noqa: F401 (gpu: a fixture)


def inputs(dtype, B, N, H, Hkv, D, rot, il=False, gap=0, seed=1):
    """Projection rows (with a gap, rows that are not 16-byte aligned), weights,
    tables, positions and gradients."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")
    row = draw(B, N, (H + 2 * Hkv) * D + gap).to(dt)
    q, k, v, _ = row.split([H * D, Hkv * D, Hkv * D, gap], -1)
    cos, sin = tables(N + 9, rot)
    x = dict(q=q.unflatten(-1, (H, D)), k=k.unflatten(-1, (Hkv, D)), v=v.unflatten(-1, (Hkv, D)),
             wq=(1 + 0.3 * draw(D)).to(dt), wk=(1 + 0.3 * draw(D)).to(dt), cos=cos.cuda(), sin=sin.cuda(),
             pos=(torch.arange(N, device="cuda") + torch.randint(0, 9, (B, 1), generator=g, device="cuda")).int())
    d = dict(dq=draw(B, H, N, D), dk=draw(B, Hkv, N, D), dv=draw(B, Hkv, N, D))
    return x, d, il, dt


def at(x):
    p = x["pos"].long()
    return x["cos"].double()[p][:, :, None], x["sin"].double()[p][:, :, None]


def within(got, want, bound, dt, what):
    """As test_norm_rope's close, on the GPU."""
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    room = bound + half_step(dt) * (want.abs() + bound) + tiny
    over = ((got.double() - want).abs() / room).max().item()
    assert math.isfinite(over) and over <= 1.0, f"{what}: {over:.3f} of the bound"


def check_forward(x, il, dt, eps):
    q, k, v = binding.qk_norm_rope(**x, eps=eps, interleaved=il)
    cos, sin = at(x)
    for name, y, w in (("q", q, x["wq"]), ("k", k, x["wk"])):
        want, bound = ref_forward(x[name], w, cos, sin, il, eps)
        within(y, want.movedim(2, 1), bound.movedim(2, 1), dt, name)
    assert torch.equal(v, x["v"].transpose(1, 2))


def check_gradient(x, d, il, dt, eps, depth):
    """depth: additions one after another of a column's terms, of q and of k."""
    x = {n: t for n, t in x.items() if n != "v"}
    gq, gk, gv, gwq, gwk = binding.qk_norm_rope_backward(**d, **x, eps=eps, interleaved=il)
    cos, sin = at(x)
    for name, g, gw, n in (("q", gq, gwq, depth[0]), ("k", gk, gwk, depth[1])):
        want, bound, dw, terms = ref_backward(d["d" + name].movedim(1, 2), x[name], x["w" + name], cos, sin, il, eps)
        within(g, want, bound, dt, "g" + name)
        over = ((gw.double() - dw).abs() / ((64 + n) * U32 * terms)).max().item()
        assert math.isfinite(over) and over <= 1.0, f"gw{name}: {over:.3f} of the bound"
    assert torch.equal(gv, d["dv"].transpose(1, 2).to(dt))


def launch(dtype, tokens, H, Hkv, D, rot, il):
    """What the 16-byte kernels' launches make of a call: the forward's heads a
    CTA and rows a step, the gradient's (items, blocks, heads an item) of q and of k."""
    R = rot // 8
    slots = (D // 8 + 1) // 2 if il else R // 2 + (D // 8 - R + 1) // 2
    L = 4 if slots <= 4 else 8 if slots <= 8 else 16
    tb = -(-tokens // (128 // L))
    hb = 32
    while hb > 1 and tb * (-(-H // hb) + 2 * -(-Hkv // hb)) < 1216:
        hb //= 2
    gb = 32
    while gb > 1 and tb * (-(-H // gb) + 2 * -(-Hkv // gb)) < 456:
        gb //= 2
    items = [tb * -(-h // gb) for h in (H, Hkv)]
    blocks = [min(n, -(-1216 * h // (H + 2 * Hkv))) for n, h in zip(items, (H, Hkv))]
    return hb, 1 if dtype == "f32" else 2, [(n, b, gb) for n, b in zip(items, blocks)]


def depths(items):
    """A lane's rows, lanes, warps, rows of partial sums, lanes."""
    return [-(-n // b) * gb + 3 + 4 + -(-b // 32) + 5 for n, b, gb in items]


# ------------------------------------------------------------------ no epsilon

# dtype, B, N, H, Hkv, D, rot, interleaved, gap: single heads beside an empty
# second step, odd heads, tokens that do not fill a block, each of the three
# widths of a group of lanes, the kernels of a warp per row
WITHOUT_EPS = [
    ("bf16", 1, 1, 1, 1, 64, 64, False, 0),
    ("bf16", 1, 16, 2, 2, 128, 128, False, 0),
    ("f16", 1, 13, 3, 1, 64, 64, True, 0),
    ("f16", 3, 777, 12, 4, 80, 32, False, 0),
    ("bf16", 2, 1500, 9, 3, 128, 128, False, 0),
    ("bf16", 1, 29, 5, 5, 256, 256, True, 0),
    ("f32", 1, 13, 3, 1, 64, 64, False, 0),
    ("f32", 2, 75, 8, 2, 128, 128, True, 0),
    ("bf16", 2, 31, 3, 1, 64, 64, False, 3),
    ("f32", 1, 13, 3, 1, 37, 22, False, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WITHOUT_EPS, ids=str)
def test_without_epsilon(gpu, case):
    # eps = 0 is accepted: what stands beside the rows must not enter the weights' gradients
    x, d, il, dt = inputs(*case)
    check_forward(x, il, dt, 0.0)
    tokens = case[1] * case[2]
    check_gradient(x, d, il, dt, 0.0, [tokens * h / 8 + 64 for h in case[3:5]])


# ------------------------------------------------------------------ a token's row past 2^31 elements


@pytest.mark.gpu
def test_a_row_past_31_bits(gpu):
    # one token of 2^25 + 2 heads of width 64: offsets inside its row pass 2^31
    H, Hkv, D = (1 << 25) + 2, 2, 64
    assert H * D > 1 << 31
    x, d, il, dt = inputs("bf16", 1, 1, H, Hkv, D, 64)
    q, k, v = binding.qk_norm_rope(x["q"], x["k"], x["v"])
    assert torch.equal(q[0, :, 0], x["q"][0, 0]) and torch.equal(k[0, :, 0], x["k"][0, 0])
    del q
    gq, gk, _, _, _ = binding.qk_norm_rope_backward(d["dq"], d["dk"], None, x["q"], x["k"])
    assert torch.equal(gq[0, 0], d["dq"][0, :, 0].to(dt)) and torch.equal(gk[0, 0], d["dk"][0, :, 0].to(dt))
    del gq
    q, k, v = binding.qk_norm_rope(**x)
    gq, _, _, gwq, _ = binding.qk_norm_rope_backward(d["dq"], d["dk"], None, x["q"], x["k"], x["wq"], x["wk"], x["cos"],
                                                     x["sin"], x["pos"])
    cos, sin = at(x)
    dw, terms = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    step = 1 << 21
    for h0 in range(0, H, step):
        part = slice(h0, h0 + step)
        rows = x["q"][:, :, part]
        want, bound = ref_forward(rows, x["wq"], cos, sin, il, 1e-6)
        within(q[:, part], want.movedim(2, 1), bound.movedim(2, 1), dt, f"q from head {h0}")
        want, bound, w, t = ref_backward(d["dq"][:, part].movedim(1, 2), rows, x["wq"], cos, sin, il, 1e-6)
        within(gq[:, :, part], want, bound, dt, f"gq from head {h0}")
        dw, terms = dw + w, terms + t
    _, _, items = launch("bf16", 1, H, Hkv, D, 64, il)
    assert ((gwq.double() - dw).abs() <= (64 + depths(items)[0]) * U32 * terms).all()


# ------------------------------------------------------------------ sizes at which the kernels loop

# a training step's 4 x 2,048 tokens of 32 and 8 heads, and an odd neighbour
LOOPS = [(dtype, B, N, H, Hkv, 128, 128, il, 0) for dtype in ("bf16", "f16", "f32")
         for B, N, H, Hkv, il in ((4, 2048, 32, 8, False), (1, 8191, 33, 11, True))]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LOOPS, ids=str)
def test_steps_and_items(gpu, case):
    dtype, B, N, H, Hkv, D, rot, il, _ = case
    heads, step, items = launch(dtype, B * N, H, Hkv, D, rot, il)
    assert heads > 2 * step and any(n > b for n, b, _ in items)
    x, d, il, dt = inputs(*case)
    check_forward(x, il, dt, 1e-6)
    check_gradient(x, d, il, dt, 1e-6, depths(items))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_one_another(gpu, dtype):
    # rows at odd places, more of them than 768 (q) and 256 (k) blocks of eight warps
    N, H, Hkv = 1024, 9, 3
    assert N * H > 768 * 8 and N * Hkv > 256 * 8
    x, d, il, dt = inputs(dtype, 1, N, H, Hkv, 64, 64, gap=3)
    check_forward(x, il, dt, 1e-6)
    # a warp's rows, warps, rows of partial sums, lanes
    check_gradient(x, d, il, dt, 1e-6, [-(-N * h // (8 * b)) + 8 + -(-b // 32) + 5 for h, b in ((H, 768), (Hkv, 256))])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [("bf16", 1, 40, 4, 2, 256, 256, True, 0), ("f32", 3, 300, 6, 2, 96, 64, False, 0)], ids=str)
def test_wide_pairs_and_f32(gpu, case):
    x, d, il, dt = inputs(*case)
    check_forward(x, il, dt, 1e-6)
    check_gradient(x, d, il, dt, 1e-6, [case[1] * case[2] * h / 8 for h in case[3:5]])


@pytest.mark.gpu
def test_more_heads_than_a_grid_has_rows(gpu):
    # the heads of a CTA are doubled until a grid's second dimension holds the blocks
    H, Hkv, D = 2200000, 2, 8
    assert -(-H // 32) > 65535
    x, d, il, dt = inputs("bf16", 1, 3, H, Hkv, D, 0)
    x.update(cos=None, sin=None, wq=None, wk=None, pos=None)
    q, k, v = binding.qk_norm_rope(**x)
    assert all(torch.equal(a, x[n].transpose(1, 2)) for n, a in (("q", q), ("k", k), ("v", v)))
    gq, gk, gv, _, _ = binding.qk_norm_rope_backward(**d, q=None, k=None, dtype=dt)
    assert all(torch.equal(a, d["d" + n].transpose(1, 2).to(dt)) for n, a in (("q", gq), ("k", gk), ("v", gv)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_at_size(gpu, dtype):
    # prompts whose heads a CTA walks over: the same bits as from the tokens by themselves
    H, Hkv, D, page, new, past = 32, 8, 128, 64, [2048, 1, 3001, 0, 2500, 900], [0, 70, 3, 10, 129, 64]
    N = sum(new)
    heads, step, _ = launch(dtype, N, H, Hkv, D, D, False)
    assert heads > 2 * step
    x, _, il, dt = inputs(dtype, 1, N, H, Hkv, D, D)
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)])
    x["pos"] = pos[None].int().cuda()
    want = binding.qk_norm_rope(**x)
    count = [-(-(n + p) // page) for n, p in zip(new, past)]
    table = torch.zeros((len(new), max(count)), dtype=torch.int32)
    order = torch.randperm(sum(count), generator=torch.Generator().manual_seed(4)).int()
    for b, c in enumerate(order.split(count)):
        table[b, : len(c)] = c
    kc = torch.full((sum(count), Hkv, page, D), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    starts = torch.tensor([0] + new).cumsum(0).int().cuda()
    lens = torch.tensor([n + p for n, p in zip(new, past)]).int().cuda()
    q = binding.paged_append(x["q"][0], x["k"][0], x["v"][0], x["wq"], x["wk"], x["cos"], x["sin"], starts, lens,
                             table.cuda(), kc, vc)
    assert torch.equal(q, want[0][0].transpose(0, 1))
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    where = table[seq, pos // page].long()
    slot = pos % page
    assert torch.equal(kc[where.cuda(), :, slot.cuda()], want[1][0].transpose(0, 1))
    assert torch.equal(vc[where.cuda(), :, slot.cuda()], want[2][0].transpose(0, 1))
    untouched = torch.ones(kc.shape[0], page, dtype=torch.bool)
    untouched[where, slot] = False
    for cache in (kc, vc):
        assert cache.transpose(1, 2)[untouched.cuda()].isnan().all()
