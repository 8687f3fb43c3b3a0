"""Query/key norms with rotation and their gradient where the kernels step and
loop: rows that are not there beside rows that are, heads by the million.
Against the formulas in 64 bits, computed on the GPU.

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
