"""Query/key norms with the position rotation, and their gradient, against the
formulas in 64 bits.

Tolerances count roundings: a result's own (half a step of its type) and those
of the f32 arithmetic before it, bounded by a number of f32 half steps (2^-24)
times the magnitudes that enter the sum.
"""
import ctypes
import math

import pytest
import torch

from attention_backward_tcgen05_gb300 import binding

U32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ the formulas, 64 bits


def pair_columns(rot, interleaved):
    """Columns (a, b) of the rotated pairs, in order of their angle."""
    if interleaved:
        return list(range(0, rot, 2)), list(range(1, rot, 2))
    return list(range(rot // 2)), list(range(rot // 2, rot))


def turn(x, cos, sin, interleaved):
    a, b = pair_columns(2 * cos.shape[-1], interleaved)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def pair_size(x, rot, interleaved):
    """|x| with both columns of a pair replaced by |a| + |b|."""
    a, b = pair_columns(rot, interleaved)
    y = x.abs()
    z = y.clone()
    z[..., a] = y[..., a] + y[..., b]
    z[..., b] = y[..., a] + y[..., b]
    return z


def ref_forward(x, w, cos, sin, interleaved, eps):
    """(y, f32 error bound) of rows x (..., heads, D); cos, sin broadcast."""
    x = x.double()
    n = x
    if w is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    # a sum of D squares in a tree or a short chain, a reciprocal root, and
    # five products and sums: below 48 half steps
    return turn(n, cos, sin, interleaved), 48 * U32 * pair_size(n, 2 * cos.shape[-1], interleaved)


def ref_backward(dy, x, w, cos, sin, interleaved, eps):
    """(dx, its f32 bound, dw, sum of |terms| of dw), rows (..., heads, D)."""
    dy = dy.double()
    g = turn(dy, cos, -sin, interleaved)
    if w is None:
        return g, 8 * U32 * pair_size(dy, 2 * cos.shape[-1], interleaved), None, None
    x = x.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, u = x * r, g * w.double()
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    size = pair_size(dy, 2 * cos.shape[-1], interleaved)
    usize = size * w.double().abs()
    bound = 64 * U32 * r * (usize + n.abs() * (usize * n.abs()).mean(-1, keepdim=True))
    terms = size * n.abs()
    return dx, bound, (g * n).flatten(0, -2).sum(0), terms.flatten(0, -2).sum(0)


def tables(P, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


# name: dtype, B, N, H, Hkv, DK, DV, rot, interleaved, norm q, norm k, with v, layout
CASES = {
    "bf16_d128": ("bf16", 2, 75, 8, 2, 128, 128, 128, False, True, True, True, "fused"),
    "bf16_d128_pairs": ("bf16", 2, 33, 4, 4, 128, 128, 128, True, True, True, True, "fused"),
    "f16_d64": ("f16", 1, 130, 6, 3, 64, 64, 64, False, True, True, True, "apart"),
    "f32_d64_pairs": ("f32", 3, 17, 2, 1, 64, 64, 64, True, True, True, True, "fused"),
    "bf16_d80_part": ("bf16", 2, 41, 6, 2, 80, 80, 32, False, True, True, True, "fused"),
    "f16_d96": ("f16", 1, 29, 5, 5, 96, 96, 96, False, True, True, True, "fused"),
    "f16_d72_pairs_part": ("f16", 2, 19, 4, 2, 72, 72, 24, True, True, True, True, "fused"),
    "f32_d256": ("f32", 1, 21, 3, 1, 256, 256, 256, False, True, True, True, "fused"),
    "bf16_d256_part": ("bf16", 1, 21, 3, 3, 256, 128, 64, False, True, True, True, "fused"),
    "bf16_no_norm": ("bf16", 2, 23, 4, 2, 128, 128, 128, False, False, False, True, "fused"),
    "f16_norm_q_only": ("f16", 2, 23, 4, 2, 64, 64, 64, False, True, False, True, "fused"),
    "bf16_norm_k_only_no_v": ("bf16", 2, 23, 4, 2, 64, 64, 64, False, False, True, False, "fused"),
    "bf16_no_rot": ("bf16", 2, 23, 4, 2, 128, 128, 0, False, True, True, True, "fused"),
    "f32_odd_widths": ("f32", 2, 13, 4, 2, 3, 5, 2, False, True, True, True, "fused"),
    "bf16_odd_widths_pairs": ("bf16", 1, 13, 2, 2, 37, 11, 22, True, True, True, True, "fused"),
    "f16_rot_of_no_chunk": ("f16", 1, 13, 2, 2, 64, 64, 20, False, True, True, True, "fused"),
    "bf16_odd_distance": ("bf16", 2, 31, 4, 2, 64, 64, 64, False, True, True, True, "odd"),
    "bf16_one_token": ("bf16", 1, 1, 32, 8, 128, 128, 128, False, True, True, True, "fused"),
    "bf16_one_token_each": ("bf16", 5, 1, 3, 1, 128, 128, 128, False, True, True, True, "apart"),
    "bf16_width_one": ("bf16", 2, 5, 2, 1, 1, 1, 0, False, True, True, True, "fused"),
    "bf16_many_tokens": ("bf16", 2, 1500, 9, 3, 128, 128, 128, False, True, True, True, "fused"),
}


def make(name):
    dtype, B, N, H, Hkv, DK, DV, rot, il, nq, nk, wv, layout = CASES[name]
    dt = DT[dtype]
    g = torch.Generator().manual_seed(sum(map(ord, name)))
    widths = [H * DK, Hkv * DK, Hkv * DV if wv else 0]
    rows = lambda w: torch.randn((B, N, w), generator=g).to(dt).cuda()
    if layout == "fused":
        parts = list(rows(sum(widths)).split(widths, -1))
    elif layout == "odd":  # rows 3 elements longer than what they hold: no row but the first is aligned
        parts = [rows(w + 3)[..., :w] for w in widths]
    else:
        parts = [rows(w) for w in widths]
    q, k = parts[0].unflatten(-1, (H, DK)), parts[1].unflatten(-1, (Hkv, DK))
    v = parts[2].unflatten(-1, (Hkv, DV)) if wv else None
    weight = lambda on: (1 + 0.3 * torch.randn((DK,), generator=g)).to(dt).cuda() if on else None
    cos, sin = tables(2 * N + 3, rot)
    pos = (torch.randint(0, N + 3, (B, 1), generator=g) + torch.arange(N)).to(torch.int32)
    return dict(q=q, k=k, v=v, wq=weight(nq), wk=weight(nk), cos=cos.cuda() if rot else None,
                sin=sin.cuda() if rot else None, pos=pos.cuda(), il=il, dt=dt, rot=rot, gen=g)


def at(x):
    """cos, sin in 64 bits on the CPU, broadcast over heads: (B, N, 1, rot/2)."""
    if not x["rot"]:
        z = torch.zeros(x["pos"].shape + (1, 0), dtype=torch.float64)
        return z, z
    p = x["pos"].cpu().long()
    return x["cos"].cpu().double()[p][:, :, None], x["sin"].cpu().double()[p][:, :, None]


def cpu(t):
    return None if t is None else t.cpu()


def close(got, want, bound, dt, what):
    """|got - want| <= the bound and the final rounding (of the value or, at
    the bottom of the type's range, of its smallest step)."""
    got = got.double().cpu()
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    room = bound + half_step(dt) * (want.abs() + bound) + tiny
    over = ((got - want).abs() / room).max().item()
    assert math.isfinite(over) and over <= 1.0, f"{what}: {over:.3f} of the bound"


# ------------------------------------------------------------------ refusals (CPU)


def rope_dims(**kw):
    d = dict(B=2, N=10, H=4, Hkv=2, DK=64, DV=64, rot=64, P=10, ldq=512, ldk=512, ldv=512, ldgq=512, ldgk=512, ldgv=512)
    d.update(kw)
    return binding.fab_rope_dims(*[d[n] for n, _ in binding.fab_rope_dims._fields_])


A = 1 << 20  # an address that is never read: every call below is refused


def call_forward(dims, q=A, k=A, v=A, wq=A, wk=A, cos=A, sin=A, pos=A, eps=1e-6, dtype=1, qo=A, ko=A, vo=A):
    return binding.lib().fab_qk_norm_rope(q, k, v, wq, wk, cos, sin, pos, eps, 0, dtype, ctypes.byref(dims), qo, ko,
                                          vo, None)


def call_backward(dims, dq=A, dk=A, dv=A, q=A, k=A, wq=A, wk=A, cos=A, sin=A, pos=A, eps=1e-6, dtype=1, ws=A,
                  wsb=1 << 40, gq=A, gk=A, gv=A, gwq=A, gwk=A):
    return binding.lib().fab_qk_norm_rope_backward(dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, 0, dtype,
                                                   ctypes.byref(dims), ws, wsb, gq, gk, gv, gwq, gwk, None)


BAD_DIMS = [dict(B=0), dict(N=0), dict(N=-1), dict(H=3), dict(Hkv=0), dict(DK=0), dict(DV=0), dict(rot=-2),
            dict(rot=63), dict(rot=66), dict(P=0), dict(ldq=255), dict(ldk=127), dict(ldv=127), dict(ldq=1 << 60),
            dict(B=1 << 30, N=1 << 30), dict(P=1 << 31), dict(B=1, N=1, H=1 << 31, DK=8, DV=8, rot=8, ldq=1 << 35)]


@pytest.mark.parametrize("bad", BAD_DIMS, ids=str)
def test_forward_refuses_dims(bad):
    assert call_forward(rope_dims(**bad)) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(ldgq=255), dict(ldgk=0), dict(ldgv=127), dict(ldq=0), dict(rot=5), dict(N=0)],
                         ids=str)
def test_backward_refuses_dims(bad):
    assert call_backward(rope_dims(**bad)) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=None), dict(vo=None), dict(qo=None), dict(ko=A + 8),
                                 dict(q=A + 1), dict(cos=None), dict(sin=A + 2), dict(pos=A + 2), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=3), dict(wq=A + 1)],
                         ids=str)
def test_forward_refuses_arguments(bad):
    assert call_forward(rope_dims(), **bad) == binding.FAB_ERR_INVALID


def test_forward_without_positions_needs_a_table_as_long():
    assert call_forward(rope_dims(P=9), pos=None) == binding.FAB_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(dq=None), dict(dk=A + 4), dict(dv=None), dict(gv=None), dict(gq=A + 1),
                                 dict(q=None), dict(k=A + 1), dict(gwq=None), dict(wq=None), dict(gwk=A + 4),
                                 dict(eps=-0.5), dict(dtype=-1)], ids=str)
def test_backward_refuses_arguments(bad):
    assert call_backward(rope_dims(), **bad) == binding.FAB_ERR_INVALID


def test_backward_refuses_a_short_workspace():
    need = binding.fab_qk_norm_rope_backward_workspace_bytes(rope_dims())
    assert need > 0 and binding.fab_qk_norm_rope_backward_workspace_bytes(rope_dims(H=3)) == 0
    assert call_backward(rope_dims(), wsb=need - 1) == binding.FAB_ERR_WORKSPACE
    assert call_backward(rope_dims(), ws=None) == binding.FAB_ERR_WORKSPACE


def test_widths_past_256_are_unsupported():
    wide = rope_dims(DK=264, DV=264, ldq=4096, ldk=4096, ldv=4096, ldgq=4096, ldgk=4096, ldgv=4096)
    assert call_forward(wide) == binding.FAB_ERR_UNSUPPORTED
    assert call_backward(wide) == binding.FAB_ERR_UNSUPPORTED


def test_binding_refuses_what_does_not_fit():
    q, k, v = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 2, 64)
    for args in ((q, k, v), (q[0], k, v), (q, k[0], v)):  # CPU tensors, ranks
        with pytest.raises(ValueError):
            binding.qk_norm_rope(*args)
    with pytest.raises(ValueError):
        binding.qk_norm_rope_backward(q[0], k, v, q, k)
    with pytest.raises(ValueError):
        binding.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2), None, q, k)


# ------------------------------------------------------------------ GPU


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()
    yield
    assert binding.fab_last_device_error() == binding.FAB_OK


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_forward(gpu, name):
    x = make(name)
    got = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], 1e-6, x["il"])
    cos, sin = at(x)
    for key, y, w in (("q", got[0], x["wq"]), ("k", got[1], x["wk"])):
        want, bound = ref_forward(cpu(x[key]), cpu(w), cos, sin, x["il"], 1e-6)
        close(y, want.movedim(2, 1), bound.movedim(2, 1), x["dt"], key)
    if x["v"] is None:
        assert got[2] is None
    else:
        assert torch.equal(got[2], x["v"].transpose(1, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_backward(gpu, name):
    x = make(name)
    B, N, H, DK = x["q"].shape
    Hkv = x["k"].shape[2]
    draw = lambda *s: torch.randn(s, generator=x["gen"]).cuda()
    dq, dk = draw(B, H, N, DK), draw(B, Hkv, N, DK)
    dv = None if x["v"] is None else draw(B, Hkv, N, x["v"].shape[3])
    args = (dq, dk, dv, x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], 1e-6, x["il"])
    gq, gk, gv, gwq, gwk = binding.qk_norm_rope_backward(*args)
    cos, sin = at(x)
    for key, dy, g, w, gw in (("q", dq, gq, x["wq"], gwq), ("k", dk, gk, x["wk"], gwk)):
        want, bound, dw, terms = ref_backward(dy.cpu().movedim(1, 2), cpu(x[key]), cpu(w), cos, sin, x["il"], 1e-6)
        close(g, want, bound, x["dt"], "g" + key)
        if w is None:
            assert gw is None
            continue
        # each term carries the f32 error of g r x; a column's terms are added
        # in chains of at most rows / 8 and a tree
        rows = B * N * (H if key == "q" else Hkv)
        room = (64 + rows / 8) * U32 * terms
        assert ((gw.double().cpu() - dw).abs() <= room).all(), "gw" + key
    if dv is None:
        assert gv is None
    else:
        assert torch.equal(gv, dv.transpose(1, 2).to(x["dt"]))
    again = binding.qk_norm_rope_backward(*args)
    for a, b in zip((gq, gk, gv, gwq, gwk), again):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.gpu
def test_gradient_against_differences(gpu):
    # d/dt sum(dy * forward(x + t e)) by central differences of the 64-bit
    # formula, for random directions, against the kernel's f32 gradient
    x = make("f32_d64_pairs")
    cos, sin = at(x)
    dq, dk = torch.randn_like(x["q"].transpose(1, 2)).contiguous(), torch.randn_like(x["k"].transpose(1, 2)).contiguous()
    gq, gk, _, gwq, gwk = binding.qk_norm_rope_backward(dq, dk, None, x["q"], x["k"], x["wq"], x["wk"], x["cos"],
                                                        x["sin"], x["pos"], 1e-6, x["il"])
    for xx, w, dy, g, gw in ((x["q"], x["wq"], dq, gq, gwq), (x["k"], x["wk"], dk, gk, gwk)):
        xd, wd, dyd = xx.cpu().double(), w.cpu().double(), dy.cpu().double().movedim(1, 2)
        f = lambda a, b: (ref_forward(a, b, cos, sin, x["il"], 1e-6)[0] * dyd).sum().item()
        h = 1e-5
        for trial in range(3):
            e = torch.randn(xd.shape, generator=x["gen"], dtype=torch.float64)
            slope = (f(xd + h * e, wd) - f(xd - h * e, wd)) / (2 * h)
            ours = (g.cpu().double() * e).sum().item()
            # differences: h^2 of the third derivative, about 1e-9 of the terms; f32: 64 half steps of them
            size = (g.cpu().double() * e).abs().sum().item()
            assert abs(slope - ours) <= 1e-5 * size
            e = torch.randn(wd.shape, generator=x["gen"], dtype=torch.float64)
            slope = (f(xd, wd + h * e) - f(xd, wd - h * e)) / (2 * h)
            ours = (gw.cpu().double() * e).sum().item()
            terms = (dyd.abs().sum().item())
            assert abs(slope - ours) <= 1e-5 * terms


@pytest.mark.gpu
def test_a_position_out_of_the_tables_is_reported(gpu):
    x = make("bf16_d128")
    pos = x["pos"].clone()
    pos[1, 3], pos[0, 5] = x["cos"].shape[0], -1
    q, k, v = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], pos)
    assert binding.fab_last_device_error() == binding.FAB_ERR_INVALID
    want = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"])
    for a, b in zip((q, k, v), want):  # every other token is as ever
        keep = torch.ones(a.shape[0], a.shape[2], dtype=torch.bool)
        keep[1, 3] = keep[0, 5] = False
        assert torch.equal(a.transpose(1, 2).cpu()[keep], b.transpose(1, 2).cpu()[keep])


@pytest.mark.gpu
def test_operands_that_do_not_match_are_refused(gpu):
    x = make("bf16_d128")
    a = dict(q=x["q"], k=x["k"], v=x["v"], wq=x["wq"], wk=x["wk"], cos=x["cos"], sin=x["sin"], pos=x["pos"])
    for bad in (dict(k=x["k"].half()), dict(k=x["k"][:, :5]), dict(v=x["v"][:1]), dict(wq=x["wq"].float()),
                dict(wq=x["wq"][:5]), dict(cos=x["cos"].double()), dict(sin=None), dict(sin=x["sin"][:5]),
                dict(pos=x["pos"].long()), dict(pos=x["pos"][:, :5]), dict(pos=x["pos"].cpu()),
                dict(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2)),  # heads apart
                dict(q=x["q"][:, :1].expand_as(x["q"])),                      # one row for all tokens
                dict(cos=x["cos"][:, :3], sin=x["sin"][:, :3].contiguous())):
        with pytest.raises((ValueError, binding.FabError)):
            binding.qk_norm_rope(**{**a, **bad})


@pytest.mark.gpu
def test_many_heads(gpu):
    # more blocks of heads than a grid's second dimension holds at first
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((1, 1, 300000, 8), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((1, 1, 2, 8), generator=g, device="cuda").to(torch.bfloat16)
    qo, ko, _ = binding.qk_norm_rope(q, k, None)
    assert torch.equal(qo[:, :, 0], q[:, 0]) and torch.equal(ko[:, :, 0], k[:, 0])


@pytest.mark.gpu
def test_default_positions_and_a_side_stream(gpu):
    x = make("f16_d64")
    B, N = x["pos"].shape
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    a = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], None, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.gpu
def test_only_the_heads_columns_are_written(gpu):
    # gradients into rows that hold other values too
    x = make("bf16_d128")
    B, N, H, DK = x["q"].shape
    Hkv = x["k"].shape[2]
    draw = lambda *s: torch.randn(s, generator=x["gen"]).cuda()
    dq, dk, dv = draw(B, H, N, DK), draw(B, Hkv, N, DK), draw(B, Hkv, N, DK)
    want = binding.qk_norm_rope_backward(dq, dk, dv, x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"])
    for gap in (5, 8):  # rows at odd places, and aligned ones
        wide = [torch.full((B, N, h * DK + gap), 7.0, dtype=x["dt"], device="cuda") for h in (H, Hkv, Hkv)]
        g = [w[..., : w.shape[2] - gap].unflatten(-1, (-1, DK)) for w in wide]
        gw = [torch.empty(DK, device="cuda") for _ in range(2)]
        ws = torch.empty(binding.fab_qk_norm_rope_backward_workspace_bytes(rope_dims(DK=DK)), dtype=torch.uint8,
                         device="cuda")
        binding.fab_qk_norm_rope_backward(dq, dk, dv, x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"],
                                          1e-6, False, ws, *g, *gw)
        for a, b, w in zip(g, want, wide):
            assert (w[..., w.shape[2] - gap:] == 7).all()
            # another kernel may take these rows: both are within a rounding of the formula
            d = (a.double() - b.double()).abs()
            assert (d <= 2 * torch.finfo(x["dt"]).eps * b.double().abs() + 1e-5).all()


@pytest.mark.gpu
def test_norm_rope_attention_and_back(gpu):
    # a projection through norm, rotation, attention and all the way back,
    # against the same in 64 bits by autograd
    x = make("f32_d64_pairs")
    B, N, H, DK = x["q"].shape
    q, k, v = binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], 1e-6, x["il"])
    o, lse = binding.forward(q, k, v, None, True, 0.125)
    d = torch.randn(o.shape, generator=x["gen"]).cuda()
    packed = binding.backward(q, k, v, d, o, lse, None, True, 0.125)
    dq, dk, dv = binding.unpack(packed, binding.dims_of(q, k, v))
    got = binding.qk_norm_rope_backward(dq, dk, dv, x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"],
                                        1e-6, x["il"])
    leaves = [t.cpu().double().requires_grad_() for t in (x["q"], x["k"], x["v"], x["wq"], x["wk"])]
    cos, sin = at(x)
    Q = ref_forward(leaves[0], leaves[3], cos, sin, x["il"], 1e-6)[0].transpose(1, 2)
    K = ref_forward(leaves[1], leaves[4], cos, sin, x["il"], 1e-6)[0].transpose(1, 2).repeat_interleave(H // x["k"].shape[2], 1)
    V = leaves[2].transpose(1, 2).repeat_interleave(H // x["k"].shape[2], 1)
    s = (0.125 * Q @ K.transpose(2, 3)).masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    O = (s.softmax(-1) @ V).transpose(1, 2)
    (O * d.cpu().double()).sum().backward()
    for a, leaf in zip(got, leaves):
        err = (a.double().cpu() - leaf.grad).abs().max() / leaf.grad.abs().max()
        # f32 throughout: some hundreds of half steps over sums of 17 keys and 64 columns
        assert err <= 2e-5, err


@pytest.mark.gpu
def test_captured_and_replayed(gpu):
    x = make("bf16_d128")
    B, N, H, DK = x["q"].shape
    Hkv = x["k"].shape[2]
    dq = torch.randn(B, H, N, DK, device="cuda")
    dk = torch.randn(B, Hkv, N, DK, device="cuda")
    run = lambda: (binding.qk_norm_rope(x["q"], x["k"], x["v"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"]),
                   binding.qk_norm_rope_backward(dq, dk, None, x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"],
                                                 x["pos"]))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(2):
        x["q"].normal_()
        x["pos"].copy_(torch.randint(0, x["cos"].shape[0], x["pos"].shape))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip((*out[0], *out[1]), (*want[0], *want[1])):
            assert a is b is None or torch.equal(a, b)
