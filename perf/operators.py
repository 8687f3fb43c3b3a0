"""Workloads of the operators around the attention: query/key norms with the
position rotation (forward and gradient), appending to a paged key/value
cache, and attention over that cache.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges,
``prepare(case, seed)`` builds what a program holds before the call and
``run(state)`` makes one pass: in elementary torch operations in 32 bits, or,
where ``own`` is true, through the library.  ``exact(case, seed)`` computes the
same outputs in 64 bits and ``work(case)`` counts what a pass cannot do without.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # the projection of one training step of the grouped-query causal
        # workload (4 sequences of 2048 tokens, 32 query and 8 key heads)
        dict(name="norm_rope_train", op="norm_rope", dtype="bf16", B=4, N=2048, H=32, Hkv=8, DK=128, DV=128, rot=128,
             interleaved=False, norm=True),
        # the library's smallest workload: one f32 head of 128 tokens, adjacent
        # pairs rotated; launch latency
        dict(name="norm_rope_tiny", op="norm_rope", dtype="f32", B=1, N=128, H=1, Hkv=1, DK=64, DV=64, rot=64,
             interleaved=True, norm=True),
        # the gradient of norm_rope_train, from the packed f32 result of the
        # attention backward to the gradient of the projection
        dict(name="norm_rope_grad_train", op="norm_rope_grad", dtype="bf16", B=4, N=2048, H=32, Hkv=8, DK=128, DV=128,
             rot=128, interleaved=False, norm=True),
        # an odd length, a head width that is no power of two and a partial
        # rotation, as small models have
        dict(name="norm_rope_grad_odd", op="norm_rope_grad", dtype="f16", B=3, N=777, H=12, Hkv=4, DK=80, DV=80,
             rot=32, interleaved=False, norm=True),
        # one token for each of 64 sequences: a decoding step
        dict(name="append_decode", op="append", dtype="bf16", B=64, H=32, Hkv=8, DK=128, DV=128, rot=128, page=16,
             new_lo=1, new_hi=1, past_lo=0, past_hi=2047, ragged=1, interleaved=False, norm=True),
        # prompts of odd lengths entering the cache, 8 sequences at once
        dict(name="append_prompts", op="append", dtype="f16", B=8, H=16, Hkv=16, DK=64, DV=64, rot=64, page=64,
             new_lo=200, new_hi=1999, past_lo=0, past_hi=500, ragged=2, interleaved=False, norm=False),
        # a decoding step of 64 sequences of unequal length
        dict(name="decode_batch", op="attention", dtype="bf16", B=64, H=32, Hkv=8, DK=128, DV=128, page=16,
             new_lo=1, new_hi=1, past_lo=64, past_hi=4095, ragged=3, causal=True),
        # one sequence with a very long cache: the split of one row's keys
        dict(name="decode_long", op="attention", dtype="bf16", B=1, H=32, Hkv=8, DK=128, DV=128, page=64,
             new_lo=1, new_hi=1, past_lo=131000, past_hi=131000, ragged=4, causal=True),
        # one short sequence: launch latency
        dict(name="decode_short", op="attention", dtype="f16", B=1, H=8, Hkv=8, DK=64, DV=64, page=16,
             new_lo=1, new_hi=1, past_lo=499, past_hi=499, ragged=5, causal=True),
        # chunks of a long prompt over what is cached already: matrix products
        dict(name="chunk_long", op="attention", dtype="bf16", B=2, H=32, Hkv=8, DK=128, DV=128, page=128,
             new_lo=2048, new_hi=2048, past_lo=14336, past_hi=14336, ragged=6, causal=True),
        # single tokens and chunks of odd lengths in one batch
        dict(name="chunk_mixed", op="attention", dtype="f16", B=24, H=16, Hkv=4, DK=64, DV=64, page=32,
             new_lo=1, new_hi=500, past_lo=0, past_hi=3500, ragged=7, causal=True),
        # 32-bit values and a head width of 80, every key visible
        dict(name="chunk_f32", op="attention", dtype="f32", B=6, H=8, Hkv=2, DK=80, DV=80, page=24,
             new_lo=1, new_hi=40, past_lo=0, past_hi=1000, ragged=8, causal=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "attention", "attention", "attention"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 7, 8]) if op == "attention" else Hkv * rng.choice([1, 2, 3, 4])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm_rope", "norm_rope_grad", "append"):
        D = rng.choice([64, 80, 96, 128])
        c = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, DK=D, DV=D, rot=rng.choice([D, D, 32]),
                 interleaved=rng.random() < 0.3, norm=rng.random() < 0.8)
        if op != "append":
            return dict(c, B=rng.randint(1, 4), N=_spread(rng, 1, 2048))
        new = _spread(rng, 1, 1000)
        return dict(c, B=_spread(rng, 1, 64) if new < 50 else rng.randint(1, 8), page=rng.choice([16, 32, 64, 128]),
                    new_lo=max(1, new // 3), new_hi=new, past_lo=0, past_hi=_spread(rng, 1, 2000),
                    ragged=rng.randint(0, 1 << 30))
    D = rng.choice([64, 128, 128, 80] if dtype != "f32" else [64, 80, 128])
    c = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, DK=D, DV=D, page=rng.choice([16, 16, 24, 32, 64, 128]),
             causal=rng.random() < 0.8, ragged=rng.randint(0, 1 << 30))
    shape = rng.choice(["decode", "decode", "chunk"])
    if shape == "decode":
        B = _spread(rng, 1, 64)
        past = _spread(rng, 1, 100000 if B == 1 else 30000 if B < 8 else 4000)
        return dict(c, B=B, new_lo=1, new_hi=rng.choice([1, 1, 1, 4]), past_lo=past // 10, past_hi=past)
    new = _spread(rng, 2, 1500 if dtype != "f32" else 60)
    past = _spread(rng, 1, 8000 if dtype != "f32" else 2000)
    return dict(c, B=rng.randint(1, 4 if H <= 16 else 2), new_lo=max(1, new // 4), new_hi=new, past_lo=past // 4,
                past_hi=past)


def _lengths(case):
    """New tokens and tokens held after them, of each sequence."""
    r = random.Random(case["ragged"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return new, [n + r.randint(case["past_lo"], case["past_hi"]) for n in new]


def _tables(length, rot, device):
    """Cosines and sines of every position, angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return a.cos().float(), a.sin().float()


def _cache(case, total, g, draw_values):
    """Caches, page table and lengths: pages in no order, two spare ones."""
    page, need = case["page"], [-(-t // case["page"]) for t in total]
    width = max(need)
    count = sum(need) + 2
    order = torch.randperm(count, generator=g, device="cuda")
    table = torch.zeros((case["B"], width), dtype=torch.int32, device="cuda")
    used = torch.tensor(need, device="cuda")
    live = torch.arange(width, device="cuda") < used[:, None]
    table.masked_scatter_(live, order[: sum(need)].to(torch.int32))
    k = draw_values((count, case["Hkv"], page, case["DK"]))
    v = draw_values((count, case["Hkv"], page, case["DV"]))
    return k, v, table, torch.tensor(total, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    H, Hkv, DK, DV = case["H"], case["Hkv"], case["DK"], case["DV"]

    def normal(shape, t=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    def projection(rows):
        # one row of the projection holds the token's queries, keys and values
        x = normal((*rows, H * DK + Hkv * DK + Hkv * DV))
        q, k, v = x.split([H * DK, Hkv * DK, Hkv * DV], dim=-1)
        return q.unflatten(-1, (H, DK)), k.unflatten(-1, (Hkv, DK)), v.unflatten(-1, (Hkv, DV))

    s = dict(case=case)
    if case["op"] != "attention":
        s["wq"] = (1 + 0.2 * normal((DK,), torch.float32)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * normal((DK,), torch.float32)).to(dt) if case["norm"] else None
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        B, N = case["B"], case["N"]
        s["q"], s["k"], s["v"] = projection((B, N))
        s["cos"], s["sin"] = _tables(2 * N + 7, case["rot"], "cuda")
        # sequences start at positions of their own
        start = torch.randint(0, N + 7, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        if case["op"] == "norm_rope_grad":
            # slices of one packed f32 buffer, as the attention backward leaves them
            sizes = [B * H * N * DK, B * Hkv * N * DK, B * Hkv * N * DV]
            pad = [-(-n // 4) * 4 for n in sizes]
            packed = normal((sum(pad),), torch.float32)
            s["dq"] = packed[: sizes[0]].view(B, H, N, DK)
            s["dk"] = packed[pad[0]: pad[0] + sizes[1]].view(B, Hkv, N, DK)
            s["dv"] = packed[pad[0] + pad[1]: pad[0] + pad[1] + sizes[2]].view(B, Hkv, N, DV)
        return s
    new, total = _lengths(case)
    s["k_cache"], s["v_cache"], s["table"], s["lens"] = _cache(case, total, g, normal)
    ends = torch.tensor([0] + new).cumsum(0)
    s["starts"] = ends.to(torch.int32).cuda()
    s["T"], s["most_new"], s["most_keys"] = sum(new), max(new), max(total)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = projection((s["T"],))
        s["cos"], s["sin"] = _tables(s["most_keys"], case["rot"], "cuda")
    else:
        s["q"] = normal((s["T"], H, DK))
        s["scale"] = DK ** -0.5
    return s


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


def _plain_norm_rope(s):
    il, dt = s["case"]["interleaved"], s["q"].dtype
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    q = _turn(_norm(s["q"].float(), s["wq"]), cos, sin, il).to(dt).transpose(1, 2).contiguous()
    k = _turn(_norm(s["k"].float(), s["wk"]), cos, sin, il).to(dt).transpose(1, 2).contiguous()
    return q, k, s["v"].transpose(1, 2).contiguous()


def _plain_norm_grad(dy, x, w, cos, sin, il):
    """Gradient of one operand's rows (dy as the output, x as the input) and of its weights."""
    g = _turn(dy.transpose(1, 2), cos, -sin, il)
    if w is None:
        return g.to(x.dtype), None
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    xr = xf * r
    u = g * w.float()
    dx = r * (u - xr * (u * xr).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xr).sum((0, 1, 2))


def _plain_norm_rope_grad(s):
    il = s["case"]["interleaved"]
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    gq, dwq = _plain_norm_grad(s["dq"], s["q"], s["wq"], cos, sin, il)
    gk, dwk = _plain_norm_grad(s["dk"], s["k"], s["wk"], cos, sin, il)
    gv = s["dv"].transpose(1, 2).to(s["v"].dtype).contiguous()
    return gq, gk, gv, dwq, dwk


def _plain_append(s):
    il, page, dt = s["case"]["interleaved"], s["case"]["page"], s["q"].dtype
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), new, output_size=s["T"])
    at = torch.arange(s["T"], device=lens.device) - starts[seq] + (lens - new)[seq]
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _turn(_norm(s["q"].float(), s["wq"]), cos, sin, il).to(dt)
    k = _turn(_norm(s["k"].float(), s["wk"]), cos, sin, il).to(dt)
    where = s["table"][seq, at // page].long()
    s["k_cache"][where, :, at % page] = k
    s["v_cache"][where, :, at % page] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    B, H, Hkv, DK, DV, page = c["B"], c["H"], c["Hkv"], c["DK"], c["DV"], c["page"]
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(s["most_new"], device=lens.device)
    token = (starts[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][token].float().view(B, s["most_new"], Hkv, H // Hkv, DK)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, DK)
    pages = s["table"].long()
    L = pages.shape[1] * page
    m = torch.arange(L, device=lens.device)
    held = (m < lens[:, None])[:, None, :, None]
    k = s["k_cache"][pages].float().transpose(1, 2).reshape(B, Hkv, L, DK)
    v = s["v_cache"][pages].float().transpose(1, 2).reshape(B, Hkv, L, DV).masked_fill(~held, 0.0)
    last = (lens - new)[:, None] + i if c["causal"] else (lens - 1)[:, None].expand(B, s["most_new"])
    seen = (m <= last[:, :, None]) & (m < lens[:, None, None])
    seen = seen[:, None, :, None].expand(B, 1, s["most_new"], H // Hkv, L).reshape(B, 1, -1, L)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = ((x @ v) / total).view(B, Hkv, s["most_new"], H // Hkv, DV).permute(0, 2, 1, 3, 4)
    lse = (top + total.log()).view(B, Hkv, s["most_new"], H // Hkv).permute(0, 2, 1, 3)
    seq = torch.repeat_interleave(torch.arange(B, device=lens.device), new, output_size=s["T"])
    row = torch.arange(s["T"], device=lens.device) - starts[seq]
    o = o[seq, row].reshape(s["T"], H, DV).to(s["q"].dtype)
    return o, lse[seq, row].reshape(s["T"], H).t().contiguous()


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        plain = {"norm_rope": _plain_norm_rope, "norm_rope_grad": _plain_norm_rope_grad, "append": _plain_append,
                 "attention": _plain_attention}
        return plain[op](s)
    from attention_backward_tcgen05_gb300 import binding

    if op == "norm_rope":
        return binding.qk_norm_rope(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS,
                                    s["case"]["interleaved"])
    if op == "norm_rope_grad":
        return binding.qk_norm_rope_backward(s["dq"], s["dk"], s["dv"], s["q"], s["k"], s["wq"], s["wk"], s["cos"],
                                             s["sin"], s["pos"], EPS, s["case"]["interleaved"])
    if op == "append":
        q = binding.paged_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["starts"],
                                 s["lens"], s["table"], s["k_cache"], s["v_cache"], EPS, s["case"]["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    return binding.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["starts"], s["lens"], s["table"],
                                   s["case"]["causal"], s["scale"])


def _exact_rows(x, w, cos, sin, interleaved, back=None):
    """Rows x in 64 bits, normalised and rotated as complex pairs; with `back`,
    the gradients of x and w for that gradient of the result."""
    x = x.double()
    rot = 2 * cos.shape[-1]
    turn = torch.complex(cos.double(), sin.double())

    def rotate(y, by):
        a = y[..., :rot]
        if interleaved:
            z = torch.view_as_complex(a.unflatten(-1, (-1, 2)).contiguous()) * by
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(a[..., : rot // 2].contiguous(), a[..., rot // 2:].contiguous()) * by
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, y[..., rot:]], -1)

    if w is not None:
        length = ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        unit = x / length
    if back is None:
        return rotate(x if w is None else unit * w.double(), turn)
    g = rotate(back.double(), turn.conj())
    if w is None:
        return g, None
    gw = g * w.double()
    inner = (gw * unit).sum(-1, keepdim=True) / x.shape[-1]
    return (gw - unit * inner) / length, (g * unit).flatten(0, -2).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        cos, sin = (t[s["pos"].long()].unsqueeze(2) for t in (s["cos"], s["sin"]))
        il = case["interleaved"]
        if case["op"] == "norm_rope":
            q = _exact_rows(s["q"], s["wq"], cos, sin, il).movedim(2, 1)
            k = _exact_rows(s["k"], s["wk"], cos, sin, il).movedim(2, 1)
            return q, k, s["v"].double().movedim(2, 1)
        gq, dwq = _exact_rows(s["q"], s["wq"], cos, sin, il, s["dq"].movedim(1, 2))
        gk, dwk = _exact_rows(s["k"], s["wk"], cos, sin, il, s["dk"].movedim(1, 2))
        return gq, gk, s["dv"].double().movedim(1, 2), dwq, dwk
    new, total = _lengths(case)
    page, G = case["page"], case["H"] // case["Hkv"]
    table = s["table"].cpu()
    if case["op"] == "append":
        at = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).cuda()
        cos, sin = s["cos"][at].unsqueeze(1), s["sin"][at].unsqueeze(1)
        q = _exact_rows(s["q"], s["wq"], cos, sin, case["interleaved"])
        k = _exact_rows(s["k"], s["wk"], cos, sin, case["interleaved"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        t0 = 0
        for b, (n, t) in enumerate(zip(new, total)):
            p = torch.arange(t - n, t)
            slot = (table[b][p // page].long().cuda(), slice(None), (p % page).cuda())
            kc[slot] = k[t0: t0 + n]
            vc[slot] = s["v"][t0: t0 + n].double()
            t0 += n
        return q, kc, vc
    o = torch.empty((s["T"], case["H"], case["DV"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((case["H"], s["T"]), dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, t) in enumerate(zip(new, total)):
        at = table[b][: -(-t // page)].long().cuda()
        last = torch.arange(t - n, t, device="cuda") if case["causal"] else torch.full((n,), t - 1, device="cuda")
        hidden = torch.arange(t, device="cuda") > last[:, None]
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


def work(case):
    e, H, Hkv, DK, DV = _SIZE[case["dtype"]], case["H"], case["Hkv"], case["DK"], case["DV"]
    heads = H * DK + Hkv * DK  # normalised and rotated values of a token
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        T = case["B"] * case["N"]
        table = min(T, 2 * case["N"] + 7) * case["rot"] * 4 + T * 4
        if case["op"] == "norm_rope":
            return dict(bytes=2 * T * (heads + Hkv * DV) * e + table, flops=10 * T * heads)
        read = T * (heads + Hkv * DV) * 4 + (T * heads * e if case["norm"] else 0)
        return dict(bytes=read + T * (heads + Hkv * DV) * e + table, flops=20 * T * heads)
    new, total = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        table = min(T, max(total)) * case["rot"] * 4 + 8 * case["B"] + 4 * T
        return dict(bytes=2 * T * (heads + Hkv * DV) * e + table, flops=10 * T * heads)
    held = sum(total)
    if case["causal"]:
        pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
    else:
        pairs = sum(n * t for n, t in zip(new, total))
    nbytes = held * Hkv * (DK + DV) * e + T * H * (DK + DV) * e + T * H * 4
    nbytes += sum(-(-t // case["page"]) for t in total) * 4
    return dict(bytes=nbytes, flops=2 * pairs * H * (DK + DV))
