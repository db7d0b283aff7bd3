"""The operators of a block with rotary positions, as cases to be measured.

Residual addition with LayerNorm (a gain and a bias of the model's or of each batch item's own) and
its backward; rotary positions on several axes, with or without the QK-RMSNorm before them, and their
backward; attention of packed sequences with grouped heads, causal or full, and its backward.  With
``own`` false ``run`` computes them from elementary torch operations in 32 bits (angles in 64); with
``own`` true it calls the library."""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one token of each of 8 requests through a 768-wide block: latency
        dict(name="ln_8_tokens", op="ln", items=1, rows=8, C=768, res=True, bias=True),
        # a 512 px training step's image and caption tokens, modulated by each item's own scale and shift
        dict(name="ln_512px", op="ln", items=16, rows=1101, C=768, res=True, bias=True),
        # backward of a first block's norm (no gradient from a later path, no bias), odd sizes
        dict(name="ln_bwd_333", op="ln_bwd", items=1, rows=333, C=1096, dh=False, bias=False),
        # a wide model's long batch, backward: the largest pass over memory
        dict(name="ln_bwd_wide", op="ln_bwd", items=1, rows=32768, C=4096, dh=True, bias=True),
        # one new token of each of 32 requests, far into their sequences, grouped heads: latency
        dict(name="rope_32_tokens", op="rope", B=32, Hq=16, Hk=4, N=1, d=128, pairs="64", norm=False,
             interleaved=False, per_item=True, far=1000000),
        # a 512 px training step, height and width, with the QK-RMSNorm
        dict(name="rope_512px", op="rope", B=16, Hq=12, Hk=12, N=1101, d=64, pairs="16,16", norm=True,
             interleaved=True, per_item=False, far=32),
        # backward of plain rotary positions of one packed batch of videos (time, height, width), grouped heads
        dict(name="rope_bwd_video", op="rope_bwd", B=1, Hq=8, Hk=2, N=4033, d=128, pairs="8,28,28", norm=False,
             interleaved=True, per_item=False, far=64),
        # backward of a 768 px step with the QK-RMSNorm and its gains' gradients: the largest
        dict(name="rope_bwd_768px", op="rope_bwd", B=4, Hq=24, Hk=24, N=2381, d=128, pairs="16,24,24", norm=True,
             interleaved=False, per_item=True, far=48),
        # the captions of a batch through a causal text tower: 16 x 77 tokens
        dict(name="attn_captions", op="attn", lens=",".join(["77"] * 16), Hq=12, Hk=12, d=64, causal=True),
        # prompts of very different lengths in one batch, grouped heads: the largest product
        dict(name="attn_prompts", op="attn", lens="16001,1,333,2381", Hq=16, Hk=4, d=128, causal=True),
        # joint sequences of several image sizes in one training batch, rotary positions, every row sees every row
        dict(name="attn_bwd_buckets", op="attn_bwd", lens="1101,333,2381,1101,1101,333,589", Hq=12, Hk=12, d=64,
             causal=False),
        # training on long documents, causal, grouped heads
        dict(name="attn_bwd_long", op="attn_bwd", lens="8192,1777", Hq=16, Hk=4, d=128, causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "rope", "rope_bwd", "attn", "attn_bwd"])
    if op in ("ln", "ln_bwd"):
        C = 8 * _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, min(32768, (1 << 27) // C))
        items = rng.choice([1, 1, rng.randint(2, 32)])
        case = dict(op=op, items=items, rows=max(1, T // items), C=C, bias=rng.random() < 0.7)
        case["res" if op == "ln" else "dh"] = rng.random() < 0.7
        return case
    d = rng.choice([64, 128])
    Hk = rng.randint(1, 12)
    Hq = Hk * rng.choice([1, 1, 2, 4])
    if op in ("rope", "rope_bwd"):
        total = rng.choice([d // 2, d // 2, 8 * rng.randint(1, d // 16)])
        axes = rng.randint(1, 3)
        cuts = sorted(rng.randint(0, total) for _ in range(axes - 1))
        pairs = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        N = _log_int(rng, 1, 4096)
        B = max(1, min(_log_int(rng, 1, 32), (1 << 26) // (N * d * (Hq + Hk))))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, N=N, d=d, pairs=",".join(map(str, pairs)), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, per_item=rng.random() < 0.5, far=_log_int(rng, 16, 1000000))
    T = _log_int(rng, 1, 8192)
    n = rng.randint(1, min(8, T))
    cuts = sorted(rng.sample(range(1, T), n - 1)) if n > 1 else []
    lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    case = dict(op=op, lens=",".join(map(str, lens)), Hq=Hq, Hk=Hk, d=d, causal=rng.random() < 0.7)
    while work(case)["flops"] > 0.9e12:
        case["Hk"], case["Hq"] = max(1, case["Hk"] // 2), max(1, case["Hk"] // 2) * (case["Hq"] // case["Hk"])
    return case


def _ints(text):
    return [int(x) for x in text.split(",")]


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op in ("ln", "ln_bwd"):
        items, rows, C = case["items"], case["rows"], case["C"]
        # a residual stream grows with depth, has a few large channels and a mean of its own
        big = 1.0 + 7.0 * (_rand(gen, C) < 0.02).float()
        stream = ((torch.randn((items, rows, C), generator=gen, device="cuda") + 0.3) * (2.0 * big)).to(torch.bfloat16)
        s["g"] = _rand(gen, items, C) + 0.5
        s["b"] = torch.randn((items, C), generator=gen, device="cuda") * 0.2 if case["bias"] else None
        if items == 1:  # the model's own gain and bias
            s["g"], s["b"] = s["g"][0], s["b"][0] if case["bias"] else None
        if op == "ln":
            s["x"] = _randn(gen, items, rows, C) if case["res"] else stream
            s["residual"] = stream if case["res"] else None
            return s
        f = stream.float()
        s["h"], s["mean"] = stream, f.mean(-1)
        s["r"] = ((f - s["mean"][..., None]).square().mean(-1) + EPS).rsqrt()
        s["dy"] = _randn(gen, items, rows, C, scale=0.1)
        s["dres"] = _randn(gen, items, rows, C, scale=0.1) if case["dh"] else None
        return s
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if op in ("rope", "rope_bwd"):
        B, N = case["B"], case["N"]
        s["axis_pairs"] = _ints(case["pairs"])
        # each axis with frequencies of its own from 1 down to 1 / 10000; positions are whole numbers
        s["freq"] = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / max(p, 1))
                               for p in s["axis_pairs"]]).float().cuda()
        shape = (B, N, len(s["axis_pairs"])) if case["per_item"] else (N, len(s["axis_pairs"]))
        s["pos"] = torch.randint(0, case["far"], shape, generator=gen, device="cuda").float()
        s["gq"], s["gk"] = (_rand(gen, d) + 0.5, _rand(gen, d) + 0.5) if case["norm"] else (None, None)
        q, k = _randn(gen, B, Hq, N, d), _randn(gen, B, Hk, N, d)
        if op == "rope":
            return dict(s, q=q, k=k)
        s["q"], s["k"] = (q, k) if case["norm"] else (None, None)
        return dict(s, dq_rot=_randn(gen, B, Hq, N, d, scale=0.1), dk_rot=_randn(gen, B, Hk, N, d, scale=0.1))
    lens = _ints(case["lens"])
    s["cu"] = [0]
    for n in lens:
        s["cu"].append(s["cu"][-1] + n)
    T = s["cu"][-1]
    s["q"], s["k"], s["v"] = _randn(gen, Hq, T, d, scale=1.5), _randn(gen, Hk, T, d), _randn(gen, Hk, T, d)
    if op == "attn_bwd":
        s["out"], s["lse"] = _attn_plain(s)
        s["dout"] = _randn(gen, Hq, T, d, scale=0.1)
    return s


def _ln_plain(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    f = h.float()
    mean = f.mean(-1)
    c = f - mean[..., None]
    r = (c.square().mean(-1) + EPS).rsqrt()
    y = c * r[..., None] * s["g"].unsqueeze(-2)
    if s["b"] is not None:
        y = y + s["b"].unsqueeze(-2)
    out = dict(y=y.to(torch.bfloat16), mean=mean, r=r)
    return out if s["residual"] is None else dict(out, h=h)


def _ln_bwd_plain(s):
    n = (s["h"].float() - s["mean"][..., None]) * s["r"][..., None]
    dy = s["dy"].float()
    u = dy * s["g"].unsqueeze(-2)
    dx = s["r"][..., None] * (u - u.mean(-1, keepdim=True) - n * (u * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = dict(dx=dx.to(torch.bfloat16), dg=(dy * n).sum(1).view(s["g"].shape))
    return dict(out, db=dy.sum(1).view(s["g"].shape)) if s["bias"] else out


def _turns(s):
    """cos and sin of every row's pairs, [B or 1, 1, N, P], from angles in 64 bits."""
    axis = [a for a, p in enumerate(s["axis_pairs"]) for _ in range(p)]
    pos = s["pos"] if s["per_item"] else s["pos"][None]
    angle = pos[..., axis].double() * s["freq"].double()
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(s, x, cos, sin):
    P = cos.shape[-1]
    out = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        out[..., 0:2 * P:2], out[..., 1:2 * P:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        out[..., :P], out[..., P:2 * P] = a * cos - b * sin, a * sin + b * cos
    return out


def _rope_plain(s):
    cos, sin = _turns(s)
    out = []
    for x, g in ((s["q"], s["gq"]), (s["k"], s["gk"])):
        x = x.float()
        if g is not None:
            x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * g
        out.append(_rotate(s, x, cos, sin).to(torch.bfloat16))
    return dict(q=out[0], k=out[1])


def _rope_bwd_plain(s):
    cos, sin = _turns(s)
    out = {}
    for name, x, g in (("q", s["q"], s["gq"]), ("k", s["k"], s["gk"])):
        du = _rotate(s, s["d" + name + "_rot"].float(), cos, -sin)
        if g is not None:
            x = x.float()
            r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
            n = x * r
            out["dg" + name] = (du * n).sum((0, 1, 2))
            u = du * g
            du = r * (u - n * (u * n).mean(-1, keepdim=True))
        out["d" + name] = du.to(torch.bfloat16)
    return out


def _parts(s):
    """(rows, kv heads, query heads) of one sequence's heads at a time, few enough for the memory."""
    group = s["Hq"] // s["Hk"]
    for a, b in zip(s["cu"], s["cu"][1:]):
        step = max(1, (1 << 29) // (group * (b - a) ** 2))
        for h in range(0, s["Hk"], step):
            e = min(s["Hk"], h + step)
            yield slice(a, b), slice(h, e), slice(h * group, e * group)


def _scores(s, rows, hk, hq):
    """Scaled, masked scores [kv heads, group, n, n] in 32 bits."""
    n, d = rows.stop - rows.start, s["d"]
    q, k = s["q"][hq, rows].float(), s["k"][hk, rows].float()
    w = (q.view(k.shape[0], -1, n, d) @ k[:, None].transpose(2, 3)).mul_(d ** -0.5)
    if s["causal"]:
        at = torch.arange(n, device=w.device)
        w.masked_fill_(at[None] > at[:, None], float("-inf"))
    return w


def _attn_plain(s):
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    for rows, hk, hq in _parts(s):
        w = _scores(s, rows, hk, hq)
        m = w.amax(-1, keepdim=True)
        w.sub_(m).exp_()
        l = w.sum(-1, keepdim=True)
        o = (w @ s["v"][hk, rows].float()[:, None]) / l
        out[hq, rows] = o.flatten(0, 1).to(torch.bfloat16)
        lse[hq, rows] = (m + l.log()).flatten(0, 1).squeeze(-1)
    return out, lse


def _attn_bwd_plain(s):
    dq, dk, dv = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    for rows, hk, hq in _parts(s):
        p = _scores(s, rows, hk, hq)
        shape = p.shape[:3]
        p.sub_(s["lse"][hq, rows].view(*shape, 1)).exp_()
        dout = s["dout"][hq, rows].float().view(*shape, -1)
        delta = (dout * s["out"][hq, rows].float().view(*shape, -1)).sum(-1, keepdim=True)
        dv[hk, rows] = (p.transpose(2, 3) @ dout).sum(1).to(torch.bfloat16)
        ds = (dout @ s["v"][hk, rows].float()[:, None].transpose(2, 3)).sub_(delta).mul_(p).mul_(s["d"] ** -0.5)
        dq[hq, rows] = (ds @ s["k"][hk, rows].float()[:, None]).flatten(0, 1).to(torch.bfloat16)
        dk[hk, rows] = (ds.transpose(2, 3) @ s["q"][hq, rows].float().view(*shape, -1)).sum(1).to(torch.bfloat16)
    return dq, dk, dv


def _run_own(s):
    import joint_attention_gb300 as ja

    op = s["op"]
    if op == "ln":
        y, h, mean, r = ja.layer_norm(s["x"], s["g"], s["b"], s["residual"], EPS)
        out = dict(y=y, mean=mean, r=r)
        return out if s["residual"] is None else dict(out, h=h)
    if op == "ln_bwd":
        dx, dg, db = ja.layer_norm_backward(s["dy"], s["h"], s["mean"], s["r"], s["g"], s["dres"], s["bias"])
        return dict(dx=dx, dg=dg, db=db) if s["bias"] else dict(dx=dx, dg=dg)
    if op == "rope":
        q, k = ja.rope(s["q"], s["k"], s["pos"], s["freq"], s["axis_pairs"], s["gq"], s["gk"], s["interleaved"], EPS)
        return dict(q=q, k=k)
    if op == "rope_bwd":
        dq, dk, dgq, dgk = ja.rope_backward(s["dq_rot"], s["dk_rot"], s["pos"], s["freq"], s["axis_pairs"], s["q"],
                                            s["k"], s["gq"], s["gk"], s["interleaved"], EPS)
        return dict(dq=dq, dk=dk, dgq=dgq, dgk=dgk) if s["norm"] else dict(dq=dq, dk=dk)
    if op == "attn":
        out, lse = ja.forward_grouped(s["q"], s["k"], s["v"], s["cu"], s["causal"])
        return dict(out=out, lse=lse)
    dq, dk, dv = ja.backward_grouped(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu"], s["causal"])
    return dict(dq=dq, dk=dk, dv=dv)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "attn":
        out, lse = _attn_plain(state)
        return dict(out=out, lse=lse)
    if op == "attn_bwd":
        dq, dk, dv = _attn_bwd_plain(state)
        return dict(dq=dq, dk=dk, dv=dv)
    return dict(ln=_ln_plain, ln_bwd=_ln_bwd_plain, rope=_rope_plain, rope_bwd=_rope_bwd_plain)[op](state)


def work(case):
    op = case["op"]
    if op in ("ln", "ln_bwd"):
        T, C, params = case["items"] * case["rows"], case["C"], 4 * case["items"] * case["C"]
        biases = 1 if case["bias"] else 0
        if op == "ln":
            return dict(bytes=T * C * (4 + (4 if case["res"] else 0)) + 8 * T + params * (1 + biases), flops=9 * T * C)
        return dict(bytes=T * C * (8 if case["dh"] else 6) + 8 * T + params * (2 + biases), flops=13 * T * C)
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if op in ("rope", "rope_bwd"):
        B, N, P = case["B"], case["N"], sum(_ints(case["pairs"]))
        values = B * (Hq + Hk) * N * d
        each = 6 if op == "rope_bwd" and case["norm"] else 4
        where = 4 * len(_ints(case["pairs"])) * N * (B if case["per_item"] else 1)
        flops = 3 * values * 2 * P // d + (0 if not case["norm"] else values * (4 if op == "rope" else 11))
        return dict(bytes=values * each + where + 4 * P + (16 * d if case["norm"] else 0), flops=flops)
    T = sum(_ints(case["lens"]))
    seen = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _ints(case["lens"]))
    heads = 4 * (Hq + Hk) if op == "attn" else 2 * (4 * Hq + 4 * Hk)
    return dict(bytes=T * d * heads + 4 * Hq * T, flops=(4 if op == "attn" else 10) * d * Hq * seen)


def _rope_factor(s):
    """e^(i angle) of every row's pairs in 64 bits, [B or 1, 1, N, P]."""
    where = s["pos"].double() if s["per_item"] else s["pos"].double().unsqueeze(0)
    cols, at = [], 0
    for a, p in enumerate(s["axis_pairs"]):
        cols.append(where[:, :, a, None] * s["freq"][at:at + p].double())
        at += p
    angle = torch.cat(cols, -1).unsqueeze(1)
    return torch.polar(torch.ones_like(angle), angle)


def _turned(s, x, factor):
    """The rotary channels of x (64 bits) as complex numbers times factor; the others as they are."""
    P = factor.shape[-1]
    turned, rest = x[..., :2 * P], x[..., 2 * P:]
    if s["interleaved"]:
        z = torch.view_as_complex(turned.reshape(*turned.shape[:-1], P, 2).contiguous())
        turned = torch.view_as_real(z * factor).flatten(-2)
    else:
        z = torch.complex(turned[..., :P].contiguous(), turned[..., P:].contiguous()) * factor
        turned = torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, rest], -1)


def _rope_exact(s, q, k, gq, gk):
    factor = _rope_factor(s)
    out = []
    for x, g in ((q, gq), (k, gk)):
        if g is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["d"] + EPS) * g
        out.append(_turned(s, x, factor))
    return out


def _attn_exact(s, q, k, v, rows, head):
    """One query head of one sequence in 64 bits."""
    w = torch.einsum("id,jd->ij", q, k) / math.sqrt(s["d"])
    if s["causal"]:
        w = w + torch.full_like(w, float("-inf")).triu(1)
    lse = torch.logsumexp(w, 1)
    return torch.einsum("ij,jd->id", torch.exp(w - lse[:, None]), v), lse


def exact(case, seed):
    """The definitions in 64 bits; gradients by automatic differentiation where that is the simplest."""
    s = prepare(case, seed)
    op = s["op"]
    if op in ("ln", "ln_bwd"):
        C = s["C"]
        g = s["g"].double().view(-1, 1, C)
        if op == "ln":
            out = {}
            x = s["x"].double()
            if s["residual"] is not None:
                x = (x + s["residual"].double()).to(torch.bfloat16).double()
                out["h"] = x
            out["mean"] = torch.einsum("bnc->bn", x) / C
            var = torch.einsum("bnc,bnc->bn", x - out["mean"].unsqueeze(2), x - out["mean"].unsqueeze(2)) / C
            out["r"] = 1.0 / torch.sqrt(var + EPS)
            out["y"] = (x - out["mean"].unsqueeze(2)) * out["r"].unsqueeze(2) * g
            if s["b"] is not None:
                out["y"] += s["b"].double().view(-1, 1, C)
            return out
        n = (s["h"].double() - s["mean"].double().unsqueeze(2)) * s["r"].double().unsqueeze(2)
        dy = s["dy"].double()
        out = dict(dg=torch.einsum("bnc,bnc->bc", dy, n).view(s["g"].shape))
        if s["bias"]:
            out["db"] = torch.einsum("bnc->bc", dy).view(s["g"].shape)
        u = dy * g
        along = torch.einsum("bnc,bnc->bn", u, n).unsqueeze(2) / C
        dx = (u - torch.einsum("bnc->bn", u).unsqueeze(2) / C - n * along) * s["r"].double().unsqueeze(2)
        out["dx"] = dx if s["dres"] is None else dx + s["dres"].double()
        return out
    if op == "rope":
        gains = [None if t is None else t.double() for t in (s["gq"], s["gk"])]
        q, k = _rope_exact(s, s["q"].double(), s["k"].double(), *gains)
        return dict(q=q, k=k)
    if op == "rope_bwd":
        if not s["norm"]:
            factor = _rope_factor(s).conj()
            return dict(dq=_turned(s, s["dq_rot"].double(), factor), dk=_turned(s, s["dk_rot"].double(), factor))
        leaves = [s[n].double().requires_grad_() for n in ("q", "k", "gq", "gk")]
        grads = torch.autograd.grad(_rope_exact(s, *leaves), leaves, [s["dq_rot"].double(), s["dk_rot"].double()])
        return dict(zip(("dq", "dk", "dgq", "dgk"), grads))
    group = s["Hq"] // s["Hk"]
    shape = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    spans = [slice(a, b) for a, b in zip(s["cu"], s["cu"][1:])]
    if op == "attn":
        out, lse = shape(s["q"]), shape(s["q"][..., 0])
        for rows in spans:
            for h in range(s["Hq"]):
                q, k, v = s["q"][h, rows], s["k"][h // group, rows], s["v"][h // group, rows]
                out[h, rows], lse[h, rows] = _attn_exact(s, q.double(), k.double(), v.double(), rows, h)
        return dict(out=out, lse=lse)
    dq, dk, dv = shape(s["q"]), shape(s["k"]), shape(s["v"])
    for rows in spans:
        for h in range(s["Hq"]):
            leaves = [t.double().requires_grad_() for t in (s["q"][h, rows], s["k"][h // group, rows],
                                                            s["v"][h // group, rows])]
            o, _ = _attn_exact(s, *leaves, rows, h)
            gq, gk, gv = torch.autograd.grad(o, leaves, s["dout"][h, rows].double())
            dq[h, rows] = gq
            dk[h // group, rows] += gk
            dv[h // group, rows] += gv
    return dict(dq=dq, dk=dk, dv=dv)
