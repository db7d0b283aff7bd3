"""The operators around the QKV projection, as cases to be measured.

Residual addition with RMSNorm (bf16 or 8-bit output) and its backward, 8-bit rows with scales, the
QKV projection from 8-bit tokens and weights, and the QKV projection with low-rank adapters of the
batch items' own.  With ``own`` false ``run`` computes them from elementary torch operations in 32
bits; with ``own`` true it calls the library."""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -80  # the smallest row maximum that a scale is made from


def listed():
    return [
        # one token of each of 8 requests through a 768-wide block: latency
        dict(name="norm_8_tokens", op="norm", T=8, C=768, res=True, fp8=False),
        # a 512 px training step's tokens, both streams (16 x 1101), width 768
        dict(name="norm_512px", op="norm", T=17616, C=768, res=True, fp8=False),
        # 768 px sampling (4 x 2381 tokens), the 8-bit output that the projection reads
        dict(name="norm_fp8_768px", op="norm", T=9524, C=2048, res=True, fp8=True),
        # a wide model's long batch: the largest pass over memory
        dict(name="norm_wide", op="norm", T=32768, C=4096, res=True, fp8=False),
        # backward of a first block's norm (no gradient from a later path), odd sizes
        dict(name="norm_bwd_333", op="norm_bwd", T=333, C=1096, dh=False),
        # backward of the 512 px training step
        dict(name="norm_bwd_512px", op="norm_bwd", T=17616, C=768, dh=True),
        # a stream's QKV weight, rows scaled once when a model is loaded
        dict(name="quant_weight", op="quant", T=2304, C=768),
        # 768 px tokens that another norm made, into 8 bits
        dict(name="quant_768px", op="quant", T=9524, C=2048),
        # 512 px sampling from 8-bit tokens and weights
        dict(name="qkv_fp8_512px", op="qkv_fp8", B=16, H=12, N_img=1024, N_txt=77, d=64, C=768, bias=True),
        # 768 px sampling, heads of 128: the largest product
        dict(name="qkv_fp8_768px", op="qkv_fp8", B=4, H=16, N_img=2304, N_txt=77, d=128, C=2048, bias=False),
        # 32 requests of one token in each stream, adapters of their own
        dict(name="lora_32_tokens", op="lora", B=32, H=12, N_img=1, N_txt=1, d=64, C=768, rank=16, n=32, bias=True),
        # 512 px sampling of 16 requests, an adapter each (one has none)
        dict(name="lora_512px", op="lora", B=16, H=12, N_img=1024, N_txt=77, d=64, C=768, rank=16, n=16, bias=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "quant", "qkv_fp8", "qkv_fp8", "lora", "lora"])
    if op in ("norm", "norm_bwd", "quant"):
        C = 8 * _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, min(32768, (1 << 27) // C))
        if op == "norm":
            return dict(op=op, T=T, C=C, res=rng.random() < 0.75, fp8=rng.random() < 0.5)
        if op == "norm_bwd":
            return dict(op=op, T=T, C=C, dh=rng.random() < 0.75)
        return dict(op=op, T=T, C=C)
    d = rng.choice([64, 128])
    H = rng.randint(1, 16)
    N_img = _log_int(rng, 1, 2304)
    N_txt = rng.choice([0, 1, 77, rng.randint(2, 154)])
    B = _log_int(rng, 1, 16 if N_img > 64 else 64)
    if op == "qkv_fp8":
        C = 16 * _log_int(rng, 4, 128)
        case = dict(op=op, B=B, H=H, N_img=N_img, N_txt=N_txt, d=d, C=C, bias=rng.random() < 0.5)
    else:
        C = 8 * _log_int(rng, 8, 256)
        case = dict(op=op, B=B, H=H, N_img=N_img, N_txt=N_txt, d=d, C=C, rank=8 * rng.randint(1, 16),
                    n=rng.randint(1, 24), bias=rng.random() < 0.5)
    while work(case)["flops"] > 2.3e11:
        case["B"] = max(1, case["B"] // 2)
    return case


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _gain(gen, n):
    return torch.rand(n, generator=gen, device="cuda") + 0.5


def _rows_e4m3(x):
    """8-bit rows and their scales, as a program that loads a model makes them."""
    s = x.float().abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)
    C = case["C"]
    if op in ("norm", "norm_bwd", "quant"):
        T = case["T"]
        if op == "quant":
            s["x"] = _randn(gen, T, C, scale=C ** -0.5)
            return s
        # a residual stream grows with depth and has a few large channels
        big = 1.0 + 7.0 * (torch.rand(C, generator=gen, device="cuda") < 0.02).float()
        stream = (torch.randn(T, C, generator=gen, device="cuda") * (3.0 * big)).to(torch.bfloat16)
        s["g"] = _gain(gen, C)
        if op == "norm":
            s["x"] = _randn(gen, T, C) if case["res"] else stream
            s["residual"] = stream if case["res"] else None
            return s
        s["h"] = stream
        s["r"] = (stream.float().square().mean(-1) + EPS).rsqrt()
        s["dy"] = _randn(gen, T, C, scale=0.1)
        s["dres"] = _randn(gen, T, C, scale=0.1) if case["dh"] else None
        return s
    B, H, d = case["B"], case["H"], case["d"]
    for stream, n in (("img", case["N_img"]), ("txt", case["N_txt"])):
        x = _randn(gen, B, n, C)
        w = _randn(gen, 3 * H * d, C, scale=C ** -0.5)
        s["b_" + stream] = torch.randn(3 * H * d, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        if op == "qkv_fp8":
            s["x_" + stream], s["sx_" + stream] = _rows_e4m3(x)
            s["w_" + stream], s["sw_" + stream] = _rows_e4m3(w)
        else:
            s["x_" + stream], s["w_" + stream] = x, w
            s["down_" + stream] = _randn(gen, case["n"], 3 * case["rank"], C, scale=C ** -0.5)
            s["up_" + stream] = _randn(gen, case["n"], 3 * H * d, case["rank"], scale=0.3 * case["rank"] ** -0.5)
    s["gq"], s["gk"] = _gain(gen, d), _gain(gen, d)
    if op == "lora":
        s["scale"] = torch.rand(case["n"], generator=gen, device="cuda") + 0.5
        # every request its adapter; about one in eight has none
        own_adapter = torch.arange(B, device="cuda") % case["n"]
        none = torch.rand(B, generator=gen, device="cuda") < 0.125
        s["index"] = torch.where(none, -1, own_adapter).to(torch.int32)
    return s


def _norm_plain(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    f = h.float()
    r = (f.square().mean(-1) + EPS).rsqrt()
    z = f * r[:, None] * s["g"]
    out = dict(r=r) if s["residual"] is None else dict(r=r, h=h)
    if not s["fp8"]:
        return dict(out, y=z.to(torch.bfloat16))
    scale = z.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return dict(out, y=(z / scale[:, None]).to(torch.float8_e4m3fn), scale=scale)


def _norm_bwd_plain(s):
    n = s["h"].float() * s["r"][:, None]
    dy = s["dy"].float()
    u = dy * s["g"]
    dx = s["r"][:, None] * (u - n * (u * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(torch.bfloat16), dg=(dy * n).sum(0))


def _quant_plain(x):
    x = x.float()
    scale = x.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return dict(y=(x / scale[:, None]).to(torch.float8_e4m3fn), scale=scale)


def _product_plain(s, stream):
    """One stream's projection [B, N_s, 3 H d] in 32 bits."""
    x, w = s["x_" + stream].float(), s["w_" + stream].float()
    y = x @ w.t()
    if s["op"] == "qkv_fp8":
        y = y * s["sx_" + stream][..., None] * s["sw_" + stream]
    else:
        B, n, rank, hd = s["B"], x.shape[1], s["rank"], s["H"] * s["d"]
        at = s["index"].clamp_min(0).long()
        a = torch.where(s["index"] >= 0, s["scale"][at], 0.0)
        down, up = s["down_" + stream][at].float(), s["up_" + stream][at].float()
        u = (x @ down.transpose(1, 2)) * a[:, None, None]
        u = u.view(B, n, 3, rank).transpose(1, 2)
        y = y + (u @ up.view(B, 3, hd, rank).transpose(2, 3)).transpose(1, 2).reshape(B, n, 3 * hd)
    return y if s["b_" + stream] is None else y + s["b_" + stream]


def _qkv_plain(s):
    B, H, d = s["B"], s["H"], s["d"]
    y = torch.cat([_product_plain(s, "txt"), _product_plain(s, "img")], 1).to(torch.bfloat16)
    q, k, v = (t.transpose(1, 2).contiguous() for t in y.view(B, -1, 3, H, d).unbind(2))
    hat = [(t.float() * (t.float().square().mean(-1, keepdim=True) + EPS).rsqrt() * g).to(torch.bfloat16)
           for t, g in ((q, s["gq"]), (k, s["gk"]))]
    return dict(q=q, k=k, v=v, q_hat=hat[0], k_hat=hat[1])


def _hats(saved, q):
    """q_hat and k_hat of the activations that a projection keeps (each part at a multiple of 256 bytes)."""
    size = 2 * q.numel()
    at = (size + 255) // 256 * 256
    return [saved[o:o + size].view(torch.bfloat16).view(q.shape) for o in (0, at)]


def _run_own(s):
    import joint_attention_gb300 as ja

    op = s["op"]
    if op == "norm":
        if s["fp8"]:
            y, scale, h, r = ja.add_norm_fp8(s["x"], s["g"], s["residual"], EPS)
            out = dict(y=y, scale=scale, r=r)
        else:
            y, h, r = ja.add_norm(s["x"], s["g"], s["residual"], EPS)
            out = dict(y=y, r=r)
        return out if s["residual"] is None else dict(out, h=h)
    if op == "norm_bwd":
        dx, dg = ja.add_norm_backward(s["dy"], s["h"], s["r"], s["g"], s["dres"])
        return dict(dx=dx, dg=dg)
    if op == "quant":
        y, scale = ja.quant_rows(s["x"])
        return dict(y=y, scale=scale)
    if op == "qkv_fp8":
        q, k, v, saved = ja.qkv_norm_fp8(s["x_img"], s["sx_img"], s["w_img"], s["sw_img"], s["b_img"], s["x_txt"],
                                         s["sx_txt"], s["w_txt"], s["sw_txt"], s["b_txt"], s["gq"], s["gk"], s["H"])
    else:
        q, k, v, saved = ja.qkv_norm_lora(s["x_img"], s["w_img"], s["b_img"], s["x_txt"], s["w_txt"], s["b_txt"],
                                          s["gq"], s["gk"], s["H"], s["down_img"], s["up_img"], s["down_txt"],
                                          s["up_txt"], s["scale"], s["index"])
    q_hat, k_hat = _hats(saved, q)
    return dict(q=q, k=k, v=v, q_hat=q_hat, k_hat=k_hat)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "quant":
        return _quant_plain(state["x"])
    return _qkv_plain(state)


def work(case):
    op, C = case["op"], case["C"]
    if op in ("norm", "norm_bwd", "quant"):
        T = case["T"]
        if op == "norm":
            each = 2 + (4 if case["res"] else 0) + (1 if case["fp8"] else 2)
            return dict(bytes=T * C * each + T * (8 if case["fp8"] else 4) + 4 * C, flops=8 * T * C)
        if op == "norm_bwd":
            return dict(bytes=T * C * (8 if case["dh"] else 6) + 4 * T + 8 * C, flops=10 * T * C)
        return dict(bytes=3 * T * C + 4 * T, flops=2 * T * C)
    B, H, d = case["B"], case["H"], case["d"]
    hd, n_all = H * d, case["N_img"] + case["N_txt"]
    streams = 1 if case["N_txt"] == 0 else 2
    tokens = B * n_all
    size = 1 if op == "qkv_fp8" else 2
    total = size * C * (tokens + streams * 3 * hd) + 5 * 2 * tokens * hd + 2 * 4 * tokens * H
    if case["bias"]:
        total += streams * 4 * 3 * hd
    flops = 2 * tokens * 3 * hd * C
    if op == "qkv_fp8":
        total += 4 * (tokens + streams * 3 * hd)
    else:
        rank = case["rank"]
        total += 2 * streams * min(B, case["n"]) * 3 * rank * (C + hd)
        flops += 2 * tokens * 3 * rank * (C + hd)
    return dict(bytes=total, flops=flops)


def exact(case, seed):
    """The definitions in 64 bits, one output at a time."""
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        out = {}
        x = s["x"].double()
        if s["residual"] is not None:
            x = (x + s["residual"].double()).to(torch.bfloat16).double()
            out["h"] = x
        mean_sq = torch.einsum("tc,tc->t", x, x) / s["C"]
        out["r"] = 1.0 / torch.sqrt(mean_sq + EPS)
        z = torch.einsum("tc,t,c->tc", x, out["r"], s["g"].double())
        if not s["fp8"]:
            return dict(out, y=z)
        out["scale"] = torch.clamp(z.abs().max(dim=1).values, min=AMAX_FLOOR) / E4M3_MAX
        out["y"] = (z / out["scale"].unsqueeze(1)).to(torch.float8_e4m3fn).double()
        return out
    if op == "norm_bwd":
        h, r, dy, g = (s[k].double() for k in ("h", "r", "dy", "g"))
        along = torch.einsum("tc,tc,c->t", dy, h, g) * r / s["C"]  # mean of u n
        dx = torch.einsum("tc,c,t->tc", dy, g, r) - h * (along * r * r)[:, None]
        if s["dres"] is not None:
            dx += s["dres"].double()
        return dict(dx=dx, dg=torch.einsum("tc,tc,t->c", dy, h, r))
    if op == "quant":
        x = s["x"].double()
        scale = torch.clamp(x.abs().max(dim=1).values, min=AMAX_FLOOR) / E4M3_MAX
        return dict(y=(x / scale.unsqueeze(1)).to(torch.float8_e4m3fn).double(), scale=scale)
    B, H, d, C = s["B"], s["H"], s["d"], s["C"]
    parts = {}
    for stream in ("img", "txt"):
        x, w = s["x_" + stream].double(), s["w_" + stream].double()
        if op == "qkv_fp8":
            x = x * s["sx_" + stream].double().unsqueeze(2)
            w = w * s["sw_" + stream].double().unsqueeze(1)
        y = torch.einsum("bnc,phec->pbhne", x, w.view(3, H, d, C))
        if s["b_" + stream] is not None:
            y += s["b_" + stream].double().view(3, 1, H, 1, d)
        if op == "lora":
            for b, a in enumerate(s["index"].tolist()):
                if a < 0:
                    continue
                down = s["down_" + stream][a].double().view(3, s["rank"], C)
                up = s["up_" + stream][a].double().view(3, H, d, s["rank"])
                u = torch.einsum("nc,pjc->pnj", x[b], down) * s["scale"][a].double()
                y[:, b] += torch.einsum("pnj,phej->phne", u, up)
        parts[stream] = y
    y = torch.cat([parts["txt"], parts["img"]], dim=3)
    out = dict(q=y[0], k=y[1], v=y[2])
    for name, g in (("q", s["gq"]), ("k", s["gk"])):
        t = out[name].to(torch.bfloat16).double()
        r = 1.0 / torch.sqrt((t * t).sum(-1, keepdim=True) / d + EPS)
        out[name + "_hat"] = g.double() * t * r
    return out
