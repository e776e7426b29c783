"""Cases of the operators around the expert products: the norms of a block, the FP8 block product, the decode layer.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded
once at the end; the router's logits in 64, because the choice of experts is decided by
their order) and, with ``own`` true, as a user calls the framework's kernels:

* ``norm``   residual_norm: r' = r + s * gate * rmsnorm(y) * post_weight, rounded to the
             residual's type, and n = rmsnorm(r') * norm_weight; the training cases also
             return the gradients of every input.
* ``fp8``    linear_fp8_block: tokens quantised to E4M3 per row and group of 128, the
             weight per block of 128 x 128, the product of both; the training cases
             quantise the weight too and return dx (from the E4M3 codes of dy and of the
             weight) and dw (a bf16 product).
* ``decode`` moe_decode: a whole mixture-of-experts layer for a few tokens: router,
             top-k, up-projection, SwiGLU, down-projection, weighted sum; bf16 weights or
             E4M3 weights with one scale per block of 128 x 128.
"""

import math

import torch

own = False

GROUP = 128
E4M3_MAX = 448.0


def _norm(name, T, H, train, gate, res, post=True, scale=1.0):
    return {"name": name, "op": "norm", "T": T, "H": H, "train": train, "gate": gate, "res": res, "post": post,
            "scale": scale}


def _fp8(name, T, H, N, train):
    return {"name": name, "op": "fp8", "T": T, "H": H, "N": N, "train": train}


def _decode(name, T, H, I, E, K, router, fp8, renorm=True):
    return {"name": name, "op": "decode", "T": T, "H": H, "I": I, "E": E, "K": K, "router": router, "fp8": fp8,
            "renorm": renorm}


def listed():
    return [
        # one token between two blocks while serving: nothing but latency
        _norm("norm one token", 1, 7168, False, "none", "bf16"),
        # a training step's norms at the largest hidden size, each token's block scaled by its own gate
        _norm("norm train large", 8192, 7168, True, "token", "bf16"),
        # a float32 residual stream with one learned gate per channel, a ragged number of tokens
        _norm("norm train f32", 4001, 2048, True, "channel", "f32", scale=0.5),
        # a dense projection while serving a handful of sequences: the weight's bytes count
        _fp8("fp8 few rows", 5, 7168, 4096, False),
        # the same projection of a long prompt: the matrix instructions count
        _fp8("fp8 prompt", 8192, 7168, 4096, False),
        # a ragged batch of prompts, a width that ends inside a block
        _fp8("fp8 ragged", 1003, 2048, 1552, False),
        # a training step of a projection, both quantisers and all three products
        _fp8("fp8 train", 4096, 4096, 2048, True),
        # the smallest layer, already routed, for a few sequences: latency
        _decode("decode small", 4, 512, 128, 4, 2, False, False),
        # one sequence's next token through the large layer: eight experts' weights
        _decode("decode one token", 1, 7168, 2048, 32, 8, True, False),
        # a batch of sequences over many narrow experts
        _decode("decode many experts", 17, 2048, 768, 128, 8, True, False, renorm=False),
        # a full batch of sequences: every expert's weights, tens of tokens each
        _decode("decode full batch", 64, 7168, 2048, 32, 8, True, False),
        # the large layer with E4M3 weights, half the bytes
        _decode("decode fp8", 8, 7168, 2048, 32, 8, True, True),
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], a multiple of step, uniform in its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "fp8", "decode"])
    if op == "norm":
        H = _log(rng, 64, 8192, 8)
        T = _log(rng, 1, min(32768, 8192 * 7168 // H))
        c = _norm("", T, H, rng.random() < 0.6, rng.choice(["none", "token", "channel", "full"]),
                  rng.choice(["bf16", "f32"]), rng.random() < 0.8, rng.choice([1.0, 0.5, 0.22]))
    elif op == "fp8":
        train = rng.random() < 0.4
        H = _log(rng, 256, 7168, GROUP)
        N = _log(rng, 128, 4096, GROUP if train else 16)
        T = _log(rng, 1, 4096 if train else 8192)
        c = _fp8("", T, H, N, train)
    else:
        fp8 = rng.random() < 0.4
        step = GROUP if fp8 else 64
        H = _log(rng, 512, 7168, step)
        I = _log(rng, 128, 2048, step)
        E = _log(rng, 4, max(4, min(160, 32 * 7168 * 2048 // (H * I))))
        K = min(E, rng.choice([1, 2, 4, 6, 8]))
        c = _decode("", _log(rng, 1, 64), H, I, E, K, rng.random() < 0.7, fp8, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------------ inputs

def _randn(gen, shape, std=1.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return t.mul_(std) if std != 1.0 else t


def _scales(amax):
    """448 / amax in float32 (1 where amax is 0), kept finite, and its reciprocal."""
    s = torch.where(amax > 0, (E4M3_MAX / amax).clamp(max=torch.finfo(torch.float32).max), torch.ones_like(amax))
    return s, 1.0 / s


def _quant_rows(x):
    """x [T, H] -> E4M3 values (float32) and one descale per row and group of 128."""
    T, H = x.shape
    v = x.float().view(T, H // GROUP, GROUP)
    s, d = _scales(v.abs().amax(dim=2))
    q = (v * s[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(T, H), d


def _quant_block(w):
    """w [H, N] -> E4M3 codes [N, H] and one descale per block of 128 x 128, [ceil(N/128), H/128]."""
    H, N = w.shape
    nb = (N + GROUP - 1) // GROUP
    v = torch.zeros((nb * GROUP, H), device=w.device, dtype=torch.float32)
    v[:N] = w.t().float()
    v = v.view(nb, GROUP, H // GROUP, GROUP)
    s, d = _scales(v.abs().amax(dim=(1, 3)))
    q = (v * s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(nb * GROUP, H)[:N].contiguous(), d.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, H, op = case["T"], case["H"], case["op"]
    s = {"case": case}
    if op == "norm":
        rt = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        s["y"] = _randn(gen, (T, H), 0.7)
        # a residual stream with a few channels far larger than the others
        s["residual"] = _randn(gen, (T, H), 1.0, rt)
        s["residual"][:, :: max(1, H // 5)] *= 30.0
        s["norm_weight"] = (1.0 + _randn(gen, (H,), 0.2, torch.float32)).to(rt)
        s["post_weight"] = (1.0 + _randn(gen, (H,), 0.2, torch.float32)).to(rt) if case["post"] else None
        shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_randn(gen, shape, 1.0, torch.float32)).to(torch.bfloat16)
        if case["train"]:
            s["d_residual"] = _randn(gen, (T, H), 1.0, rt)
            s["d_normed"] = _randn(gen, (T, H), 1.0)
            for k in ("y", "residual", "norm_weight", "post_weight", "gate"):
                if s[k] is not None:
                    s[k].requires_grad_(True)
    elif op == "fp8":
        N = case["N"]
        s["x"] = _randn(gen, (T, H))
        s["x"][:: 97] *= 20.0  # a few outlier tokens
        w = _randn(gen, (H, N), 1.0 / math.sqrt(H))
        if case["train"]:
            s["w"] = w.requires_grad_(True)
            s["x"].requires_grad_(True)
            s["dy"] = _randn(gen, (T, N))
        else:
            q, s["descale"] = _quant_block(w)
            s["codes"] = q.view(torch.uint8)
    else:
        I, E, K = case["I"], case["E"], case["K"]
        s["x"] = _randn(gen, (T, H))
        if case["router"]:
            s["router_weight"] = _randn(gen, (E, H), 1.0 / math.sqrt(H))
        else:
            keys = torch.rand((T, E), generator=gen, device="cuda")
            s["topk_ids"] = keys.argsort(dim=1)[:, :K].to(torch.int32).contiguous()
            s["topk_weights"] = torch.softmax(_randn(gen, (T, K), 1.0, torch.float32), dim=1)
        if case["fp8"]:
            for name, shape in (("up", (E, H, 2 * I)), ("down", (E, I, H))):
                codes = torch.empty((E, shape[2], shape[1]), device="cuda", dtype=torch.uint8)
                desc = torch.empty((E, shape[2] // GROUP, shape[1] // GROUP), device="cuda")
                for e in range(E):
                    q, desc[e] = _quant_block(_randn(gen, shape[1:], 1.0 / math.sqrt(shape[1])))
                    codes[e] = q.view(torch.uint8)
                s[name], s[name + "_descale"] = codes, desc
        else:
            s["up"] = _randn(gen, (E, H, 2 * I), 1.0 / math.sqrt(H))
            s["down"] = _randn(gen, (E, I, H), 1.0 / math.sqrt(I))
    return s


# ------------------------------------------------------------------- plain forms

def _rms(v, weight, eps):
    n = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    return n if weight is None else n * weight


def _norm_plain(s):
    c = s["case"]
    names = [k for k in ("y", "residual", "norm_weight", "post_weight", "gate") if s[k] is not None]
    a = {k: s[k].detach().float().requires_grad_(c["train"]) for k in names}
    z = _rms(a["y"], a["post_weight"], 1e-6) if c["post"] else a["y"]
    if "gate" in a:
        z = z * a["gate"]
    r = a["residual"] + c["scale"] * z
    rt = s["residual"].dtype
    r = r + (r.to(rt).float() - r).detach()  # the stored stream: rounded, with the gradient of the sum
    n = _rms(r, a["norm_weight"], 1e-6)
    out = {"residual": r.detach().to(rt), "normed": n.detach().to(torch.bfloat16)}
    if c["train"]:
        g = torch.autograd.grad((r, n), [a[k] for k in names], (s["d_residual"].float(), s["d_normed"].float()))
        out.update({"d_" + k: v.to(s[k].dtype) for k, v in zip(names, g)})
    return out


def _fp8_plain(s):
    c = s["case"]
    N = c["N"]
    xq, xd = _quant_rows(s["x"].detach())
    if c["train"]:
        wq, wd = _quant_block(s["w"].detach())
    else:
        wq, wd = s["codes"].view(torch.float8_e4m3fn), s["descale"]
    xv = xq.float() * xd.repeat_interleave(GROUP, dim=1)
    wv = wq.float() * wd.repeat_interleave(GROUP, dim=0)[:N].repeat_interleave(GROUP, dim=1)
    y = (xv @ wv.t()).to(torch.bfloat16)
    if not c["train"]:
        return y
    gq, gd = _quant_rows(s["dy"])
    dx = (gq.float() * gd.repeat_interleave(GROUP, dim=1)) @ wv
    dw = s["x"].detach().float().t() @ s["dy"].float()
    return y, dx.to(torch.bfloat16), dw.to(torch.bfloat16)


def _route(x, router_weight, K, renorm):
    """The K largest logits of a token (ties to the lower index) and their weights."""
    logits = x.double() @ router_weight.double().t()
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp((v - v[:, :1]).float())
    w = e[:, :K] / (e[:, :K] if renorm else e).sum(dim=1, keepdim=True)
    return ids[:, :K].to(torch.int32), w


def _decode_plain(s):
    c = s["case"]
    T, I, E, K, x = c["T"], c["I"], c["E"], c["K"], s["x"]
    if c["router"]:
        ids, w = _route(x, s["router_weight"], K, c["renorm"])
    else:
        ids, w = s["topk_ids"], s["topk_weights"]
    slots = T * K <= E  # one product per slot, or every expert for every token
    at = ids.reshape(-1).long() if slots else slice(None)
    if c["fp8"]:
        def weight(k):
            q, d = s[k][at], s[k + "_descale"][at]
            v = q.view(torch.float8_e4m3fn).float().view(-1, d.shape[1], GROUP, d.shape[2], GROUP)
            return (v * d[:, :, None, :, None]).view(q.shape).transpose(1, 2).contiguous()
    else:
        def weight(k):
            return s[k][at].float()
    xs = x.float().repeat_interleave(K, dim=0)[:, None] if slots else x.float()[None].expand(E, T, c["H"])
    h = torch.bmm(xs, weight("up"))
    g, u = h[..., :I], h[..., I:]
    o = torch.bmm(g / (1.0 + torch.exp(-g)) * u, weight("down"))
    if slots:
        y = (o.view(T, K, c["H"]) * w[:, :, None]).sum(dim=1)
    else:
        full = torch.zeros((T, E), device=x.device).scatter_add_(1, ids.long(), w)
        y = (o * full.t()[:, :, None]).sum(dim=0)
    y = y.to(torch.bfloat16)
    return (y, ids, w) if c["router"] else y


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm_plain, "fp8": _fp8_plain, "decode": _decode_plain}[c["op"]](s)
    import mixture_experts_ffn_int32_amd as hmm
    if c["op"] == "norm":
        r, n = hmm.residual_norm(s["y"], s["residual"], s["norm_weight"], post_weight=s["post_weight"],
                                 gate=s["gate"], residual_scale=c["scale"], eps=1e-6)
        out = {"residual": r.detach(), "normed": n.detach()}
        if c["train"]:
            names = [k for k in ("y", "residual", "norm_weight", "post_weight", "gate") if s[k] is not None]
            g = torch.autograd.grad((r, n), [s[k] for k in names], (s["d_residual"], s["d_normed"]))
            out.update({"d_" + k: v for k, v in zip(names, g)})
        return out
    if c["op"] == "fp8":
        if not c["train"]:
            return hmm.linear_fp8_block(s["x"], (s["codes"], s["descale"]))
        y = hmm.linear_fp8_block(s["x"], s["w"])
        return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    scales = {"up_descale": s["up_descale"], "down_descale": s["down_descale"]} if c["fp8"] else {}
    if c["router"]:
        return hmm.moe_decode(s["x"], s["up"], s["down"], router_weight=s["router_weight"], top_k=c["K"],
                              renormalize=c["renorm"], **scales)
    return hmm.moe_decode(s["x"], s["up"], s["down"], topk_ids=s["topk_ids"], topk_weights=s["topk_weights"], **scales)


# ------------------------------------------------------------------ work, exact

def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        rb = 2 if case["res"] == "bf16" else 4
        gate = {"none": 0, "token": 2 * T, "channel": 2 * H, "full": 2 * T * H}[case["gate"]]
        ws = rb * H * (2 if case["post"] else 1)
        n = T * H
        b = n * (2 + rb + rb + 2) + gate + ws  # y, r in; r', n out
        f = 10 * n
        if case["train"]:
            b += n * (rb + 2 + 2 + rb) + gate + ws  # dr', dn in; dy, dr out, and the weights' gradients
            f += 25 * n
        return {"bytes": b, "flops": f}
    if case["op"] == "fp8":
        N = case["N"]
        f = 2 * T * H * N
        if not case["train"]:
            return {"bytes": 2 * T * H + N * H + 4 * (-(-N // GROUP)) * (H // GROUP) + 2 * T * N, "flops": f}
        return {"bytes": 2 * (T * H + H * N + T * N) + 2 * (T * N + T * H + H * N), "flops": 3 * f}
    I, E, K = case["I"], case["E"], case["K"]
    active = E * (1.0 - (1.0 - K / E) ** T)  # experts that some token goes to, on average
    per = 3 * H * I
    b = active * (per * (1 + 4 / GROUP ** 2) if case["fp8"] else 2 * per) + 4 * T * H + 8 * T * K
    f = 6 * T * K * H * I
    if case["router"]:
        b += 2 * E * H
        f += 2 * T * E * H
    return {"bytes": int(b), "flops": int(f)}



def exact(case, seed):
    s = prepare(case, seed)
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        y, r0 = s["y"].detach().double(), s["residual"].detach().double()
        w = s["norm_weight"].detach().double()
        one = torch.ones((), device=y.device, dtype=torch.float64)
        wp = s["post_weight"].detach().double() if case["post"] else one
        g = s["gate"].detach().double() if s["gate"] is not None else one
        rho_y = (y.square().mean(1, keepdim=True) + 1e-6).rsqrt() if case["post"] else one
        u = y * rho_y
        r = r0 + case["scale"] * g * u * wp
        rs = r.float().to(s["residual"].dtype).double()  # the stream as stored
        rho = (rs.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        out = {"residual": r, "normed": rs * rho * w}
        if not case["train"]:
            return out
        dn, t = s["d_normed"].double(), s["d_residual"].double()
        a = dn * w
        t = t + rho * a - rs * rho ** 3 * (a * rs).mean(1, keepdim=True)
        dz = case["scale"] * t
        b = dz * g * wp
        out["d_y"] = rho_y * b - y * rho_y ** 3 * (b * y).mean(1, keepdim=True) if case["post"] else b
        out["d_residual"] = t
        out["d_norm_weight"] = (dn * rs * rho).sum(0)
        if case["post"]:
            out["d_post_weight"] = (dz * g * u).sum(0)
        if s["gate"] is not None:
            dg = dz * u * wp
            out["d_gate"] = {"token": lambda: dg.sum(1, keepdim=True), "channel": lambda: dg.sum(0),
                             "full": lambda: dg}[case["gate"]]()
        return out
    if case["op"] == "fp8":
        N, G = case["N"], H // GROUP

        def values(q, d, rows):
            """codes and descales, spread over blocks of ``rows`` x 128, as 64-bit values"""
            v = q.view(torch.float8_e4m3fn).double() if q.dtype == torch.uint8 else q.double()
            i = torch.arange(v.shape[0], device=v.device) // rows
            j = torch.arange(v.shape[1], device=v.device) // GROUP
            return v * d.double()[i][:, j]

        x = s["x"].detach()
        xv = values(*_quant_rows(x), 1)
        codes, desc = _quant_block(s["w"].detach()) if case["train"] else (s["codes"], s["descale"])
        wv = values(codes, desc, GROUP)
        if not case["train"]:
            return torch.matmul(xv, wv.t())
        return (torch.matmul(xv, wv.t()), torch.matmul(values(*_quant_rows(s["dy"]), 1), wv),
                torch.matmul(x.double().t(), s["dy"].double()))
    I, E, K = case["I"], case["E"], case["K"]
    x = s["x"].double()
    if case["router"]:
        logits = x @ s["router_weight"].double().t()
        order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :K]
        p = torch.softmax(logits, dim=1).gather(1, order)
        weights = p / p.sum(1, keepdim=True) if case["renorm"] else p
    else:
        order, weights = s["topk_ids"].long(), s["topk_weights"].double()
    y = torch.zeros((T, H), device=x.device, dtype=torch.float64)
    for e in range(E):
        share = (weights * (order == e)).sum(1, keepdim=True)
        mats = []
        for k in ("up", "down"):
            m = s[k][e]
            if case["fp8"]:
                d = s[k + "_descale"][e].double()
                i = torch.arange(m.shape[0], device=x.device) // GROUP
                j = torch.arange(m.shape[1], device=x.device) // GROUP
                mats.append((m.view(torch.float8_e4m3fn).double() * d[i][:, j]).t())
            else:
                mats.append(m.double())
        h = x @ mats[0]
        y += share * ((h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]) @ mats[1])
    return (y, None, weights) if case["router"] else y
