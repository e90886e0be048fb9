"""Measured cases of the router and of the feed-forward operators' 8-bit forms.

``run`` computes a case in elementary torch operations where ``own`` is false (in 32
bits; the router's choice in 64, since two experts may be next to each other), and
through ``comm_matmul_tensor_amd`` where it is true.  Widths are those of the
library's other workloads (4096, 1792, 7168; 8192, 1024 and 517 tokens; 32, 64 and
160 experts) or generic ones.

Operators (``op`` of a case):
  route       scores of the experts (softmax or sigmoid), a bias on the choice, groups of experts, the `top`
              best experts of each token and their weights
  route_grad  its gradient for the scores' logits
  quant       rows to int8 codes with a scale for each row or each 128 columns, and back, through an activation
  i8          residual + act(x @ w^T * scales + bias) of int8 codes, of one matrix or of row ranges with a matrix
              each (experts)
  i8_grad     gradients for x, w and bias of act(x_act(x) @ w^T + bias) where x and the pre-activation were kept
              as int8 codes with a scale for each 128 columns
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small decoding batch's router: latency
        dict(name="route_16_tokens", op="route", rows=16, experts=64, top=4, dtype="bf16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0),
        # a ragged training batch's router with balanced experts in groups
        dict(name="route_8191_groups", op="route", rows=8191, experts=256, top=8, dtype="f32", score="sigmoid",
             bias=True, groups=16, top_groups=6, group_top=2, renorm=True, scale=2.0),
        # the backward of a training batch's router: every expert's score takes part in the softmax
        dict(name="route_grad_8192", op="route_grad", rows=8192, experts=160, top=4, dtype="f32", score="softmax",
             renorm=False, scale=1.0),
        # the backward of a few tokens' router: latency
        dict(name="route_grad_33", op="route_grad", rows=33, experts=64, top=4, dtype="bf16", score="sigmoid",
             renorm=True, scale=1.0),
        # a decoding batch's rows on their way into an int8 product
        dict(name="quant_16_tokens", op="quant", rows=16, h=4096, dtype="bf16", group=0, act="none"),
        # a training batch's pre-activations kept in 8 bits, and the activations from them in the backward
        dict(name="quant_8191_kept", op="quant", rows=8191, h=7168, dtype="bf16", group=128, act="gelu"),
        # one generated token through a layer's wide linear: the codes of the weight are read once
        dict(name="i8_1_token", op="i8", rows=1, k=4096, n=7168, groups=0, dtype="bf16", act="silu", bias=True,
             residual=False),
        # a prompt or a full serving batch through the feed-forward's first linear
        dict(name="i8_4096_tokens", op="i8", rows=4096, k=4096, n=7168, groups=0, dtype="bf16", act="gelu", bias=True,
             residual=False),
        # a prompt's rows by expert
        dict(name="i8_experts_16384", op="i8", rows=16384, k=4096, n=1792, groups=32, dtype="bf16", act="silu",
             bias=False, residual=False),
        # a small decoding batch's rows by expert: about one row for each of many matrices
        dict(name="i8_experts_64", op="i8", rows=64, k=1792, n=4096, groups=64, dtype="f16", act="none", bias=True,
             residual=False),
        # the backward of a ragged batch's second linear, whose input is the activation of what was kept
        dict(name="i8_grad_517", op="i8_grad", rows=517, k=4096, n=1792, groups=0, dtype="f16", act="none",
             x_act="gelu", bias=True),
        # the backward of a training batch's first linear from what was kept
        dict(name="i8_grad_4096", op="i8_grad", rows=4096, k=4096, n=7168, groups=0, dtype="bf16", act="gelu",
             x_act="none", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """An odd multiple of 64 (a model's width), of 8 or of 1 (ragged)."""
    step = rng.choice([64, 64, 64, 8, 8, 1])
    w = max(1, _log(rng, lo, hi) // step)
    return step * (w - 1 + w % 2) if w > 1 else step


def _rows(rng, hi):
    r = _log(rng, 1, hi)
    return r - 1 + r % 2 if r > 1 else 1


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "quant", "quant", "i8", "i8", "i8", "i8_grad", "i8_grad"])
    if op in ("route", "route_grad"):
        e = rng.choice([5, 8, 32, 64, 96, 160, 256, 512])
        case = dict(op=op, rows=_rows(rng, 8192 if e <= 256 else 4096), experts=e, top=rng.choice([1, 2, 4, 6, 8]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.0]))
        case["top"] = min(case["top"], e - 1)
        if op == "route":
            g = rng.choice([1, 1, 4, 8])
            if e % g or e // g < 3:
                g = 1
            least = -(-case["top"] // (e // g - 1))
            case.update(bias=rng.random() < 0.6, groups=g, top_groups=rng.randint(least, g) if least < g else g,
                        group_top=rng.choice([1, 2]))
        return case
    dtype = rng.choice(["bf16", "f16"])
    if op == "quant":
        return dict(op=op, rows=_rows(rng, 8192), h=_width(rng, 64, 7168), dtype=dtype, group=rng.choice([0, 128]),
                    act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]))
    groups = rng.choice([0, 0, 4, 13, 32])
    case = dict(op=op, rows=_rows(rng, 4096 if not groups else 8192), k=_width(rng, 256, 4096),
                n=_width(rng, 256, 7168 if not groups else 2048), groups=groups, dtype=dtype,
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.6)
    if op == "i8":
        case["residual"] = rng.random() < 0.4
    else:
        case["x_act"] = rng.choice(["none", "none", "relu", "gelu", "silu"])
    return case


# ------------------------------------------------------------------ inputs
def _ranges(case, g):
    """Row ranges of the groups: uneven, one of them empty, the last rows in none."""
    part = torch.rand((case["groups"],), generator=g, device="cuda") + 0.2
    part[1] = 0.0
    end = (part.cumsum(0) / part.sum() * max(1, case["rows"] - case["rows"] // 64)).floor().to(torch.int32)
    return torch.cat([torch.zeros((1,), dtype=torch.int32, device="cuda"), end])


def _codes(v, group):
    """int8 codes of the rows of v with a scale for each row (group 0) or each `group` columns."""
    r, c = v.shape
    width = group or c
    pad = -c % width
    b = torch.nn.functional.pad(v, (0, pad)).view(r, -1, width)
    scale = b.abs().amax(2, keepdim=True) / 127.0
    q = torch.where(scale > 0, b / scale, torch.zeros_like(b)).round().clamp(-127, 127)
    return q.to(torch.int8).view(r, -1)[:, :c].contiguous(), scale[:, :, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    s = dict(case=case)
    op, rows = case["op"], case["rows"]
    if op in ("route", "route_grad"):
        e, top = case["experts"], case["top"]
        liked = 0.5 * normal(e)  # experts that most tokens like
        logits = (normal(rows, e) + liked).to(dt)
        logits[:, e // 2] = -math.inf  # an expert that is switched off
        s["logits"] = logits
        if op == "route":
            s["bias"] = 0.05 * normal(e) if case["bias"] else None
        else:
            pick = torch.rand((rows, e), generator=g, device="cuda") + 0.2 * logits.float().clamp(min=-4.0)
            pick[:, e // 2] = -math.inf
            ids = pick.topk(top, dim=1).indices.to(torch.int32)
            lost = torch.rand((rows, top), generator=g, device="cuda") < 0.02  # choices there was no expert for
            s["ids"] = torch.where(lost, torch.full_like(ids, -1), ids)
            s["dweights"] = normal(rows, top)
    elif op == "quant":
        h = case["h"]
        loud = 1.0 + 15.0 * (torch.rand((h,), generator=g, device="cuda") < 0.004)  # a stream's few loud channels
        s["x"] = (normal(rows, h) * loud).to(dt)
    else:
        k, n, e = case["k"], case["n"], case["groups"]
        s["offsets"] = _ranges(case, g) if e else None
        s["bias"] = normal(*((e, n) if e else (n,)), std=0.5).to(dt) if case["bias"] else None
        if op == "i8":
            s["x"], s["x_scale"] = _codes(normal(rows, k), 0)
            w, ws = _codes(normal(max(e, 1) * n, k, std=k ** -0.5), 0)
            s["w"], s["w_scale"] = (w.view(e, n, k), ws.view(e, n)) if e else (w, ws.view(n))
            s["residual"] = normal(rows, n).to(dt) if case["residual"] else None
        else:
            s["x"], s["x_scale"] = _codes(normal(rows, k), 128)
            s["z"], s["z_scale"] = _codes(normal(rows, n), 128) if case["act"] != "none" else (None, None)
            s["w"] = normal(*((e, n, k) if e else (n, k)), std=k ** -0.5).to(dt)
            s["dout"] = normal(rows, n).to(dt)
        if e:
            # where the plain form puts each row: its group's block of `most` rows, the rows of none past them
            at = torch.arange(rows, device="cuda")
            of = torch.searchsorted(s["offsets"][1:].contiguous().long(), at, right=True)
            most = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
            inside = at - s["offsets"].long()[of]
            s["most"] = most
            s["slot"] = torch.where(of < e, of * most + inside, e * most)
    return s


# ------------------------------------------------------------------ the plain form
def _act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _values(codes, scale, group):
    """What codes stand for, in 32 bits."""
    r, c = codes.shape
    width = group or c
    return codes.float() * scale.repeat_interleave(width, dim=1)[:, :c]


def _blocks(s, a):
    """Rows `a` in their groups' blocks of `most` rows, zeros elsewhere: (groups, most, columns)."""
    e, most = s["case"]["groups"], s["most"]
    b = torch.zeros((e * most + 1, a.shape[1]), dtype=a.dtype, device=a.device)
    b[s["slot"]] = a
    return b[:-1].view(e, most, a.shape[1])


def _rows_of(s, b):
    """The rows of the blocks `b` in their own order, zeros for rows of no group."""
    flat = torch.cat([b.reshape(-1, b.shape[2]), torch.zeros((1, b.shape[2]), dtype=b.dtype, device=b.device)])
    return flat[s["slot"]]


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op == "route":
        l = s["logits"].double()
        if case["score"] == "softmax":
            p = torch.exp(l - l.amax(1, keepdim=True))
            p = p / p.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-l))
        choice = p if s["bias"] is None else p + s["bias"].double()
        choice = torch.where(l > -math.inf, choice, torch.full_like(choice, -math.inf))
        groups, per = case["groups"], case["experts"] // case["groups"]
        if groups > 1:
            of = choice.view(-1, groups, per)
            best = torch.sort(of, dim=2, descending=True).values[:, :, :case["group_top"]]
            value = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
            value = torch.where(best[:, :, 0] > -math.inf, value, torch.full_like(value, -math.inf))
            rank = torch.argsort(torch.argsort(value, dim=1, descending=True, stable=True), dim=1)
            choice = torch.where((rank < case["top_groups"])[:, :, None], of, torch.full_like(of, -math.inf)).view(l.shape)
        ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :case["top"]]
        there = choice.gather(1, ids) > -math.inf
        w = p.gather(1, ids) * there
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return [torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32), (case["scale"] * w).float()]
    if op == "route_grad":
        l, ids = s["logits"].float(), s["ids"].long()
        there = ids >= 0
        at = ids.clamp(min=0)
        dw = case["scale"] * s["dweights"] * there
        if case["score"] == "softmax":
            p = torch.exp(l - l.amax(1, keepdim=True))
            p = p / p.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-l))
        if case["renorm"]:
            chosen = p.gather(1, at) * there
            total = chosen.sum(1, keepdim=True)
            share = torch.where(total > 0, chosen / total, torch.zeros_like(chosen))
            dchosen = torch.where(total > 0, (dw - (dw * share).sum(1, keepdim=True)) / total, torch.zeros_like(dw)) * there
        else:
            dchosen = dw
        dp = torch.zeros_like(p).scatter_add_(1, at, dchosen)
        if case["score"] == "softmax":
            dl = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dl = dp * p * (1.0 - p)
        return [dl.to(dt)]
    if op == "quant":
        r, h = s["x"].shape
        width = case["group"] or h
        b = torch.nn.functional.pad(s["x"].float(), (0, -h % width)).view(r, -1, width)
        scale = b.abs().amax(2, keepdim=True) / 127.0
        q = torch.where(scale > 0, b / scale, torch.zeros_like(b)).round().clamp(-127, 127)
        return [_act((q * scale).view(r, -1)[:, :h], case["act"]).to(dt), scale[:, :, 0].contiguous()]
    if op == "i8":
        x = s["x"].float()
        w = s["w"].float()
        if case["groups"]:
            z = torch.bmm(_blocks(s, x * s["x_scale"]), w.transpose(1, 2).contiguous()) * s["w_scale"][:, None]
            if case["bias"]:
                z = z + s["bias"].float()[:, None]
            z = _rows_of(s, z)
        else:
            z = (x @ w.t()) * s["x_scale"] * s["w_scale"]
            if case["bias"]:
                z = z + s["bias"].float()
        out = _act(z, case["act"])
        if case["residual"]:
            out = out + s["residual"].float()
        return [out.to(dt)]
    x = _act(_values(s["x"], s["x_scale"], 128), case["x_act"])
    w, dz = s["w"].float(), s["dout"].float()
    if case["act"] != "none":
        dz = dz * _act_slope(_values(s["z"], s["z_scale"], 128), case["act"])
    if case["groups"]:
        db = _blocks(s, dz)
        dx = _rows_of(s, torch.bmm(db, w))
        dw = torch.bmm(db.transpose(1, 2).contiguous(), _blocks(s, x))
        dbias = db.sum(1)
    else:
        dx, dw, dbias = dz @ w, dz.t() @ x, dz.sum(0)
    return [dx.to(dt), dw.to(dt)] + ([dbias.to(dt)] if case["bias"] else [])


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import comm_matmul_tensor_amd as mc2
    case = s["case"]
    op = case["op"]
    acts = {"none": mc2.MC2_ACT_NONE, "relu": mc2.MC2_ACT_RELU, "gelu": mc2.MC2_ACT_GELU,
            "gelu_tanh": mc2.MC2_ACT_GELU_TANH, "silu": mc2.MC2_ACT_SILU}
    if op in ("route", "route_grad"):
        score = mc2.MC2_SCORE_SOFTMAX if case["score"] == "softmax" else mc2.MC2_SCORE_SIGMOID
        if op == "route":
            return list(mc2.mc2_moe_route(s["logits"], case["top"], s["bias"], score=score, groups=case["groups"],
                                          top_groups=case["top_groups"], group_top=case["group_top"],
                                          renormalise=case["renorm"], scale=case["scale"]))
        return [mc2.mc2_moe_route_grad(s["dweights"], s["logits"], s["ids"], score=score, renormalise=case["renorm"],
                                       scale=case["scale"])]
    if op == "quant":
        codes, scale = mc2.mc2_quant_rows(s["x"], group=case["group"])
        return [mc2.mc2_dequant_rows(codes, scale, group=case["group"], act=acts[case["act"]], dtype=s["x"].dtype), scale]
    if op == "i8":
        return [mc2.mc2_linear_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["bias"], s["residual"],
                                  dtype=DT[case["dtype"]], act=acts[case["act"]], group_offsets=s["offsets"])]
    dx, dw, dbias = mc2.mc2_linear_act_grad_i8(s["dout"], s["x"], s["x_scale"], s["w"], s["z"], s["z_scale"],
                                               act=acts[case["act"]], x_act=acts[case["x_act"]],
                                               group_offsets=s["offsets"], need_dbias=case["bias"])
    return [dx, dw] + ([dbias] if case["bias"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, r = case["op"], case["rows"]
    if op in ("route", "route_grad"):
        e, top = case["experts"], case["top"]
        logits = r * e * (4 if case["dtype"] == "f32" else 2)
        if op == "route":
            return dict(bytes=logits + 8 * r * top + (4 * e if case["bias"] else 0), flops=5 * r * e)
        return dict(bytes=2 * logits + 8 * r * top, flops=8 * r * e)
    if op == "quant":  # the codes are written and read once: they are what is kept in between
        scales = r * (-(-case["h"] // case["group"]) if case["group"] else 1)
        return dict(bytes=r * case["h"] * (2 + 1 + 1 + 2) + 8 * scales, flops=4 * r * case["h"])
    k, n = case["k"], case["n"]
    e = min(max(1, case["groups"]), r)  # a group without rows needs no matrix
    if op == "i8":
        return dict(bytes=r * k + e * n * k + 2 * r * n * (1 + case["residual"]) + 4 * r + 4 * e * n
                    + (2 * e * n if case["bias"] else 0), flops=2 * r * k * n)
    act = 0 if case["act"] == "none" else 1
    return dict(bytes=r * k * 3 + 4 * e * n * k + r * n * (2 + act) + 4 * r * (k + n * act) // 128, flops=4 * r * k * n)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_act(z, name):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0 * z), (z > 0).double()
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh u) = expit(2 u)
    c = 2 * math.sqrt(2 / math.pi)
    p = torch.special.expit(c * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z ** 2)


def _exact_codes(codes, scale):
    """codes times their scales, a block of columns at a time."""
    v = codes.double()
    for i in range(scale.shape[1]):
        v[:, 128 * i:128 * (i + 1)] *= scale[:, i:i + 1].double()
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op in ("route", "route_grad"):
        l = s["logits"].double()
        p = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.special.expit(l)
        if op == "route_grad":
            # the weights' own derivative, by hand of autograd in 64 bits
            leaf = l.clone().requires_grad_()
            q = torch.softmax(leaf, dim=1) if case["score"] == "softmax" else torch.sigmoid(leaf)
            keep = s["ids"] >= 0
            w = torch.where(keep, q.gather(1, s["ids"].long().clamp(min=0)), torch.zeros((), dtype=torch.float64, device="cuda"))
            if case["renorm"]:
                w = w / torch.where(keep.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones_like(w[:, :1]))
            (grad,) = torch.autograd.grad((w * s["dweights"].double()).sum() * case["scale"], leaf)
            return [torch.nan_to_num(grad)]
        left = p + (s["bias"].double() if s["bias"] is not None else 0.0)
        left[l == -math.inf] = -math.inf
        g, per = case["groups"], case["experts"] // case["groups"]
        if g > 1:
            worth = torch.zeros((rows, g), dtype=torch.float64, device="cuda")
            of = left.view(rows, g, per).clone()
            none = (of == -math.inf).all(2)
            for _ in range(case["group_top"]):
                m, i = of.max(2)
                worth += torch.where(m > -math.inf, m, torch.zeros_like(m))
                of.scatter_(2, i[:, :, None], -math.inf)
            worth[none] = -math.inf
            # a group is kept if fewer than top_groups stand before it
            idx = torch.arange(g, device="cuda")
            before = (worth[:, None, :] > worth[:, :, None]) | (
                (worth[:, None, :] == worth[:, :, None]) & (idx[None, None, :] < idx[None, :, None]))
            out = before.sum(2) >= case["top_groups"]
            left = left.masked_fill(out[:, :, None].expand(rows, g, per).reshape(rows, -1), -math.inf)
        w = torch.zeros((rows, case["top"]), dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            m = left.amax(1, keepdim=True)
            i = (left == m).to(torch.int8).argmax(1, keepdim=True)
            w[:, j:j + 1] = torch.where(m > -math.inf, p.gather(1, i), torch.zeros_like(m))
            left.scatter_(1, i, -math.inf)
        if case["renorm"]:
            w /= w.sum(1, keepdim=True)
        return [None, w * case["scale"]]
    if op == "quant":
        # scale and quotient are 32-bit numbers by definition, the rest is in 64
        x = s["x"].double()
        step = case["group"] or case["h"]
        out, scales = torch.empty_like(x), []
        for c in range(0, case["h"], step):
            b = x[:, c:c + step]
            scale = (b.abs().max(1, keepdim=True).values / 127).float().double()
            q = (b / torch.where(scale > 0, scale, torch.ones_like(scale))).float().double()
            out[:, c:c + step] = torch.round(q).clamp(-127, 127) * scale
            scales.append(scale)
        return [_exact_act(out, case["act"])[0], torch.cat(scales, dim=1)]
    n = case["n"]
    if case["groups"]:
        ends = s["offsets"].tolist()
        spans = [(i, ends[i], ends[i + 1]) for i in range(case["groups"])]
    else:
        spans = [(0, 0, rows)]
    w = s["w"].double().view(-1, n, case["k"])
    if op == "i8":
        x = s["x"].double() * s["x_scale"].double()
        w = w * s["w_scale"].double().view(-1, n, 1)
        z = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
        for i, a, b in spans:
            z[a:b] = x[a:b] @ w[i].T
            if case["bias"]:
                z[a:b] += s["bias"].double().view(-1, n)[i]
        out = _exact_act(z, case["act"])[0]
        return [out + s["residual"].double() if case["residual"] else out]
    x = _exact_act(_exact_codes(s["x"], s["x_scale"]), case["x_act"])[0]
    dz = s["dout"].double()
    if case["act"] != "none":
        dz = dz * _exact_act(_exact_codes(s["z"], s["z_scale"]), case["act"])[1]
    dx = torch.zeros((rows, case["k"]), dtype=torch.float64, device="cuda")
    dw, db = torch.zeros_like(w), torch.zeros((w.shape[0], n), dtype=torch.float64, device="cuda")
    for i, a, b in spans:
        dx[a:b] = dz[a:b] @ w[i]
        dw[i] = dz[a:b].T @ x[a:b]
        db[i] = dz[a:b].sum(0)
    if not case["groups"]:
        dw, db = dw[0], db[0]
    return [dx, dw] + ([db] if case["bias"] else [])
