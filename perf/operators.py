"""The feed-forward operators' measured cases: normalisation, linear with its epilogue, tokens by expert.

``run`` computes a case in elementary torch operations in 32 bits where ``own`` is
false, and through ``comm_matmul_tensor_amd`` where it is true.  Widths are the
library's own workloads' (4096, 1792, 7168; 8192 and 1024 tokens) or generic ones.

Operators (``op`` of a case):
  norm         s = x + residual, y = s rsqrt(mean(s^2) + eps) weight; y in 16 bits or in 8 with scales
  norm_grad    its gradients for x (= residual) and weight
  linear       residual + act(x @ w^T + bias), of one matrix or of row ranges with a matrix each (experts)
  linear_grad  gradients for x, w and bias
  sort         tokens' rows sorted by expert, with the map of rows and the experts' ranges
  unsort       the experts' rows back in token order, summed with the router's weights
  unsort_grad  its gradients for the rows and the weights
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one generated token through the norm of a decoder layer: latency
        dict(name="norm_1_token", op="norm", rows=1, h=4096, dtype="bf16", out="bf16", group=0, residual=True),
        # a prompt or training batch through a wide layer's norm, the residual stream kept
        dict(name="norm_8192_tokens", op="norm", rows=8192, h=7168, dtype="bf16", out="bf16", group=0, residual=True),
        # a ragged serving batch whose normed rows go to an int8 product: codes with a scale for each token
        dict(name="norm_int8_1023", op="norm", rows=1023, h=7168, dtype="f16", out="int8", group=0, residual=True),
        # the backward of a training batch's norm
        dict(name="norm_grad_8192", op="norm_grad", rows=8192, h=4096, dtype="bf16", residual=True),
        # one generated token through a layer's wide linear: the weight is read once
        dict(name="linear_1_token", op="linear", rows=1, k=4096, n=7168, groups=0, dtype="bf16", act="silu", bias=True,
             residual=False, keep_z=False),
        # a training batch's first linear of the feed-forward, its pre-activation kept for the backward
        dict(name="linear_gelu_4096", op="linear", rows=4096, k=4096, n=7168, groups=0, dtype="bf16", act="gelu",
             bias=True, residual=False, keep_z=True),
        # a ragged prompt through the second linear, added to the residual stream
        dict(name="linear_residual_517", op="linear", rows=517, k=1792, n=4096, groups=0, dtype="f16", act="none",
             bias=True, residual=True, keep_z=False),
        # the backward of the training batch's first linear
        dict(name="linear_grad_4096", op="linear_grad", rows=4096, k=4096, n=7168, groups=0, dtype="bf16", act="gelu",
             bias=True),
        # a training batch's experts: each range of rows by its own matrix
        dict(name="experts_16384", op="linear", rows=16384, k=4096, n=1792, groups=32, dtype="bf16", act="silu",
             bias=False, residual=False, keep_z=True),
        # a training batch's tokens sorted by expert
        dict(name="sort_8192", op="sort", rows=8192, h=4096, experts=64, top=4, dtype="bf16"),
        # a small decoding batch's expert rows back in token order: latency
        dict(name="unsort_16", op="unsort", rows=16, h=4096, experts=64, top=4, dtype="bf16", weights=True),
        # the backward of the training batch's weighted sum
        dict(name="unsort_grad_8192", op="unsort_grad", rows=8192, h=4096, experts=64, top=4, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """An odd multiple of 64 (a model's width), of 8 (rows still 16-byte aligned) or of 1 (ragged)."""
    step = rng.choice([64, 64, 64, 8, 8, 1])
    w = max(1, _log(rng, lo, hi) // step)
    return step * (w - 1 + w % 2) if w > 1 else step


def _rows(rng, hi):
    r = _log(rng, 1, hi)
    return r - 1 + r % 2 if r > 1 else 1


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "linear", "linear", "linear_grad", "sort", "unsort", "unsort_grad"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm":
        h = _width(rng, 64, 8192)
        out = rng.choice([dtype, "int8", "fp8"])
        group = 128 if out != dtype and rng.random() < 0.4 else 0
        if group:
            h = 128 * max(1, h // 128)
            h += 128 * (h // 128 % 2 == 0)
        return dict(op=op, rows=_rows(rng, 8192), h=h, dtype=dtype, out=out, group=group, residual=rng.random() < 0.7)
    if op == "norm_grad":
        return dict(op=op, rows=_rows(rng, 8192), h=_width(rng, 64, 4096), dtype=dtype, residual=rng.random() < 0.7)
    if op in ("linear", "linear_grad"):
        groups = rng.choice([0, 0, 4, 13, 32])
        k, n = _width(rng, 256, 4096), _width(rng, 256, 7168 if not groups else 2048)
        rows = _rows(rng, 4096 if not groups else 8192)
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        case = dict(op=op, rows=rows, k=k, n=n, groups=groups, dtype=dtype, act=act, bias=rng.random() < 0.6)
        if op == "linear":
            case.update(residual=rng.random() < 0.4, keep_z=rng.random() < 0.4)
        return case
    case = dict(op=op, rows=_rows(rng, 8192), h=_width(rng, 64, 4096), experts=rng.choice([5, 8, 32, 64, 160]),
                top=rng.choice([1, 2, 4]), dtype=dtype)
    if op == "unsort":
        case["weights"] = rng.random() < 0.8
    return case


# ------------------------------------------------------------------ inputs
def _routing(case, g):
    """Each token's distinct experts, popular ones oftener; one choice in 50 is dropped (-1)."""
    t, e, top = case["rows"], case["experts"], case["top"]
    score = torch.rand((t, e), generator=g, device="cuda") + 0.3 * torch.rand((e,), generator=g, device="cuda")
    ids = score.topk(top, dim=1).indices.to(torch.int32)
    drop = torch.rand((t, top), generator=g, device="cuda") < 0.02
    return torch.where(drop, torch.full_like(ids, -1), ids)


def _ranges(case, g):
    """Row ranges of the groups: uneven, one of them empty, the last rows in none."""
    part = torch.rand((case["groups"],), generator=g, device="cuda") + 0.2
    part[1] = 0.0
    end = (part.cumsum(0) / part.sum() * max(1, case["rows"] - case["rows"] // 64)).floor().to(torch.int32)
    return torch.cat([torch.zeros((1,), dtype=torch.int32, device="cuda"), end])


def _sorted_map(ids, experts):
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    return torch.where(flat < 0, torch.full_like(row, -1), row).to(torch.int32).view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    s = dict(case=case)
    op, rows = case["op"], case["rows"]
    if op in ("norm", "norm_grad"):
        h = case["h"]
        loud = 1.0 + 15.0 * (torch.rand((h,), generator=g, device="cuda") < 0.004)  # a stream's few loud channels
        s["weight"] = (1.0 + 0.1 * torch.randn((h,), generator=g, device="cuda")).to(dt)
        s["residual"] = (torch.randn((rows, h), generator=g, device="cuda") * loud).to(dt) if case["residual"] else None
        s["x"] = normal(rows, h)
        if op == "norm_grad":
            if case["residual"]:
                s["x"] = s["x"] + s["residual"]
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dout"] = normal(rows, h)
            s["dh"] = normal(rows, h) if case["residual"] else None
        elif case["out"] in ("int8", "fp8"):
            s["values"] = torch.empty((rows, h), dtype=dt, device="cuda")
    elif op in ("linear", "linear_grad"):
        k, n, e = case["k"], case["n"], case["groups"]
        s["x"] = normal(rows, k)
        s["w"] = normal(*((e, n, k) if e else (n, k)), std=k ** -0.5)
        s["bias"] = normal(*((e, n) if e else (n,)), std=0.5) if case["bias"] else None
        s["offsets"] = _ranges(case, g) if e else None
        if op == "linear":
            s["residual"] = normal(rows, n) if case["residual"] else None
        else:
            s["dout"], s["z"] = normal(rows, n), normal(rows, n)
        if e:
            # where the plain form puts each row: its group's block of `most` rows, the rows of none past them
            at = torch.arange(rows, device="cuda")
            of = torch.searchsorted(s["offsets"][1:].contiguous().long(), at, right=True)
            most = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
            inside = at - s["offsets"].long()[of]
            s["group_of"], s["most"] = of, most
            s["slot"] = torch.where(of < e, of * most + inside, e * most)
    else:
        ids = _routing(case, g)
        s["ids"] = ids
        if op == "sort":
            s["x"] = normal(rows, case["h"])
        else:
            s["map"] = _sorted_map(ids, case["experts"])
            s["y"] = normal(rows * case["top"], case["h"])
            p = torch.rand((rows, case["top"]), generator=g, device="cuda") + 0.05
            s["weights"] = p / p.sum(1, keepdim=True) if case.get("weights", True) else None
            if op == "unsort_grad":
                s["dout"] = normal(rows, case["h"])
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
    if name == "none":
        return torch.ones_like(z)
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
    if op == "norm":
        v = s["x"].float()
        if case["residual"]:
            v = v + s["residual"].float()
        rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
        y = v * rstd * s["weight"].float()
        kept = [v.to(dt)] if case["residual"] else []
        if case["out"] not in ("int8", "fp8"):
            return [y.to(dt), rstd[:, 0]] + kept
        top = 127.0 if case["out"] == "int8" else 448.0
        yg = y.view(y.shape[0], -1, case["group"] or y.shape[1])
        scale = yg.abs().amax(2, keepdim=True) / top
        c = torch.where(scale > 0, yg / scale, torch.zeros_like(yg)).clamp(-top, top)
        c = torch.round(c) if case["out"] == "int8" else c.to(torch.float8_e4m3fn).float()
        return [(c * scale).view_as(y).to(dt), scale[:, :, 0], rstd[:, 0]] + kept
    if op == "norm_grad":
        v, dy, w, rstd = s["x"].float(), s["dout"].float(), s["weight"].float(), s["rstd"][:, None]
        gw = dy * w
        dv = rstd * (gw - v * rstd * rstd * (gw * v).mean(1, keepdim=True))
        if case["residual"]:
            dv = dv + s["dh"].float()
        return [dv.to(dt), (dy * v * rstd).sum(0).to(dt)]
    if op == "linear":
        x, w = s["x"].float(), s["w"].float()
        if case["groups"]:
            z = torch.bmm(_blocks(s, x), w.transpose(1, 2).contiguous())
            if case["bias"]:
                z = z + s["bias"].float()[:, None]
            z = _rows_of(s, z)
        else:
            z = x @ w.t()
            if case["bias"]:
                z = z + s["bias"].float()
        out = _act(z, case["act"])
        if case["residual"]:
            out = out + s["residual"].float()
        return [out.to(dt)] + ([z.to(dt)] if case["keep_z"] else [])
    if op == "linear_grad":
        x, w, dz = s["x"].float(), s["w"].float(), s["dout"].float() * _act_slope(s["z"].float(), case["act"])
        if case["groups"]:
            db = _blocks(s, dz)
            dx = _rows_of(s, torch.bmm(db, w))
            dw = torch.bmm(db.transpose(1, 2).contiguous(), _blocks(s, x))
            dbias = db.sum(1)
        else:
            dx, dw, dbias = dz @ w, dz.t() @ x, dz.sum(0)
        return [dx.to(dt), dw.to(dt)] + ([dbias.to(dt)] if case["bias"] else [])
    if op == "sort":
        ids, e, top = s["ids"].reshape(-1).long(), case["experts"], case["top"]
        key = torch.where(ids < 0, torch.full_like(ids, e), ids)
        order = torch.argsort(key, stable=True)
        row = torch.empty_like(order)
        row[order] = torch.arange(order.numel(), device=order.device)
        out = s["x"][order // top] * (key[order] < e)[:, None]
        ends = (key[None, :] <= torch.arange(e, device=key.device)[:, None]).sum(1)
        offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
        return [out, torch.where(ids < 0, torch.full_like(row, -1), row).to(torch.int32).view(s["ids"].shape),
                offsets.to(torch.int32)]
    m = s["map"].long()
    rows = s["y"].float()[m.clamp(min=0)] * (m >= 0)[:, :, None]
    if op == "unsort":
        if s["weights"] is not None:
            rows = rows * s["weights"][:, :, None]
        return [rows.sum(1).to(dt)]
    dout = s["dout"].float()
    dy = torch.zeros((s["y"].shape[0] + 1, dout.shape[1]), device=dout.device)
    dy[torch.where(m >= 0, m, torch.full_like(m, s["y"].shape[0])).view(-1)] = (
        dout[:, None, :] * s["weights"][:, :, None]).view(-1, dout.shape[1])
    return [dy[:-1].to(dt), (rows * dout[:, None, :]).sum(2)]


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import comm_matmul_tensor_amd as mc2
    case = s["case"]
    op = case["op"]
    if op == "norm":
        out_dtype = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}.get(case["out"])
        y, scale, v, rstd = mc2.mc2_add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, out_dtype=out_dtype,
                                                 group=case["group"], need_rstd=True)
        kept = [v] if case["residual"] else []
        if scale is None:
            return [y, rstd] + kept
        if case["out"] == "fp8":
            y = y.to(torch.float32)
        g = scale.shape[1]
        values = s["values"]
        torch.mul(y.view(y.shape[0], g, -1), scale[:, :, None], out=values.view(y.shape[0], g, -1))
        return [values, scale, rstd] + kept
    if op == "norm_grad":
        return list(mc2.mc2_add_rms_norm_grad(s["dout"], s["x"], s["weight"], s["rstd"], s["dh"]))
    if op in ("linear", "linear_grad"):
        act = {"none": mc2.MC2_ACT_NONE, "relu": mc2.MC2_ACT_RELU, "gelu": mc2.MC2_ACT_GELU,
               "gelu_tanh": mc2.MC2_ACT_GELU_TANH, "silu": mc2.MC2_ACT_SILU}[case["act"]]
        if op == "linear":
            out, z = mc2.mc2_linear_act(s["x"], s["w"], s["bias"], s["residual"], act=act, group_offsets=s["offsets"],
                                        need_z=case["keep_z"])
            return [out] + ([z] if case["keep_z"] else [])
        dx, dw, dbias = mc2.mc2_linear_act_grad(s["dout"], s["x"], s["w"], s["z"], act=act, group_offsets=s["offsets"],
                                                need_dbias=case["bias"])
        return [dx, dw] + ([dbias] if case["bias"] else [])
    if op == "sort":
        return list(mc2.mc2_moe_permute(s["x"], s["ids"], case["experts"]))
    if op == "unsort":
        return [mc2.mc2_moe_unpermute(s["y"], s["map"], s["weights"])]
    return list(mc2.mc2_moe_unpermute_grad(s["dout"], s["y"], s["map"], s["weights"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, r = case["op"], case["rows"]
    if op == "norm":
        h = case["h"]
        eight = case["out"] in ("int8", "fp8")
        per_scale = 4 * r * (h // case["group"] if case["group"] else 1)
        b = r * h * (2 + (4 if case["residual"] else 0) + (1 if eight else 2)) + 2 * h + 4 * r + (per_scale if eight else 0)
        return dict(bytes=b, flops=4 * r * h)
    if op == "norm_grad":
        h = case["h"]
        return dict(bytes=r * h * (6 + (2 if case["residual"] else 0)) + 4 * h + 4 * r, flops=10 * r * h)
    if op in ("linear", "linear_grad"):
        k, n, e = case["k"], case["n"], max(1, case["groups"])
        if case["groups"]:
            e = min(e, r)  # a group without rows needs no matrix
        w = e * n * k * 2
        if op == "linear":
            b = 2 * r * k + w + 2 * r * n * (1 + case["residual"] + case["keep_z"]) + (2 * e * n if case["bias"] else 0)
            return dict(bytes=b, flops=2 * r * k * n)
        act = 0 if case["act"] == "none" else 2
        return dict(bytes=2 * r * k * 2 + 2 * w + r * n * (2 + act), flops=4 * r * k * n)
    h, top = case["h"], case["top"]
    if op == "sort":
        return dict(bytes=2 * r * h * (1 + top) + 8 * r * top, flops=0)
    if op == "unsort":
        return dict(bytes=2 * r * h * (1 + top) + 4 * r * top * (1 + case["weights"]), flops=2 * r * h * top)
    return dict(bytes=2 * r * h * (1 + 2 * top) + 12 * r * top, flops=3 * r * h * top)


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


def exact(case, seed):
    s = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op in ("norm", "norm_grad"):
        v = s["x"].double()
        w = s["weight"].double()
        if op == "norm":
            if case["residual"]:
                v = v + s["residual"].double()
            rstd = 1.0 / (torch.linalg.vector_norm(v, dim=1) ** 2 / case["h"] + EPS).sqrt()
            y = torch.einsum("rh,r,h->rh", v, rstd, w)
            kept = [v] if case["residual"] else []
            if case["out"] not in ("int8", "fp8"):
                return [y, rstd] + kept
            # the codes' rounding is part of the definition: values are compared without it, scales with
            g = case["group"] or case["h"]
            return [y, y.unflatten(1, (-1, g)).abs().max(2).values / (127 if case["out"] == "int8" else 448), rstd] + kept
        dy, r = s["dout"].double(), s["rstd"].double()
        n = v * r[:, None]
        dn = dy * w
        dv = (dn - n * ((dn * n).sum(1) / case["h"])[:, None]) * r[:, None]
        return [dv + s["dh"].double() if case["residual"] else dv, torch.einsum("rh,rh->h", dy, n)]
    if op in ("linear", "linear_grad"):
        x, w = s["x"].double(), s["w"].double()
        n, act = case["n"], case["act"]
        if case["groups"]:
            ends = s["offsets"].tolist()
            spans = [(i, ends[i], ends[i + 1]) for i in range(case["groups"])]
        else:
            w = w[None]
            spans = [(0, 0, rows)]
        if op == "linear":
            z = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
            for i, a, b in spans:
                z[a:b] = x[a:b] @ w[i].T
                if case["bias"]:
                    z[a:b] += s["bias"].double().view(-1, n)[i]
            out = _exact_act(z, act)[0]
            if case["residual"]:
                out = out + s["residual"].double()
            return [out] + ([z] if case["keep_z"] else [])
        dz = s["dout"].double() * _exact_act(s["z"].double(), act)[1]
        dx = torch.zeros((rows, case["k"]), dtype=torch.float64, device="cuda")
        dw, db = torch.zeros_like(w), torch.zeros((w.shape[0], n), dtype=torch.float64, device="cuda")
        for i, a, b in spans:
            dx[a:b] = dz[a:b] @ w[i]
            dw[i] = dz[a:b].T @ x[a:b]
            db[i] = dz[a:b].sum(0)
        if not case["groups"]:
            dw, db = dw[0], db[0]
        return [dx, dw] + ([db] if case["bias"] else [])
    if op == "sort":
        ids = s["ids"].cpu().view(-1).tolist()
        order = [i for _, i in sorted((e, i) for i, e in enumerate(ids) if e >= 0)]
        out = torch.zeros((len(ids), case["h"]), dtype=torch.float64, device="cuda")
        token = torch.tensor(order, dtype=torch.long, device="cuda") // case["top"]
        out[:len(order)] = s["x"].double()[token]
        return [out, None, None]
    out = torch.zeros((rows, case["h"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((rows, case["top"]), dtype=torch.float64, device="cuda")
    dy = torch.zeros((s["y"].shape[0], case["h"]), dtype=torch.float64, device="cuda")
    for j in range(case["top"]):
        m = s["map"][:, j].long()
        t = torch.nonzero(m >= 0)[:, 0]
        y = s["y"][m[t]].double()
        p = s["weights"][t, j].double() if s["weights"] is not None else torch.ones(t.shape, dtype=torch.float64, device="cuda")
        if op == "unsort":
            out[t] += p[:, None] * y
        else:
            d = s["dout"][t].double()
            dy[m[t]] = p[:, None] * d
            dw[t, j] = (y * d).sum(1)
    return [out] if op == "unsort" else [dy, dw]
