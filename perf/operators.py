"""Cases for the operators that stand beside the layer: layer norm in front of or behind it,
products grouped by expert (forward and both gradients), and the orthogonalised update of its
weight gradients.

`own` false: the operators in their plain form (elementary torch operations in float32, rounded
once at the end).  `own` true: the library's entry points, called as a user's program calls them.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one projection of the 16B layer's 64 routed experts over a prefill batch: 8192 tokens,
        # top-6, rows grouped by expert
        dict(name="grouped_prefill_bf16", op="grouped", dtype="bf16", rows=49152, tail=0,
             groups=64, n=1408, k=2048, skew=0.0),
        # the same layer's down projection for a decode batch of 64 tokens: six rows an expert
        dict(name="grouped_decode_bf16", op="grouped", dtype="bf16", rows=384, tail=0, groups=64,
             n=2048, k=1408, skew=0.0),
        # float32 experts of the 2B-class layer under skewed routing, in a buffer with rows left over
        dict(name="grouped_f32", op="grouped", dtype="f32", rows=8190, tail=66, groups=16, n=896,
             k=1280, skew=0.7),
        # training step of the 2B-class layer: both gradients of one projection, 4096 tokens, top-7
        dict(name="grouped_backward_bf16", op="grouped_backward", dtype="bf16", rows=28672, tail=0,
             groups=63, n=896, k=1280, skew=0.3),
        # a small float32 model with odd widths, an odd row count and experts without tokens
        dict(name="grouped_backward_f32_odd", op="grouped_backward", dtype="f32", rows=1021, tail=3,
             groups=16, n=136, k=267, skew=1.5),
        # the update of one projection of all 64 routed experts of the 16B layer
        dict(name="orthogonalize_16b_f32", op="orthogonalize", dtype="f32", batch=64, m=1408,
             n=2048),
        # tall bfloat16 gradients (a down projection of the 2B-class layer), four experts
        dict(name="orthogonalize_tall_bf16", op="orthogonalize", dtype="bf16", batch=4, m=1280,
             n=896),
        # the tiny model's 16 experts, where launches count
        dict(name="orthogonalize_tiny_f32", op="orthogonalize", dtype="f32", batch=16, m=128,
             n=256),
        # one decoded token
        dict(name="layer_norm_token_bf16", op="layer_norm", dtype="bf16", rows=1, d=2048),
        # the 16B layer's prefill batch
        dict(name="layer_norm_prefill_bf16", op="layer_norm", dtype="bf16", rows=8192, d=2048),
        # training step of the 145B-class layer
        dict(name="layer_norm_backward_bf16", op="layer_norm_backward", dtype="bf16", rows=16384,
             d=4096),
        # float32 with an odd width and an odd batch
        dict(name="layer_norm_backward_f32_odd", op="layer_norm_backward", dtype="f32", rows=3001,
             d=1283),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_backward", "orthogonalize", "layer_norm",
                     "layer_norm_backward"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f32"]))
    if op in ("grouped", "grouped_backward"):
        width = rng.choice([1, 8, 64])  # odd widths, whole 16-byte rows, the layer's own widths
        groups = _spread(rng, 1, 128)
        n, k = (max(width, _spread(rng, 24, 2048) // width * width) for _ in range(2))
        rows = _spread(rng, 1, 16384)
        case |= dict(rows=rows, tail=rng.choice([0, 0, rng.randint(1, 40)]), groups=groups, n=n,
                     k=k, skew=rng.choice([0.0, rng.uniform(0.0, 1.5)]))
    elif op == "orthogonalize":
        m, n = _spread(rng, 8, 2048), _spread(rng, 8, 2048)
        most = max(1, min(64, int(4e8 / (min(m, n) * (m + n)))))
        case |= dict(batch=_spread(rng, 1, most), m=m, n=n)
    else:
        rows, d = _spread(rng, 1, 16384), _spread(rng, 64, 8192)
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        case |= dict(rows=rows, d=d)
    return case


# ---------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _group_sizes(case, seed):
    """Rows of each expert: a draw of the routing with probabilities ~ 1 / rank^skew."""
    gen = torch.Generator().manual_seed(seed * 7919 + 11)
    groups = case["groups"]
    p = (1.0 + torch.randperm(groups, generator=gen).double()) ** -case["skew"]
    of_row = torch.multinomial(p, case["rows"], replacement=True, generator=gen)
    return torch.bincount(of_row, minlength=groups)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _T[case["dtype"]], case["op"]
    s = dict(op=op, dtype=dt)
    if op in ("grouped", "grouped_backward"):
        sizes = _group_sizes(case, seed)
        M, E, n, k = case["rows"] + case["tail"], case["groups"], case["n"], case["k"]
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(
            torch.int32).cuda()
        s["most"] = int(sizes.max())  # the largest group, which the plain form pads to
        s["x"] = _normal(gen, M, k).to(dt)
        s["w"] = (_normal(gen, E, n, k) * 0.02).to(dt)
        if op == "grouped_backward":
            s["dy"] = _normal(gen, M, n).to(dt)
    elif op == "orthogonalize":
        # weight gradients: dy^T x over more tokens than the smaller side, channels of uneven size
        B, m, n = case["batch"], case["m"], case["n"]
        tokens = 2 * min(m, n) + 8
        g = torch.empty(B, m, n, device="cuda", dtype=dt)
        scale = torch.exp(0.5 * _normal(gen, 1, n))
        for i in range(B):
            g[i] = (_normal(gen, m, tokens) @ (_normal(gen, tokens, n) * scale) * 1e-3).to(dt)
        s["x"] = g
    else:
        R, d = case["rows"], case["d"]
        channel = _normal(gen, d)
        s["x"] = (_normal(gen, R, d) * (1.0 + 0.5 * channel.abs()) + 0.3 * channel).to(dt)
        s["weight"] = (1.0 + 0.1 * _normal(gen, d)).to(dt)
        s["bias"] = (0.1 * _normal(gen, d)).to(dt)
        if op == "layer_norm_backward":
            s["dy"] = _normal(gen, R, d).to(dt)
            # what the forward pass kept
            xf = s["x"].double()
            mean = xf.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xf - mean[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    return s


# ---------------------------------------------------------------- plain forms
def _padded(t, e, pos, E, most):
    """Rows of a group at [group, position]; zeros behind a group's last row."""
    out = torch.zeros(E, most, t.shape[1], device=t.device, dtype=torch.float32)
    out[e, pos] = t.float()
    return out


def _plain_places(s):
    off = s["offsets"].long()
    rows = torch.arange(s["x"].shape[0], device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    return off, rows, e


def _plain_grouped(s):
    off, rows, e = _plain_places(s)
    E, most = s["w"].shape[0], max(1, s["most"])
    inside = e < E
    e, rows = e[inside], rows[inside]
    pos = rows - off[e]
    xp = _padded(s["x"][rows], e, pos, E, most)
    yp = torch.matmul(xp, s["w"].float().transpose(1, 2))
    y = torch.zeros(s["x"].shape[0], s["w"].shape[1], device=xp.device, dtype=s["dtype"])
    y[rows] = yp[e, pos].to(s["dtype"])
    return y


def _plain_grouped_backward(s):
    off, rows, e = _plain_places(s)
    E, most = s["w"].shape[0], max(1, s["most"])
    inside = e < E
    e, rows = e[inside], rows[inside]
    pos = rows - off[e]
    xp = _padded(s["x"][rows], e, pos, E, most)
    dyp = _padded(s["dy"][rows], e, pos, E, most)
    dw = torch.matmul(dyp.transpose(1, 2), xp)
    dxp = torch.matmul(dyp, s["w"].float())
    dx = torch.zeros(s["x"].shape, device=xp.device, dtype=s["dtype"])
    dx[rows] = dxp[e, pos].to(s["dtype"])
    return dict(dx=dx, dw=dw)


def _plain_orthogonalize(s):
    x = s["x"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt().float() + 1e-7)
    a, b, c = COEFFICIENTS
    for _ in range(5):
        g = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.to(s["dtype"])


def _plain_layer_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = (xc.square().mean(1) + 1e-5).rsqrt()
    y = xc * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return dict(y=y.to(s["dtype"]), mean=mean, rstd=rstd)


def _plain_layer_norm_backward(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    return dict(dx=dx.to(s["dtype"]), dweight=(dy * xh).sum(0), dbias=dy.sum(0))


# ---------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if own:
        import mixture_experts_ffn_fp32_amd as moe

        if op == "grouped":
            return moe.grouped_matmul(s["x"], s["w"], s["offsets"])
        if op == "grouped_backward":
            dx, dw = moe.grouped_matmul_backward(s["x"], s["w"], s["offsets"], s["dy"])
            return dict(dx=dx, dw=dw)
        if op == "orthogonalize":
            return moe.orthogonalize(s["x"])
        if op == "layer_norm":
            y, mean, rstd = moe.layer_norm(s["x"], s["weight"], s["bias"])
            return dict(y=y, mean=mean, rstd=rstd)
        dx, dweight, dbias = moe.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"],
                                                     s["rstd"])
        return dict(dx=dx, dweight=dweight, dbias=dbias)
    return {"grouped": _plain_grouped, "grouped_backward": _plain_grouped_backward,
            "orthogonalize": _plain_orthogonalize, "layer_norm": _plain_layer_norm,
            "layer_norm_backward": _plain_layer_norm_backward}[op](s)


# ---------------------------------------------------------------- work and exact values
def work(case):
    es, op = _SIZE[case["dtype"]], case["op"]
    if op in ("grouped", "grouped_backward"):
        R, E, n, k = case["rows"], min(case["groups"], case["rows"]), case["n"], case["k"]
        if op == "grouped":
            return dict(bytes=es * (R * k + E * n * k + R * n), flops=2 * R * n * k)
        return dict(bytes=es * (2 * R * k + R * n + E * n * k) + 4 * case["groups"] * n * k,
                    flops=4 * R * n * k)
    if op == "orthogonalize":
        # the Gram matrix and its square are symmetric: half of each product
        B, p, q = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
        return dict(bytes=2 * es * B * p * q, flops=5 * B * (p * p * q + p ** 3 + 2 * p * p * q))
    R, d = case["rows"], case["d"]
    if op == "layer_norm":
        return dict(bytes=es * (2 * R * d + 2 * d) + 8 * R, flops=8 * R * d)
    return dict(bytes=es * (3 * R * d + d) + 8 * R + 8 * d, flops=14 * R * d)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("grouped", "grouped_backward"):
        off = s["offsets"].tolist()
        x, n = s["x"], s["w"].shape[1]
        y = torch.zeros(x.shape[0], n, dtype=torch.float64, device=x.device)
        dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        dw = []
        for e in range(len(off) - 1):
            at = slice(off[e], off[e + 1])
            we, xe = s["w"][e].double(), x[at].double()
            if op == "grouped":
                y[at] = xe @ we.t()
            else:
                dye = s["dy"][at].double()
                dx[at] = dye @ we
                dw.append(dye.t().contiguous() @ xe)
        return y if op == "grouped" else dict(dx=dx, dw=torch.stack(dw))
    if op == "orthogonalize":
        a, b, c = COEFFICIENTS
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        eye = torch.eye(min(case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for i in range(out.shape[0]):
            g = s["x"][i].double()
            g = g.t().contiguous() if case["m"] > case["n"] else g
            g = g / (torch.linalg.norm(g) + 1e-7)
            for _ in range(5):
                gram = g @ g.t()
                g = (a * eye + gram @ (b * eye + c * gram)) @ g
            out[i] = g.t() if case["m"] > case["n"] else g
        return out
    x, w = s["x"].double(), s["weight"].double()
    if op == "layer_norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + 1e-5)
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w)
        return dict(y=y, mean=mean, rstd=rstd)
    mean, rstd, dy = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["dy"].double()
    xh = (x - mean) * rstd
    d = x.shape[1]
    along = torch.stack([(dy @ w), ((dy * xh) @ w)], 1) / d
    dx = rstd * (dy * w - along[:, :1] - xh * along[:, 1:])
    return dict(dx=dx, dweight=torch.einsum("rd,rd->d", dy, xh),
                dbias=torch.ones(len(dy), dtype=torch.float64, device=dy.device) @ dy)
