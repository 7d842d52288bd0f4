"""Cases for experts held in 8 bits and what stands around them: root-mean-square norm with the
residual's addition (and an output in 8 bits), quantising to 8 bits, products of 8-bit operands
grouped by expert, and the balance loss of the routing with its gradient.

`own` false: the operators in their plain form (elementary torch operations in float32, sums over
a batch in float64, rounded once at the end).  `own` true: the library's entry points, called as
a user's program calls them.

8-bit values are e4m3 or e5m2 with one float32 scale for each block of 128: the block's largest
magnitude over the type's largest value.  A row has a scale for each 128 of its elements, an
expert's weight matrix for each 128 x 128.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_MOST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token on its way into 8-bit experts
        dict(name="rms_norm_token_f8", op="rms_norm", dtype="bf16", rows=1, d=2048, residual=True,
             f8="e4m3"),
        # the 16B layer's prefill batch on its way into 8-bit experts
        dict(name="rms_norm_prefill_f8", op="rms_norm", dtype="bf16", rows=8192, d=2048,
             residual=True, f8="e4m3"),
        # float32 with an odd width and an odd batch
        dict(name="rms_norm_f32_odd", op="rms_norm", dtype="f32", rows=3001, d=1283, residual=True,
             f8=""),
        # training step of the 145B-class layer: the norm's gradient joins the residual stream's
        dict(name="rms_norm_backward_bf16", op="rms_norm_backward", dtype="bf16", rows=16384,
             d=4096, residual=True),
        # gradients of the 2B-class layer's rows on their way into the 8-bit input gradient
        dict(name="quantize_rows_e5m2", op="quantize_rows", dtype="bf16", rows=28672, d=896,
             f8="e5m2"),
        # one projection of all 64 experts of the 16B layer after an update of the float32 weights
        dict(name="quantize_blocks_f32", op="quantize_blocks", dtype="f32", groups=64, n=1408,
             k=2048, f8="e4m3"),
        # one projection of the 16B layer's 64 experts over a prefill batch: 8192 tokens, top-6
        dict(name="f8_prefill", op="f8", f8="e4m3", dtype="bf16", rows=49152, tail=0, groups=64,
             n=1408, k=2048, skew=0.0),
        # the same layer's down projection for a decode batch of 64 tokens: six rows an expert
        dict(name="f8_decode", op="f8", f8="e4m3", dtype="bf16", rows=384, tail=0, groups=64,
             n=2048, k=1408, skew=0.0),
        # a small model with odd widths, an odd row count, experts without tokens, float32 results
        dict(name="f8_odd_f32", op="f8", f8="e4m3", dtype="f32", rows=1021, tail=3, groups=16,
             n=136, k=267, skew=1.5),
        # training step of the 2B-class layer: input gradient of one projection, 4096 tokens, top-7
        dict(name="f8_dx_e5m2", op="f8_dx", f8="e5m2", dtype="bf16", rows=28672, tail=0, groups=63,
             n=896, k=1280, skew=0.3),
        # balance loss of the 2B-class layer's training batch and its gradient
        dict(name="balance_2b", op="balance", rows=4096, experts=63, top=7, sequences=1,
             padded=0.0, devices=0),
        # the 145B-class layer: eight padded sequences, each with a loss of its own, eight devices
        dict(name="balance_145b", op="balance", rows=16384, experts=128, top=12, sequences=8,
             padded=0.2, devices=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """Odd widths, whole 16-byte rows of 8-bit values, whole blocks."""
    unit = rng.choice([1, 16, 128])
    return max(unit, _spread(rng, lo, hi) // unit * unit)


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm_backward", "quantize_rows", "quantize_blocks", "f8",
                     "f8", "f8_dx", "balance"])
    if op == "balance":
        experts = rng.randint(2, 256)
        return dict(op=op, rows=_spread(rng, 1, 16384), experts=experts,
                    top=rng.randint(1, min(16, experts)), sequences=_spread(rng, 1, 64),
                    padded=rng.choice([0.0, rng.uniform(0.0, 0.9)]),
                    devices=rng.choice([0, rng.randint(1, experts)]))
    case = dict(op=op, dtype=rng.choice(["bf16", "f32"]))
    if op in ("f8", "f8_dx"):
        case |= dict(f8=rng.choice(["e4m3", "e5m2"]), rows=_spread(rng, 1, 16384),
                     tail=rng.choice([0, 0, rng.randint(1, 40)]), groups=_spread(rng, 1, 128),
                     n=_width(rng, 24, 2048), k=_width(rng, 24, 2048),
                     skew=rng.choice([0.0, rng.uniform(0.0, 1.5)]))
    elif op == "quantize_blocks":
        case |= dict(groups=_spread(rng, 1, 32), n=_width(rng, 24, 2048), k=_width(rng, 24, 2048),
                     f8=rng.choice(["e4m3", "e5m2"]))
    else:
        case |= dict(rows=_spread(rng, 1, 16384), d=_width(rng, 64, 8192))
        if op == "quantize_rows":
            case |= dict(f8=rng.choice(["e4m3", "e5m2"]))
        else:
            case |= dict(residual=rng.random() < 0.7)
            if op == "rms_norm":
                case |= dict(f8=rng.choice(["", "e4m3", "e5m2"]))
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


def _activations(gen, rows, d):
    """Rows whose channels differ in size, as those of a trained model do."""
    return _normal(gen, rows, d) * torch.exp(0.5 * _normal(gen, 1, d))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op, dtype=_T[case.get("dtype", "f32")], f8=_F8.get(case.get("f8")))
    dt = s["dtype"]
    if op in ("f8", "f8_dx"):
        sizes = _group_sizes(case, seed)
        M, E, n, k = case["rows"] + case["tail"], case["groups"], case["n"], case["k"]
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(
            torch.int32).cuda()
        s["most"] = int(sizes.max())  # the largest group, which the plain form pads to
        rows = _activations(gen, M, k if op == "f8" else n)
        if op == "f8_dx":             # gradients: rows under gates of any size
            rows = rows * torch.exp(2.0 * _normal(gen, M, 1)) * 1e-4
        s["x"], s["xs"] = _quantize_rows(rows, s["f8"])
        s["w"], s["ws"] = _quantize_blocks(_normal(gen, E, n, k) * 0.02, torch.float8_e4m3fn)
    elif op == "quantize_blocks":
        s["x"] = (_normal(gen, case["groups"], case["n"], case["k"]) * 0.02).to(dt)
    elif op == "quantize_rows":
        s["x"] = (_activations(gen, case["rows"], case["d"]) *
                  torch.exp(2.0 * _normal(gen, case["rows"], 1)) * 1e-4).to(dt)
    elif op == "balance":
        T, N, K, S = case["rows"], case["experts"], case["top"], case["sequences"]
        logits = _normal(gen, T, N) + 0.7 * _normal(gen, 1, N)
        s["scores"] = torch.softmax(logits.double(), 1).float()
        s["idx"] = torch.topk(s["scores"], K, dim=1).indices.to(torch.int32)
        host = torch.Generator().manual_seed(seed + 5)
        cuts = torch.randint(0, T + 1, (S - 1,), generator=host).sort().values
        ends = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.full((1,), T)])
        s["offsets"] = ends.to(torch.int32).cuda() if S > 1 else None
        # a sequence's padding stands behind its tokens
        s["mask"] = None
        if case["padded"]:
            of = torch.bucketize(torch.arange(T), ends[1:], right=True)
            at = torch.arange(T) - ends[of]
            s["mask"] = (at < ((1 - case["padded"]) * (ends[1:] - ends[:-1]))[of]).cuda()
        D = case["devices"]
        s["devices"] = D
        s["device_of"] = None
        if D:
            s["device_of"] = (torch.arange(N) * D // N).to(torch.int32).cuda()
        s["K"], s["alpha"] = K, (0.003, 0.05)
        s["dlosses"] = torch.rand(S, 2, generator=gen, device="cuda") / S
    else:
        R, d = case["rows"], case["d"]
        s["weight"] = (1.0 + 0.1 * _normal(gen, d)).to(dt)
        s["x"] = _activations(gen, R, d).to(dt)
        if op == "rms_norm":
            s["residual"] = (3.0 * _activations(gen, R, d)).to(dt) if case["residual"] else None
        else:
            s["dy"] = _normal(gen, R, d).to(dt)
            s["dh"] = _normal(gen, R, d).to(dt) if case["residual"] else None
            # what the forward pass kept
            s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(v):
    return -(-v // BLOCK)


def _scale(values, dims, most):
    """The scale of the finite values along dims; one for a block of zeros."""
    top = torch.where(torch.isfinite(values), values.abs(), 0.0).amax(dims, keepdim=True)
    return torch.where(top > 0, (top / most).clamp_min(2.0 ** -126), 1.0)


def _held(values, f8):
    return torch.where(torch.isfinite(values), values, math.nan).to(f8)


def _quantize_rows(x, f8):
    """(q, scales) of float32 rows."""
    rows, d = x.shape
    b = _blocks(d)
    if b * BLOCK != d:
        wide = torch.zeros(rows, b * BLOCK, device=x.device)
        wide[:, :d] = x
        x = wide
    x = x.view(rows, b, BLOCK)
    scale = _scale(x, -1, _MOST[f8])
    return _held(x / scale, f8).view(rows, -1)[:, :d].contiguous(), scale.view(rows, b)


def _quantize_blocks(w, f8):
    """(q, scales) of float32 matrices."""
    E, n, k = w.shape
    nb, kb = _blocks(n), _blocks(k)
    if (nb * BLOCK, kb * BLOCK) != (n, k):
        wide = torch.zeros(E, nb * BLOCK, kb * BLOCK, device=w.device)
        wide[:, :n, :k] = w
        w = wide
    w = w.view(E, nb, BLOCK, kb, BLOCK)
    scale = _scale(w, (2, 4), _MOST[f8])
    q = _held(w / scale, f8).view(E, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous()
    return q, scale.view(E, nb, kb)


def _rows_of(q, scales, dtype=torch.float32):
    return q.to(dtype) * scales.to(dtype).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _matrices_of(q, scales, dtype=torch.float32):
    wide = scales.to(dtype).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.to(dtype) * wide.repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]


def _plain_f8(s):
    off = s["offsets"].long()
    M, E, most = s["x"].shape[0], s["w"].shape[0], max(1, s["most"])
    rows = torch.arange(M, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    inside = e < E
    e, rows = e[inside], rows[inside]
    pos = rows - off[e]
    x, w = _rows_of(s["x"], s["xs"]), _matrices_of(s["w"], s["ws"])
    xp = torch.zeros(E, most, x.shape[1], device=x.device)
    xp[e, pos] = x[rows]
    yp = torch.matmul(xp, w.transpose(1, 2) if s["op"] == "f8" else w)
    y = torch.zeros(M, yp.shape[2], device=x.device, dtype=s["dtype"])
    y[rows] = yp[e, pos].to(s["dtype"])
    return y


def _plain_rms_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (s["x"].float() + s["residual"].float()).to(s["dtype"])
    hf = h.float()
    rstd = (hf.square().mean(1) + EPS).rsqrt()
    y = hf * rstd[:, None] * s["weight"].float()
    out = dict(h=h, rstd=rstd)
    if s["f8"] is None:
        return out | dict(y=y.to(s["dtype"]))
    q, scales = _quantize_rows(y, s["f8"])
    return out | dict(q=q, scales=scales)


def _plain_rms_norm_backward(s):
    r = s["rstd"][:, None]
    xh, dy = s["x"].float() * r, s["dy"].float()
    g = dy * s["weight"].float()
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * r
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(s["dtype"]), dweight=(dy * xh).sum(0))


def _plain_balance(s):
    scores, idx, K = s["scores"], s["idx"].long(), s["K"]
    T, N = scores.shape
    S = s["dlosses"].shape[0]
    rows = torch.arange(T, device=scores.device)
    seq = torch.zeros_like(rows)
    if s["offsets"] is not None:
        seq = torch.searchsorted(s["offsets"][1:].long().contiguous(), rows, right=True)
    real = torch.ones_like(rows) if s["mask"] is None else s["mask"].double()
    # sums over a sequence's rows as products with its membership, whole numbers exact in float64
    of = (seq == torch.arange(S, device=rows.device)[:, None]).double() * real
    n = of.sum(1)
    most = n.clamp_min(1)[:, None]
    picked = torch.zeros(T, N, dtype=torch.float64, device=rows.device)
    picked.scatter_add_(1, idx, torch.ones(T, K, dtype=torch.float64, device=rows.device))
    counts = of @ picked
    P = of @ scores.double() / most
    f = N * counts / (K * most)
    expert = s["alpha"][0] * f
    device = torch.zeros_like(f)
    if s["devices"]:
        member = (s["device_of"][:, None] == torch.arange(s["devices"], device=rows.device)).double()
        device = s["alpha"][1] * ((f @ member) / member.sum(0)) @ member.t()
    losses = torch.stack([(expert * P).sum(1), (device * P).sum(1)], 1)
    d = s["dlosses"].double()
    slope = ((d[:, :1] * expert + d[:, 1:] * device) / most).float()[seq]
    dlogits = scores * (slope - (scores * slope).sum(1, keepdim=True)) * real.float()[:, None]
    return dict(losses=losses.float(), counts=counts.to(torch.int32), P=P.float(), dlogits=dlogits)


# ---------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if own:
        import mixture_experts_ffn_fp32_amd as moe

        if op == "f8":
            return moe.grouped_matmul_quantized(s["x"], s["xs"], s["w"], s["ws"], s["offsets"],
                                                out_dtype=s["dtype"])
        if op == "f8_dx":
            return moe.grouped_matmul_quantized_dx(s["x"], s["xs"], s["w"], s["ws"], s["offsets"],
                                                   out_dtype=s["dtype"])
        if op == "quantize_rows":
            q, scales = moe.quantize_rows(s["x"], s["f8"])
            return dict(q=q, scales=scales)
        if op == "quantize_blocks":
            q, scales = moe.quantize_blocks(s["x"], s["f8"])
            return dict(q=q, scales=scales)
        if op == "rms_norm":
            if s["f8"] is None:
                y, h, rstd = moe.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
                return dict(y=y, h=h, rstd=rstd)
            q, scales, h, rstd = moe.rms_norm_quantized(s["x"], s["weight"], s["residual"], eps=EPS,
                                                        q_dtype=s["f8"])
            return dict(q=q, scales=scales, h=h, rstd=rstd)
        if op == "rms_norm_backward":
            dx, dweight = moe.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dh"])
            return dict(dx=dx, dweight=dweight)
        b = moe.balance_loss(s["scores"], s["idx"], offsets=s["offsets"], mask=s["mask"],
                             device_of=s["device_of"], devices=s["devices"], alpha1=s["alpha"][0],
                             alpha2=s["alpha"][1])
        dlogits = moe.balance_loss_backward(s["scores"], b["slopes"], s["dlosses"],
                                            offsets=s["offsets"], mask=s["mask"])
        return dict(losses=b["losses"], counts=b["counts"], P=b["P"], dlogits=dlogits)
    if op == "quantize_rows":
        q, scales = _quantize_rows(s["x"].float(), s["f8"])
        return dict(q=q, scales=scales)
    if op == "quantize_blocks":
        q, scales = _quantize_blocks(s["x"].float(), s["f8"])
        return dict(q=q, scales=scales)
    return {"f8": _plain_f8, "f8_dx": _plain_f8, "rms_norm": _plain_rms_norm,
            "rms_norm_backward": _plain_rms_norm_backward, "balance": _plain_balance}[op](s)


# ---------------------------------------------------------------- work and exact values
def work(case):
    op = case["op"]
    if op == "balance":
        T, N, K, S = case["rows"], case["experts"], case["top"], case["sequences"]
        return dict(bytes=8 * T * N + 4 * T * K + 8 * S * N + 16 * S, flops=5 * T * N)
    es = _SIZE[case["dtype"]]
    if op in ("f8", "f8_dx"):
        R, E, n, k = case["rows"], min(case["groups"], case["rows"]), case["n"], case["k"]
        into, out = (k, n) if op == "f8" else (n, k)
        return dict(bytes=R * (into + 4 * _blocks(into) + es * out) +
                    E * (n * k + 4 * _blocks(n) * _blocks(k)), flops=2 * R * n * k)
    if op == "quantize_blocks":
        E, n, k = case["groups"], case["n"], case["k"]
        return dict(bytes=E * ((es + 1) * n * k + 4 * _blocks(n) * _blocks(k)), flops=3 * E * n * k)
    R, d = case["rows"], case["d"]
    if op == "quantize_rows":
        return dict(bytes=R * ((es + 1) * d + 4 * _blocks(d)), flops=3 * R * d)
    extra = 1 if case["residual"] else 0
    if op == "rms_norm":
        # without a residual h is x itself
        out = 1 + 4 / BLOCK if case["f8"] else es
        return dict(bytes=R * d * (es * (1 + 2 * extra) + out) + es * d + 4 * R, flops=6 * R * d)
    return dict(bytes=es * ((3 + extra) * R * d + d) + 4 * R + 4 * d, flops=9 * R * d)


def _exact_quantized(v, f8):
    """(values before they are rounded, scales) along the rows of v, in float64.  None for the
    values in e5m2: their two bits of mantissa are rounded away by more than says anything."""
    rows, d = v.shape
    scale = torch.ones(rows, _blocks(d), dtype=torch.float64, device=v.device)
    for b in range(_blocks(d)):
        scale[:, b] = v[:, b * BLOCK:(b + 1) * BLOCK].abs().max(dim=1).values / _MOST[f8]
    scale[scale == 0] = 1.0
    at = torch.arange(d, device=v.device) // BLOCK
    return None if f8 == torch.float8_e5m2 else v / scale[:, at], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("f8", "f8_dx"):
        off = s["offsets"].tolist()
        x = s["x"].double()
        at = torch.arange(x.shape[1], device=x.device) // BLOCK
        x *= s["xs"].double()[:, at]
        n, k = s["w"].shape[1:]
        rn, rk = (torch.arange(v, device=x.device) // BLOCK for v in (n, k))
        y = torch.zeros(x.shape[0], n if op == "f8" else k, dtype=torch.float64, device=x.device)
        for e in range(len(off) - 1):
            w = s["w"][e].double() * s["ws"][e].double()[rn][:, rk]
            y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ (w.t() if op == "f8" else w)
        return y
    if op == "quantize_rows":
        q, scales = _exact_quantized(s["x"].double(), s["f8"])
        return dict(q=q, scales=scales)
    if op == "quantize_blocks":
        E, n, k = s["x"].shape
        scale = torch.empty(E, _blocks(n), _blocks(k), dtype=torch.float64, device="cuda")
        for i in range(_blocks(n)):
            for j in range(_blocks(k)):
                part = s["x"][:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                scale[:, i, j] = part.abs().amax((1, 2)).double() / _MOST[s["f8"]]
        rn, rk = (torch.arange(v, device="cuda") // BLOCK for v in (n, k))
        q = None if s["f8"] == torch.float8_e5m2 else s["x"].double() / scale[:, rn][:, :, rk]
        return dict(q=q, scales=scale)
    if op == "balance":
        N, K = s["scores"].shape[1], s["K"]
        T, S = s["scores"].shape[0], s["dlosses"].shape[0]
        ends = [0, T] if s["offsets"] is None else s["offsets"].tolist()
        z = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        P, losses = torch.zeros(S, N, dtype=torch.float64), torch.zeros(S, 2, dtype=torch.float64)
        counts = torch.zeros(S, N, dtype=torch.int32)
        for q in range(S):
            rows = torch.arange(ends[q], ends[q + 1], device="cuda")
            if s["mask"] is not None:
                rows = rows[s["mask"][rows]]
            if not len(rows):
                continue
            sc = s["scores"][rows].double()
            picked = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=N)
            f = N / (K * len(rows)) * picked.double()
            c = [s["alpha"][0] * f, torch.zeros_like(f)]
            for g in range(s["devices"]):
                of = s["device_of"] == g
                c[1][of] = s["alpha"][1] * f[of].mean()
            mean = sc.mean(0)
            P[q], counts[q] = mean.cpu(), picked.to(torch.int32).cpu()
            losses[q, 0], losses[q, 1] = float(c[0] @ mean), float(c[1] @ mean)
            d = s["dlosses"][q].double()
            ds = (d[0] * c[0] + d[1] * c[1]) / len(rows)
            z[rows] = sc * (ds - (sc @ ds)[:, None])
        return dict(losses=losses, counts=counts, P=P, dlogits=z)
    x, w = s["x"].double(), s["weight"].double()
    if op == "rms_norm":
        h = x
        if s["residual"] is not None:
            h = x + s["residual"].double()
        kept = h.to(s["dtype"]).double()  # the stream is what the next layer reads: rounded
        rstd = 1.0 / torch.sqrt((kept * kept).sum(1) / kept.shape[1] + EPS)
        y = kept * w * rstd[:, None]
        if s["f8"] is None:
            return dict(h=h, rstd=rstd, y=y)
        q, scales = _exact_quantized(y, s["f8"])
        return dict(h=h, rstd=rstd, q=q, scales=scales)
    r, dy = s["rstd"].double()[:, None], s["dy"].double()
    xh = x * r
    dx = r * (dy * w - xh * (((dy * xh) @ w) / x.shape[1])[:, None])
    if s["dh"] is not None:
        dx += s["dh"].double()
    return dict(dx=dx, dweight=torch.einsum("rd,rd->d", dy, xh))
