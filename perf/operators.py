"""What is measured of the operators around the expert layer, and on which sizes.

Four operators of a trainable (or served) Mixture-of-Experts block, each as a user's program calls
it, beside its plain form in elementary torch operations:

  norm     layer norm over the hidden dimension, forward and backward with the sums of the
           weight's and the bias's gradients; for serving, the form that writes the FP8 rows and
           1x128 scales that the fused expert layer reads
  route    the router: top-k experts of each token with their gate weights, the expert-major
           order of the chosen (token, slot) pairs, and the gradient of the logits
  rows     rows moved into that order and weighted back out of it, with the gradients of the rows
           and of the gate weights
  grouped  matrix products with one weight per expert over ragged groups of rows: the forward
           product, the gradient of the rows and the gradient of the weights

`own` says which side run() computes: False is the plain form, True the framework's kernels.
"""
import math

import torch

own = False

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------------------- cases ----
def listed():
    return [
        # one decode step of 128 sequences at the framework's decode sizes: the norm ahead of the
        # fused expert layer, written as the FP8 rows and scales that it reads
        dict(name="norm fp8 decode", op="norm_fp8", T=128, H=7168, dtype="bfloat16"),
        # a training step on the large batch: forward and backward
        dict(name="norm train large", op="norm_train", T=16384, H=4096, dtype="bfloat16"),
        # a training step on a batch of odd length and a hidden size with unaligned rows, in 32 bits
        dict(name="norm train odd", op="norm_train", T=4099, H=1001, dtype="float32"),
        # the router of a decode step: 32 experts, top 8
        dict(name="route decode", op="route_fwd", T=128, E=32, topk=8, dtype="float32", masked=0.0),
        # the router of a training step on the large batch, part of its tokens padding; forward,
        # order and the logits' gradient
        dict(name="route train large", op="route_train", T=16384, E=128, topk=8, dtype="bfloat16", masked=0.05),
        # a decode step's expert outputs weighted back into token order
        dict(name="rows combine decode", op="rows_combine", T=128, E=32, topk=8, H=7168, dtype="bfloat16", skew=0.0, skip=0.0),
        # the large batch's rows gathered into expert order
        dict(name="rows gather large", op="rows_gather", T=16384, E=128, topk=8, H=4096, dtype="bfloat16", skew=0.0, skip=0.0),
        # a training step on the skewed batch, 5% of its slots skipped: combine and its gradients
        dict(name="rows train skewed", op="rows_train", T=8192, E=64, topk=8, H=7168, dtype="bfloat16", skew=1.2, skip=0.05),
        # a decode step's products: about 32 rows for each of 32 experts, bound by reading the weights
        dict(name="grouped decode", op="grouped_y", T=128, E=32, topk=8, N=4096, K=7168, dtype="bfloat16", skew=0.0, skip=0.0),
        # the prefill batch's gate and up product
        dict(name="grouped prefill", op="grouped_y", T=4096, E=32, topk=8, N=4096, K=7168, dtype="bfloat16", skew=0.0, skip=0.0),
        # the gradient of the down product's rows, ragged groups of odd lengths, skipped slots, fp16
        dict(name="grouped dx ragged", op="grouped_dx", T=8192, E=64, topk=8, N=7168, K=2048, dtype="float16", skew=0.4, skip=0.05),
        # the gradient of the down weights on the large batch
        dict(name="grouped dw large", op="grouped_dw", T=16384, E=128, topk=8, N=4096, K=1536, dtype="bfloat16", skew=0.0, skip=0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _not_3072(n, step):
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm_fp8", "norm_train", "route_fwd", "route_train", "rows_combine", "rows_gather",
                     "rows_train", "grouped_y", "grouped_y", "grouped_dx", "grouped_dx", "grouped_dw", "grouped_dw"])
    half = rng.choice(["bfloat16", "float16"])
    while True:
        T = _log(rng, 1, 16384)
        E = _log(rng, 1, 128)
        k = rng.randint(1, min(8, E))
        if op == "norm_fp8":
            c = dict(op=op, T=T, H=_not_3072(128 * _log(rng, 1, 56), 128), dtype=half)
        elif op == "norm_train":
            c = dict(op=op, T=T, H=_not_3072(_log(rng, 32, 8192), 1), dtype=rng.choice([half, half, "float32"]))
            if c["T"] * c["H"] > 16384 * 4096:
                continue
        elif op in ("route_fwd", "route_train"):
            E = _log(rng, 2, 256)
            c = dict(op=op, T=T, E=E, topk=rng.randint(1, min(8, E)), dtype=rng.choice(["float32", half]), masked=rng.choice([0.0, 0.1]))
        elif op.startswith("rows"):
            H = _not_3072(rng.choice([8 * _log(rng, 4, 896), _log(rng, 32, 7168)]), 8)
            c = dict(op=op, T=T, E=E, topk=k, H=H, dtype=rng.choice([half, half, "float32"]), skew=rng.choice([0.0, 0.8]), skip=rng.choice([0.0, 0.05]))
            if T * k * H * (2 if c["dtype"] == "float32" else 1) > 65536 * 7168:
                continue
        else:
            N, K = (_not_3072(8 * _log(rng, 8, 896), 8) for _ in range(2))
            c = dict(op=op, T=T, E=E, topk=k, N=N, K=K, dtype=half, skew=rng.choice([0.0, 0.4]), skip=rng.choice([0.0, 0.05]))
            if T * k * N * K > 32768 * 4096 * 7168 or E * N * K > 32 * 4096 * 7168:
                continue
        return c


# ------------------------------------------------------------------------------ inputs ----
def _gen(seed, n):
    return torch.Generator(device="cuda").manual_seed(seed * 1009 + n)


def _normal(g, *shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _routing(case, seed):
    """Chosen experts [T, topk] without repeats inside a token (-1: skipped), and gate weights."""
    g = _gen(seed, 77)
    T, E, k = case["T"], case["E"], case["topk"]
    s = torch.randn(T, E, generator=g, device="cuda")
    if case["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        s = s - case["skew"] * rank.log()
    s = s - torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-6)))
    top = s.topk(k, dim=1)
    idx = top.indices
    w = torch.softmax(top.values, dim=1)
    if case["skip"]:
        idx = idx.masked_fill(torch.rand(T, k, generator=g, device="cuda") < case["skip"], -1)
    return idx.contiguous(), w.contiguous()


def _expert_major(idx, E):
    """offsets [E+1] and the row [T, k] of each (token, slot) in expert-major order: by expert,
    then token, then slot; -1 for a skipped slot."""
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    at = torch.argsort(key, stable=True)
    rows = torch.empty_like(at)
    rows[at] = torch.arange(at.numel(), device=at.device)
    rows = torch.where(flat < 0, -1, rows).view_as(idx).to(torch.int32)
    counts = (key[None, :] == torch.arange(E, device=idx.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, rows


def prepare(case, seed):
    op, dt = case["op"], DT[case["dtype"]]
    T = case["T"]
    g = _gen(seed, 1)
    s = {"case": case}
    if op.startswith("norm"):
        H = case["H"]
        # a residual stream: channels of different spread, a mean of its own
        s["x"] = _normal(g, T, H, dtype=torch.float32) * (0.5 + torch.rand(H, generator=g, device="cuda"))
        s["x"] = (s["x"] + 0.3).to(dt)
        s["weight"] = _normal(g, H, dtype=dt, std=0.1, mean=1.0)
        s["bias"] = _normal(g, H, dtype=dt, std=0.1)
        if op == "norm_train":
            s["dy"] = _normal(g, T, H, dtype=dt)
    elif op.startswith("route"):
        E, k = case["E"], case["topk"]
        s["logits"] = _normal(g, T, E, dtype=dt, std=1.5)
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"] if case["masked"] else None
        if op == "route_train":
            s["dw"] = _normal(g, T, k, dtype=torch.float32)
    else:
        E, k = case["E"], case["topk"]
        idx, w = _routing(case, seed)
        s["offsets"], s["rows"] = _expert_major(idx, E)
        sizes = s["offsets"].diff().cpu()
        s["total"], s["largest"] = int(sizes.sum()), int(sizes.max())
        if op == "rows_gather":
            s["x"] = _normal(g, T, case["H"], dtype=dt)
        elif op.startswith("rows"):
            s["w"] = w
            s["y"] = _normal(g, T * k, case["H"], dtype=dt)
            if op == "rows_train":
                s["dout"] = _normal(g, T, case["H"], dtype=dt)
        else:
            N, K = case["N"], case["K"]
            if op != "grouped_dw":
                s["weights"] = torch.empty(E, N, K, dtype=dt, device="cuda").normal_(0.0, 0.02, generator=g)
            if op != "grouped_dx":
                s["x"] = _normal(g, T * k, K, dtype=dt)
            if op != "grouped_y":
                s["dy"] = _normal(g, T * k, N, dtype=dt)
    return s


# --------------------------------------------------------------------- the plain forms ----
def _plain_norm(x, weight, bias):
    xf = x.float()
    mean = xf.mean(1)
    c = xf - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * weight.float() + bias.float()
    return y, mean, rstd


def _plain_norm_fp8(x, weight, bias):
    y, _, _ = _plain_norm(x, weight, bias)
    y = y.view(y.shape[0], -1, 128)
    sf = y.abs().amax(2).clamp_min(1e-4) / 448.0
    q = (y / sf[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(x.shape), sf


def _plain_norm_backward(dy, x, weight, mean, rstd):
    d = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    g = d * weight.float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd[:, None]
    return dx.to(x.dtype), (d * xhat).sum(0).to(weight.dtype), d.sum(0).to(weight.dtype)


def _plain_route(logits, topk, mask):
    lf = logits.float()
    val, idx = torch.sort(lf, dim=1, descending=True, stable=True)
    val, idx = val[:, :topk], idx[:, :topk]
    p = torch.exp(val - val[:, :1])
    w = p / p.sum(1, keepdim=True)
    if mask is not None:
        idx = torch.where(mask[:, None], idx, -1)
        w = torch.where(mask[:, None], w, 0.0)
    return idx, w


def _plain_route_backward(dw, idx, w, logits):
    ds = w * (dw - (w * dw).sum(1, keepdim=True))
    d = torch.zeros(logits.shape, dtype=torch.float32, device=logits.device)
    ds = torch.where(idx < 0, 0.0, ds)
    return d.scatter_add_(1, idx.clamp_min(0), ds).to(logits.dtype)


def _plain_gather(x, rows):
    T, k = rows.shape
    out = torch.zeros(T * k + 1, x.shape[1], dtype=x.dtype, device=x.device)
    flat = rows.reshape(-1).long()
    out[torch.where(flat < 0, T * k, flat)] = x.repeat_interleave(k, 0)
    out[T * k] = 0
    return out[: T * k]


def _plain_combine(y, rows, w):
    flat = rows.long()
    v = y[flat.clamp_min(0)].float() * w[:, :, None]
    return torch.where((flat < 0)[:, :, None], 0.0, v).sum(1).to(y.dtype)


def _plain_combine_backward(dout, y, rows, w):
    T, k = rows.shape
    flat = rows.reshape(-1).long()
    d = dout.float()
    dw = (y[flat.clamp_min(0)].float().view(T, k, -1) * d[:, None, :]).sum(2)
    dw = torch.where(rows < 0, 0.0, dw)
    dy = torch.zeros(T * k + 1, y.shape[1], dtype=y.dtype, device=y.device)
    dy[torch.where(flat < 0, T * k, flat)] = (w[:, :, None] * d[:, None, :]).to(y.dtype).view(T * k, -1)
    dy[T * k] = 0
    return dy[: T * k], dw


def _place(s):
    """The (expert, place in its group) of every row, for a batch padded to the largest group."""
    r = torch.arange(s["total"], device=s["offsets"].device)
    off = s["offsets"].long()
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return e, r - off[e]


def _padded(v, s, e, at):
    E = s["offsets"].numel() - 1
    p = torch.zeros(E, max(1, s["largest"]), v.shape[1], dtype=torch.float32, device=v.device)
    p[e, at] = v[: s["total"]].float()
    return p


def _plain_grouped(v, w, s):
    """rows of v times w[expert], w [E, in, out] in 32 bits, over groups padded to the largest."""
    e, at = _place(s)
    out = torch.zeros(v.shape[0], w.shape[2], dtype=v.dtype, device=v.device)
    out[: s["total"]] = torch.bmm(_padded(v, s, e, at), w)[e, at].to(v.dtype)
    return out


def _plain_grouped_dw(dy, x, s):
    e, at = _place(s)
    return torch.bmm(_padded(dy, s, e, at).transpose(1, 2), _padded(x, s, e, at)).to(x.dtype)


# ------------------------------------------------------------------------------- a pass ----
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from combine_persistent_warp_gb300 import ops
        if op == "norm_fp8":
            q, sf = ops.layer_norm_fp8(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"q": q.view(torch.float8_e4m3fn), "sf": sf}
        if op == "norm_train":
            y, mean, rstd = ops.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
            dx, dweight, dbias = ops.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
            return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dweight, "dbias": dbias}
        if op in ("route_fwd", "route_train"):
            idx, w = ops.route_topk(s["logits"], case["topk"], token_mask=s["mask"])
            order = ops.expert_order(idx, case["E"])
            r = {"idx": idx, "w": w, "offsets": order.offsets, "rows": order.rows}
            if op == "route_train":
                r["dlogits"] = ops.route_topk_backward(s["dw"], idx, w, s["logits"])
            return r
        if op == "rows_gather":
            return ops.gather_rows(s["x"], s["rows"], s["offsets"])
        if op == "rows_combine":
            return ops.combine_rows(s["y"], s["rows"], s["w"])
        if op == "rows_train":
            out = ops.combine_rows(s["y"], s["rows"], s["w"])
            dy, dw = ops.combine_rows_backward(s["dout"], s["y"], s["rows"], s["w"], s["offsets"])
            return {"out": out, "dy": dy, "dw": dw}
        if op == "grouped_y":
            return ops.grouped_mm(s["x"], s["weights"], s["offsets"])
        if op == "grouped_dx":
            return ops.grouped_mm_dx(s["dy"], s["weights"], s["offsets"])
        return ops.grouped_mm_dw(s["dy"], s["x"], s["offsets"])
    if op == "norm_fp8":
        q, sf = _plain_norm_fp8(s["x"], s["weight"], s["bias"])
        return {"q": q, "sf": sf}
    if op == "norm_train":
        y, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        dx, dweight, dbias = _plain_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd, "dx": dx, "dweight": dweight, "dbias": dbias}
    if op in ("route_fwd", "route_train"):
        idx, w = _plain_route(s["logits"], case["topk"], s["mask"])
        offsets, rows = _expert_major(idx, case["E"])
        r = {"idx": idx, "w": w, "offsets": offsets, "rows": rows}
        if op == "route_train":
            r["dlogits"] = _plain_route_backward(s["dw"], idx, w, s["logits"])
        return r
    if op == "rows_gather":
        return _plain_gather(s["x"], s["rows"])
    if op == "rows_combine":
        return _plain_combine(s["y"], s["rows"], s["w"])
    if op == "rows_train":
        out = _plain_combine(s["y"], s["rows"], s["w"])
        dy, dw = _plain_combine_backward(s["dout"], s["y"], s["rows"], s["w"])
        return {"out": out, "dy": dy, "dw": dw}
    if op == "grouped_y":
        return _plain_grouped(s["x"], s["weights"].float().transpose(1, 2), s)
    if op == "grouped_dx":
        return _plain_grouped(s["dy"], s["weights"].float(), s)
    return _plain_grouped_dw(s["dy"], s["x"], s)


# ------------------------------------------------------------------- what it cannot avoid ----
def work(case):
    op, T, b = case["op"], case["T"], DT[case["dtype"]].itemsize
    if op == "norm_fp8":
        n = T * case["H"]
        return {"bytes": n * b + n + n // 128 * 4 + 2 * case["H"] * b, "flops": 10 * n}
    if op == "norm_train":
        n = T * case["H"]  # x read and y written; dy and x read and dx written
        return {"bytes": 5 * n * b + 5 * case["H"] * b + 8 * T, "flops": 22 * n}
    if op in ("route_fwd", "route_train"):
        n, m = T * case["E"], T * case["topk"]
        by = n * b + m * (8 + 4 + 4) + 4 * (case["E"] + 1)
        return {"bytes": by + (m * 4 + n * b if op == "route_train" else 0), "flops": 4 * n + 8 * m}
    k = case["topk"]
    M = int(round(T * k * (1 - case["skip"])))
    if op.startswith("rows"):
        H = case["H"]
        if op == "rows_gather":
            return {"bytes": T * H * b + T * k * H * b + 4 * T * k, "flops": 0}
        if op == "rows_combine":
            return {"bytes": M * H * b + T * H * b + 8 * T * k, "flops": 2 * M * H}
        # combine, then dout and the rows read once more and the rows' gradient written
        return {"bytes": M * H * b + T * H * b + T * H * b + M * H * b + T * k * H * b + 20 * T * k, "flops": 5 * M * H}
    N, K, E = case["N"], case["K"], case["E"]
    used = min(E, M)
    if op == "grouped_dw":
        by = M * (N + K) * b + E * N * K * b
    else:
        by = used * N * K * b + M * (N + K) * b
    return {"bytes": by + 4 * (E + 1), "flops": 2 * M * N * K}


# -------------------------------------------------------------------- in 64 bits, apart ----
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op.startswith("norm"):
        x, g, c = s["x"].to(D), s["weight"].to(D), s["bias"].to(D)
        n = x.shape[1]
        mu = x.sum(1, keepdim=True) / n
        var = (x * x).sum(1, keepdim=True) / n - mu * mu
        r = 1.0 / torch.sqrt(var + EPS)
        h = (x - mu) * r
        y = h * g + c
        if op == "norm_fp8":
            peak = y.abs().reshape(-1, n // 128, 128).max(2).values
            return {"q": None, "sf": torch.maximum(peak, torch.full_like(peak, 1e-4)) / 448.0}
        d = s["dy"].to(D)
        a = d * g
        dx = r * (a - a.sum(1, keepdim=True) / n - h * ((a * h).sum(1, keepdim=True) / n))
        return {"y": y, "mean": mu[:, 0], "rstd": r[:, 0], "dx": dx, "dweight": torch.einsum("th,th->h", d, h), "dbias": d.sum(0)}
    if op.startswith("route"):
        k, E = case["topk"], case["E"]
        l = s["logits"].to(D)
        left = l.clone()
        seen = []
        for _ in range(k):  # the largest that is left, at its lowest index
            m = left.max(1, keepdim=True).values
            at = torch.where(left == m, torch.arange(E, device=l.device), E).min(1).values
            seen.append(at)
            left.scatter_(1, at[:, None], -math.inf)
        idx = torch.stack(seen, 1)
        w = torch.softmax(l.gather(1, idx), 1)
        keep = torch.ones(case["T"], dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"]
        idx = idx.masked_fill(~keep[:, None], -1)
        w = w.masked_fill(~keep[:, None], 0.0)
        r = {"idx": None, "w": w, "offsets": None, "rows": None}
        if op == "route_train":
            dw = s["dw"].to(D)
            eye = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
            part = (eye @ dw[:, :, None])[:, :, 0]
            hot = torch.zeros(case["T"], E + 1, dtype=D, device=l.device)
            hot.scatter_(1, torch.where(idx < 0, E, idx), part)
            r["dlogits"] = hot[:, :E]
        return r
    rows, off = s["rows"].long(), s["offsets"].tolist()
    T, k = rows.shape
    named = rows >= 0
    token = torch.full((T * k,), -1, dtype=torch.long, device=rows.device)
    token[rows[named]] = torch.nonzero(named)[:, 0]
    if op == "rows_gather":
        return torch.where(token[:, None] >= 0, s["x"][token.clamp_min(0)], torch.zeros((), dtype=s["x"].dtype, device=rows.device)).to(D)
    if op in ("rows_combine", "rows_train"):
        y = s["y"]
        gate = torch.zeros(T * k, dtype=D, device=rows.device)
        gate[rows[named]] = s["w"].to(D)[named]
        some = token >= 0
        out = torch.zeros(T, y.shape[1], dtype=D, device=rows.device)
        for j in range(k):
            hit = named[:, j]
            out[hit] += s["w"].to(D)[hit, j, None] * y[rows[hit, j]].to(D)
        if op == "rows_combine":
            return out
        dout = s["dout"]
        dy = torch.zeros(T * k, y.shape[1], dtype=D, device=rows.device)
        dw = torch.zeros(T, k, dtype=D, device=rows.device)
        dy[some] = gate[some, None] * dout[token[some]].to(D)
        for j in range(k):
            hit = named[:, j]
            dw[hit, j] = (y[rows[hit, j]].to(D) * dout[hit].to(D)).sum(1)
        return {"out": out, "dy": dy, "dw": dw}
    E, N, K = case["E"], case["N"], case["K"]
    if op == "grouped_dw":
        out = torch.zeros(E, N, K, dtype=D, device=rows.device)
        for e in range(E):
            a, b = off[e], off[e + 1]
            out[e] = s["dy"][a:b].to(D).t() @ s["x"][a:b].to(D)
        return out
    v = s["x"] if op == "grouped_y" else s["dy"]
    out = torch.zeros(T * k, N if op == "grouped_y" else K, dtype=D, device=rows.device)
    for e in range(E):
        a, b = off[e], off[e + 1]
        we = s["weights"][e].to(D)
        out[a:b] = v[a:b].to(D) @ (we.t() if op == "grouped_y" else we)
    return out
