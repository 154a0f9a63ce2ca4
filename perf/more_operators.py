"""What is measured of the operators for an expert block with RMS norms, scored routing and 8-bit
activation checkpoints, and on which sizes.

Four operators, each as a user's program calls it, beside its plain form in elementary torch operations:

  rms         RMS norm with the residual's addition, forward and backward with the weight's gradient;
              for serving, the form that writes the FP8 rows and 1x128 scales of the fused expert layer
  scores      the router over sigmoid or softmax scores: a bias for balance, groups of experts, top-k,
              renormalised and scaled gate weights, and the gradient of the logits
  swiglu      silu(gate) * up over the experts' gate and up rows, with its gradient; with a checkpoint in
              8 bits, from which the backward pass takes the gradient and the activation again
  checkpoint  rows kept in 8 bits for the backward pass, and restored there

The checkpoints' format: 32 neighbours of a row share the power of two X = 2^floor(log2(largest
magnitude)), not below 2^-120, and each is a whole number of X/64 between -127 and 127 (nearest, ties to even).

`own` says which side run() computes: False is the plain form, True the framework's kernels.
"""
import math

import torch

own = False

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases ----
def listed():
    return [
        # one decode step of 128 sequences: the norm ahead of the fused expert layer, the residual stream
        # updated on the way
        dict(name="rms fp8 decode", op="rms_fp8", T=128, H=7168, dtype="bfloat16", residual=True),
        # a training step on the large batch: forward, and backward with the stream's own gradient
        dict(name="rms train large", op="rms_train", T=16384, H=4096, dtype="bfloat16", residual=True),
        # a training step on an odd number of tokens, rows off 16-byte boundaries
        dict(name="rms train odd", op="rms_train", T=6001, H=2003, dtype="float16", residual=True),
        # the router of a decode step: 32 experts in 4 groups, 2 of them kept, top 8, sigmoid scores
        dict(name="scores decode", op="scores_fwd", T=128, E=32, topk=8, groups=4, kept=2, top=2, dtype="float32", score="sigmoid",
             bias=True, renormalize=True, scale=2.5, masked=0.0),
        # the router of a training step on the large batch, part of its tokens padding
        dict(name="scores train large", op="scores_train", T=16384, E=128, topk=8, groups=8, kept=4, top=2, dtype="bfloat16",
             score="sigmoid", bias=True, renormalize=True, scale=2.5, masked=0.05),
        # softmax scores of the skewed batch's experts less one token, kept as they are, one group
        dict(name="scores train softmax", op="scores_train", T=8191, E=64, topk=6, groups=1, kept=1, top=1, dtype="float32",
             score="softmax", bias=False, renormalize=False, scale=1.0, masked=0.0),
        # the expert rows of a decode step
        dict(name="swiglu decode", op="swiglu_fwd", M=1024, I=2048, dtype="bfloat16"),
        # a training step on the skewed batch's expert rows, kept in 8 bits between forward and backward
        dict(name="swiglu train checkpoint", op="swiglu_checkpoint", M=65536, I=2048, dtype="bfloat16"),
        # a training step that keeps the rows themselves; odd width, rows off 16-byte boundaries
        dict(name="swiglu train odd", op="swiglu_train", M=7001, I=1403, dtype="float16"),
        # the down products' rows of the prefill batch through the 8-bit form
        dict(name="checkpoint prefill", op="checkpoint", M=32768, H=7168, dtype="bfloat16"),
        # the same for a ragged batch in 32 bits, groups that end inside 32 values
        dict(name="checkpoint ragged", op="checkpoint", M=5003, H=1500, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fp8", "rms_train", "rms_train", "scores_fwd", "scores_train", "scores_train", "swiglu_fwd",
                     "swiglu_train", "swiglu_checkpoint", "swiglu_checkpoint", "checkpoint", "checkpoint"])
    half = rng.choice(["bfloat16", "float16"])
    any_type = rng.choice([half, half, "float32"])
    while True:
        if op == "rms_fp8":
            return dict(op=op, T=_log(rng, 1, 16384), H=128 * _log(rng, 1, 56), dtype=half, residual=rng.random() < 0.7)
        if op == "rms_train":
            H = rng.choice([8 * _log(rng, 4, 1024), _log(rng, 32, 8192)])
            c = dict(op=op, T=_log(rng, 1, 16384), H=H, dtype=any_type, residual=rng.random() < 0.7)
            if c["T"] * H > 16384 * 4096:
                continue
            return c
        if op.startswith("scores"):
            groups = rng.choice([1, 1, 2, 4, 8])
            per = _log(rng, 2, 256 // groups)
            kept = rng.randint(1, groups)
            return dict(op=op, T=_log(rng, 1, 16384), E=groups * per, topk=rng.randint(1, min(8, kept * per)), groups=groups, kept=kept,
                        top=rng.randint(1, 2), dtype=rng.choice(["float32", half]), score=rng.choice(["sigmoid", "sigmoid", "softmax"]),
                        bias=rng.random() < 0.7, renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]))
        if op.startswith("swiglu"):
            I = rng.choice([8 * _log(rng, 4, 512), _log(rng, 32, 4096)])
            c = dict(op=op, M=_log(rng, 1, 65536), I=I, dtype=any_type)
            if c["M"] * I * (2 if any_type == "float32" else 1) > 65536 * 2048:
                continue
            return c
        H = rng.choice([8 * _log(rng, 4, 1024), _log(rng, 32, 8192)])
        c = dict(op=op, M=_log(rng, 1, 65536), H=H, dtype=any_type)
        if c["M"] * H * (2 if any_type == "float32" else 1) > 32768 * 7168:
            continue
        return c


# ------------------------------------------------------------------------------ inputs ----
def _gen(seed, n):
    return torch.Generator(device="cuda").manual_seed(seed * 1013 + n)


def _normal(g, *shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def prepare(case, seed):
    op, dt = case["op"], DT[case["dtype"]]
    g = _gen(seed, 3)
    s = {"case": case}
    if op.startswith("rms"):
        T, H = case["T"], case["H"]
        # a residual stream whose channels differ in spread, and a block's output to be added to it
        s["x"] = _normal(g, T, H, dtype=dt, std=0.7)
        s["residual"] = None
        if case["residual"]:
            s["residual"] = (_normal(g, T, H, dtype=torch.float32) * (0.5 + 2 * torch.rand(H, generator=g, device="cuda"))).to(dt)
        s["weight"] = _normal(g, H, dtype=dt, std=0.1, mean=1.0)
        if op == "rms_train":
            s["dy"] = _normal(g, T, H, dtype=dt)
            s["dh"] = _normal(g, T, H, dtype=dt) if case["residual"] else None
    elif op.startswith("scores"):
        T, E = case["T"], case["E"]
        s["logits"] = _normal(g, T, E, dtype=dt, std=1.5)
        # what steps of 0.001 against the experts' loads leave after some hundred batches
        s["bias"] = (torch.randint(-200, 201, (E,), generator=g, device="cuda").float() * 0.001) if case["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"] if case["masked"] else None
        if op == "scores_train":
            s["dw"] = _normal(g, T, case["topk"], dtype=torch.float32)
    elif op.startswith("swiglu"):
        M, I = case["M"], case["I"]
        s["gu"] = _normal(g, M, 2 * I, dtype=dt, std=1.5)
        if op != "swiglu_fwd":
            s["dact"] = _normal(g, M, I, dtype=dt)
    else:
        # rows of different size, as experts give them
        size = torch.exp(_normal(g, case["M"], 1, dtype=torch.float32, std=1.0))
        s["x"] = (_normal(g, case["M"], case["H"], dtype=torch.float32) * size).to(dt)
    return s


# --------------------------------------------------------------------- the plain forms ----
def _plain_rms(x, residual, weight):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hf = h.float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(1) + EPS)
    return h, rstd, hf * rstd[:, None] * weight.float()


def _plain_fp8(y):
    v = y.view(y.shape[0], -1, 128)
    sf = v.abs().amax(2).clamp_min(1e-4) / 448.0
    return (v / sf[:, :, None]).to(torch.float8_e4m3fn).view(y.shape), sf


def _plain_rms_backward(dy, dh, h, weight, rstd):
    d = dy.float()
    xh = h.float() * rstd[:, None]
    a = d * weight.float()
    dx = (a - xh * (a * xh).mean(1, keepdim=True)) * rstd[:, None]
    if dh is not None:
        dx = dx + dh.float()
    return dx.to(h.dtype), (d * xh).sum(0).to(weight.dtype)


def _plain_scores(case, logits, bias, mask):
    T, E = logits.shape
    G, k = case["groups"], case["topk"]
    l = logits.double()   # the choice is made next to borders between nearly equal values
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        s = p / p.sum(1, keepdim=True)
    c = s if bias is None else s + bias.double()
    if G > 1:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[:, :, : case["top"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        c = torch.where(keep[:, :, None], c.view(T, G, E // G), -math.inf).view(T, E)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.float().gather(1, idx)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    if mask is not None:
        idx = torch.where(mask[:, None], idx, -1)
        w = torch.where(mask[:, None], w, 0.0)
    return idx, w


def _plain_scores_backward(case, dw, idx, w, logits):
    l = logits.float()
    at = idx.clamp_min(0)
    dot = (w * dw).sum(1, keepdim=True)
    if case["score"] == "softmax" and not case["renormalize"]:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        d = torch.where(idx < 0, 0.0, dw) * case["scale"]
        dl = p * (torch.zeros_like(l).scatter_add_(1, at, d) - dot)
        return torch.where((idx < 0).all(1, keepdim=True), 0.0, dl).to(logits.dtype)
    d = w * (dw - dot / case["scale"]) if case["renormalize"] else w * dw
    if case["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(l.gather(1, at)))
    return torch.zeros_like(l).scatter_add_(1, at, torch.where(idx < 0, 0.0, d)).to(logits.dtype)


def _plain_silu(g):
    return 1.0 / (1.0 + torch.exp(-g))


def _plain_swiglu(gu):
    g, u = gu.float().chunk(2, dim=1)
    return g * _plain_silu(g) * u


def _plain_swiglu_backward(dact, gu):
    g, u = gu.float().chunk(2, dim=1)
    d, s = dact.float(), _plain_silu(g)
    return torch.cat([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], 1).to(dact.dtype)


def _plain_checkpoint(x):
    """The values that rows stand for in 8 bits."""
    M, H = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -H % 32)).view(M, -1, 32)
    big = v.abs().amax(2, keepdim=True)
    fraction, _ = torch.frexp(big)   # in [1/2, 1)
    step = torch.where(big > 0, big / (2.0 * fraction), 0.0).clamp_min(2.0 ** -120) / 64.0
    return ((v / step).round().clamp(-127, 127) * step).view(M, -1)[:, :H]


# ------------------------------------------------------------------------------- a pass ----
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from combine_persistent_warp_gb300 import ops
        if op == "rms_fp8":
            q, sf, h = ops.rms_norm_fp8(s["x"], s["weight"], EPS, residual=s["residual"])
            return {"q": q.view(torch.float8_e4m3fn), "sf": sf, "h": h}
        if op == "rms_train":
            y, rstd, h = ops.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
            dx, dweight = ops.rms_norm_backward(s["dy"], h, s["weight"], rstd, dh=s["dh"])
            return {"y": y, "rstd": rstd, "h": h, "dx": dx, "dweight": dweight}
        if op.startswith("scores"):
            idx, w = ops.route_scores(s["logits"], case["topk"], score=case["score"], bias=s["bias"], groups=case["groups"],
                                      topk_groups=case["kept"], group_top=case["top"], renormalize=case["renormalize"],
                                      scale=case["scale"], token_mask=s["mask"])
            r = {"idx": idx, "w": w}
            if op == "scores_train":
                r["dlogits"] = ops.route_scores_backward(s["dw"], idx, w, s["logits"], score=case["score"],
                                                         renormalize=case["renormalize"], scale=case["scale"])
            return r
        if op == "swiglu_fwd":
            return ops.swiglu(s["gu"])
        if op == "swiglu_train":
            return {"act": ops.swiglu(s["gu"]), "dgu": ops.swiglu_backward(s["dact"], s["gu"])}
        if op == "swiglu_checkpoint":
            act, codes, scales = ops.swiglu_checkpoint(s["gu"])
            dgu, again = ops.swiglu_checkpoint_backward(s["dact"], codes, scales)
            return {"act": act, "dgu": dgu, "again": again}
        codes, scales = ops.checkpoint_rows(s["x"])
        return ops.restore_rows(codes, scales, s["x"].dtype)
    if op.startswith("rms"):
        h, rstd, y = _plain_rms(s["x"], s["residual"], s["weight"])
        if op == "rms_fp8":
            q, sf = _plain_fp8(y)
            return {"q": q, "sf": sf, "h": h}
        dx, dweight = _plain_rms_backward(s["dy"], s["dh"], h, s["weight"], rstd)
        return {"y": y.to(h.dtype), "rstd": rstd, "h": h, "dx": dx, "dweight": dweight}
    if op.startswith("scores"):
        idx, w = _plain_scores(case, s["logits"], s["bias"], s["mask"])
        r = {"idx": idx, "w": w}
        if op == "scores_train":
            r["dlogits"] = _plain_scores_backward(case, s["dw"], idx, w, s["logits"])
        return r
    if op == "swiglu_fwd":
        return _plain_swiglu(s["gu"]).to(s["gu"].dtype)
    if op == "swiglu_train":
        return {"act": _plain_swiglu(s["gu"]).to(s["gu"].dtype), "dgu": _plain_swiglu_backward(s["dact"], s["gu"])}
    if op == "swiglu_checkpoint":
        kept = torch.cat([_plain_checkpoint(half) for half in s["gu"].chunk(2, dim=1)], 1)
        return {"act": _plain_swiglu(s["gu"]).to(s["gu"].dtype), "dgu": _plain_swiglu_backward(s["dact"], kept),
                "again": _plain_swiglu(kept).to(s["gu"].dtype)}
    return _plain_checkpoint(s["x"]).to(s["x"].dtype)


# ------------------------------------------------------------------- what it cannot avoid ----
def work(case):
    op, b = case["op"], DT[case["dtype"]].itemsize
    if op.startswith("rms"):
        T, H = case["T"], case["H"]
        n, r = T * H, int(case["residual"])
        if op == "rms_fp8":   # x and the residual read, the stream, codes and scales written
            return {"bytes": n * b * (1 + 2 * r) + n + n // 128 * 4 + H * b, "flops": (7 + r) * n}
        # the same with y and rstd; dy, h and the stream's gradient read, dx written
        return {"bytes": n * b * (2 + 2 * r) + n * b * (3 + r) + 4 * H * b + 8 * T, "flops": (15 + 2 * r) * n}
    if op.startswith("scores"):
        n, m = case["T"] * case["E"], case["T"] * case["topk"]
        by = n * b + m * 12
        return {"bytes": by + (m * 4 + n * b if op == "scores_train" else 0), "flops": 6 * n + 10 * m}
    if op.startswith("swiglu"):
        n = case["M"] * case["I"]
        if op == "swiglu_fwd":
            return {"bytes": 3 * n * b, "flops": 5 * n}
        if op == "swiglu_train":   # gate and up once forward; they and the gradient read, theirs written
            return {"bytes": 8 * n * b, "flops": 16 * n}
        kept = 2 * n + 2 * n // 32   # 8-bit gate and up with a byte for 32 of them
        return {"bytes": 3 * n * b + kept + n * b + kept + 3 * n * b, "flops": 26 * n}
    n = case["M"] * case["H"]
    return {"bytes": 2 * n * b + 2 * (n + n // 32), "flops": 5 * n}


# -------------------------------------------------------------------- in 64 bits, apart ----
def _exact_kept(x):
    """Rows in 8 bits: the power of two is the largest magnitude's 64-bit word without its fraction."""
    M, H = x.shape
    pad = torch.zeros(M, (H + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    pad[:, :H] = x.double()
    v = pad.view(M, -1, 32)
    big = v.abs().max(2, keepdim=True).values.clamp_min(2.0 ** -120)
    power = (big.view(torch.int64) >> 52 << 52).view(torch.float64)
    n = torch.round(v * 64.0 / power)
    return (torch.minimum(torch.maximum(n, torch.full_like(n, -127.0)), torch.full_like(n, 127.0)) * power / 64.0).view(M, -1)[:, :H]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op.startswith("rms"):
        h = s["x"].to(D)
        if s["residual"] is not None:
            h = (h + s["residual"].to(D)).to(s["x"].dtype).to(D)   # the stream is kept in its type
        n = h.shape[1]
        g = s["weight"].to(D)
        r = torch.rsqrt(torch.einsum("th,th->t", h, h) / n + EPS)
        y = r[:, None] * h * g
        if op == "rms_fp8":
            peak = y.abs().reshape(-1, n // 128, 128).max(2).values
            return {"q": None, "sf": torch.maximum(peak, torch.full_like(peak, 1e-4)) / 448.0, "h": h}
        d = s["dy"].to(D)
        dot = torch.einsum("th,th,h->t", d, h, g)
        dx = r[:, None] * d * g - (r * r * r * dot / n)[:, None] * h
        if s["dh"] is not None:
            dx = dx + s["dh"].to(D)
        return {"y": y, "rstd": r, "h": h, "dx": dx, "dweight": torch.einsum("th,th,t->h", d, h, r)}
    if op.startswith("scores"):
        T, E, k, G = case["T"], case["E"], case["topk"], case["groups"]
        l = s["logits"].to(D)
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        c = score.clone() if s["bias"] is None else score + s["bias"].to(D)[None, :]
        ids = torch.arange(E, device=l.device)

        def first_largest(v, count):
            left, seen = v.clone(), []
            for _ in range(count):
                m = left.max(1, keepdim=True).values
                at = torch.where(left == m, torch.arange(v.shape[1], device=v.device), v.shape[1]).min(1).values
                seen.append(at)
                left.scatter_(1, at[:, None], -math.inf)
            return torch.stack(seen, 1)

        if G > 1:
            parts = torch.stack([c[:, i * (E // G): (i + 1) * (E // G)].topk(case["top"], 1).values.sum(1) for i in range(G)], 1)
            groups = first_largest(parts, case["kept"])
            c = c.masked_fill(~(groups[:, :, None] == (ids // (E // G))[None, None, :]).any(1), -math.inf)
        idx = first_largest(c, k)
        chosen = score.gather(1, idx)
        total = chosen.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(chosen[:, :1])
        w = case["scale"] * chosen / total
        keep = torch.ones(T, dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"]
        r = {"idx": None, "w": w.masked_fill(~keep[:, None], 0.0)}
        if op == "scores_train":
            dw = s["dw"].to(D)
            # by the chain: to the chosen scores, then to the logits
            ds = case["scale"] * dw / total
            if case["renormalize"]:
                ds = ds - (ds * chosen).sum(1, keepdim=True) / total
            full = torch.zeros(T, E, dtype=D, device=l.device).scatter_(1, idx, ds)
            if case["score"] == "sigmoid":
                dl = full * score * (1 - score)
            else:
                dl = score * (full - (full * score).sum(1, keepdim=True))
            r["dlogits"] = dl.masked_fill(~keep[:, None], 0.0)
        return r
    if op == "checkpoint":
        return _exact_kept(s["x"])
    I = case["I"]

    def act(a):
        return a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]

    gu = s["gu"].to(D)
    if op == "swiglu_fwd":
        return act(gu)
    at = gu if op == "swiglu_train" else torch.cat([_exact_kept(s["gu"][:, :I]), _exact_kept(s["gu"][:, I:])], 1)
    g, d = at[:, :I], s["dact"].to(D)
    p = torch.sigmoid(g)
    dgu = torch.cat([d * at[:, I:] * (p + g * p * (1 - p)), d * g * p], 1)
    if op == "swiglu_train":
        return {"act": act(gu), "dgu": dgu}
    return {"act": act(gu), "dgu": dgu, "again": act(at)}
