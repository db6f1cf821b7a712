"""The operators of a mixture-of-experts layer in FP8, as cases to time and compare.

Each case is one pass through an operator, in its plain form (elementary torch operations in 32 bits,
64 where a choice between near scores hangs on the last digits) or, with ``own`` set, through the calls
of this package:

  route     scores of the experts, the choice of top_k of them for each token, the order of the rows by
            expert, and the gradient of the logits
  combine   the weighted sum of the chosen experts' rows for each token, forward and backward
  mm        the matrix product of FP8 codes under 1x128 groups and 128x128 blocks of scales: a linear
            layer forward, its input gradient and its weight gradient
  experts   the same product with one weight for each expert, rows gathered by expert; and the two
            gradients of a training step

Scales follow the package's convention: codes hold fl(x * S), so a value is decode(code) / S.
"""
import math

import torch

own = False

GROUP = 128
DEV = "cuda"
E4M3, E5M2 = "e4m3", "e5m2"
_F8 = {E4M3: (torch.float8_e4m3fn, 448.0), E5M2: (torch.float8_e5m2, 57344.0)}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of 64 sequences: sigmoid scores, balance bias, 4 of 8 groups; latency counts
        {"name": "route_tokens", "op": "route", "tokens": 64, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "renorm": True, "scale": 2.5, "dtype": "fp32", "align": 1,
         "backward": False},
        # a training step's batch: softmax over 128 experts, bf16 logits, rows padded to groups of 128
        {"name": "route_step", "op": "route", "tokens": 16384, "experts": 128, "top_k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0, "dtype": "bf16", "align": 128,
         "backward": True},
        # the same decoding step's sum over its experts' rows
        {"name": "combine_tokens", "op": "combine", "tokens": 64, "experts": 64, "top_k": 8, "dim": 7168, "align": 1,
         "backward": False},
        # a training step: sum, and the gradients of rows and weights
        {"name": "combine_step", "op": "combine", "tokens": 8192, "experts": 64, "top_k": 8, "dim": 4096,
         "align": 128, "backward": True},
        # one token through a large linear layer: the weight is read once
        {"name": "mm_token", "op": "mm", "kind": "nk", "m": 1, "n": 7168, "k": 18432, "fmt_a": E4M3, "fmt_b": E4M3,
         "pow2": False, "out": "bf16"},
        # a few sequences' worth of rows and sizes that divide by nothing
        {"name": "mm_odd", "op": "mm", "kind": "nk", "m": 333, "n": 4101, "k": 4104, "fmt_a": E4M3, "fmt_b": E4M3,
         "pow2": False, "out": "bf16"},
        # forward of a large linear layer on a batch of 8192 tokens
        {"name": "mm_forward", "op": "mm", "kind": "nk", "m": 8192, "n": 7168, "k": 18432, "fmt_a": E4M3,
         "fmt_b": E4M3, "pow2": False, "out": "bf16"},
        # input gradient: E5M2 gradients times the weight as the forward pass stored it
        {"name": "mm_input_grad", "op": "mm", "kind": "kn", "m": 4096, "n": 4096, "k": 14336, "fmt_a": E5M2,
         "fmt_b": E4M3, "pow2": False, "out": "bf16"},
        # weight gradient in fp32: both operands in 1x128 groups along the tokens
        {"name": "mm_weight_grad", "op": "mm", "kind": "groups", "m": 7168, "n": 4096, "k": 8192, "fmt_a": E5M2,
         "fmt_b": E4M3, "pow2": False, "out": "fp32"},
        # 64 decoded tokens, 8 of 64 experts each: about 8 rows to a weight
        {"name": "experts_tokens", "op": "experts", "tokens": 64, "experts": 64, "top_k": 8, "n": 4096, "k": 7168,
         "fmt_a": E4M3, "fmt_b": E4M3, "pow2": False},
        # a prompt of 4096 tokens
        {"name": "experts_prompt", "op": "experts", "tokens": 4096, "experts": 64, "top_k": 8, "n": 4096, "k": 7168,
         "fmt_a": E4M3, "fmt_b": E4M3, "pow2": False},
        # a training step's two gradients of the experts' product, power-of-two scales
        {"name": "experts_grad", "op": "experts_grad", "tokens": 4096, "experts": 32, "top_k": 4, "n": 4096,
         "k": 4096, "fmt_a": E5M2, "fmt_b": E4M3, "pow2": True},
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["route", "combine", "mm", "mm", "experts", "experts_grad"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 16, 20, 32]) if groups > 1 else rng.choice([8, 60, 64, 128, 160, 256])
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "tokens": _log_int(rng, 16, 16384), "experts": experts,
                "top_k": rng.choice([1, 2, 4, 6, 8]), "score": score, "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": max(1, groups // 2), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "dtype": rng.choice(["bf16", "fp32"]), "align": rng.choice([1, 16, 128]),
                "backward": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "tokens": _log_int(rng, 16, 8192), "experts": rng.choice([8, 32, 64]),
                "top_k": rng.choice([1, 2, 4, 8]), "dim": _log_int(rng, 256, 4096, 8), "align": rng.choice([1, 128]),
                "backward": rng.random() < 0.5}
    if op == "mm":
        kind = rng.choice(["nk", "nk", "kn", "groups"])
        m = _log_int(rng, 1, 8192)
        n = _log_int(rng, 512, 8192, 8 if kind == "kn" else 1)
        k = _log_int(rng, 512, 16384, rng.choice([8, 16, 128]))
        if kind == "groups":
            m = _log_int(rng, 512, 8192)
        return {"op": op, "kind": kind, "m": m, "n": n, "k": k, "fmt_a": E4M3 if kind == "nk" else E5M2,
                "fmt_b": E4M3, "pow2": rng.random() < 0.4, "out": "fp32" if kind == "groups" else "bf16"}
    if op == "experts":
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "experts": rng.choice([8, 16, 40]),
                "top_k": rng.choice([1, 2, 4, 6]), "n": _log_int(rng, 512, 4096, 8), "k": _log_int(rng, 512, 7168, 16),
                "fmt_a": E4M3, "fmt_b": E4M3, "pow2": rng.random() < 0.4}
    return {"op": op, "tokens": _log_int(rng, 64, 4096), "experts": rng.choice([4, 8, 16]),
            "top_k": rng.choice([1, 2, 4]), "n": _log_int(rng, 512, 4096, 16), "k": _log_int(rng, 512, 4096, 16),
            "fmt_a": E5M2, "fmt_b": E4M3, "pow2": rng.random() < 0.6}


# ---- inputs ----------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _activation(gen, rows, cols):
    """Tokens with heavy tails: a magnitude for each row, rare large channels."""
    x = _normal(gen, rows, cols)
    x *= torch.exp(0.6 * _normal(gen, rows, 1))
    x *= 1.0 + 15.0 * (torch.rand(1, cols, generator=gen, device=DEV) < 0.002)
    return x


def _quantize(x, fmt, block_rows, pow2):
    """Codes (uint8) and scales S of groups of block_rows x 128; partial groups at the edges."""
    dt, top = _F8[fmt]
    r, c = x.shape
    gr, gc = -(-r // block_rows), -(-c // GROUP)
    pad = torch.zeros(gr * block_rows, gc * GROUP, device=x.device, dtype=x.dtype)
    pad[:r, :c] = x
    pad = pad.view(gr, block_rows, gc, GROUP)
    amax = pad.abs().amax(dim=(1, 3))
    s = torch.where(amax > 0, top / amax, torch.ones_like(amax))
    if pow2:
        s = (s.view(torch.int32) & 0x7F800000).view(torch.float32)      # the power of two below
    q = (pad * s[:, None, :, None]).clamp_(-top, top).to(dt).view(torch.uint8)
    return q.view(gr * block_rows, gc * GROUP)[:r, :c].contiguous(), s.contiguous()


def _weights(gen, experts, n, k, fmt, pow2):
    """[experts][n][k] codes and their 128x128 scales, one expert at a time."""
    q = torch.empty(experts, n, k, dtype=torch.uint8, device=DEV)
    s = torch.empty(experts, -(-n // GROUP), -(-k // GROUP), dtype=torch.float32, device=DEV)
    for e in range(experts):
        q[e], s[e] = _quantize(0.02 * _normal(gen, n, k), fmt, GROUP, pow2)
    return q, s


def _choices(gen, tokens, experts, top_k):
    """Distinct experts for each token, some experts chosen more often than others."""
    popularity = 0.7 * _normal(gen, 1, experts)
    u = torch.rand(tokens, experts, generator=gen, device=DEV).clamp_min_(1e-9)
    return torch.sort(popularity - torch.log(-torch.log(u)), dim=1, descending=True)[1][:, :top_k].to(torch.int32).contiguous()


def _padded_rows(choices, experts, align):
    return -(-(choices + min(experts, choices) * (align - 1)) // align) * align


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["logits"] = (1.5 * _normal(gen, t, e) + 0.5 * _normal(gen, 1, e)).to(dt)
        st["bias"] = 0.05 * _normal(gen, e) if case["bias"] else None
        if case["backward"]:
            st["dweights"] = _normal(gen, t, case["top_k"])
    elif op == "combine":
        ids = _choices(gen, case["tokens"], case["experts"], case["top_k"])
        _, st["rows"], st["slots"] = _plain_order(ids, case["experts"], case["align"])
        st["x"] = _normal(gen, st["rows"].numel(), case["dim"]).to(torch.bfloat16)
        st["x"][st["rows"] < 0] = 0
        st["weights"] = torch.softmax(_normal(gen, case["tokens"], case["top_k"]), dim=1)
        if case["backward"]:
            st["dy"] = (1e-2 * _normal(gen, case["tokens"], case["dim"])).to(torch.bfloat16)
    elif op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        if case["fmt_a"] == E5M2:
            xa = _normal(gen, m, k) * torch.exp(1.5 * _normal(gen, m, 1)) * 1e-3
        else:
            xa = _activation(gen, m, k)
        st["a"], st["sa"] = _quantize(xa, case["fmt_a"], 1, case["pow2"])
        del xa
        if case["kind"] == "groups":
            st["b"], st["sb"] = _quantize(_activation(gen, n, k), case["fmt_b"], 1, case["pow2"])
        else:
            shape = (n, k) if case["kind"] == "nk" else (k, n)
            st["b"], st["sb"] = _quantize(0.02 * _normal(gen, *shape), case["fmt_b"], GROUP, case["pow2"])
    elif op == "experts":
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        ids = _choices(gen, t, e, case["top_k"])
        st["offsets"], st["rows"], _ = _plain_order(ids, e, 1)
        st["bounds"] = st["offsets"].tolist()
        st["a"], st["sa"] = _quantize(_activation(gen, t, k), case["fmt_a"], 1, case["pow2"])
        st["b"], st["sb"] = _weights(gen, e, n, k, case["fmt_b"], case["pow2"])
    else:  # experts_grad: dy [rows][n], x [rows][k], w [e][n][k]; dx = dy w, dw = dy^T x
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        ids = _choices(gen, t, e, case["top_k"])
        st["offsets"], rows, _ = _plain_order(ids, e, GROUP)
        st["bounds"] = st["offsets"].tolist()
        keep = (rows >= 0)[:, None]
        r = rows.numel()
        dy = torch.where(keep, 1e-3 * _normal(gen, r, n) * torch.exp(_normal(gen, r, 1)), 0.0)
        st["dy"], st["sdy"] = _quantize(dy, case["fmt_a"], 1, case["pow2"])
        st["dyt"], st["sdyt"] = _quantize(dy.t().contiguous(), case["fmt_a"], 1, case["pow2"])
        del dy
        x = torch.where(keep, _activation(gen, r, k), 0.0)
        st["xt"], st["sxt"] = _quantize(x.t().contiguous(), case["fmt_b"], 1, case["pow2"])
        del x
        st["w"], st["sw"] = _weights(gen, e, n, k, case["fmt_b"], case["pow2"])
    return st


# ---- plain forms -----------------------------------------------------------------------------

def _values(q, s, fmt, block_rows):
    """decode(q) / S in fp32; S holds groups of block_rows x 128."""
    v = q.view(_F8[fmt][0]).to(torch.float32)
    r, c = q.shape
    return v / s.repeat_interleave(block_rows, dim=0)[:r].repeat_interleave(GROUP, dim=1)[:, :c]


def _plain_route(case, logits, bias):
    l64 = logits.to(torch.float64)
    s = torch.softmax(l64, dim=1) if case["score"] == "softmax" else torch.sigmoid(l64)
    if bias is None and case["groups"] == 1:
        choice = l64                                 # scores rise with the logits
    else:
        choice = s if bias is None else s + bias.to(torch.float64)
    if case["groups"] > 1:
        t, e = choice.shape
        by_group = choice.view(t, case["groups"], e // case["groups"])
        two = torch.sort(by_group, dim=2, descending=True)[0][:, :, :2].sum(dim=2)
        best = torch.sort(two, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        kept = torch.zeros_like(two, dtype=torch.bool).scatter_(1, best, True)
        choice = by_group.masked_fill(~kept[:, :, None], -math.inf).view(t, e)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :case["top_k"]]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * case["scale"]).to(torch.float32)


def _plain_route_backward(case, logits, ids, dweights):
    l32 = logits.to(torch.float32)
    idx = ids.to(torch.int64)
    s = torch.softmax(l32, dim=1) if case["score"] == "softmax" else torch.sigmoid(l32)
    g = dweights * case["scale"]
    chosen = s.gather(1, idx)
    if case["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        g = (g - (g * chosen).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, g)
    if case["score"] == "softmax":
        d = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    else:
        d = ds * s * (1.0 - s)
    return d.to(logits.dtype)


def _plain_order(ids, experts, align):
    """Rows by expert, in the order of the tokens; each expert's rows start at a multiple of align."""
    t, k = ids.shape
    flat = ids.reshape(-1).to(torch.int64)
    key, perm = torch.sort(flat, stable=True)
    counts = torch.zeros(experts, dtype=torch.int64, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    padded = (counts + align - 1) // align * align
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(padded, 0)
    first = torch.cumsum(counts, 0) - counts
    slot_sorted = offsets[key] + torch.arange(t * k, device=ids.device) - first[key]
    slots = torch.empty_like(flat).scatter_(0, perm, slot_sorted)
    rows = torch.full((_padded_rows(t * k, experts, align),), -1, dtype=torch.int64, device=ids.device)
    rows.scatter_(0, slot_sorted, perm // k)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.view(t, k).to(torch.int32)


def _plain_combine(x, weights, slots):
    y = torch.zeros(slots.shape[0], x.shape[1], dtype=torch.float32, device=x.device)
    for j in range(slots.shape[1]):
        y += weights[:, j:j + 1] * x[slots[:, j].to(torch.int64)].to(torch.float32)
    return y.to(x.dtype)


def _plain_combine_backward(dy, x, weights, slots):
    d32 = dy.to(torch.float32)
    dx = torch.zeros_like(x)
    dw = []
    for j in range(slots.shape[1]):
        at = slots[:, j].to(torch.int64)
        dw.append((d32 * x[at].to(torch.float32)).sum(dim=1))
        dx[at] = (weights[:, j:j + 1] * d32).to(x.dtype)
    return dx, torch.stack(dw, dim=1)


def _plain_mm(st, case):
    a = _values(st["a"], st["sa"], case["fmt_a"], 1)
    if case["kind"] == "groups":
        y = a @ _values(st["b"], st["sb"], case["fmt_b"], 1).t()
    else:
        b = _values(st["b"], st["sb"], case["fmt_b"], GROUP)
        y = a @ (b.t() if case["kind"] == "nk" else b)
    return y.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)


def _plain_experts(st, case):
    a = _values(st["a"], st["sa"], case["fmt_a"], 1)[st["rows"].to(torch.int64)]
    y = torch.zeros(a.shape[0], case["n"], dtype=torch.bfloat16, device=a.device)
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if hi > lo:
            y[lo:hi] = (a[lo:hi] @ _values(st["b"][e], st["sb"][e], case["fmt_b"], GROUP).t()).to(torch.bfloat16)
    return y


def _plain_experts_grad(st, case):
    dy = _values(st["dy"], st["sdy"], case["fmt_a"], 1)
    dyt = _values(st["dyt"], st["sdyt"], case["fmt_a"], 1)
    xt = _values(st["xt"], st["sxt"], case["fmt_b"], 1)
    dx = torch.zeros(dy.shape[0], case["k"], dtype=torch.bfloat16, device=dy.device)
    dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float32, device=dy.device)
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if hi > lo:
            dx[lo:hi] = (dy[lo:hi] @ _values(st["w"][e], st["sw"][e], case["fmt_b"], GROUP)).to(torch.bfloat16)
            dw[e] = dyt[:, lo:hi] @ xt[:, lo:hi].t()
    return dx, dw


# ---- one pass --------------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        ids, w = _plain_route(case, st["logits"], st["bias"])
        out = (ids, w) + _plain_order(ids, case["experts"], case["align"])
        if case["backward"]:
            out += (_plain_route_backward(case, st["logits"], ids, st["dweights"]),)
        return out
    if op == "combine":
        y = _plain_combine(st["x"], st["weights"], st["slots"])
        if not case["backward"]:
            return (y,)
        return (y,) + _plain_combine_backward(st["dy"], st["x"], st["weights"], st["slots"])
    if op == "mm":
        return (_plain_mm(st, case),)
    if op == "experts":
        return (_plain_experts(st, case),)
    return _plain_experts_grad(st, case)


def _run_own(st):
    import mx_block_scaled_amax_amd as qf8
    case = st["case"]
    op = case["op"]
    fmt = {E4M3: qf8.E4M3, E5M2: qf8.E5M2}
    if op == "route":
        score = qf8.SCORE_SOFTMAX if case["score"] == "softmax" else qf8.SCORE_SIGMOID
        ids, w = qf8.route_experts(st["logits"], case["top_k"], score=score, bias=st["bias"], groups=case["groups"],
                                   top_groups=case["top_groups"], renorm=case["renorm"], scale=case["scale"])
        out = (ids, w) + tuple(qf8.order_experts(ids, case["experts"], align=case["align"]))
        if case["backward"]:
            out += (qf8.route_experts_backward(st["logits"], ids, st["dweights"], score=score,
                                               renorm=case["renorm"], scale=case["scale"]),)
        return out
    if op == "combine":
        y = qf8.combine_experts(st["x"], st["weights"], st["slots"])
        if not case["backward"]:
            return (y,)
        return (y,) + tuple(qf8.combine_experts_backward(st["dy"], st["x"], st["weights"], st["slots"], st["rows"]))
    if op == "mm":
        kind = {"nk": qf8.WEIGHT_NK, "kn": qf8.WEIGHT_KN, "groups": qf8.GROUPS_NK}[case["kind"]]
        out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        return (qf8.matmul_block(st["a"], st["sa"], st["b"], st["sb"], fmt[case["fmt_a"]], fmt[case["fmt_b"]], kind,
                                 pow2_scales=case["pow2"], out_dtype=out),)
    if op == "experts":
        return (qf8.matmul_block_experts(st["a"], st["sa"], st["b"], st["sb"], st["offsets"], fmt[case["fmt_a"]],
                                         fmt[case["fmt_b"]], qf8.WEIGHT_NK, rows=st["rows"],
                                         pow2_scales=case["pow2"]),)
    fa, fb = fmt[case["fmt_a"]], fmt[case["fmt_b"]]
    dx = qf8.matmul_block_experts(st["dy"], st["sdy"], st["w"], st["sw"], st["offsets"], fa, fb, qf8.WEIGHT_KN,
                                  pow2_scales=case["pow2"])
    dw = qf8.matmul_block_experts_wgrad(st["dyt"], st["sdyt"], st["xt"], st["sxt"], st["offsets"], fa, fb,
                                        pow2_scales=case["pow2"])
    return dx, dw


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        el = 2 if case["dtype"] == "bf16" else 4
        rows = _padded_rows(t * k, e, case["align"])
        nbytes = t * e * el + (4 * e if case["bias"] else 0) + t * k * 8 + (e + 1) * 4 + rows * 4 + t * k * 4
        flops = t * e * 4
        if case["backward"]:
            nbytes += t * e * el + t * k * 4
            flops += t * e * 4
        return {"bytes": nbytes, "flops": flops}
    if op == "combine":
        t, k, d = case["tokens"], case["top_k"], case["dim"]
        nbytes = t * k * d * 2 + t * k * 8 + t * d * 2
        flops = 2 * t * k * d
        if case["backward"]:
            rows = _padded_rows(t * k, case["experts"], case["align"])
            nbytes += t * d * 2 + rows * d * 2 + t * k * 4
            flops += 3 * t * k * d
        return {"bytes": nbytes, "flops": flops}
    n, k = case["n"], case["k"]
    gk = -(-k // GROUP)
    if op == "mm":
        m = case["m"]
        sb = n * gk if case["kind"] == "groups" else -(-n // GROUP) * gk
        return {"bytes": m * k + n * k + 4 * (m * gk + sb) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    rows = case["tokens"] * case["top_k"]
    used = min(case["experts"], rows)
    weight = used * (n * k + 4 * -(-n // GROUP) * gk)
    if op == "experts":
        return {"bytes": case["tokens"] * (k + 4 * gk) + weight + rows * n * 2 + rows * 4 + 4 * (case["experts"] + 1),
                "flops": 2 * rows * n * k}
    padded = _padded_rows(rows, case["experts"], GROUP)
    return {"bytes": rows * (n + 4 * -(-n // GROUP)) + weight + padded * k * 2 + rows * (n + k) * (1 + 4 / GROUP)
                     + case["experts"] * n * k * 4,
            "flops": 4 * rows * n * k}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_values(q, s, fmt, block_rows):
    """The values that the codes stand for, in fp64: every block divided by its own scale."""
    v = q.view(_F8[fmt][0]).to(torch.float64)
    for g in range(s.shape[1]):
        cols = slice(g * GROUP, min((g + 1) * GROUP, q.shape[1]))
        if block_rows == 1:
            v[:, cols] /= s[:, g:g + 1].to(torch.float64)
        else:
            per_row = s[:, g].to(torch.float64)[torch.arange(q.shape[0], device=q.device) // block_rows]
            v[:, cols] /= per_row[:, None]
    return v


def _exact_route(case, st):
    x = st["logits"].to(torch.float64)
    t, e = x.shape
    if case["score"] == "softmax":
        p = torch.exp(x - x.max(dim=1, keepdim=True)[0])
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = p.clone() if st["bias"] is None else p + st["bias"].to(torch.float64)
    lane = torch.arange(e, device=x.device)
    if case["groups"] > 1:
        size = e // case["groups"]
        g1, at = c.view(t, -1, size).max(dim=2)
        rest = c.view(t, -1, size).clone().scatter_(2, at[:, :, None], -math.inf)
        value = g1 + rest.max(dim=2)[0]
        open_ = torch.zeros(t, case["groups"], dtype=torch.bool, device=x.device)
        index = torch.arange(case["groups"], device=x.device)
        for _ in range(case["top_groups"]):
            top = value.max(dim=1, keepdim=True)[0]
            pick = torch.where(value == top, index, case["groups"]).min(dim=1)[0]
            open_[torch.arange(t, device=x.device), pick] = True
            value[torch.arange(t, device=x.device), pick] = -math.inf
        c = torch.where(open_[:, lane // size], c, -math.inf)
    ids = torch.empty(t, case["top_k"], dtype=torch.int64, device=x.device)
    for j in range(case["top_k"]):
        top = c.max(dim=1, keepdim=True)[0]
        ids[:, j] = torch.where(c == top, lane, e).min(dim=1)[0]
        c.scatter_(1, ids[:, j:j + 1], -math.inf)
    chosen = p.gather(1, ids)
    norm = chosen.sum(dim=1, keepdim=True) if case["renorm"] else torch.ones(t, 1, dtype=torch.float64, device=x.device)
    out = [ids.to(torch.int32), case["scale"] * chosen / norm]
    # the order of the rows, expert by expert
    flat = ids.reshape(-1)
    offsets = [0]
    rows = torch.full((_padded_rows(t * case["top_k"], e, case["align"]),), -1, dtype=torch.int32, device=x.device)
    slots = torch.empty(t * case["top_k"], dtype=torch.int32, device=x.device)
    for i in range(e):
        at = torch.nonzero(flat == i)[:, 0]
        lo = offsets[-1]
        rows[lo:lo + at.numel()] = (at // case["top_k"]).to(torch.int32)
        slots[at] = torch.arange(lo, lo + at.numel(), dtype=torch.int32, device=x.device)
        offsets.append(lo + -(-at.numel() // case["align"]) * case["align"])
    out += [torch.tensor(offsets, dtype=torch.int32, device=x.device), rows, slots.view(t, case["top_k"])]
    if case["backward"]:
        # w_j = scale * p_j / norm, so dL/dp_j follows by the quotient rule, then the score's own slope
        g = case["scale"] * st["dweights"].to(torch.float64)
        w = chosen / norm
        dp = (g - (g * w).sum(dim=1, keepdim=True)) / norm if case["renorm"] else g
        full = torch.zeros_like(p).scatter_(1, ids, dp)
        if case["score"] == "softmax":
            out.append(p * full - p * (p * full).sum(dim=1, keepdim=True))
        else:
            out.append(full * p / (1.0 + torch.exp(x)))
    return tuple(out)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "combine":
        x, w, at = st["x"].to(torch.float64), st["weights"].to(torch.float64), st["slots"].to(torch.int64)
        t, k = at.shape
        y = torch.cat([torch.bmm(w[i:i + 256, None, :], x[at[i:i + 256]])[:, 0] for i in range(0, t, 256)])
        if not case["backward"]:
            return (y,)
        dy = st["dy"].to(torch.float64)
        flat = at.reshape(-1)
        dw = torch.cat([torch.bmm(x[at[i:i + 256]], dy[i:i + 256, :, None])[:, :, 0] for i in range(0, t, 256)])
        del x
        dx = torch.zeros(st["x"].shape, dtype=torch.float64, device=DEV)
        dx[flat] = w.reshape(-1, 1) * dy[torch.arange(t * k, device=DEV) // k]
        return y, dx, dw
    if op == "mm":
        a = _exact_values(st["a"], st["sa"], case["fmt_a"], 1)
        b = _exact_values(st["b"], st["sb"], case["fmt_b"], 1 if case["kind"] == "groups" else GROUP)
        return (torch.matmul(a, b if case["kind"] == "kn" else b.t()),)
    lo_hi = list(zip(st["bounds"], st["bounds"][1:]))
    if op == "experts":
        a = _exact_values(st["a"], st["sa"], case["fmt_a"], 1)
        y = torch.zeros(st["rows"].numel(), case["n"], dtype=torch.float64, device=DEV)
        for e, (lo, hi) in enumerate(lo_hi):
            token = st["rows"][lo:hi].to(torch.int64)
            y[lo:hi] = torch.matmul(a[token], _exact_values(st["b"][e], st["sb"][e], case["fmt_b"], GROUP).t())
        return (y,)
    dy = _exact_values(st["dy"], st["sdy"], case["fmt_a"], 1)
    dyt = _exact_values(st["dyt"], st["sdyt"], case["fmt_a"], 1)
    xt = _exact_values(st["xt"], st["sxt"], case["fmt_b"], 1)
    dx = torch.zeros(dy.shape[0], case["k"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(lo_hi):
        dx[lo:hi] = torch.matmul(dy[lo:hi], _exact_values(st["w"][e], st["sw"][e], case["fmt_b"], GROUP))
        dw[e] = torch.matmul(dyt[:, lo:hi], xt[:, lo:hi].t())
    return dx, dw
