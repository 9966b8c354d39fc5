"""Measured cases of the matrix products with block scales and of the expert layer around them.

Five operators:
  mm        one product of blockwise FP8 tensors (the Fprop, Dgrad and Wgrad of a linear layer)
  grouped   the experts' products: rows sorted by expert, one weight matrix each; and their Wgrad
  route     scores of the experts, top-k with groups and a balance bias, weights, and the gradient
  dispatch  the sorted order of the rows, and the rows gathered and quantized in that order
  combine   the weighted sum of the experts' rows for each token, and its gradients

`run` computes the plain form with elementary torch operations in 32 bits, or, where `own` is true, calls the
package's operators.  Shapes come from the linear layer (16384 x 4096 -> 14336) and the 64-expert
activations (65536 rows, hidden 7168) that bench.py quantizes.
"""
import math

import torch

own = False

E4M3, E5M2 = 0, 1
MAXIMUM = (448.0, 57344.0)
TYPES = (torch.float8_e4m3fn, torch.float8_e5m2)
NEG_INF = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token through the linear layer while serving: the weights' bytes bound it
        {"name": "mm token 1x14336x4096", "op": "mm", "kind": "fprop", "m": 1, "n": 14336, "k": 4096},
        # the layer's Dgrad for a batch whose token count is no multiple of anything; gradients in E5M2
        {"name": "mm dgrad 12345x4096x14336", "op": "mm", "kind": "dgrad", "m": 12345, "n": 4096, "k": 14336},
        # the layer's Wgrad over 16384 tokens, gradient of the weights in FP32
        {"name": "mm wgrad 14336x4096x16384", "op": "mm", "kind": "wgrad", "m": 14336, "n": 4096, "k": 16384},
        # 16 tokens with 8 experts each while serving: nearly every expert's weights are read for a few rows
        {"name": "grouped decode 128r 64e", "op": "grouped", "kind": "fprop", "rows": 128, "experts": 64, "n": 4096, "k": 7168},
        # the experts' first product for 65536 ragged rows in training
        {"name": "grouped fprop 65536r 64e", "op": "grouped", "kind": "fprop", "rows": 65536, "experts": 64, "n": 4096, "k": 7168},
        # the experts' Wgrad, rows padded to 128 for each expert
        {"name": "grouped wgrad 16384r 16e", "op": "grouped", "kind": "wgrad", "rows": 16384, "experts": 16, "n": 4096, "k": 7168},
        # routing of 16 tokens while serving: sigmoid scores, a bias, 4 of 8 groups
        {"name": "route decode 16t 64e", "op": "route", "tokens": 16, "experts": 64, "top": 8, "score": "sigmoid", "groups": 8, "top_groups": 4, "backward": False, "type": "bf16"},
        # routing of a training batch, with the gradient of the logits
        {"name": "route train 65536t 256e", "op": "route", "tokens": 65536, "experts": 256, "top": 8, "score": "softmax", "groups": 1, "top_groups": 1, "backward": True, "type": "fp32"},
        # the rows of 16 tokens sorted by expert and quantized, no padding
        {"name": "dispatch decode 16t", "op": "dispatch", "tokens": 16, "experts": 64, "top": 8, "hidden": 7168, "align": 1, "both": False},
        # a training batch: 65536 rows, padded to 128 for each expert, both copies
        {"name": "dispatch train 8192t", "op": "dispatch", "tokens": 8192, "experts": 64, "top": 8, "hidden": 7168, "align": 128, "both": True},
        # the weighted sum for 16 tokens
        {"name": "combine decode 16t", "op": "combine", "tokens": 16, "experts": 64, "top": 8, "hidden": 7168, "align": 1, "backward": False},
        # the weighted sum of a training batch, with the gradients of the rows and the weights
        {"name": "combine train 8192t", "op": "combine", "tokens": 8192, "experts": 64, "top": 8, "hidden": 7168, "align": 128, "backward": True},
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over the logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["mm", "mm", "grouped", "grouped", "route", "dispatch", "combine"])
    if op == "mm":
        kind = rng.choice(["fprop", "dgrad", "wgrad"])
        n, k = _log(rng, 256, 14336, 16), _log(rng, 256, 14336, 16)
        return {"op": op, "kind": kind, "m": _log(rng, 256, 14336, 16) if kind == "wgrad" else _log(rng, 1, 16384), "n": n, "k": k}
    if op == "grouped":
        kind = rng.choice(["fprop", "fprop", "wgrad"])
        e = _log(rng, 2, 16) if kind == "wgrad" else _log(rng, 2, 64)
        return {"op": op, "kind": kind, "rows": _log(rng, 16, 16384) if kind == "wgrad" else _log(rng, 1, 65536), "experts": e,
                "n": _log(rng, 256, 4096, 16), "k": _log(rng, 512, 7168, 16)}
    score = rng.choice(["softmax", "sigmoid"])
    top = rng.randint(1, 8)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8]) if score == "sigmoid" else 1
        e = groups * rng.randint(8, 32) if groups > 1 else _log(rng, 8, 256)
        return {"op": op, "tokens": _log(rng, 1, 65536), "experts": e, "top": top, "score": score, "groups": groups,
                "top_groups": max(1, groups // 2), "backward": rng.random() < 0.6, "type": rng.choice(["bf16", "fp32"])}
    e = _log(rng, 8, 256)
    both = rng.random() < 0.5
    case = {"op": op, "tokens": _log(rng, 1, 8192), "experts": e, "top": top, "hidden": _log(rng, 256, 7168, 16), "align": 128 if both else 1}
    case["both" if op == "dispatch" else "backward"] = both
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _blockwise(x, fmt, block_rows):
    """Codes and 1/scale of x [rows, cols] in blocks of block_rows x 128."""
    rows, cols = x.shape
    r, c = -(-rows // block_rows), -(-cols // 128)
    p = torch.zeros(r * block_rows, c * 128, device=x.device)
    p[:rows, :cols] = x
    v = p.view(r, block_rows, c, 128)
    amax = v.abs().amax((1, 3))
    scale = torch.where(amax > 0, MAXIMUM[fmt] / amax, torch.ones_like(amax))
    q = (v * scale[:, None, :, None]).clamp(-MAXIMUM[fmt], MAXIMUM[fmt]).to(TYPES[fmt])
    return q.view(torch.uint8).view(r * block_rows, c * 128)[:rows, :cols].contiguous(), 1.0 / scale


def _random(g, rows, cols, heavy):
    """Activations, weights: normal values; gradients: Student-t values with 3 degrees of freedom."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    if heavy:
        x /= (torch.randn(3, rows, 1, device="cuda", generator=g).square().sum(0) / 3).sqrt().clamp_min(0.05)
    return x.bfloat16().float()


def _top_random(g, tokens, experts, top):
    """Each token's `top` experts, some experts more wanted than others."""
    want = torch.randn(tokens, experts, device="cuda", generator=g) + 0.5 * torch.randn(1, experts, device="cuda", generator=g)
    return want.sort(1, descending=True).indices[:, :min(top, experts)].int().contiguous()


def _capacity(slots, experts, align):
    """Rows that hold `slots` rows when each expert's are padded to `align`."""
    return (slots + min(experts, slots) * (align - 1)) // align * align


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        grad = case["kind"] != "fprop"
        s["a_fmt"], s["b_fmt"] = (E5M2 if grad else E4M3), E4M3
        s["a"], s["sa"] = _blockwise(_random(g, m, k, grad), s["a_fmt"], 1)
        s["b"], s["sb"] = _blockwise(0.02 * _random(g, n, k, False), E4M3, 1 if case["kind"] == "wgrad" else 128)
    elif case["op"] == "grouped":
        e, n, k, rows = case["experts"], case["n"], case["k"], case["rows"]
        share = torch.rand(e, device="cuda", generator=g) + 0.5
        of = torch.multinomial(share, rows, replacement=True, generator=g)
        count = torch.bincount(of, minlength=e)
        if case["kind"] == "wgrad":
            count = (count + 127) // 128 * 128
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)])
        total = int(s["offsets"][-1])
        s["most"] = int(count.max())
        if case["kind"] == "wgrad":
            s["a_fmt"], s["b_fmt"] = E5M2, E4M3
            s["a"], s["sa"] = _blockwise(_random(g, n, total, True), E5M2, 1)
            s["b"], s["sb"] = _blockwise(_random(g, k, total, False), E4M3, 1)
        else:
            s["a_fmt"], s["b_fmt"] = E4M3, E4M3
            s["a"], s["sa"] = _blockwise(_random(g, total, k, False), E4M3, 1)
            s["b"] = torch.empty(e, n, k, dtype=torch.uint8, device="cuda")
            s["sb"] = torch.empty(e, -(-n // 128), -(-k // 128), device="cuda")
            for i in range(e):
                s["b"][i], s["sb"][i] = _blockwise(0.02 * _random(g, n, k, False), E4M3, 128)
    elif case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        x = torch.randn(t, e, device="cuda", generator=g) + 0.5 * torch.randn(1, e, device="cuda", generator=g)
        s["logits"] = x.bfloat16() if case["type"] == "bf16" else x
        s["bias"] = 0.05 * torch.randn(e, device="cuda", generator=g) if case["score"] == "sigmoid" else None
        s["d_weights"] = torch.randn(t, min(case["top"], e), device="cuda", generator=g)
    else:
        t, e, h = case["tokens"], case["experts"], case["hidden"]
        s["ids"] = _top_random(g, t, e, case["top"])
        slots = s["ids"].numel()
        rows = _capacity(slots, e, case["align"])
        if case["op"] == "dispatch":
            s["x"] = _random(g, t, h, True).bfloat16()
        else:
            s["offsets"], s["row_of"], s["src"] = _order(s["ids"], e, case["align"], rows)
            s["y"] = _random(g, rows, h, False).bfloat16()
            w = torch.rand(t, s["ids"].shape[1], device="cuda", generator=g) + 0.1
            s["weights"] = w / w.sum(1, keepdim=True)
            s["d_out"] = (0.01 * _random(g, t, h, True)).bfloat16()
        s["rows"] = rows
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _spread(scale, rows, cols, block_rows):
    """The scale of each element of [..., rows, cols]."""
    r = torch.arange(rows, device=scale.device) // block_rows
    c = torch.arange(cols, device=scale.device) // 128
    return scale[..., r, :][..., c]


def _values(q, scale, fmt, block_rows):
    return q.view(TYPES[fmt]).float() * _spread(scale, q.shape[-2], q.shape[-1], block_rows)


def _mm(s):
    a = _values(s["a"], s["sa"], s["a_fmt"], 1)
    if s["case"]["kind"] == "wgrad":
        return a @ _values(s["b"], s["sb"], s["b_fmt"], 1).t()
    return (a @ _values(s["b"], s["sb"], s["b_fmt"], 128).t()).bfloat16()


def _grouped(s):
    """Each expert's rows in a slab of the largest expert's size, one batched product, and back."""
    off, most = s["offsets"], s["most"]
    e = off.numel() - 1
    if s["case"]["kind"] == "wgrad":
        a, b = _values(s["a"], s["sa"], s["a_fmt"], 1), _values(s["b"], s["sb"], s["b_fmt"], 1)
        at = off[:-1, None] + torch.arange(most, device="cuda")
        inside = at < off[1:, None]
        at = at.clamp_max(a.shape[1] - 1)
        a, b = a.t()[at] * inside[:, :, None], b.t()[at]
        return torch.bmm(a.transpose(1, 2), b)
    a = _values(s["a"], s["sa"], s["a_fmt"], 1)
    row = torch.arange(a.shape[0], device="cuda")
    of = torch.searchsorted(off[1:], row, right=True)
    place = of * most + row - off[of]
    slab = torch.zeros(e * most, a.shape[1], device="cuda")
    slab[place] = a
    out = torch.bmm(slab.view(e, most, -1), _values(s["b"], s["sb"], s["b_fmt"], 128).transpose(1, 2))
    return out.view(e * most, -1)[place].bfloat16()


def _route(s):
    """Scores, the k best of the best groups (ties to the lowest index), renormalised weights, d logits."""
    c, x = s["case"], s["logits"].float()
    t, e = x.shape
    if c["score"] == "softmax":
        p = (x - x.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
        key = x
    else:
        p = 1.0 / (1.0 + (-x).exp())
        key = p + s["bias"]
    if c["groups"] > 1:
        best = key.view(t, c["groups"], -1).sort(2, descending=True).values
        of_group = best[:, :, 0] + best[:, :, 1]
        rank = of_group.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        out = (rank >= c["top_groups"]).repeat_interleave(e // c["groups"], 1)
        key = key.masked_fill(out, NEG_INF)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :min(c["top"], e)]
    chosen = p.gather(1, ids)
    total = chosen.sum(1, keepdim=True)
    w = chosen / total
    if not c["backward"]:
        return {"weights": w, "ids": ids.int()}
    d = s["d_weights"]
    d_p = torch.zeros_like(p).scatter(1, ids, (d - (d * w).sum(1, keepdim=True)) / total)
    d_x = p * (d_p - (d_p * p).sum(1, keepdim=True)) if c["score"] == "softmax" else d_p * p * (1.0 - p)
    return {"weights": w, "ids": ids.int(), "d_logits": d_x.to(s["logits"].dtype)}


def _order(ids, experts, align, rows):
    """Offsets of the experts' padded segments, the row of each slot, the slot of each row (-1: padding)."""
    flat = ids.reshape(-1).long()
    e, slot = flat.sort(stable=True)
    count = torch.zeros(experts, dtype=torch.int64, device=ids.device).index_add_(0, flat, torch.ones_like(flat))
    padded = (count + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    first = count.cumsum(0) - count
    row = offsets[e] + torch.arange(flat.numel(), device=ids.device) - first[e]
    src = torch.full((rows,), -1, dtype=torch.int32, device=ids.device)
    src[row] = slot.int()
    row_of = torch.empty_like(flat, dtype=torch.int32)
    row_of[slot] = row.int()
    return offsets, row_of.view(ids.shape), src


def _dispatch(s):
    c = s["case"]
    offsets, row_of, src = _order(s["ids"], c["experts"], c["align"], s["rows"])
    x = s["x"].float()[(src // s["ids"].shape[1]).clamp_min(0).long()] * (src >= 0)[:, None]
    q, scale_inv = _blockwise(x, E4M3, 1)
    out = {"offsets": offsets, "row_of": row_of, "src": src, "q": q.view(TYPES[E4M3]), "scale_inv": scale_inv}
    if c["both"]:
        q_t, out["scale_inv_t"] = _blockwise(x.t(), E4M3, 1)
        out["q_t"] = q_t.view(TYPES[E4M3])
    return out


def _combine(s):
    c, h = s["case"], s["case"]["hidden"]
    rows = s["y"].float()[s["row_of"].reshape(-1).long()].view(c["tokens"], -1, h)
    out = {"out": (rows * s["weights"][:, :, None]).sum(1).bfloat16()}
    if c["backward"]:
        d = s["d_out"].float()
        out["d_weights"] = (rows * d[:, None, :]).sum(2)
        src = s["src"].clamp_min(0).long()
        w = s["weights"].reshape(-1)[src] * (s["src"] >= 0)
        out["d_y"] = (d[src // s["weights"].shape[1]] * w[:, None]).bfloat16()
    return out


def _run_own(s):
    import mxfp8_quantization_amax_gb300 as fq

    c = s["case"]
    if c["op"] == "mm":
        wgrad = c["kind"] == "wgrad"
        return fq.fp8q_matmul_blockwise(s["a"], s["sa"], s["b"], s["sb"], a_fmt=s["a_fmt"], b_fmt=s["b_fmt"],
                                        b_block=fq.BLOCK_1X128 if wgrad else fq.BLOCK_128X128,
                                        out_dtype=torch.float32 if wgrad else torch.bfloat16)
    if c["op"] == "grouped":
        if c["kind"] == "wgrad":
            return fq.fp8q_matmul_grouped_wgrad(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], a_fmt=s["a_fmt"], b_fmt=s["b_fmt"])
        return fq.fp8q_matmul_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], a_fmt=s["a_fmt"], b_fmt=s["b_fmt"])
    if c["op"] == "route":
        score = fq.SCORE_SOFTMAX if c["score"] == "softmax" else fq.SCORE_SIGMOID
        top = min(c["top"], c["experts"])
        r = fq.fp8q_moe_route(s["logits"], top, score=score, bias=s["bias"], num_groups=c["groups"], top_groups=c["top_groups"])
        if c["backward"]:
            r["d_logits"] = fq.fp8q_moe_route_backward(s["logits"], r["ids"], s["d_weights"], score=score)
        return r
    if c["op"] == "dispatch":
        plan = fq.fp8q_moe_plan(s["ids"], c["experts"], align=c["align"])
        r = fq.fp8q_moe_dispatch(s["x"], plan, direction=fq.BOTH if c["both"] else fq.ROW)
        out = {"offsets": plan["offsets"], "row_of": plan["row_of"], "src": plan["src"],
               "q": r["q"].view(TYPES[E4M3]), "scale_inv": r["scale_inv"]}
        if c["both"]:
            out["q_t"], out["scale_inv_t"] = r["q_t"].view(TYPES[E4M3]), r["scale_inv_t"]
        return out
    plan = {"row_of": s["row_of"], "src": s["src"]}
    out = {"out": fq.fp8q_moe_combine(s["y"], plan, s["weights"])}
    if c["backward"]:
        out.update(fq.fp8q_moe_combine_backward(s["d_out"], s["y"], plan, s["weights"]))
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"mm": _mm, "grouped": _grouped, "route": _route, "dispatch": _dispatch, "combine": _combine}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        kb, wgrad = -(-k // 128), case["kind"] == "wgrad"
        scales = m * kb + (n if wgrad else -(-n // 128)) * kb
        return {"bytes": m * k + n * k + 4 * scales + m * n * (4 if wgrad else 2), "flops": 2 * m * n * k}
    if op == "grouped":
        e, n, k, rows = case["experts"], case["n"], case["k"], case["rows"]
        if case["kind"] == "wgrad":
            return {"bytes": rows * (n + k) * (1 + 4 / 128) + 4 * e * n * k, "flops": 2 * rows * n * k}
        hit = e * (1 - (1 - 1 / e) ** rows)  # experts that some row reaches
        return {"bytes": hit * (n * k + n * k / 4096) + rows * (k * (1 + 4 / 128) + 2 * n), "flops": 2 * rows * n * k}
    t, top = case["tokens"], min(case["top"], case["experts"])
    if op == "route":
        size = 2 if case["type"] == "bf16" else 4
        passes = 3 if case["backward"] else 1  # logits in; logits in again and their gradient out
        return {"bytes": t * case["experts"] * size * passes + t * top * (8 + (8 if case["backward"] else 0)), "flops": 8 * t * case["experts"]}
    h, slots = case["hidden"], t * top
    rows = slots if case["align"] == 1 else slots + min(case["experts"], slots) * case["align"] / 2
    if op == "dispatch":
        copies = 2 if case["both"] else 1
        return {"bytes": 2 * t * h + copies * rows * h * (1 + 4 / 128) + 12 * slots, "flops": 3 * copies * rows * h}
    out = slots * h * 2 + t * h * 2 + 8 * slots  # rows, weights and their places in, the sum out
    if case["backward"]:
        out += t * h * 2 + slots * h * 2 + rows * h * 2 + 12 * slots  # d_out and rows in, d_y and d_weights out
    return {"bytes": out, "flops": 2 * slots * h * (3 if case["backward"] else 1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _table(fmt):
    """The value of each of the 256 codes: sign, exponent, mantissa."""
    bits, bias = ((3, 7), (2, 15))[fmt]
    out = []
    for code in range(256):
        e, m = (code & 127) >> bits, code & ((1 << bits) - 1)
        v = (m / (1 << bits)) * 2.0 ** (1 - bias) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias)
        out.append(-v if code & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _decode(q, scale, fmt, block_rows):
    v = _table(fmt)[q.long()]
    for i in range(0, q.shape[1], 128):  # one column of blocks at a time
        v[:, i:i + 128] *= scale[:, i // 128].double().repeat_interleave(block_rows)[:q.shape[0], None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "mm":
        a = _decode(s["a"], s["sa"], s["a_fmt"], 1)
        return a @ _decode(s["b"], s["sb"], s["b_fmt"], 1 if case["kind"] == "wgrad" else 128).T
    if case["op"] == "grouped":
        off, parts = s["offsets"].tolist(), []
        for i in range(case["experts"]):
            lo, hi = off[i], off[i + 1]
            if case["kind"] == "wgrad":
                a = _decode(s["a"][:, lo:hi], s["sa"][:, lo // 128:hi // 128], s["a_fmt"], 1)
                parts.append(a @ _decode(s["b"][:, lo:hi], s["sb"][:, lo // 128:hi // 128], s["b_fmt"], 1).T)
            elif hi > lo:
                parts.append(_decode(s["a"][lo:hi], s["sa"][lo:hi], s["a_fmt"], 1) @ _decode(s["b"][i], s["sb"][i], s["b_fmt"], 128).T)
        return torch.stack(parts) if case["kind"] == "wgrad" else torch.cat(parts)
    if case["op"] == "route":
        return _exact_route(case, s)
    ids = s["ids"].tolist()
    order = sorted((e, t, j) for t, row in enumerate(ids) for j, e in enumerate(row))
    place, row, last = {}, -1, None
    for e, t, j in order:
        row = row + 1 if e == last or last is None else -(-(row + 1) // case["align"]) * case["align"]
        place[t, j], last = row, e
    top = len(ids[0])
    at = torch.tensor([place[t, j] for t in range(len(ids)) for j in range(top)], device="cuda")
    if case["op"] == "dispatch":
        x = torch.zeros(s["rows"], case["hidden"], dtype=torch.float64, device="cuda")
        x[at] = s["x"].double().repeat_interleave(top, 0)
        out = {"offsets": None, "row_of": None, "src": None}
        for name, v in (("", x), ("_t", x.T)) if case["both"] else (("", x),):
            q, inv = torch.zeros_like(v), torch.empty(v.shape[0], -(-v.shape[1] // 128), dtype=torch.float64, device="cuda")
            for i in range(inv.shape[1]):
                block = v[:, 128 * i:128 * i + 128]
                big = block.abs().amax(1)
                inv[:, i] = torch.where(big > 0, big / 448.0, 1.0)
                q[:, 128 * i:128 * i + 128] = block / inv[:, i, None]
            out["q" + name], out["scale_inv" + name] = q, inv
        return out
    y, w, d = s["y"].double()[at].view(-1, top, case["hidden"]), s["weights"].double(), s["d_out"].double()
    out = {"out": torch.einsum("tjh,tj->th", y, w)}
    if case["backward"]:
        out["d_weights"] = torch.einsum("tjh,th->tj", y, d)
        out["d_y"] = torch.zeros(s["rows"], case["hidden"], dtype=torch.float64, device="cuda")
        out["d_y"][at] = torch.einsum("th,tj->tjh", d, w).reshape(-1, case["hidden"])
    return out


def _exact_route(case, s):
    x = s["logits"].double()
    t, e = x.shape
    p = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    key = x if s["bias"] is None else p + s["bias"].double()
    if case["groups"] > 1:
        of = key.view(t, case["groups"], -1).topk(2, 2).values.sum(2)
        keep = torch.zeros_like(of, dtype=torch.bool).scatter(1, of.topk(case["top_groups"], 1).indices, True)
        key = torch.where(keep[:, :, None], key.view(t, case["groups"], -1), NEG_INF).view(t, e)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :min(case["top"], e)]
    leaf = x.clone().requires_grad_(True)
    chosen = (torch.softmax(leaf, 1) if case["score"] == "softmax" else torch.sigmoid(leaf)).gather(1, ids)
    w = chosen / chosen.sum(1, keepdim=True)
    out = {"weights": w.detach(), "ids": None}
    if case["backward"]:
        w.backward(s["d_weights"].double())
        out["d_logits"] = leaf.grad
    return out
