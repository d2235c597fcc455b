"""The operators around the MoE expert LoRA fold, as cases to be measured.

Three groups, the path of a MoE projection in its order: the router's top-k weights ("route" and
its gradient "route_grad"), rows brought into expert order ("dispatch") and back with the router's
weights ("combine", and its gradient "combine_grad"; "combine" without weights is the gradient of
"dispatch"), and the decode-side product of gathered rows with 4-bit expert weights ("q4").

Sizes are those of this repository's workloads (64 x top-8 and 256 x top-8 decode batches over 128
experts with k/n of 768 and 2048, the 16384-token top-10 prefill over 512 experts) and odd ones
between them.  ``run`` computes the plain form with elementary torch operations in 32 bits, or,
where ``own`` is set, calls the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's router: 64 requests, 128 experts; latency
        {"name": "route_decode", "op": "route", "tokens": 64, "experts": 128, "top_k": 8,
         "dtype": "bf16", "renorm": True, "masked": 0.0},
        # the large prefill's router over 512 experts
        {"name": "route_prefill", "op": "route", "tokens": 16384, "experts": 512, "top_k": 10,
         "dtype": "bf16", "renorm": True, "masked": 0.0},
        # training: the router's gradient with plain softmax weights, odd sizes, fp32 logits,
        # some experts masked out
        {"name": "route_grad_odd", "op": "route_grad", "tokens": 4099, "experts": 97, "top_k": 6,
         "dtype": "f32", "renorm": False, "masked": 0.05},
        # a decode batch brought into expert order; latency
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 64, "experts": 128, "top_k": 8,
         "width": 2048, "dtype": "bf16", "adapters": 0, "drop": 0.0, "skew": 0.0},
        # packed prefill streams of several adapters: rows sorted by (adapter, expert), some
        # requests without adapter, x a slice of a wider activation
        {"name": "dispatch_adapters", "op": "dispatch", "tokens": 4093, "experts": 128, "top_k": 8,
         "width": 776, "dtype": "bf16", "adapters": 4, "drop": 0.02, "skew": 1.5},
        # the large prefill's rows into expert order
        {"name": "dispatch_prefill", "op": "dispatch", "tokens": 16384, "experts": 512,
         "top_k": 10, "width": 2048, "dtype": "bf16", "adapters": 0, "drop": 0.0, "skew": 1.5},
        # a decode batch's expert outputs weighted and summed; latency
        {"name": "combine_decode", "op": "combine", "tokens": 64, "experts": 128, "top_k": 8,
         "width": 2048, "dtype": "bf16", "weighted": True, "drop": 0.0, "skew": 0.0},
        # the large prefill's expert outputs weighted and summed
        {"name": "combine_prefill", "op": "combine", "tokens": 16384, "experts": 512, "top_k": 10,
         "width": 2048, "dtype": "bf16", "weighted": True, "drop": 0.0, "skew": 1.5},
        # training: the gradient of the weighted sum, 30K rows, some slots without expert
        {"name": "combine_grad", "op": "combine_grad", "tokens": 4001, "experts": 128, "top_k": 8,
         "width": 2048, "dtype": "bf16", "weighted": True, "drop": 0.01, "skew": 1.5},
        # one token's 8 experts, gate/up shape: the smallest decode product
        {"name": "q4_one_token", "op": "q4", "tokens": 1, "experts": 128, "top_k": 8, "k_in": 2048,
         "n_out": 768, "group": 128, "zeros": False, "per_row": False, "drop": 0.0},
        # a decode batch's down projection (one input row per expert row), zero points, groups of 32
        {"name": "q4_down", "op": "q4", "tokens": 64, "experts": 128, "top_k": 8, "k_in": 768,
         "n_out": 2048, "group": 32, "zeros": True, "per_row": True, "drop": 0.02},
        # the largest decode batch, gate/up shape
        {"name": "q4_gate_up", "op": "q4", "tokens": 256, "experts": 128, "top_k": 8,
         "k_in": 2048, "n_out": 768, "group": 128, "zeros": False, "per_row": False, "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "combine", "combine_grad", "q4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("route", "route_grad"):
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts,
                "top_k": rng.randint(1, min(10, experts)), "dtype": dtype,
                "renorm": rng.random() < 0.5, "masked": rng.choice([0.0, 0.05, 0.5])}
    if op == "q4":
        group = rng.choice([32, 64, 128])
        experts, top_k = _log(rng, 1, 128), rng.randint(1, 8)
        return {"op": op, "tokens": _log(rng, 1, 256), "experts": experts,
                "top_k": min(top_k, experts), "k_in": group * _log(rng, 1, 2048 // group),
                "n_out": 8 * _log(rng, 1, 96), "group": group, "zeros": rng.random() < 0.5,
                "per_row": rng.random() < 0.5, "drop": rng.choice([0.0, 0.02])}
    experts = _log(rng, 4, 512)
    size = 2 if dtype == "bf16" else 4
    case = {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts,
            "top_k": rng.randint(1, min(10, experts)), "width": 8 * _log(rng, 8, 512 // size * 2),
            "dtype": dtype, "drop": rng.choice([0.0, 0.02, 0.3]), "skew": rng.choice([0.0, 1.5])}
    if op == "dispatch":
        case["adapters"] = rng.choice([0, 0, 1, 4])
    else:
        case["weighted"] = op == "combine_grad" or rng.random() < 0.7
    most = work(listed()[5])["bytes"]  # no more than the large prefill's dispatch
    case["tokens"] = min(case["tokens"], max(1, int(most * case["tokens"] / work(case)["bytes"])))
    return case


# ------------------------------------------------------------------ the inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _routing(case, g):
    """Expert ids [tokens, top_k] as a router picks them: top_k of normal logits, with a
    per-expert bias of variance `skew`; a share `drop` of the ids is out of range."""
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case.get("skew"):
        logits += torch.randn(E, generator=g, device="cuda") * math.sqrt(case["skew"])
    ids = torch.topk(logits, K, dim=1).indices.to(torch.int32)
    if case["drop"]:
        lost = torch.rand(T, K, generator=g, device="cuda")
        ids = torch.where(lost < case["drop"] / 2, torch.full_like(ids, -1), ids)
        ids = torch.where(lost > 1 - case["drop"] / 2, torch.full_like(ids, E), ids)
    return ids.contiguous()


def _wide(T, W, dtype, g):
    """[T, W] activations that are a slice of a wider tensor (row stride W + 8)."""
    return torch.randn(T, W + 8, generator=g, device="cuda").to(dtype)[:, :W]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, E, K = case["op"], case["tokens"], case["experts"], case["top_k"]
    s = {"case": dict(case)}
    i32 = {"dtype": torch.int32, "device": "cuda"}
    f32 = {"dtype": torch.float32, "device": "cuda"}
    if op in ("route", "route_grad"):
        logits = torch.randn(T, E, generator=g, device="cuda") * 2
        if case["masked"]:
            hide = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
            hide |= torch.rand(T, 1, generator=g, device="cuda") < 0.01  # padding rows
            logits = torch.where(hide, torch.full_like(logits, -math.inf), logits)
        s["logits"] = logits.to(_type(case)).contiguous()
        s["indices"], s["weights"] = torch.empty(T, K, **i32), torch.empty(T, K, **f32)
        if op == "route_grad":
            s["indices"], s["weights"] = _route_plain(s["logits"], K, case["renorm"])
            s["dweights"] = torch.randn(T, K, generator=g, device="cuda")
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    s["indices"] = _routing(case, g)
    if op == "q4":
        k, n, G = case["k_in"], case["n_out"], case["group"]
        rows = T * K if case["per_row"] else T
        s["x"] = torch.randn(rows, k, generator=g, device="cuda").to(torch.bfloat16)
        s["codes"] = torch.randint(0, 256, (E, n, k // 2), generator=g, device="cuda",
                                   dtype=torch.uint8)
        s["scales"] = ((torch.rand(E, n, k // G, generator=g, device="cuda") + 0.5)
                       / (4 * math.sqrt(k))).to(torch.bfloat16)
        s["zeros"] = (torch.randint(5, 11, (E, n, k // G), generator=g, device="cuda",
                                    dtype=torch.uint8) if case["zeros"] else None)
        s["out"] = torch.empty(T * K, n, dtype=torch.bfloat16, device="cuda")
        return s
    W, dt, rows = case["width"], _type(case), T * K
    if op == "dispatch":
        s["x"] = _wide(T, W, dt, g)
        s["row_adapter"] = (torch.randint(-1, case["adapters"], (T,), generator=g, device="cuda",
                                          dtype=torch.int32) if case["adapters"] else None)
        cells = E * max(1, case["adapters"])
        s["offsets"] = torch.empty(cells + 1, **i32)
        s["src"], s["pos"] = torch.empty(rows, **i32), torch.empty(rows, **i32)
        s["x_rows"] = torch.empty(rows, W, dtype=dt, device="cuda")
        return s
    s["offsets"], _, s["pos"] = _sort_plain(s["indices"], None, E, 0)
    s["held"] = s["offsets"][-1:]  # the rows that belong to an expert, on the device
    y = torch.randn(rows, W, generator=g, device="cuda").to(dt)
    if case["drop"]:  # rows of no expert were never written by the experts' product
        y[torch.arange(rows, device="cuda") >= s["offsets"][-1]] = math.nan
    s["y_rows"] = y
    w = torch.rand(T, K, generator=g, device="cuda") + 0.1
    s["weights"] = (w / w.sum(1, keepdim=True)) if case["weighted"] else None
    if op == "combine":
        s["out"] = torch.empty(T, W, dtype=dt, device="cuda")
    else:
        s["dout"] = torch.randn(T, W, generator=g, device="cuda").to(dt)
        s["dy_rows"] = torch.empty(rows, W, dtype=dt, device="cuda")
        s["dweights"] = torch.empty(T, K, **f32)
    return s


# ------------------------------------------------------------------ the plain forms
def _eligible(logits):
    """fp32 logits with everything that cannot be chosen (-inf, NaN) at -inf, +inf at the largest
    finite value, and which can be chosen."""
    v = logits.float()
    ok = v > -math.inf
    return torch.where(ok, v.clamp(max=_FLT_MAX), torch.full_like(v, -math.inf)), ok


def _softmax_parts(logits):
    v, ok = _eligible(logits)
    m = v.max(1, keepdim=True).values
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = torch.where(ok, torch.exp(v - m), torch.zeros_like(v))
    return v, ok, e


def _route_plain(logits, top_k, renorm):
    v, ok, e = _softmax_parts(logits)
    order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top_k]
    there = torch.gather(ok, 1, order)
    top = torch.gather(e, 1, order)
    total = (top if renorm else e).sum(1, keepdim=True)
    weights = torch.where(there, top / total, torch.zeros_like(top))
    indices = torch.where(there, order, torch.full_like(order, -1)).to(torch.int32)
    return indices, weights


def _route_grad_plain(s):
    case, w, dw = s["case"], s["weights"], s["dweights"]
    at = s["indices"].clamp(min=0).long()
    wdw = w * dw  # zero where the slot has no expert
    total = wdw.sum(1, keepdim=True)
    if case["renorm"]:
        grad = torch.zeros(s["logits"].shape, dtype=torch.float32, device="cuda")
        grad.scatter_add_(1, at, wdw - w * total)
    else:
        _, _, e = _softmax_parts(s["logits"])
        z = e.sum(1, keepdim=True)
        grad = -(e / torch.where(z > 0, z, torch.ones_like(z))) * total
        grad.scatter_add_(1, at, wdw)
    return grad.to(s["logits"].dtype)


def _sort_plain(indices, row_adapter, E, adapters):
    """(offsets, src, pos): the slots in the order of their cells (stable), those of no cell last."""
    T, K = indices.shape
    cells = E * max(1, adapters)
    cell, ok = indices, (indices >= 0) & (indices < E)
    if row_adapter is not None:
        a = row_adapter[:, None]
        ok = ok & (a >= 0) & (a < adapters)
        cell = a * E + indices
    cell = torch.where(ok, cell, torch.full_like(cell, cells)).reshape(-1)
    sorted_cells, src = torch.sort(cell, stable=True)
    edges = torch.arange(cells + 1, device="cuda", dtype=cell.dtype)
    offsets = torch.searchsorted(sorted_cells, edges).to(torch.int32)
    pos = torch.empty_like(src)
    pos[src] = torch.arange(T * K, device="cuda")
    pos = torch.where(ok.reshape(-1), pos, torch.full_like(pos, -1)).to(torch.int32)
    return offsets, src.to(torch.int32), pos


def _dispatch_plain(s):
    case, x = s["case"], s["x"]
    offsets, src, pos = _sort_plain(s["indices"], s["row_adapter"], case["experts"],
                                    case["adapters"])
    held = torch.arange(src.numel(), device="cuda") < offsets[-1]
    x_rows = torch.where(held[:, None], x[src.long() // case["top_k"]],
                         torch.zeros((), dtype=x.dtype, device="cuda"))
    return {"offsets": offsets, "src": src, "pos": pos, "x_rows": x_rows}


def _rows_of(s):
    """The tokens' rows [tokens, top_k, width] in fp32, zero where a slot has none, and which have."""
    case = s["case"]
    pos = s["pos"].reshape(case["tokens"], case["top_k"]).long()
    there = (pos >= 0)[:, :, None]
    y = s["y_rows"][pos.clamp(min=0)].float()
    return torch.where(there, y, torch.zeros((), device="cuda")), there


def _combine_plain(s):
    y, _ = _rows_of(s)
    if s["weights"] is not None:
        y = y * s["weights"][:, :, None]
    return y.sum(1).to(s["y_rows"].dtype)


def _combine_grad_plain(s):
    case = s["case"]
    y, there = _rows_of(s)
    dout = s["dout"].float()[:, None, :]
    dweights = (y * dout).sum(2)
    rows = s["y_rows"].shape[0]
    dy = torch.zeros(rows + 1, case["width"], dtype=s["y_rows"].dtype, device="cuda")
    at = torch.where(s["pos"] >= 0, s["pos"], torch.full_like(s["pos"], rows)).long()
    dy[at] = (s["weights"][:, :, None] * dout).to(dy.dtype).reshape(rows, -1)
    return {"dy_rows": dy[:rows], "dweights": dweights}


def _dequantised(codes, scales, zeros, group):
    """fp32 weights of 4-bit codes [..., n, k/2], low nibble first, by groups along k."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    zero = 8.0 if zeros is None else zeros.float()[..., None]
    return ((q.unflatten(-1, (-1, group)) - zero) * scales.float()[..., None]).flatten(-2)


def _q4_plain(s):
    case, idx = s["case"], s["indices"].reshape(-1).long()
    E, K, n, k = case["experts"], case["top_k"], case["n_out"], case["k_in"]
    rows = idx.numel()
    ok = ((idx >= 0) & (idx < E))[:, None]
    at = idx.clamp(0, E - 1)
    x = s["x"].float()
    if rows <= E:  # the rows' own experts
        w = _dequantised(s["codes"][at], s["scales"][at],
                         None if s["zeros"] is None else s["zeros"][at], case["group"])
        x_rows = x if case["per_row"] else x.repeat_interleave(K, 0)
        out = torch.bmm(w, x_rows[:, :, None])[:, :, 0]
    else:  # every expert's product with every input row, then the rows' own
        w = _dequantised(s["codes"], s["scales"], s["zeros"], case["group"])
        full = (x @ w.reshape(E * n, k).t()).reshape(x.shape[0], E, n)
        row = torch.arange(rows, device="cuda")
        out = full[row if case["per_row"] else row // K, at]
    return torch.where(ok, out, torch.zeros((), device="cuda")).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op, T, K, E = case["op"], case["tokens"], case["top_k"], case["experts"]
    if not own:
        if op == "route":
            return dict(zip(("indices", "weights"), _route_plain(s["logits"], K, case["renorm"])))
        return {"route_grad": _route_grad_plain, "dispatch": _dispatch_plain,
                "combine": _combine_plain, "combine_grad": _combine_grad_plain,
                "q4": _q4_plain}[op](s)

    import lora_moe_expert_gb300 as mlg

    if op == "route":
        mlg.mlg_route_topk(s["logits"], s["indices"], s["weights"], T, E, K, case["renorm"])
        return {"indices": s["indices"], "weights": s["weights"]}
    if op == "route_grad":
        mlg.mlg_route_topk_backward(s["logits"], s["indices"], s["weights"], s["dweights"],
                                    s["dlogits"], T, E, K, case["renorm"])
        return s["dlogits"]
    if op == "dispatch":
        mlg.mlg_dispatch(s["x"], s["indices"], s["row_adapter"], s["offsets"], s["src"], s["pos"],
                         s["x_rows"], T * K, case["width"], K, E, max(1, case["adapters"]))
        return {"offsets": s["offsets"], "src": s["src"], "pos": s["pos"], "x_rows": s["x_rows"]}
    if op == "combine":
        mlg.mlg_combine(s["y_rows"], s["pos"], s["weights"], s["out"], T, case["width"], K, T * K)
        return s["out"]
    if op == "combine_grad":
        mlg.mlg_combine_backward(s["dout"], s["y_rows"], s["pos"], s["weights"],
                                 s["held"], s["dy_rows"], s["dweights"], T, case["width"], K, T * K)
        return {"dy_rows": s["dy_rows"], "dweights": s["dweights"]}
    mlg.mlg_gather_q4(s["x"], s["indices"], s["codes"], s["scales"], s["zeros"], s["out"], T * K,
                      case["k_in"], case["n_out"], 1 if case["per_row"] else K, E, case["group"])
    return s["out"]


def work(case):
    op, T, K, E = case["op"], case["tokens"], case["top_k"], case["experts"]
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    rows = T * K
    if op == "route":
        return {"bytes": T * E * size + rows * 8, "flops": 4 * T * E}
    if op == "route_grad":
        passes = 1 if case["renorm"] else 2
        return {"bytes": passes * T * E * size + rows * 12, "flops": passes * 3 * T * E}
    held = rows * (1 - case["drop"])
    if op == "q4":
        k, n = case["k_in"], case["n_out"]
        hit = E * (1 - (1 - K / E) ** T) if K < E else E
        weight = n * k / 2 + n * (k / case["group"]) * (3 if case["zeros"] else 2)
        x_rows = rows if case["per_row"] else T
        return {"bytes": hit * weight + x_rows * k * 2 + rows * (n * 2 + 4),
                "flops": 2 * held * n * k}
    W = case["width"]
    if op == "dispatch":
        cells = E * max(1, case["adapters"])
        return {"bytes": (T + rows) * W * size + rows * 12 + cells * 4, "flops": rows}
    if op == "combine":
        return {"bytes": (held + T) * W * size + rows * 8, "flops": 2 * held * W}
    return {"bytes": (held + rows + T) * W * size + rows * 12, "flops": 3 * held * W}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, T, K, E = case["op"], case["tokens"], case["top_k"], case["experts"]
    if op in ("route", "route_grad"):
        v = s["logits"].double().nan_to_num(nan=-math.inf, posinf=_FLT_MAX, neginf=-math.inf)
        p = (v - torch.logsumexp(v, 1, keepdim=True)).exp().nan_to_num(nan=0.0)
        if op == "route":
            top = p.sort(1, descending=True).values[:, :K]
            if case["renorm"]:
                top = (top / top.sum(1, keepdim=True)).nan_to_num(nan=0.0)
            return {"indices": None, "weights": top}
        chosen = torch.zeros_like(p)
        dense = torch.zeros_like(p)
        for j in range(K):
            t = torch.nonzero(s["indices"][:, j] >= 0)[:, 0]
            e = s["indices"][t, j].long()
            chosen[t, e] = 1.0
            dense[t, e] = s["dweights"][t, j].double()
        if case["renorm"]:
            p = (p * chosen / (p * chosen).sum(1, keepdim=True)).nan_to_num(nan=0.0)
        return p * (dense - (p * dense).sum(1, keepdim=True))
    if op == "q4":
        idx = s["indices"].reshape(-1).cpu().numpy()
        out = torch.zeros(T * K, case["n_out"], dtype=torch.float64, device="cuda")
        for e in np.unique(idx[(idx >= 0) & (idx < E)]).tolist():
            rows = torch.from_numpy(np.nonzero(idx == e)[0]).cuda()
            x = s["x"][rows if case["per_row"] else rows // K].double()
            c = s["codes"][e].to(torch.int64)
            q = torch.empty(case["n_out"], case["k_in"], dtype=torch.float64, device="cuda")
            q[:, 0::2], q[:, 1::2] = (c % 16).double(), (c // 16).double()
            G = case["group"]
            zero = s["zeros"][e].double().repeat_interleave(G, 1) if case["zeros"] else 8.0
            out[rows] = x @ ((q - zero) * s["scales"][e].double().repeat_interleave(G, 1)).t()
        return out
    if op == "dispatch":
        idx = s["indices"].cpu().numpy().astype(np.int64)
        ok = (idx >= 0) & (idx < E)
        cell = idx
        if case["adapters"]:
            a = s["row_adapter"].cpu().numpy().astype(np.int64)[:, None]
            ok &= a >= 0
            cell = cell + a * E
        flat = np.flatnonzero(ok)
        flat = flat[np.argsort(cell.reshape(-1)[flat], kind="stable")]
        x_rows = torch.zeros(T * K, case["width"], dtype=torch.float64, device="cuda")
        x_rows[: flat.size] = s["x"][torch.from_numpy(flat // K).cuda()].double()
        return {"offsets": None, "src": None, "pos": None, "x_rows": x_rows}
    pos = s["pos"].reshape(T, K).long()
    if op == "combine":
        out = torch.zeros(T, case["width"], dtype=torch.float64, device="cuda")
        for j in range(K):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            row = s["y_rows"][pos[t, j]].double()
            out[t] += row if s["weights"] is None else row * s["weights"][t, j, None].double()
        return out
    dy = torch.zeros(T * K, case["width"], dtype=torch.float64, device="cuda")
    dweights = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for j in range(K):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        d = s["dout"][t].double()
        dy[pos[t, j]] = d * s["weights"][t, j, None].double()
        dweights[t, j] = (d * s["y_rows"][pos[t, j]].double()).sum(1)
    return {"dy_rows": dy, "dweights": dweights}
