"""The operators around the expert FFN and the dense projections, as cases with
sizes: the router's gate projection (hidden states -> expert logits), the
routing itself (logits -> expert ids and weights) and the low-rank adapters of
many requests beside a shared projection.

With ``own`` false every operator runs in its plain form (elementary torch
operations); with ``own`` true through the framework's entry points.  ``exact``
gives the definitions in 64 bits, written apart from the plain forms.
"""
import math

import numpy as np
import torch

own = False

FLT_MAX = float(torch.finfo(torch.float32).max)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, logits, scoring, bias, n_group, topk_group, group_top, renorm, scale, masked):
    c = {"op": "route", "T": T, "E": E, "k": k, "logits": logits, "scoring": scoring, "bias": bias,
         "n_group": n_group, "topk_group": topk_group, "group_top": group_top, "renorm": renorm, "scale": scale,
         "masked": masked}
    return {"name": name, **c} if name else c


def _logits(name, T, H, E, weight, bias):
    c = {"op": "router_logits", "T": T, "H": H, "E": E, "weight": weight, "bias": bias}
    return {"name": name, **c} if name else c


def _lora(name, T, K, N, r, L, requests, plain, dtype):
    c = {"op": "lora_add", "T": T, "K": K, "N": N, "r": r, "L": L, "requests": requests, "plain": plain,
         "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token being generated: the latency of the smallest call
        _route("route T1 grouped", 1, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, False),
        # a decode batch of the 256-expert layer, softmax over the chosen logits
        _route("route T128 softmax", 128, 256, 8, "f32", "softmax", False, 1, 1, 1, True, 1.0, False),
        # a prefill of the same layer with balance biases and expert groups
        _route("route T16384 grouped", 16384, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, False),
        # an odd number of tokens, bf16 logits (many ties), some experts masked out
        _route("route T5003 bf16 masked", 5003, 160, 6, "bf16", "softmax", False, 8, 3, 1, False, 16.0, True),
        # the gate projection of one token, of a decode batch and of a prefill
        _logits("logits T1", 1, 7168, 256, "bf16", False),
        _logits("logits T128", 128, 7168, 256, "bf16", False),
        _logits("logits T16384", 16384, 7168, 256, "bf16", False),
        # a gate kept in 32 bits with a bias, a batch that fills no whole tiles
        _logits("logits T1000 f32 E72", 1000, 4096, 72, "f32", True),
        # one request with one adapter
        _lora("lora T1", 1, 7168, 2048, 16, 4, 1, 0, "bf16"),
        # a decode batch: every token a request of its own, 64 adapters, some requests with none
        _lora("lora T128 64 adapters", 128, 4096, 16384, 16, 64, 128, 16, "bf16"),
        # a prefill batch of twelve requests
        _lora("lora T4096", 4096, 4096, 16384, 32, 8, 12, 2, "bf16"),
        # a larger rank into a 32-bit sum, an odd number of tokens
        _lora("lora T5003 f32 r64", 5003, 7168, 4096, 64, 5, 9, 1, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "router_logits", "lora_add"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * max(1, _log_int(rng, 4, 512) // n_group)
        topk_group = rng.randint(1, n_group)
        k = min(rng.randint(1, 16), E // n_group * topk_group)
        bias = rng.random() < 0.5
        return _route(None, _log_int(rng, 1, 16384), E, k, rng.choice(["f32", "bf16"]),
                      rng.choice(["sigmoid", "softmax"]), bias, n_group, topk_group,
                      rng.choice([1, 2]) if n_group > 1 else 1, rng.random() < 0.6, rng.choice([1.0, 2.5, 16.0]),
                      rng.random() < 0.3)
    if op == "router_logits":
        return _logits(None, _log_int(rng, 1, 16384), 32 * _log_int(rng, 8, 224), _log_int(rng, 4, 256),
                       rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
    T = _log_int(rng, 1, 4096)
    requests = max(1, min(T, _log_int(rng, 1, 256)))
    return _lora(None, T, 32 * _log_int(rng, 8, 128), 8 * _log_int(rng, 32, 1024), 8 * _log_int(rng, 1, 12),
                 _log_int(rng, 1, 32), requests, rng.randint(0, requests // 4), rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    if case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = normal(T, E) * 1.5 + normal(E) * 0.5  # some experts are liked more than others
        if case["masked"]:  # experts that are switched off for a token, by either kind of mask; some rows lose all
            u = torch.rand(T, E, generator=gen, device=dev)
            row = torch.rand(T, 1, generator=gen, device=dev)
            logits = torch.where(u < 0.1, torch.full_like(logits, -math.inf), logits)
            logits = torch.where(u > 0.95, torch.full_like(logits, float(torch.finfo(torch.bfloat16).min)), logits)
            logits = torch.where(row < 0.01, torch.full_like(logits, -math.inf), logits)
        # balance biases move by fixed steps of a thousandth
        bias = torch.round(normal(E) * 20.0) * 0.001 if case["bias"] else None
        return {"logits": logits.to(DTYPES[case["logits"]]), "bias": bias}
    if case["op"] == "router_logits":
        T, H, E = case["T"], case["H"], case["E"]
        return {"x": normal(T, H).to(torch.bfloat16), "w": (normal(E, H) * 0.02).to(DTYPES[case["weight"]]),
                "bias": normal(E) * 0.1 if case["bias"] else None}
    T, K, N, r, L = case["T"], case["K"], case["N"], case["r"], case["L"]
    rng = np.random.Generator(np.random.PCG64(seed))
    n, bare = case["requests"], case["plain"]
    which = rng.permutation(L)[np.arange(n - bare) % L]  # every adapter is used as often as the others
    which = rng.permutation(np.concatenate([which, np.full(bare, -1)]))
    cuts = np.sort(rng.choice(T - 1, n - 1, replace=False) + 1) if n > 1 else np.zeros(0, np.int64)
    ids = np.repeat(which, np.diff(np.concatenate([[0], cuts, [T]])))
    return {"y": normal(T, N).to(DTYPES[case["dtype"]]), "x": normal(T, K).to(torch.bfloat16),
            "a": (normal(L, r, K) / math.sqrt(K)).to(torch.bfloat16),
            "b": (normal(L, N, r) * 0.1).to(torch.bfloat16),
            "ids": torch.from_numpy(ids.astype(np.int32)).to(dev),
            "scales": torch.rand(L, generator=gen, device=dev) + 0.5}


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"route": _plain_route, "router_logits": _plain_logits, "lora_add": _plain_lora}[s["case"]["op"]](s)


def _own(s):
    import quantization_nvfp4_quantize_amd as nv
    c = s["case"]
    if c["op"] == "route":
        ids, w = nv.route(s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"], n_group=c["n_group"],
                          topk_group=c["topk_group"], group_top=c["group_top"], renormalize=c["renorm"],
                          scale=c["scale"])
        return {"ids": ids, "weights": w}
    if c["op"] == "router_logits":
        return {"logits": nv.router_logits(s["x"], s["w"], bias=s["bias"])}
    return {"y": nv.lora_add(s["y"], s["x"], s["a"], s["b"], s["ids"], scales=s["scales"])}


def _plain_route(s):
    # in 64 bits: two experts whose choice values lie next to each other are
    # told apart by their values, not by the rounding of a score
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    x = s["logits"].double()
    live = x > -math.inf  # false for -inf and NaN
    x = torch.where(live, x.clamp(max=FLT_MAX), torch.full_like(x, -math.inf))
    top = x.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    e = torch.exp(x - top)
    if c["scoring"] == "softmax":
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = torch.where(live, 1.0 / (1.0 + torch.exp(-x)), torch.zeros_like(x))
    if s["bias"] is None:
        choice = x if G == 1 or c["group_top"] == 1 else score
    else:
        choice = score + s["bias"].double()
        live = live & (choice > -math.inf)
    if G > 1:
        grouped = torch.where(live, choice, torch.full_like(x, -math.inf)).view(T, G, E // G)
        best = grouped.sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        some = best[:, :, :1] > -math.inf
        value = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2, keepdim=True)
        value = torch.where(some, value, torch.full_like(value, -math.inf)).squeeze(2)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        live = live & keep[:, :, None].expand(T, G, E // G).reshape(T, E)
    # among the experts that are left the logits decide when there is no bias
    rank = x if s["bias"] is None else choice
    ids = torch.where(live, rank, torch.full_like(x, -math.inf)).sort(dim=1, descending=True, stable=True).indices[:, :k]
    on = live.gather(1, ids)
    if not c["renorm"]:
        w = score.gather(1, ids)
    else:
        # the chosen scores over their sum, scaled so that tiny scores do not vanish
        z = torch.where(on, x.gather(1, ids), torch.full((1, 1), -math.inf, dtype=x.dtype, device=x.device))
        peak = z.amax(1, keepdim=True)
        peak = torch.where(peak > -math.inf, peak, torch.zeros_like(peak))
        if c["scoring"] == "softmax":
            w = torch.exp(z - peak)
        else:
            m = peak.clamp(max=0.0)
            w = torch.where(z > 0, 1.0 / (1.0 + torch.exp(-z)), torch.exp(z - m) / (1.0 + torch.exp(z)))
        w = torch.where(on, w, torch.zeros_like(w))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = torch.where(on, w * c["scale"], torch.zeros_like(w)).float()
    return {"ids": torch.where(on, ids, torch.full_like(ids, -1)).int(), "weights": w}


def _plain_logits(s):
    y = s["x"].float() @ s["w"].float().t()
    return {"logits": y if s["bias"] is None else y + s["bias"]}


def _plain_lora(s):
    # every token against every adapter, the others' columns set to zero
    y, x, a, b, ids = s["y"], s["x"], s["a"], s["b"], s["ids"]
    L, r, K = a.shape
    u = x.float() @ a.reshape(L * r, K).float().t()
    mine = ids[:, None] == torch.arange(L, device=ids.device, dtype=ids.dtype)[None, :]
    u = u.view(-1, L, r) * (mine * s["scales"][None, :])[:, :, None]
    d = u.view(-1, L * r) @ b.float().permute(0, 2, 1).reshape(L * r, -1)
    return {"y": (y.float() + d).to(y.dtype)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    i = _inputs(case, seed)
    if case["op"] == "router_logits":
        out = torch.matmul(i["x"].to(torch.float64), i["w"].to(torch.float64).t().contiguous())
        if i["bias"] is not None:
            out += i["bias"].to(torch.float64)
        return {"logits": out}
    if case["op"] == "lora_add":
        out = i["y"].to(torch.float64)
        for l in range(case["L"]):
            rows = torch.nonzero(i["ids"] == l).flatten()
            if rows.numel():
                t = i["x"][rows].to(torch.float64) @ i["a"][l].to(torch.float64).t().contiguous()
                out[rows] += float(i["scales"][l]) * (t @ i["b"][l].to(torch.float64).t().contiguous())
        return {"y": out}
    return _exact_route(case, i["logits"].double().cpu().numpy(),
                        None if i["bias"] is None else i["bias"].double().cpu().numpy())


def _exact_route(case, logits, bias):
    T, E, k, G, S = case["T"], case["E"], case["k"], case["n_group"], case["E"] // case["n_group"]
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k), np.float64)
    z = np.where(np.isnan(logits), -np.inf, np.minimum(logits, FLT_MAX))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore", under="ignore"):
        if case["scoring"] == "softmax":
            hi = z.max(axis=1, keepdims=True)
            num = np.exp(z - np.where(np.isfinite(hi), hi, 0.0))
            score = num / np.maximum(num.sum(axis=1, keepdims=True), 1e-300)
        else:
            score = np.exp(-np.logaddexp(0.0, -z))
        open_ = np.isfinite(z)
        key = z if bias is None else score + bias
        if G > 1:
            gkey = score if bias is None and case["group_top"] > 1 else key
            parts = np.sort(np.where(open_, gkey, -np.inf).reshape(T, G, S), axis=2)[:, :, ::-1][:, :, :case["group_top"]]
            has = np.isfinite(parts)
            value = np.where(has[:, :, 0], np.where(has, parts, 0.0).sum(axis=2), -np.inf)
            first = np.argsort(-value, axis=1, kind="stable")[:, :case["topk_group"]]
            kept = np.zeros((T, G), bool)
            np.put_along_axis(kept, first, True, axis=1)
            open_ = open_ & np.repeat(kept, S, axis=1)
        order = np.argsort(np.where(open_, -key, np.inf), axis=1, kind="stable")[:, :k]
        taken = np.take_along_axis(open_, order, axis=1)
        if case["renorm"]:
            # log of each score: the ratios of scores are exp of differences
            log = z if case["scoring"] == "softmax" else -np.logaddexp(0.0, -z)
            log = np.where(taken, np.take_along_axis(log, order, axis=1), -np.inf)
            hi = log.max(axis=1, keepdims=True)
            part = np.exp(log - np.where(np.isfinite(hi), hi, 0.0))
            part = part / np.maximum(part.sum(axis=1, keepdims=True), 1e-300)
        else:
            part = np.take_along_axis(score, order, axis=1)
    ids[taken] = order[taken]
    weights[taken] = part[taken] * case["scale"]
    return {"ids": ids, "weights": weights}


# ------------------------------------------------------------------ work
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        size = 2 if case["logits"] == "bf16" else 4
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if case["op"] == "router_logits":
        H, E = case["H"], case["E"]
        size = 2 if case["weight"] == "bf16" else 4
        return {"bytes": 2 * T * H + size * E * H + 4 * T * E + (4 * E if case["bias"] else 0), "flops": 2 * T * H * E}
    K, N, r = case["K"], case["N"], case["r"]
    n, bare = case["requests"], case["plain"]
    used, size = min(case["L"], n - bare), 2 if case["dtype"] == "bf16" else 4
    rows = T * (n - bare) / n  # tokens with an adapter, on average
    return {"bytes": int(2 * rows * K) + 2 * T * N * size + 2 * used * r * (K + N) + 4 * T,
            "flops": int(2 * rows * r * (K + N))}
