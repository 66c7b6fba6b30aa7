"""The operators of a decode step on quantized data, as cases with sizes: products
of a few tokens with 4-bit weights (the activations stay bf16), and a cache whose
rows are quantized as they are written and read back by slot or by page table.

With ``own`` false every operator runs in its plain form (elementary torch
operations); with ``own`` true through the framework's entry points.  ``exact``
gives the definitions in 64 bits, written apart from the plain forms.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HALF_STEPS = (0, 1, 2, 3, 4, 4, 5, 6, 6, 6, 6, 7, 7)  # NVFP4's index of each rounded count of half steps
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
PAGE = 64


# ------------------------------------------------------------------ cases
def _matvec(name, fmt, M, K, N, dtype):
    c = {"op": "matvec", "fmt": fmt, "M": M, "K": K, "N": N, "dtype": dtype}
    return {"name": name, **c} if name else c


def _write(name, fmt, T, heads, dim, parts, padded):
    c = {"op": "write", "fmt": fmt, "T": T, "heads": heads, "dim": dim, "parts": parts, "padded": padded}
    return {"name": name, **c} if name else c


def _read(name, fmt, seqs, most, heads, dim, parts, dtype):
    c = {"op": "read", "fmt": fmt, "seqs": seqs, "most": most, "heads": heads, "dim": dim, "parts": parts,
         "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token through a small projection: latency
        _matvec("matvec nvfp4 M1 K1024 N512", "nvfp4", 1, 1024, 512, "bf16"),
        # one token being generated, down to the width of an expert or a latent
        _matvec("matvec nvfp4 M1 K7168 N2048", "nvfp4", 1, 7168, 2048, "bf16"),
        # the dense projection of a layer, one token and a batch of eight requests
        _matvec("matvec nvfp4 M1 K4096 N16384", "nvfp4", 1, 4096, 16384, "bf16"),
        _matvec("matvec nvfp4 M8 K7168 N16384", "nvfp4", 8, 7168, 16384, "bf16"),
        # the largest decode batch, into a 32-bit result
        _matvec("matvec nvfp4 M64 K4096 N16384", "nvfp4", 64, 4096, 16384, "f32"),
        # the other 4-bit format: a batch of requests, and sizes that fill no tiles
        _matvec("matvec mxfp4 M16 K4096 N16384", "mxfp4", 16, 4096, 16384, "bf16"),
        _matvec("matvec mxfp4 M5 K1376 N4099", "mxfp4", 5, 1376, 4099, "f32"),
        # keys and values of one token, and of a prefill with some padding behind it
        _write("write mxfp8 T1", "mxfp8", 1, 8, 128, 2, 0),
        _write("write mxfp8 T16384", "mxfp8", 16384, 8, 128, 2, 100),
        # latent rows of a prefill chunk in four bits: written, and what was written read back
        _write("write and read nvfp4 T5003", "nvfp4", 5003, 1, 576, 1, 3),
        # the latent rows of a batch of sequences, for attention over all that came before
        _read("read mxfp8 24 sequences", "mxfp8", 24, 8192, 1, 576, 1, "bf16"),
        # keys and values of a few sequences in four bits, short heads, 32-bit result
        _read("read mxfp4 5 sequences", "mxfp4", 5, 1500, 4, 64, 2, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "write", "read"])
    if op == "matvec":
        K = 32 * _log_int(rng, 8, 224)
        N = _log_int(rng, 64, min(16384, 4096 * 16384 // K))
        return _matvec(None, rng.choice(["nvfp4", "nvfp4", "mxfp4"]), _log_int(rng, 1, 64), K, N,
                       rng.choice(["bf16", "bf16", "f32"]))
    heads, dim, parts = rng.choice([(1, 576, 1), (1, 128, 2), (2, 256, 2), (4, 64, 2), (4, 192, 1), (8, 128, 2),
                                    (3, 96, 2)])
    fmt = rng.choice(["mxfp8", "mxfp8", "nvfp4", "mxfp4"])
    if op == "write":
        T = _log_int(rng, 1, 16384)
        return _write(None, fmt, T, heads, dim, parts, rng.randint(0, T // 8))
    return _read(None, fmt, _log_int(rng, 1, 32), _log_int(rng, 1, 2048), heads, dim, parts,
                 rng.choice(["bf16", "bf16", "f32"]))


def _lengths(case):
    """Rows of each sequence: spread up to the longest, which comes first; some have one row or none."""
    rng = np.random.Generator(np.random.PCG64(case["seqs"] * 100003 + case["most"]))
    n = rng.integers(0, case["most"] + 1, case["seqs"])
    n[0] = case["most"]
    n[1::7] = np.minimum(n[1::7], 1)
    return n.astype(np.int64)


# ------------------------------------------------------------------ inputs
def _pack(idx):
    return (idx[..., 0::2] | (idx[..., 1::2] << 4)).to(torch.uint8)


def _e2m1_index(a):
    """The nearest E2M1 index of each |value|, ties to the even one."""
    a = a.clamp(max=6.0)
    step = torch.where(a < 2, torch.full_like(a, 0.5), torch.where(a < 4, torch.ones_like(a), torch.full_like(a, 2.0)))
    v = torch.round(a / step) * step
    return torch.where(v < 2, v * 2, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.int32)


def _power(e):
    """2^e as float32 for whole e in [-127, 127], from its bits."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantize(x, fmt, gs):
    """Blocks of the last dimension of float32 x -> (element bytes, scale bytes), in float32 as the format has it."""
    g = BLOCK[fmt]
    b = x.unflatten(-1, (-1, g))
    top = b.abs().amax(-1)
    neg = torch.signbit(b).to(torch.int32)
    if fmt == "nvfp4":
        inv = 1.0 / gs
        sf = (top / 6.0 * inv).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = sf.float()
        r = torch.where(d > 0, inv / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(d))
        half = torch.round(2.0 * (b * r[..., None]).abs().clamp(max=6.0)).to(torch.int64)
        idx = torch.tensor(HALF_STEPS, dtype=torch.int32, device=x.device)[half]
        return _pack((idx | (neg << 3)).flatten(-2)), sf.view(torch.uint8)
    mant, exp = torch.frexp(top)  # top = mant * 2^exp, mant in [0.5, 1)
    if fmt == "mxfp4":
        code = torch.where(top > 0, exp - 1 - 2 + 127, torch.zeros_like(exp)).clamp(0, 254)
        v = b * _power(127 - code)[..., None]
        return _pack((_e2m1_index(v.abs()) | (neg << 3)).flatten(-2)), code.to(torch.uint8)
    # the smallest power of two at which nothing saturates
    code = torch.where(top > 0, exp - 1 - 8 + (mant > 0.875).to(exp.dtype) + 127, torch.zeros_like(exp)).clamp(0, 254)
    v = (b * _power(127 - code)[..., None]).to(torch.float8_e4m3fn)
    return v.view(torch.uint8).flatten(-2), code.to(torch.uint8)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda:0", dtype=torch.float32)


def _rows(gen, T, heads, dim):
    """Keys, values or latents: some channels are much larger than the others."""
    channel = torch.exp(0.5 * _normal(gen, heads, dim)) * (1.0 + 7.0 * (torch.rand(heads, dim, generator=gen,
                                                                                  device="cuda:0") < 0.03))
    return (_normal(gen, T, heads, dim) * channel).to(torch.bfloat16)


def _pages_of(rng, count, pool):
    return rng.permutation(pool)[:count]


def _inputs(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    fmt = case["fmt"]
    if case["op"] == "matvec":
        w = _normal(gen, case["N"], case["K"]) * 0.02
        gs = w.abs().amax().reshape(1) / 2688.0
        q, s = _quantize(w, fmt, gs)
        del w
        x = _normal(gen, case["M"], case["K"]) * (1.0 + 9.0 * (torch.rand(case["K"], generator=gen, device=dev) < 0.01))
        return {"x": x.to(torch.bfloat16), "q": q, "s": s, "gs": gs}
    heads, dim, parts = case["heads"], case["dim"], case["parts"]
    gs = torch.full((1,), 0.03, dtype=torch.float32, device=dev)
    out = {"gs": gs}
    if case["op"] == "write":
        # the fused projection's output: queries beside keys and values
        T = case["T"]
        pool = 2 * (-(-T // PAGE)) + 2
        out["rows"] = [_rows(gen, T, heads, dim) for _ in range(parts)]
        out["fused"] = torch.cat([r.reshape(T, heads * dim) for r in [out["rows"][0]] + out["rows"]], dim=1)
        pages = _pages_of(rng, -(-T // PAGE), pool)
        at = np.arange(T)
        slots = pages[at // PAGE] * PAGE + at % PAGE
        slots[T - case["padded"]:] = -1
        out["slots"] = torch.from_numpy(slots.astype(np.int32)).to(dev)
        out["n_slots"] = pool * PAGE
        return out
    n = _lengths(case)
    need = -(-n // PAGE)
    wide = max(1, int(need.max()))
    pool = int(need.sum()) + 5
    order = _pages_of(rng, int(need.sum()), pool)
    table = np.full((case["seqs"], wide), -1, np.int64)
    table[np.arange(wide)[None, :] < need[:, None]] = order
    out["pages"] = torch.from_numpy(table.astype(np.int32)).to(dev)
    out["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev)
    out["total"] = int(n.sum())
    out["cache"] = [_quantize(_rows(gen, pool * PAGE, heads, dim).float(), fmt, gs) for _ in range(parts)]
    return out


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if case["op"] == "write":
        heads, dim, n, fmt = case["heads"], case["dim"], s["n_slots"], case["fmt"]
        wide = dim if fmt == "mxfp8" else dim // 2
        s["cache"] = [(torch.zeros(n, heads, wide, dtype=torch.uint8, device="cuda:0"),
                       torch.zeros(n, heads, dim // BLOCK[fmt], dtype=torch.uint8, device="cuda:0"))
                      for _ in range(case["parts"])]
        # keys and values are columns of one row: views, not tensors of their own
        R = heads * dim
        s["views"] = [s["fused"][:, (i + 1) * R:(i + 2) * R].unflatten(1, (heads, dim)) for i in range(case["parts"])]
        del s["rows"]
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"matvec": _plain_matvec, "write": _plain_write, "read": _plain_read}[s["case"]["op"]](s)


def _own(s):
    import quantization_nvfp4_quantize_amd as nv
    c = s["case"]
    fmt = c["fmt"]
    if c["op"] == "matvec":
        if fmt == "nvfp4":
            return {"y": nv.matvec(s["x"], s["q"], s["s"], s["gs"], out_dtype=DTYPES[c["dtype"]])}
        return {"y": nv.mx_matvec(s["x"], s["q"], s["s"], out_dtype=DTYPES[c["dtype"]])}
    cache = [(q, sc, s["gs"]) if fmt == "nvfp4" else (q, sc) for q, sc in s["cache"]]
    if c["op"] == "write":
        nv.cache_write(s["views"], s["slots"], cache, format=fmt)
        if fmt == "mxfp8":
            return _as_values(s["cache"])
        return {"rows": nv.cache_read(cache, s["slots"], format=fmt)}
    return {"rows": nv.cache_read_pages(cache, s["pages"], s["cu"], PAGE, s["total"], format=fmt,
                                        out_dtype=DTYPES[c["dtype"]])}


def _as_values(cache):
    return {"elements": [q.view(torch.float8_e4m3fn) for q, _ in cache], "codes": [sc for _, sc in cache]}


def _values(q, s, fmt, gs):
    """(element bytes, scale bytes) -> float32."""
    if fmt == "mxfp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        n = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).to(torch.int32)
        lut = torch.tensor(E2M1 + tuple(-e for e in E2M1), dtype=torch.float32, device=q.device)
        v = lut[n]
    g = BLOCK[fmt]
    if fmt == "nvfp4":
        scale = s.view(torch.float8_e4m3fn).float()
        return (v.unflatten(-1, (-1, g)) * scale[..., None]).flatten(-2) * gs
    return (v.unflatten(-1, (-1, g)) * _power(s.to(torch.int32) - 127)[..., None]).flatten(-2)


def _plain_matvec(s):
    fmt = s["case"]["fmt"]
    one = torch.ones_like(s["gs"])
    y = s["x"].float() @ _values(s["q"], s["s"], fmt, one).t()
    return {"y": (y * s["gs"] if fmt == "nvfp4" else y).to(DTYPES[s["case"]["dtype"]])}


def _plain_write(s):
    fmt = s["case"]["fmt"]
    on = s["slots"] >= 0
    at = s["slots"][on].long()
    for view, (q, sc) in zip(s["views"], s["cache"]):
        e, c = _quantize(view.float(), fmt, s["gs"])
        q[at] = e[on]
        sc[at] = c[on]
    if fmt == "mxfp8":
        return _as_values(s["cache"])
    back = s["slots"].clamp(min=0).long()
    return {"rows": [torch.where(on[:, None, None], _values(q[back], sc[back], fmt, s["gs"]),
                                 torch.zeros(1, device=q.device)).to(torch.bfloat16) for q, sc in s["cache"]]}


def _plain_read(s):
    c = s["case"]
    row = torch.arange(s["total"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = row - s["cu"][seq]
    slot = s["pages"][seq, pos // PAGE].long() * PAGE + pos % PAGE
    return {"rows": [_values(q[slot], sc[slot], c["fmt"], s["gs"]).to(DTYPES[c["dtype"]]) for q, sc in s["cache"]]}


# ------------------------------------------------------------------ 64 bits
def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(s, fmt, gs):
    c = s.to(torch.int64)
    if fmt != "nvfp4":
        return _two_to(c - 127)
    e, m = (c >> 3) & 15, (c & 7).to(torch.float64)
    return torch.where(e > 0, _two_to(e - 7) * (1 + m / 8), m * 2.0 ** -9) * gs


def _exact_values(q, s, fmt, gs):
    scale = _exact_scale(s, fmt, gs).repeat_interleave(BLOCK[fmt], dim=-1)
    b = q.to(torch.int64)
    if fmt == "mxfp8":
        e, m = (b >> 3) & 15, (b & 7).to(torch.float64)
        v = torch.where(e > 0, _two_to(e - 7) * (1 + m / 8), m * 2.0 ** -9)
        return torch.where(b >= 128, -v, v) * scale
    out = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    for k in (0, 1):
        n = (b >> (4 * k)) & 15
        e, m = (n >> 1) & 3, (n & 1).to(torch.float64)
        v = torch.where(e > 0, _two_to(e - 1) * (1 + m / 2), m / 2)
        out[..., k::2] = torch.where(n >= 8, -v, v)
    return out * scale


def _nearest(v, grid):
    """Index of the nearest entry of a rising grid, ties to the even index."""
    g = torch.tensor(grid, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(g, v).clamp(1, len(grid) - 1)
    lo = hi - 1
    d = (v - g[lo]) - (g[hi] - v)
    return torch.where(d < 0, lo, torch.where(d > 0, hi, torch.where(lo % 2 == 0, lo, hi)))


def _e4m3_grid():
    g = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        g += [2.0 ** (e - 7) * (1 + m / 8) for m in range(8)]
    return g[:-1]  # the last pattern is NaN


def _exact_rows(x, fmt, gs):
    """What the quantized form of x (float64) stands for: (elements with their sign, scale of each block)."""
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device=x.device)
        scale = grid[_nearest((top / 6 / gs).clamp(max=448.0), _e4m3_grid())] * gs
        v = torch.where(scale[..., None] > 0, b.abs() / scale.clamp(min=1e-300)[..., None], torch.zeros_like(b))
        half = _nearest(2 * v.clamp(max=6.0), [float(i) for i in range(13)])
        idx = torch.tensor(HALF_STEPS, device=x.device)[half]
        lut = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        return torch.sign(b) * lut[idx], scale
    most = 448.0 if fmt == "mxfp8" else None
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
    e = torch.where(_two_to(e) > top, e - 1, torch.where(_two_to(e + 1) <= top, e + 1, e))
    e = e - (8 if most else 2)
    if most:
        e = torch.where(top > most * _two_to(e), e + 1, e)
    scale = _two_to(e.clamp(-127, 127))
    v = b.abs() / scale[..., None]
    grid = _e4m3_grid() if most else list(E2M1)
    lut = torch.tensor(grid, dtype=torch.float64, device=x.device)
    return torch.sign(b) * lut[_nearest(v.clamp(max=grid[-1]), grid)], scale


def exact(case, seed):
    i = _inputs(case, seed)
    fmt = case["fmt"]
    gs = i["gs"].to(torch.float64)
    if case["op"] == "matvec":
        w = _exact_values(i["q"], i["s"], fmt, gs)
        return {"y": torch.matmul(i["x"].to(torch.float64), w.t().contiguous())}
    if case["op"] == "write":
        live = i["slots"] >= 0
        at = i["slots"][live].to(torch.int64)
        heads, dim = case["heads"], case["dim"]
        got = [_exact_rows(r.to(torch.float64), fmt, gs) for r in i["rows"]]
        if fmt != "mxfp8":
            return {"rows": [(e * s[..., None]).flatten(-2) * live[:, None, None] for e, s in got]}
        full = []
        for e, _ in got:
            pool = torch.zeros(i["n_slots"], heads, dim, dtype=torch.float64, device=e.device)
            pool[at] = e.flatten(-2)[live]
            full.append(pool)
        return {"elements": full, "codes": [None] * len(full)}
    n = _lengths(case)
    table = i["pages"].cpu().numpy().astype(np.int64)
    slots = [table[b, np.arange(n[b]) // PAGE] * PAGE + np.arange(n[b]) % PAGE for b in range(case["seqs"])]
    at = torch.from_numpy(np.concatenate(slots)).to(i["cu"].device)
    return {"rows": [_exact_values(q[at], s[at], fmt, gs) for q, s in i["cache"]]}


# ------------------------------------------------------------------ work
def work(case):
    fmt = case["fmt"]
    size = 2 if case.get("dtype") != "f32" else 4
    if case["op"] == "matvec":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * (K // 2 + K // BLOCK[fmt]) + 2 * M * K + size * M * N, "flops": 2 * M * K * N}
    R = case["heads"] * case["dim"] * case["parts"]
    held = (R if fmt == "mxfp8" else R // 2) + R // BLOCK[fmt]
    if case["op"] == "write":
        T, n = case["T"], case["T"] - case["padded"]
        back = 0 if fmt == "mxfp8" else n * held + 2 * T * R + 4 * T
        return {"bytes": n * (2 * R + held) + 4 * T + back, "flops": 0}
    T = int(_lengths(case).sum())
    return {"bytes": T * (held + size * R) + 4 * case["seqs"], "flops": 0}
