"""Cases of the operators around the expert layer: layer norm (forward and
backward), rows sorted by expert and back (with the gradients) and the experts'
product in microscaled 4-bit floating point.

run() computes a case in its plain form (elementary torch operations in fp32,
rounded once at the end) or, with own = True, through the package's operators.
exact() computes the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # values of the 4-bit codes 0..7; 8..15 negative
BLOCK = 32                                       # elements that share a scale


def listed():
    return [
        # one token of a decoding step through the norm in front of the Kimi-like layer: launch latency
        dict(name="norm_token", op="norm", train=False, T=1, d=7168, dtype="bf16", wdtype="bf16", pad=0),
        # a training step's norm, forward and backward, at the balanced layer's shape
        dict(name="norm_balanced", op="norm", train=True, T=2048, d=2048, dtype="bf16", wdtype="bf16", pad=0),
        # the largest: the rows of one GPU's share of an expert-parallel run, weights kept in fp32
        dict(name="norm_large", op="norm", train=True, T=16384, d=7168, dtype="bf16", wdtype="f32", pad=0),
        # odd width, rows with a stride, all fp32 (a small model in full precision)
        dict(name="norm_odd", op="norm", train=True, T=1003, d=1999, dtype="f32", wdtype="f32", pad=5),
        # one token's eight rows to their experts and back: five or so tiny steps, latency
        dict(name="sort_token", op="sort", train=False, T=1, d=7168, E=256, k=8, zipf=1.2, drop=0.0, dtype="bf16"),
        # a training step's dispatch and combine with gradients, Kimi-like with skewed routing
        dict(name="sort_large", op="sort", train=True, T=4096, d=7168, E=256, k=8, zipf=1.2, drop=0.0, dtype="bf16"),
        # odd sizes and rows without an expert (capacity or another GPU's experts), half precision
        dict(name="sort_odd", op="sort", train=True, T=1777, d=1333, E=37, k=3, zipf=0.6, drop=0.2, dtype="f16"),
        # activations of the Kimi-like layer to 4 bits and back to values
        dict(name="fp4_rows", op="fp4", what="quantize", T=4096, K=7168, N=0, E=1, k=1, zipf=0.0, act=False, dtype="bf16"),
        # one decoded token: its eight experts' gate and up products, bound by the weight stream
        dict(name="fp4_token", op="fp4", what="product", T=1, K=7168, N=4096, E=32, k=8, zipf=1.2, act=True, dtype="bf16"),
        # the balanced layer's first product with SwiGLU
        dict(name="fp4_balanced", op="fp4", what="product", T=2048, K=2048, N=1536, E=64, k=8, zipf=0.0, act=True, dtype="bf16"),
        # the largest: the Kimi-like layer's first product, about 128 rows an expert
        dict(name="fp4_large", op="fp4", what="product", T=4096, K=7168, N=4096, E=256, k=8, zipf=0.0, act=False, dtype="bf16"),
        # ragged: an odd count of blocks along K, odd N, experts without rows, half precision out
        dict(name="fp4_odd", op="fp4", what="product", T=333, K=1056, N=999, E=24, k=3, zipf=1.2, act=False, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "sort", "fp4"))
    if op == "norm":
        d = _log(rng, 96, 7168)
        T = min(_log(rng, 1, 16384), max(1, 100_000_000 // d))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        return dict(op="norm", train=rng.random() < 0.7, T=T, d=d, dtype=dtype, wdtype=rng.choice((dtype, "f32")),
                    pad=rng.choice((0, 0, 3, 8)))
    if op == "sort":
        d, E = _log(rng, 64, 7168), _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = min(_log(rng, 1, 8192), max(1, 200_000_000 // (d * k)))
        return dict(op="sort", train=rng.random() < 0.7, T=T, d=d, E=E, k=k, zipf=rng.choice((0.0, 0.6, 1.2)),
                    drop=rng.choice((0.0, 0.0, 0.2)), dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    K = BLOCK * _log(rng, 2, 224)
    if rng.random() < 0.2:
        return dict(op="fp4", what="quantize", T=_log(rng, 1, 4096), K=K, N=0, E=1, k=1, zipf=0.0, act=False,
                    dtype=rng.choice(("bf16", "f16", "f32")))
    N, E = 2 * _log(rng, 40, 2048) - rng.choice((0, 1)), _log(rng, 1, 64)
    k = rng.randint(1, min(8, E))
    return dict(op="fp4", what="product", T=_log(rng, 1, 2048), K=K, N=N, E=E, k=k, zipf=rng.choice((0.0, 0.6)),
                act=N % 2 == 0 and rng.random() < 0.5, dtype=rng.choice(("bf16", "bf16", "f16")))


# ------------------------------------------------------------------ inputs
def _route(T, E, k, zipf, gen):
    """k distinct experts of each token, by noise over a Zipf prior, as a router's top-k picks them."""
    z = torch.randn(T, E, generator=gen, device="cuda")
    if zipf > 0:
        z = z - zipf * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return z.topk(k, dim=1).indices.to(torch.int32)


def _to_fp4(x):
    """Codes (one a byte) and scale exponents of blocks of 32 along the last dimension: the smallest
    s with max |x| <= 6 * 2^s, x / 2^s rounded to the nearest of the 16 values, ties to the even code."""
    b = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                      # amax = m * 2^e, m in [0.5, 1)
    s = torch.where(m <= 0.75, e - 3, e - 2)
    s = torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(-127, 127)
    v = torch.ldexp(b, -s[..., None])
    y = v.abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    code = torch.where(y <= 2, y * 2, torch.where(y <= 4, y + 2, y / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(b).to(torch.uint8)
    return code.reshape(x.shape), s


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _scale_tiles(s):
    """Scale exponents [E, N, K/32] as bytes in the library's order: 512-byte tiles of 128 rows and four
    blocks, row r's scale of block kb at byte 16 * (r % 32) + 4 * (r % 128 // 32) + kb % 4."""
    E, N, B = s.shape
    rn, rb = -N % 128, -B % 4
    t = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, rb, 0, rn), value=127)
    t = t.reshape(E, (N + rn) // 128, 4, 32, (B + rb) // 4, 4)
    return t.permute(0, 1, 4, 3, 2, 5).contiguous().reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    st = dict(case=dict(case))
    T = case["T"]
    if case["op"] == "norm":
        d, wdt = case["d"], DTYPES[case["wdtype"]]
        ld = d + case["pad"]                     # the rows of a wider buffer
        st["x"] = normal(T, ld, std=1.5, mean=0.3)[:, :d]
        st["w"], st["b"] = normal(d, std=0.2, mean=1.0, dtype=wdt), normal(d, std=0.2, dtype=wdt)
        st["y"] = torch.empty(T, d, dtype=dt, device="cuda")
        st["mean"], st["rstd"] = (torch.empty(T, device="cuda") for _ in range(2))
        if case["train"]:
            st["dy"] = normal(T, ld)[:, :d]
            st["dx"] = torch.empty(T, d, dtype=dt, device="cuda")
            st["dw"], st["db"] = (torch.empty(d, dtype=wdt, device="cuda") for _ in range(2))
    elif case["op"] == "sort":
        d, E, k = case["d"], case["E"], case["k"]
        R = T * k
        ids = _route(T, E, k, case["zipf"], gen)
        if case["drop"] > 0:
            ids[torch.rand(T, k, generator=gen, device="cuda") < case["drop"]] = -1
        st["ids"] = ids.reshape(-1).contiguous()
        st["x"] = normal(T, d)
        st["w"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), dim=1)
        st["y"] = normal(R, d)                   # the experts' outputs, in expert order
        i32 = dict(dtype=torch.int32, device="cuda")
        st["counts"], st["offsets"] = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        st["perm"], st["inv"] = torch.empty(R, **i32), torch.empty(R, **i32)
        st["xp"] = torch.empty(R, d, dtype=dt, device="cuda")
        st["out"] = torch.empty(T, d, dtype=dt, device="cuda")
        if case["train"]:
            st["dout"], st["dxp"] = normal(T, d), normal(R, d)  # gradients of the output and of the experts' inputs
            st["dy"] = torch.empty(R, d, dtype=dt, device="cuda")
            st["dx"] = torch.empty(T, d, dtype=dt, device="cuda")
            st["dw"] = torch.empty(R, device="cuda")
    else:
        K, N, E, k = case["K"], case["N"], case["E"], case["k"]
        R = T * k
        st["x"] = normal(R, K)                   # rows in expert order
        if case["what"] == "quantize":
            st["values"] = torch.empty(R, K, dtype=dt, device="cuda")
        else:
            counts = torch.bincount(_route(T, E, k, case["zipf"], gen).reshape(-1), minlength=E)
            st["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            st["offsets"][1:] = counts.cumsum(0)
            st["most"] = int(counts.max())       # a host's bound on the rows of one expert
            wq, ws = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(E, N, K // BLOCK, dtype=torch.int32, device="cuda")
            for e in range(E):
                code, ws[e] = _to_fp4(normal(N, K, std=K ** -0.5, dtype=torch.bfloat16))
                wq[e] = _pack(code)
            st["wq"], st["wscale"], st["wtiles"] = wq, ws.to(torch.int8), _scale_tiles(ws)
            st["out"] = torch.empty(R, N // 2 if case["act"] else N, dtype=dt, device="cuda")
    return st


# ------------------------------------------------------------------ plain form
def _norm_plain(st):
    x, w, b = st["x"].float(), st["w"].float(), st["b"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    out = {"y": (xh * w + b).to(st["x"].dtype)}
    if st["case"]["train"]:
        dy = st["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        out.update(dx=dx.to(st["x"].dtype), dw=(dy * xh).sum(0).to(st["w"].dtype), db=dy.sum(0).to(st["b"].dtype))
    return out


def _sort_plain(st):
    c = st["case"]
    T, E, k, d, dt = c["T"], c["E"], c["k"], c["d"], st["x"].dtype
    ids = st["ids"].long()
    key = torch.where((ids >= 0) & (ids < E), ids, E)
    perm = torch.sort(key, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    counts = (key[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    kept = (key < E)[:, None]
    x = st["x"].float()
    xp = torch.where(kept[perm], x[perm // k], 0.0)
    w = st["w"].reshape(-1, 1)
    yt = torch.where(kept, st["y"].float()[inv], 0.0)
    out = {"offsets": offsets.to(torch.int32), "perm": perm.to(torch.int32), "xp": xp.to(dt),
           "out": (w * yt).reshape(T, k, d).sum(1).to(dt)}
    if c["train"]:
        g = st["dout"].float().repeat_interleave(k, 0)
        out["dy"] = torch.where(kept, w * g, 0.0)[perm].to(dt)
        out["dw"] = (g * yt).sum(1)
        out["dx"] = torch.where(kept, st["dxp"].float()[inv], 0.0).reshape(T, k, d).sum(1).to(dt)
    return out


def _values(q, s):
    """fp32 values of packed codes and their scale exponents."""
    v = torch.tensor(E2M1 + tuple(-t for t in E2M1), device="cuda")
    pair = torch.stack((v.repeat(16), v.repeat_interleave(16)), 1)      # both codes of a byte
    w = pair[q.int()].reshape(*s.shape, BLOCK)
    w *= torch.exp2(s.float())[..., None]
    return w.reshape(*q.shape[:-1], -1)


def _fp4_plain(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    code, s = _to_fp4(st["x"])
    x = _values(_pack(code), s)
    if c["what"] == "quantize":
        return {"values": x.to(dt)}
    off, R, E = st["offsets"].long(), x.shape[0], c["E"]
    e = torch.searchsorted(off[1:], torch.arange(R, device="cuda"), right=True)
    if R <= 32:                                   # a few rows: each with its own expert's weights
        h = torch.bmm(_values(st["wq"][e], st["wscale"][e]), x[:, :, None])[:, :, 0]
    else:                                         # every expert's rows side by side, padded to the longest
        at = e * st["most"] + torch.arange(R, device="cuda") - off[e]
        rows = x.new_zeros(E * st["most"], x.shape[1])
        rows[at] = x
        w = _values(st["wq"], st["wscale"])
        h = torch.bmm(rows.reshape(E, st["most"], -1), w.transpose(1, 2)).reshape(E * st["most"], -1)[at]
    if c["act"]:                                  # weight rows in pairs: gate, up
        g, u = h[:, 0::2], h[:, 1::2]
        h = g / (1.0 + torch.exp(-g)) * u
    return {"out": h.to(dt)}


# ------------------------------------------------------------------ the package's operators
def _norm_own(st):
    from mixture_experts_layer_stable_gb300 import ops
    T, d = st["x"].shape
    ops.moe_layernorm_forward(st["x"], st["w"], st["b"], EPS, st["y"], st["mean"], st["rstd"])
    if not st["case"]["train"]:
        return {"y": st["y"]}
    if "ws" not in st:                            # a workspace that the user's program keeps
        st["ws"] = torch.empty(ops.moe_layernorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    ops.moe_layernorm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], st["db"], st["ws"])
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"], "db": st["db"]}


def _sort_own(st):
    from mixture_experts_layer_stable_gb300 import ops
    c = st["case"]
    k = c["k"]
    if "ws" not in st:
        st["ws"] = torch.empty(ops.moe_sort_workspace_bytes(c["T"] * k, c["E"]), dtype=torch.uint8, device="cuda")
    ops.moe_sort_rows(st["ids"], st["counts"], st["offsets"], st["perm"], st["inv"], st["ws"])
    ops.moe_permute(st["x"], k, st["inv"], st["offsets"], st["xp"])
    ops.moe_unpermute(st["y"], st["w"], k, st["inv"], st["offsets"], st["out"])
    out = {"offsets": st["offsets"], "perm": st["perm"], "xp": st["xp"], "out": st["out"]}
    if c["train"]:
        ops.moe_unpermute_backward(st["dout"], st["y"], st["w"], k, st["inv"], st["offsets"], st["dy"], st["dw"])
        ops.moe_unpermute(st["dxp"], None, k, st["inv"], st["offsets"], st["dx"])
        out.update(dy=st["dy"], dw=st["dw"], dx=st["dx"])
    return out


def _fp4_own(st):
    from mixture_experts_layer_stable_gb300 import ops
    c = st["case"]
    R, K, E = st["x"].shape[0], c["K"], c["E"]
    if "q" not in st:                             # buffers that the user's program keeps
        st["q"] = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda")
        st["qs"] = torch.empty(ops.moe_mxfp4_row_scale_bytes(R, K, E), dtype=torch.uint8, device="cuda")
        if c["what"] == "product":
            st["ws"] = torch.empty(ops.moe_mxfp4_product_workspace_bytes(R, c["N"], K, E), dtype=torch.uint8, device="cuda")
    if c["what"] == "quantize":
        ops.moe_quantize_mxfp4_rows(st["x"], st["q"], st["qs"])
        ops.moe_dequantize_mxfp4_rows(st["q"], st["qs"], st["values"])
        return {"values": st["values"]}
    ops.moe_quantize_mxfp4_rows(st["x"], st["q"], st["qs"], st["offsets"])
    ops.moe_mxfp4_product(st["q"], st["qs"], st["offsets"], st["wq"], st["wtiles"],
                          ops.MOE_ACT_SWIGLU if c["act"] else ops.MOE_ACT_NONE, st["out"], st["ws"])
    return {"out": st["out"]}


PLAIN = {"norm": _norm_plain, "sort": _sort_plain, "fp4": _fp4_plain}
OWN = {"norm": _norm_own, "sort": _sort_own, "fp4": _fp4_own}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    T, b = case["T"], size[case["dtype"]]
    if case["op"] == "norm":
        d, wb = case["d"], size[case["wdtype"]]
        if not case["train"]:
            return {"bytes": 2 * T * d * b + 2 * d * wb, "flops": 8 * T * d}
        return {"bytes": 4 * T * d * b + 4 * d * wb, "flops": 24 * T * d}
    if case["op"] == "sort":
        d, R = case["d"], T * case["k"]
        n = T * d * b + R * d * b + R * d * b + T * d * b + R * 4 * 3 + case["E"] * 4  # x, xp; y, out; ids, w, perm
        f = 2 * R * d
        if case["train"]:
            n += T * d * b + R * d * b + R * d * b + T * d * b + R * 4                 # dout, dy; dxp, dx; dw (y once)
            f += 4 * R * d
        return {"bytes": n, "flops": f}
    K, N, E, k = case["K"], case["N"], case["E"], case["k"]
    R = T * k
    if case["what"] == "quantize":
        return {"bytes": 2 * R * K * b, "flops": 4 * R * K}
    touched = E * (1 - (1 - k / E) ** T)          # experts with a row, for even routing
    return {"bytes": int(R * K * b + touched * N * K * 17 / 32 + R * (N // 2 if case["act"] else N) * b), "flops": 2 * R * N * K}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_fp4(x):
    """Values of x [n, K] after quantisation, in 64 bits, by the distances to the 4-bit values."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.ceil(torch.log2(amax / 6.0)).clamp(-127, 127)
    s = torch.where(amax <= 6.0 * torch.exp2(s - 1), s - 1, s)
    s = torch.where(amax > 6.0 * torch.exp2(s), s + 1, s)
    s = torch.where(amax > 0, s, torch.full_like(s, -127.0))
    v = b / torch.exp2(s)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    up = torch.searchsorted(mid, v.abs(), right=True)     # a tie goes to the upper neighbour
    low = torch.searchsorted(mid, v.abs(), right=False)   # a tie goes to the lower one
    code = torch.where(up % 2 == 0, up, low)              # the even code of the two
    return (torch.where(v < 0, -1.0, 1.0) * grid[code] * torch.exp2(s)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    T = case["T"]
    if case["op"] == "norm":
        n, d = T, case["d"]
        x, w, b = st["x"].double(), st["w"].double(), st["b"].double()
        mu = x.sum(1) / d
        var = ((x - mu[:, None]) ** 2).sum(1) / d
        sd = torch.sqrt(var + EPS)[:, None]
        z = (x - mu[:, None]) / sd
        out = {"y": z * w + b}
        if case["train"]:
            dy = st["dy"].double()
            dz = dy * w
            out["dx"] = (dz - dz.sum(1, keepdim=True) / d - z * (dz * z).sum(1, keepdim=True) / d) / sd
            out["dw"], out["db"] = (dy * z).sum(0), dy.sum(0)
        return out
    if case["op"] == "sort":
        E, k, d = case["E"], case["k"], case["d"]
        R = T * k
        ids = st["ids"].cpu().tolist()
        order = sorted(range(R), key=lambda r: ids[r] if 0 <= ids[r] < E else E)
        off = [0] * (E + 1)
        for i in ids:
            if 0 <= i < E:
                off[i + 1] += 1
        for e in range(E):
            off[e + 1] += off[e]
        kept = off[E]
        perm = torch.tensor(order, device="cuda")
        live = perm[:kept]
        tok, wr = live // k, st["w"].reshape(-1).double()[live][:, None]
        y, x = st["y"].double()[:kept], st["x"].double()
        xp = torch.zeros(R, d, dtype=torch.float64, device="cuda")
        xp[:kept] = x[tok]
        out = {"offsets": None, "perm": None, "xp": xp,
               "out": torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add_(0, tok, wr * y)}
        if case["train"]:
            g = st["dout"].double()[tok]
            dy, dw = torch.zeros_like(xp), torch.zeros(R, dtype=torch.float64, device="cuda")
            dy[:kept] = wr * g
            dw[live] = (g * y).sum(1)
            out.update(dy=dy, dw=dw, dx=torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add_(0, tok, st["dxp"].double()[:kept]))
        return out
    x = _exact_fp4(st["x"])
    if case["what"] == "quantize":
        return {"values": x}
    off = st["offsets"].cpu().tolist()
    N = case["N"]
    h = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
    val = torch.tensor(E2M1 + tuple(-t for t in E2M1), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if off[e] < off[e + 1]:
            q = st["wq"][e].long()
            w = torch.empty(N, case["K"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = val[q % 16], val[q // 16]
            w *= torch.exp2(st["wscale"][e].double()).repeat_interleave(BLOCK, 1)
            h[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w.T
    if case["act"]:
        g, u = h[:, 0::2], h[:, 1::2]
        h = g * torch.sigmoid(g) * u
    return {"out": h}
