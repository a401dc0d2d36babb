"""Cases of the operators of a training step around an expert function: matrix
products grouped by expert with ragged row counts (forward, gradients of the rows
and of the weights) and activation checkpoints in 8 bits (rows, and SwiGLU whose
backward works from them).

run() computes a case in its plain form (elementary torch operations in fp32,
rounded once at the end) or, with own = True, through the package's operators.
exact() computes the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32                                       # elements that share a scale


def listed():
    return [
        # one decoded token's eight rows through its experts' first product: bound by the weight stream
        dict(name="prod_token", op="product", train=False, T=1, K=7168, N=4096, E=32, k=8, zipf=0.0, drop=0.0, dtype="bf16", gdtype="bf16", pad=0),
        # the smallest layer's training step, three calls of a few rows an expert: latency
        dict(name="prod_tiny", op="product", train=True, T=64, K=128, N=128, E=8, k=2, zipf=0.0, drop=0.0, dtype="bf16", gdtype="bf16", pad=0),
        # the balanced layer's first product in training: about 256 rows an expert
        dict(name="prod_balanced", op="product", train=True, T=2048, K=2048, N=1536, E=64, k=8, zipf=0.0, drop=0.0, dtype="bf16", gdtype="bf16", pad=0),
        # the Kimi-like layer's first product with skewed routing: some experts with thousands of rows, many with none
        dict(name="prod_skewed", op="product", train=False, T=4096, K=7168, N=4096, E=256, k=8, zipf=1.2, drop=0.0, dtype="bf16", gdtype="bf16", pad=0),
        # one GPU's share of an expert-parallel training run, weight gradients in fp32: bound by arithmetic, the largest
        dict(name="prod_share", op="product", train=True, T=16384, K=7168, N=4096, E=4, k=1, zipf=0.0, drop=0.0, dtype="bf16", gdtype="f32", pad=0),
        # odd sizes, rows with a stride, rows without an expert, half precision
        dict(name="prod_odd", op="product", train=True, T=333, K=1061, N=999, E=24, k=3, zipf=1.2, drop=0.1, dtype="f16", gdtype="f32", pad=3),
        # a small model in full precision
        dict(name="prod_f32", op="product", train=True, T=512, K=640, N=896, E=16, k=2, zipf=0.0, drop=0.0, dtype="f32", gdtype="f32", pad=0),
        # the activation between one decoded token's two products: launch latency
        dict(name="swiglu_token", op="checkpoint", what="swiglu", train=False, rows=8, n=2048, dtype="bf16", pad=0),
        # training steps' activation, its input kept in 8 bits: the balanced layer and the Kimi-like one
        dict(name="swiglu_balanced", op="checkpoint", what="swiglu", train=True, rows=16384, n=768, dtype="bf16", pad=0),
        dict(name="swiglu_large", op="checkpoint", what="swiglu", train=True, rows=32768, n=2048, dtype="bf16", pad=0),
        # odd sizes and strides, half precision
        dict(name="swiglu_odd", op="checkpoint", what="swiglu", train=True, rows=5331, n=1333, dtype="f16", pad=3),
        # the rows that enter the experts, kept in 8 bits and brought back for the weight gradients
        dict(name="rows_large", op="checkpoint", what="rows", train=True, rows=16384, n=7168, dtype="bf16", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    pad = rng.choice((0, 0, 3, 8))
    if rng.random() < 0.6:
        unit = rng.choice((1, 1, 8, 64))          # odd lengths, whole vectors, whole tiles
        K, N = (unit * max(1, _log(rng, 64, 7168) // unit) for _ in range(2))
        E = min(_log(rng, 1, 128), max(1, 400_000_000 // (K * N)))
        k = rng.randint(1, min(8, E))
        T = min(_log(rng, 1, 16384), max(1, (20_000_000_000 if dtype == "f32" else 200_000_000_000) // (K * N * k)),
                max(1, 120_000_000 // (k * max(K, N))))
        return dict(op="product", train=rng.random() < 0.6, T=T, K=K, N=N, E=E, k=k, zipf=rng.choice((0.0, 0.6, 1.2)),
                    drop=rng.choice((0.0, 0.0, 0.1)), dtype=dtype, gdtype=rng.choice((dtype, "f32")), pad=pad)
    n = _log(rng, 48, 7168)
    rows = min(_log(rng, 1, 32768), 60_000_000 // n)
    if rng.random() < 0.3:
        return dict(op="checkpoint", what="rows", train=True, rows=rows, n=n, dtype=dtype, pad=pad)
    return dict(op="checkpoint", what="swiglu", train=rng.random() < 0.8, rows=rows, n=n, dtype=dtype, pad=pad)


# ------------------------------------------------------------------ inputs
def _route(T, E, k, zipf, gen):
    """k distinct experts of each token, by noise over a Zipf prior, as a router's top-k picks them."""
    z = torch.randn(T, E, generator=gen, device="cuda")
    if zipf > 0:
        z = z - zipf * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return z.topk(k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, pad = DTYPES[case["dtype"]], case["pad"]

    def rows_of(n, d, std=1.0, mean=0.0):         # rows of a wider buffer
        return (torch.randn(n, d + pad, generator=gen, device="cuda") * std + mean).to(dt)[:, :d]

    def zeros(n, d, t=dt):
        return torch.zeros(n, d, dtype=t, device="cuda")

    st = dict(case=dict(case))
    if case["op"] == "product":
        T, K, N, E, k = (case[i] for i in ("T", "K", "N", "E", "k"))
        ids = _route(T, E, k, case["zipf"], gen).reshape(-1)
        if case["drop"] > 0:                      # over an expert's capacity, or another GPU's expert
            ids = ids[torch.rand(T * k, generator=gen, device="cuda") >= case["drop"]]
        R = T * k
        st["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        st["offsets"][1:] = torch.bincount(ids, minlength=E).cumsum(0)
        st["split"] = st["offsets"].tolist()      # the host's copy, for the plain form's loop
        st["x"] = rows_of(R, K)                   # rows in expert order, those without an expert last
        st["w"] = torch.empty(E, K, N, dtype=dt, device="cuda")
        for e in range(E):
            st["w"][e] = torch.randn(K, N, generator=gen, device="cuda") * K ** -0.5
        st["out"] = zeros(R, N)
        if case["train"]:
            st["dy"] = rows_of(R, N)
            st["dx"] = zeros(R, K)
            st["dw"] = torch.empty(E, K, N, dtype=DTYPES[case["gdtype"]], device="cuda")
        return st
    R, n = case["rows"], case["n"]
    if case["what"] == "rows":
        st["x"] = rows_of(R, n, 1.5, 0.3)
        st["values"] = zeros(R, n)
    else:
        st["h"] = rows_of(R, 2 * n, 1.2)          # gates, then up products
        st["a"] = zeros(R, n)
        if case["train"]:
            st["da"] = rows_of(R, n)
            st["again"], st["dh"] = zeros(R, n), zeros(R, 2 * n)
    return st


# ------------------------------------------------------------------ plain form
def _product_plain(st):
    c, x, w, off = st["case"], st["x"], st["w"], st["split"]
    out = {"out": torch.zeros_like(st["out"])}
    if c["train"]:
        out.update(dx=torch.zeros_like(st["dx"]), dw=torch.zeros_like(st["dw"]))
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        xe, we = x[a:b].float(), w[e].float()
        out["out"][a:b] = xe @ we
        if c["train"]:
            dye = st["dy"][a:b].float()
            out["dx"][a:b] = dye @ we.t()
            out["dw"][e] = xe.t() @ dye
    return out


def _int8_plain(x):
    """fp32 values of x after quantisation: blocks of 32 along the last dimension share 2^s, the smallest with
    max |x| <= 127 * 2^s (s >= -127); x / 2^s rounded to the nearest whole number, ties to the even one."""
    n = x.shape[-1]
    b = torch.nn.functional.pad(x.float(), (0, -n % BLOCK)).reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                      # amax = m * 2^e, m in [0.5, 1)
    s = torch.where(m <= 127.0 / 128.0, e - 7, e - 6)
    s = torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(min=-127)
    return torch.ldexp(torch.round(torch.ldexp(b, -s)), s).reshape(x.shape[0], -1)[:, :n]


def _swiglu_plain(h, n):
    g, u = h[:, :n], h[:, n:]
    sg = 1.0 / (1.0 + torch.exp(-g))
    return g, u, sg, g * sg


def _checkpoint_plain(st):
    c = st["case"]
    n, dt = c["n"], DTYPES[c["dtype"]]
    if c["what"] == "rows":
        return {"values": _int8_plain(st["x"]).to(dt)}
    _, u, _, silu = _swiglu_plain(st["h"].float(), n)
    out = {"a": (silu * u).to(dt)}
    if c["train"]:
        kept = torch.cat((_int8_plain(st["h"][:, :n]), _int8_plain(st["h"][:, n:])), 1)
        g, u, sg, silu = _swiglu_plain(kept, n)
        da = st["da"].float()
        dg = da * u * (sg * (1.0 + g * (1.0 - sg)))
        out.update(dh=torch.cat((dg, da * silu), 1).to(dt), again=(silu * u).to(dt))
    return out


# ------------------------------------------------------------------ the package's operators
def _workspace(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _product_own(st):
    from mixture_experts_layer_stable_gb300 import ops
    c = st["case"]
    if "ws" not in st:                            # a workspace that the user's program keeps
        st["ws"] = _workspace(ops.moe_grouped_product_workspace_bytes(c["T"] * c["k"], c["K"], c["N"], c["E"]))
    off, ws = st["offsets"], st["ws"]
    ops.moe_grouped_product(st["x"], st["w"], off, st["out"], ws)
    if not c["train"]:
        return {"out": st["out"]}
    ops.moe_grouped_product(st["dy"], st["w"], off, st["dx"], ws, transposed=True)
    ops.moe_grouped_product_dw(st["x"], st["dy"], off, st["dw"], ws)
    return {"out": st["out"], "dx": st["dx"], "dw": st["dw"]}


def _checkpoint_own(st):
    from mixture_experts_layer_stable_gb300 import ops
    c = st["case"]
    R, n = c["rows"], c["n"]
    if c["train"] and "q" not in st:              # the checkpoint, which lives from the forward to the backward
        wide = 1 if c["what"] == "rows" else 2
        st["q"] = torch.empty(R, wide * n, dtype=torch.int8, device="cuda")
        st["s"] = _workspace(ops.moe_mxint8_scale_bytes(wide * R, n))
    if c["what"] == "rows":
        ops.moe_quantize_mxint8_rows(st["x"], st["q"], st["s"])
        ops.moe_dequantize_mxint8_rows(st["q"], st["s"], st["values"])
        return {"values": st["values"]}
    if not c["train"]:
        ops.moe_swiglu_forward(st["h"], st["a"])
        return {"a": st["a"]}
    ops.moe_swiglu_forward(st["h"], st["a"], st["q"], st["s"])
    ops.moe_swiglu_backward(st["da"], None, st["dh"], st["again"], st["q"], st["s"])
    return {"a": st["a"], "dh": st["dh"], "again": st["again"]}


PLAIN = {"product": _product_plain, "checkpoint": _checkpoint_plain}
OWN = {"product": _product_own, "checkpoint": _checkpoint_own}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def _touched(T, E, k, zipf):
    """Experts with a row: expert e is among a token's k with the normal tail's probability past a
    threshold that k experts pass on average."""
    if k >= E:
        return E

    def chosen(at):
        return [0.5 * math.erfc((at + zipf * math.log(e + 1)) / math.sqrt(2.0)) for e in range(E)]

    lo, hi = -20.0, 20.0
    for _ in range(60):
        at = (lo + hi) / 2
        lo, hi = (at, hi) if sum(chosen(at)) > k else (lo, at)
    return sum(1 - (1 - p) ** T for p in chosen(lo))


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "product":
        T, K, N, E, k = (case[i] for i in ("T", "K", "N", "E", "k"))
        R = T * k * (1 - case["drop"])
        n = R * (K + N) * b + _touched(T * (1 - case["drop"]), E, k, case["zipf"]) * K * N * b  # x, out; w
        f = 2 * R * K * N
        if case["train"]:
            n += R * (K + N) * b + E * K * N * SIZE[case["gdtype"]]                             # dy, dx; dw
            f *= 3
        return {"bytes": int(n), "flops": int(f)}
    e = case["rows"] * case["n"]
    if case["what"] == "rows":
        return {"bytes": 2 * e * b, "flops": 4 * e}
    if not case["train"]:
        return {"bytes": 3 * e * b, "flops": 6 * e}
    return {"bytes": 7 * e * b, "flops": 30 * e}  # h, a; da, dh, a again


# ------------------------------------------------------------------ 64 bits, from the definitions
def _int8_exact(x):
    """Values of x after quantisation, in 64 bits: the scale by trying exponents."""
    n = x.shape[1]
    v = torch.zeros(x.shape[0], (n + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :n] = x.double()
    v = v.reshape(x.shape[0], -1, BLOCK)
    top = v.abs().max(-1, keepdim=True).values
    s = torch.floor(torch.log2(top.clamp(min=2.0 ** -160) / 127.0)) - 1
    for _ in range(3):                            # up to the first exponent that holds the block
        s = torch.where(top > 127.0 * torch.exp2(s), s + 1, s)
    step = torch.exp2(s.clamp(min=-127.0))
    y = v / step
    low = torch.floor(y)
    up = (y - low > 0.5) | ((y - low == 0.5) & (low % 2 != 0))
    return ((low + up.double()) * step).reshape(x.shape[0], -1)[:, :n]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        off, R = st["split"], case["T"] * case["k"]
        x, f64 = st["x"], dict(dtype=torch.float64, device="cuda")
        out = {"out": torch.zeros(R, case["N"], **f64)}
        if case["train"]:
            out.update(dx=torch.zeros(R, case["K"], **f64), dw=torch.zeros(case["E"], case["K"], case["N"], **f64))
        for e in range(case["E"]):
            r = slice(off[e], off[e + 1])
            if r.start < r.stop:
                out["out"][r] = torch.einsum("pk,kn->pn", x[r].double(), st["w"][e].double())
                if case["train"]:
                    out["dx"][r] = torch.einsum("pn,kn->pk", st["dy"][r].double(), st["w"][e].double())
                    out["dw"][e] = torch.einsum("pk,pn->kn", x[r].double(), st["dy"][r].double())
        return out
    n = case["n"]
    if case["what"] == "rows":
        return {"values": _int8_exact(st["x"])}
    h = st["h"].double()
    out = {"a": h[:, :n] * torch.sigmoid(h[:, :n]) * h[:, n:]}
    if case["train"]:
        g, u, da = _int8_exact(st["h"][:, :n]), _int8_exact(st["h"][:, n:]), st["da"].double()
        p = torch.sigmoid(g)
        slope = p + g * p * torch.sigmoid(-g)
        out.update(dh=torch.cat((da * u * slope, da * g * p), 1), again=g * p * u)
    return out
