"""Microscaled 4-bit floating point (MXFP4 and NVFP4) around a linear layer and a gated
feed-forward block: the measured cases, their plain forms and their 64-bit definitions.

Formats. A 4-bit element is e2m1: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, rounded to nearest, ties to the
even code, saturating at 6. Blocks run along the summed axis of the product that uses them:
  mxfp4  blocks of 32, scale 2^e with e = floor(log2(amax of the block)) - 2 (>= -127), one byte
         e + 127;
  nvfp4  blocks of 16, scale e4m3(amax of the block / (6 f)), one byte, times a power of two f
         for the whole tensor, f = 2^ceil(log2(amax of the tensor / 2688)), or a kept one.
Codes are packed two to a byte, low half first, in rows of `ld` elements (the columns rounded up
to 128, zeros behind the last). Scales lie in tiles of 128 rows by 4 blocks (512 bytes): row r,
block b at tile (r // 128, b // 4), byte 16 (r % 32) + 4 (r % 128 // 32) + b % 4.
"""
import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# kept tensor factors of nvfp4, as a calibration leaves them: activations, the gated product, its gradient
X_FACTOR, A_FACTOR, DU_FACTOR = 2.0 ** -4, 2.0 ** -6, 2.0 ** -16


def listed():
    return [
        # a prompt's activations (h = 4096), before a product
        {"name": "quantize-prompt", "op": "quantize", "fmt": "mxfp4", "dtype": "bf16",
         "rows": 2048, "cols": 4096, "pad": 0, "both": False},
        # fp32 master weights of fc2 (f = 11008) laid out for the forward and the backward product
        {"name": "quantize-weights-both", "op": "quantize", "fmt": "nvfp4", "dtype": "f32",
         "rows": 4096, "cols": 11008, "pad": 0, "both": True},
        # one token through the QKV projection
        {"name": "linear-token", "op": "linear", "fmt": "mxfp4", "out": "bf16",
         "M": 1, "N": 12288, "K": 4096},
        # a batch of sequences, one token each, through fc2
        {"name": "linear-batch", "op": "linear", "fmt": "nvfp4", "out": "bf16",
         "M": 37, "N": 4096, "K": 11008},
        # a short ragged prompt through a layer of odd sizes, fp32 out
        {"name": "linear-ragged", "op": "linear", "fmt": "mxfp4", "out": "f32",
         "M": 333, "N": 1777, "K": 1111},
        # a prompt through the QKV projection
        {"name": "linear-prompt", "op": "linear", "fmt": "mxfp4", "out": "bf16",
         "M": 2048, "N": 12288, "K": 4096},
        # fc1 of the h = 6144 layer over two sequences of 4096
        {"name": "linear-large", "op": "linear", "fmt": "nvfp4", "out": "bf16",
         "M": 8192, "N": 24576, "K": 6144},
        # both gradients of the QKV projection over one sequence
        {"name": "linear-backward", "op": "linear_bwd", "fmt": "mxfp4",
         "M": 2048, "N": 12288, "K": 4096},
        # the gated block (h = 4096, f = 11008): one token, a prompt, a training step's backward
        {"name": "gated-token", "op": "gated", "fmt": "mxfp4", "act": "silu", "keep": False,
         "M": 1, "H": 4096, "F": 11008},
        {"name": "gated-prompt", "op": "gated", "fmt": "nvfp4", "act": "silu", "keep": True,
         "M": 2048, "H": 4096, "F": 11008},
        {"name": "gated-backward", "op": "gated_bwd", "fmt": "mxfp4", "act": "silu",
         "M": 2048, "H": 4096, "F": 11008},
        # the same on a ragged batch of a small layer (h = 1024) with an odd width
        {"name": "gated-backward-ragged", "op": "gated_bwd", "fmt": "nvfp4", "act": "gelu",
         "M": 517, "H": 1024, "F": 2731},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = 2.0 * 8192 * 24576 * 6144
    fmt = rng.choice(["mxfp4", "nvfp4"])
    op = rng.choice(["quantize", "linear", "linear", "linear_bwd", "gated", "gated_bwd"])
    while True:
        if op == "quantize":
            c = {"op": op, "fmt": fmt, "dtype": rng.choice(["bf16", "f32"]), "rows": size(1, 16384),
                 "cols": size(16, 24576), "pad": rng.choice([0, 0, 8, 5]), "both": rng.random() < 0.5}
            if c["rows"] * c["cols"] <= 4096 * 11008:
                return c
        elif op in ("linear", "linear_bwd"):
            c = {"op": op, "fmt": fmt, "M": size(1, 8192), "N": size(64, 24576), "K": size(64, 12288)}
            if op == "linear":
                c["out"] = rng.choice(["bf16", "bf16", "f32"])
            if 2.0 * c["M"] * c["N"] * c["K"] * (2 if op == "linear_bwd" else 1) <= most / 2:
                return c
        else:
            c = {"op": op, "fmt": fmt, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                 "M": size(1, 4096), "H": size(128, 6144), "F": size(128, 16384)}
            if op == "gated":
                c["keep"] = rng.random() < 0.5
            if 6.0 * c["M"] * c["H"] * c["F"] * (2 if op == "gated_bwd" else 1) <= most / 2:
                return c


# ------------------------------------------------------------------------- plain form, 32 bits
def up128(n):
    return (n + 127) // 128 * 128


def two_to(e):
    """2^e for whole e from -127 to 127, put together from its bits (a power function may be off)."""
    bits = torch.where(e > -127, (e.int() + 127) << 23, 1 << 22)
    return bits.int().view(torch.float32)


def tensor_factor(x):
    """f = 2^ceil(log2(amax / 2688)), 1 for zeros: with amax = m 2^e, 0.5 <= m < 1, and
    2688 = 0.65625 * 2^12, the exponent is e - 12, one more where m > 0.65625."""
    amax = x.abs().max().float()
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, two_to((e - 12 + (m > 0.65625).int()).clamp(min=-126)), torch.ones_like(amax))


def quantize(x, fmt, factor):
    """Rows of x in blocks along the columns: (signed element values [rows, blocks, block],
    scale values [rows, blocks, 1], scale bytes [rows, blocks]) in fp32; columns padded to 128."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x.float(), (0, up128(cols) - cols)).view(rows, -1, BLOCK[fmt])
    if fmt == "mxfp4":
        amax = b.abs().amax(2, keepdim=True)
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 125)
        a, scale, byte = b * two_to(-e), two_to(e), e + 127
    else:
        b = b / factor
        six = torch.full((), 6.0, device=x.device)  # a tensor: a number would become a product with 1 / 6
        s = (b.abs().amax(2, keepdim=True) / six).clamp(max=448).to(torch.float8_e4m3fn)
        byte, scale = s.view(torch.uint8), s.float()
        a = torch.where(scale > 0, b / torch.where(scale > 0, scale, 1), 0)
        scale = scale * factor
    m = a.abs()
    level = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5))
    value = torch.tensor(GRID, device=x.device)[level.int()]
    return torch.where(a < 0, -value, value), scale, byte.to(torch.uint8).squeeze(2)


def rounded(x, fmt, factor):
    """x through 4 bits and back, fp32, without the padding."""
    value, scale, _ = quantize(x, fmt, factor)
    return (value * scale).view(x.shape[0], -1)[:, :x.shape[1]]


def pack(x, fmt, factor, rows=None, ld=None):
    """Codes [rows, ld / 2] and scale tiles of x, with rows and columns of zeros up to rows, ld."""
    n, cols = x.shape
    rows, ld = rows or n, ld or up128(cols)
    value, _, byte = quantize(torch.nn.functional.pad(x, (0, ld - cols)), fmt, factor)
    grid = torch.tensor(GRID, device=x.device)
    code = torch.bucketize(value.abs().contiguous(), grid).to(torch.uint8) + 8 * (value < 0).to(torch.uint8)
    code = torch.nn.functional.pad(code.view(n, ld), (0, 0, 0, rows - n))
    tiles = torch.nn.functional.pad(byte, (0, 0, 0, up128(rows) - n))
    tiles = tiles.view(up128(rows) // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous()
    return code[:, 0::2] | (code[:, 1::2] << 4), tiles.view(-1)


def unpack(codes, tiles, fmt, factor):
    """The fp32 values that packed codes and scale tiles stand for, [rows, ld]."""
    rows, ld = codes.shape[0], codes.shape[1] * 2
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    value = grid[torch.stack([codes & 15, codes >> 4], 2).view(rows, ld).int()]
    byte = tiles.view(up128(rows) // 128, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up128(rows), -1)[:rows]
    if fmt == "mxfp4":
        scale = two_to(byte.int() - 127)
    else:
        scale = byte.contiguous().view(torch.float8_e4m3fn).float() * factor
    return (value.view(rows, -1, BLOCK[fmt]) * scale.unsqueeze(2)).view(rows, ld)


def act_plain(z, name):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(z / math.sqrt(2.0)))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 0.134145 * z * z)


# ------------------------------------------------------------------------- inputs
def activations(rows, cols, gen, dtype, spread=1.0):
    """Rows of a residual stream: channels of different strength, a few of them strong."""
    strength = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    strength[torch.randint(cols, (max(1, cols // 256),), device="cuda", generator=gen)] *= 12
    return (spread * torch.randn(rows, cols, device="cuda", generator=gen) * strength).to(dtype)


def weight(w, fmt, **kw):
    f = tensor_factor(w) if fmt == "nvfp4" else torch.ones((), device="cuda")
    codes, tiles = pack(w, fmt, f, **kw)
    return {"codes": codes, "tiles": tiles, "factor": torch.stack([w.abs().max().float(), f])}


def factor_of(v):
    return torch.tensor([0.0, v], device="cuda")


def room(rows, cols, fmt):
    """Buffers for codes and scale tiles of [rows, cols], as a program keeps them."""
    ld = up128(cols)
    return {"codes": torch.empty(rows, ld // 2, dtype=torch.uint8, device="cuda"),
            "tiles": torch.empty(up128(rows) * ld // BLOCK[fmt], dtype=torch.uint8, device="cuda"),
            "factor": factor_of(1.0)}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    fmt, s = case["fmt"], {"case": dict(case), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    randn = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    empty = lambda *n, t=torch.bfloat16: torch.empty(*n, dtype=t, device="cuda")  # noqa: E731
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = activations(R, C + case["pad"], gen, t)
        s.update(x=wide[:, :C], q=room(R, C, fmt), y=empty(R, C))
        if case["both"]:
            s.update(qt=room(C, R, fmt), yt=empty(C, R))
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s.update(x=activations(M, K, gen, torch.bfloat16), q=room(M, K, fmt),
                 w=weight(0.02 * randn(N, K), fmt),
                 y=empty(M, N, t=torch.bfloat16 if case["out"] == "bf16" else torch.float32))
        s["q"]["factor"] = factor_of(X_FACTOR if fmt == "nvfp4" else 1.0)
    elif case["op"] == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        s.update(dy=(1e-3 * randn(M, N)).bfloat16(), q=room(M, N, fmt), qt=room(N, M, fmt),
                 wt=weight(0.02 * randn(K, N), fmt),  # the weight transposed, blocks along N
                 xt=weight(activations(M, K, gen, torch.bfloat16).t(), fmt),  # kept by the forward
                 dx=empty(M, K), dw=empty(N, K, t=torch.float32))
    else:
        M, H, F = case["M"], case["H"], case["F"]
        P = up128(F)
        wg, wu, w2 = 0.02 * randn(F, H), 0.02 * randn(F, H), 0.02 * randn(H, F)
        gap = torch.zeros(P - F, H, device="cuda")
        one = torch.cat([wg, gap, wu, gap])  # gate rows from 0, up rows from F rounded up to 128
        if case["op"] == "gated":
            s.update(x=activations(M, H, gen, torch.bfloat16, 0.5), q=room(M, H, fmt), w1=weight(one, fmt),
                     w2=weight(w2, fmt), a=room(M, F, fmt), y=empty(M, H),
                     u=empty(M, 2 * F) if case["keep"] else None)
            s["q"]["factor"] = factor_of(X_FACTOR if fmt == "nvfp4" else 1.0)
            s["a"]["factor"] = factor_of(A_FACTOR if fmt == "nvfp4" else 1.0)
        else:
            s.update(dy=(1e-3 * randn(M, H)).bfloat16(), u=(1.5 * randn(M, 2 * F)).bfloat16(),
                     w2t=weight(w2.t(), fmt), w1t=weight(one.t(), fmt),
                     xt=weight(activations(M, H, gen, torch.bfloat16, 0.5).t(), fmt),
                     q=room(M, H, fmt), qt=room(H, M, fmt), da=empty(M, F), du=room(M, 2 * P, fmt),
                     dut=room(2 * P, M, fmt), at=room(F, M, fmt), dx=empty(M, H), dwg=empty(F, H),
                     dwu=empty(F, H), dw2=empty(H, F))
            for k, v in (("du", DU_FACTOR), ("dut", DU_FACTOR), ("at", A_FACTOR)):
                s[k]["factor"] = factor_of(v if fmt == "nvfp4" else 1.0)
    return s


# ------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return run_own(state, c)
    fmt, op = c["fmt"], c["op"]
    back = lambda w: unpack(w["codes"], w["tiles"], fmt, w["factor"][1])  # noqa: E731
    fit = lambda x, n: torch.nn.functional.pad(x, (0, up128(n) - n))  # noqa: E731

    def factor(x):
        return tensor_factor(x) if fmt == "nvfp4" else None

    if op == "quantize":
        x = state["x"]
        f = factor(x)
        out = {"y": rounded(x, fmt, f).bfloat16()}
        if c["both"]:
            out["yt"] = rounded(x.t(), fmt, f).bfloat16()
        return out
    if op == "linear":
        x = fit(rounded(state["x"], fmt, state["q"]["factor"][1]), c["K"])
        return {"y": (x @ back(state["w"]).t()).to(state["y"].dtype)}
    if op == "linear_bwd":
        dy = state["dy"]
        f = factor(dy)
        dx = fit(rounded(dy, fmt, f), c["N"]) @ back(state["wt"]).t()
        dw = fit(rounded(dy.t(), fmt, f), c["M"]) @ back(state["xt"]).t()
        return {"dx": dx.bfloat16(), "dw": dw}
    M, H, F, P = c["M"], c["H"], c["F"], up128(c["F"])
    if op == "gated":
        x = fit(rounded(state["x"], fmt, state["q"]["factor"][1]), H)
        z = x @ back(state["w1"]).t()
        g, u = z[:, :F], z[:, P:P + F]
        a = act_plain(g, c["act"])[0] * u
        a = fit(rounded(a, fmt, state["a"]["factor"][1]), F)
        out = {"y": (a @ back(state["w2"]).t()).bfloat16()}
        if c["keep"]:
            out["u"] = torch.cat([g, u], 1).bfloat16()
        return out
    dy = state["dy"]
    f = factor(dy)
    da = (fit(rounded(dy, fmt, f), H) @ back(state["w2t"]).t()).bfloat16().float()
    g, u = state["u"][:, :F].float(), state["u"][:, F:].float()
    h, dh = act_plain(g, c["act"])
    du = torch.zeros(M, 2 * P, device=dy.device)
    du[:, :F], du[:, P:P + F] = da * u * dh, da * h
    dx = rounded(du, fmt, state["du"]["factor"][1]) @ back(state["w1t"]).t()
    dut = fit(rounded(du.t(), fmt, state["dut"]["factor"][1]), M)
    dw1 = dut @ back(state["xt"]).t()
    at = fit(rounded((h * u).t(), fmt, state["at"]["factor"][1]), M)
    dw2 = fit(rounded(dy.t(), fmt, f), M) @ at.t()
    return {"dx": dx.bfloat16(), "dwg": dw1[:F].bfloat16(), "dwu": dw1[P:P + F].bfloat16(), "dw2": dw2.bfloat16()}


def handles(state, c):
    """The framework's handles on the state's buffers, made once, as a program keeps them."""
    import tensor_transformer_layer_megatron_b200 as mgt
    rows = {"quantize": lambda: {"q": (c["rows"], c["cols"]), "qt": (c["cols"], c["rows"])},
            "linear": lambda: {"q": (c["M"], c["K"]), "w": (c["N"], c["K"])},
            "linear_bwd": lambda: {"q": (c["M"], c["N"]), "qt": (c["N"], c["M"]), "wt": (c["K"], c["N"]),
                                   "xt": (c["K"], c["M"])},
            "gated": lambda: {"q": (c["M"], c["H"]), "w1": (2 * up128(c["F"]), c["H"]),
                              "a": (c["M"], c["F"]), "w2": (c["H"], c["F"])},
            "gated_bwd": lambda: {"q": (c["M"], c["H"]), "qt": (c["H"], c["M"]), "w2t": (c["F"], c["H"]),
                                  "w1t": (c["H"], 2 * up128(c["F"])), "xt": (c["H"], c["M"]),
                                  "du": (c["M"], 2 * up128(c["F"])), "dut": (2 * up128(c["F"]), c["M"]),
                                  "at": (c["F"], c["M"])}}[c["op"]]()
    h = {k: mgt.Mx4(c["fmt"], *rc, codes=state[k]["codes"], scales=state[k]["tiles"], factor=state[k]["factor"])
         for k, rc in rows.items() if k in state}
    if "qt" in h:  # one factor for both layouts
        h["qt"] = mgt.Mx4(c["fmt"], *rows["qt"], codes=state["qt"]["codes"], scales=state["qt"]["tiles"],
                          factor=state["q"]["factor"])
    if c["op"] == "gated_bwd":
        h["dgt"], h["dupt"] = h["dut"].rows_view(0, c["F"]), h["dut"].rows_view(up128(c["F"]), c["F"])
    h["mgt"] = mgt
    return h


def run_own(s, c):
    h = s.get("handles") or s.setdefault("handles", handles(s, c))
    mgt, op, dynamic = h["mgt"], c["op"], c["fmt"] == "nvfp4"
    if op == "quantize":
        if dynamic:
            mgt.mx4_tensor_factor(s["x"], h["q"].factor)
        mgt.mx4_quantize(s["x"], h["q"], h.get("qt"))
        mgt.mx4_dequantize(h["q"], s["y"])
        if not c["both"]:
            return {"y": s["y"]}
        mgt.mx4_dequantize(h["qt"], s["yt"])
        return {"y": s["y"], "yt": s["yt"]}
    if op == "linear":
        mgt.mx4_quantize(s["x"], h["q"])
        mgt.gemm_mx4(h["q"], h["w"], s["y"], s["status"])
        return {"y": s["y"]}
    if op == "gated":
        mgt.mx4_quantize(s["x"], h["q"])
        mgt.gemm_mx4_gated(h["q"], h["w1"], h["a"], s["status"], act=c["act"], u=s["u"])
        mgt.gemm_mx4(h["a"], h["w2"], s["y"], s["status"])
        return {"y": s["y"], "u": s["u"]} if c["keep"] else {"y": s["y"]}
    if dynamic:
        mgt.mx4_tensor_factor(s["dy"], h["q"].factor)
    mgt.mx4_quantize(s["dy"], h["q"], h["qt"])
    if op == "linear_bwd":
        mgt.gemm_mx4(h["q"], h["wt"], s["dx"], s["status"])
        mgt.gemm_mx4(h["qt"], h["xt"], s["dw"], s["status"])
        return {"dx": s["dx"], "dw": s["dw"]}
    mgt.gemm_mx4(h["q"], h["w2t"], s["da"], s["status"])
    mgt.mx4_gated_bwd(s["da"], s["u"], h["du"], h["dut"], h["at"], act=c["act"])
    mgt.gemm_mx4(h["du"], h["w1t"], s["dx"], s["status"])
    mgt.gemm_mx4(h["dgt"], h["xt"], s["dwg"], s["status"])
    mgt.gemm_mx4(h["dupt"], h["xt"], s["dwu"], s["status"])
    mgt.gemm_mx4(h["qt"], h["at"], s["dw2"], s["status"])
    return {"dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"], "dw2": s["dw2"]}


# ------------------------------------------------------------------------- what a pass needs
def work(case):
    op = case["op"]
    four = lambda r, c: r * c * (0.5 + 1.0 / BLOCK[case["fmt"]])  # noqa: E731
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + (4 if case["both"] else 2)), "flops": 0}
    if op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":
            return {"bytes": 2 * M * K + four(N, K) + M * N * (2 if case["out"] == "bf16" else 4),
                    "flops": 2.0 * M * N * K}
        return {"bytes": 2 * M * N + four(K, N) + four(K, M) + 2 * M * K + 4 * N * K, "flops": 4.0 * M * N * K}
    M, H, F = case["M"], case["H"], case["F"]
    if op == "gated":
        return {"bytes": 2 * M * H + 3 * four(F, H) + 2 * M * H + (4 * M * F if case["keep"] else 0),
                "flops": 6.0 * M * H * F}
    return {"bytes": 2 * M * H + 4 * M * F + 3 * four(F, H) + four(H, M) + 2 * M * H + 6 * F * H,
            "flops": 12.0 * M * H * F}


# ------------------------------------------------------------------------- definition, 64 bits
def power_64(e):
    """2^e, exactly, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e2m1_64(v):
    """Nearest element: spacing 0.5 below 2, 1 below 4, 2 above; halves to the even multiple."""
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    return torch.sign(v) * torch.clamp(torch.round(m / step) * step, max=6)


def through_64(x, fmt, f):
    """x through 4 bits along its last axis, by the definition."""
    r, c = x.shape
    n = BLOCK[fmt]
    k = -(-c // n)
    z = torch.zeros(r, k * n, dtype=torch.float64, device=x.device)
    z[:, :c] = x.double()
    z = z.reshape(r, k, n)
    top = z.abs().max(2, keepdim=True).values
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        e = e + (power_64(e + 1) <= top).double() - (power_64(e) > top).double()
        s = power_64(torch.clamp(torch.where(top > 0, e - 2, -127.0), min=-127))
    else:
        t = torch.clamp(top / (6 * f), max=448.0)
        b = torch.clamp(torch.floor(torch.log2(torch.where(t > 0, t, 1.0))), min=-6)
        s = torch.clamp(torch.round(t / power_64(b - 3)) * power_64(b - 3), max=448.0) * f
    q = torch.where(s > 0, e2m1_64(z / torch.where(s > 0, s, 1.0)), 0.0)
    return (q * s).reshape(r, k * n)[:, :c]


def values_64(w, fmt, rows, cols):
    """What packed codes and scale tiles stand for, from the layout's definition."""
    code = w["codes"][:rows].long()
    table = torch.tensor([*GRID, *[-g for g in GRID]], dtype=torch.float64, device=code.device)
    v = torch.empty(rows, 2 * code.shape[1], dtype=torch.float64, device=code.device)
    v[:, 0::2], v[:, 1::2] = table[code % 16], table[code // 16]
    n = BLOCK[fmt]
    r = torch.arange(rows, device=code.device).view(-1, 1)
    b = torch.arange(v.shape[1] // n, device=code.device).view(1, -1)
    at = (r // 128 * (v.shape[1] // (4 * n)) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    byte = w["tiles"][at].long()
    if fmt == "mxfp4":
        s = power_64(byte - 127)
    else:
        e, m = byte // 8, (byte % 8).double()
        s = torch.where(e > 0, (8 + m) * power_64(e - 10), m * 2.0 ** -9) * w["factor"][1].double()
    return (v.view(rows, -1, n) * s.unsqueeze(2)).reshape(rows, -1)[:, :cols]


def act_64(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        c = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * c, c + z * torch.exp(-z * z / 2) * (1 / math.sqrt(2 * math.pi))
    y = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(2 * y)
    return z * s, s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s, fmt, op = prepare(case, seed), case["fmt"], case["op"]

    def dynamic(x):
        top = float(x.double().abs().max())
        if top == 0 or fmt == "mxfp4":
            return 1.0
        e = math.ceil(math.log2(top / 2688))
        e += (2688 * 2.0 ** e < top) - (2688 * 2.0 ** (e - 1) >= top)
        return 2.0 ** e

    kept = lambda k: float(s[k]["factor"][1])  # noqa: E731
    if op == "quantize":
        f = dynamic(s["x"])
        out = {"y": through_64(s["x"], fmt, f)}
        if case["both"]:
            out["yt"] = through_64(s["x"].t(), fmt, f)
        return out
    if op == "linear":
        w = values_64(s["w"], fmt, case["N"], case["K"])
        return {"y": through_64(s["x"], fmt, kept("q")) @ w.t()}
    f = dynamic(s["dy"]) if "dy" in s else None
    if op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        return {"dx": through_64(s["dy"], fmt, f) @ values_64(s["wt"], fmt, K, N).t(),
                "dw": through_64(s["dy"].t(), fmt, f) @ values_64(s["xt"], fmt, K, M).t()}
    M, H, F = case["M"], case["H"], case["F"]
    P = up128(F)
    if op == "gated":
        x = through_64(s["x"], fmt, kept("q"))
        w = values_64(s["w1"], fmt, 2 * P, H)
        g, u = x @ w[:F].t(), x @ w[P:P + F].t()
        a = through_64(act_64(g, case["act"])[0] * u, fmt, kept("a"))
        out = {"y": a @ values_64(s["w2"], fmt, H, F).t()}
        if case["keep"]:
            out["u"] = torch.cat([g, u], 1)
        return out
    da = (through_64(s["dy"], fmt, f) @ values_64(s["w2t"], fmt, F, H).t()).bfloat16().double()
    g, u = s["u"][:, :F].double(), s["u"][:, F:].double()
    h, dh = act_64(g, case["act"])
    dg, du = da * u * dh, da * h
    w1 = values_64(s["w1t"], fmt, H, 2 * P)
    x = values_64(s["xt"], fmt, H, M)
    fd, fa = kept("du"), kept("at")
    dx = through_64(dg, fmt, fd) @ w1[:, :F].t() + through_64(du, fmt, fd) @ w1[:, P:P + F].t()
    at = through_64((h * u).t(), fmt, fa)
    return {"dx": dx, "dwg": through_64(dg.t(), fmt, fd) @ x.t(), "dwu": through_64(du.t(), fmt, fd) @ x.t(),
            "dw2": through_64(s["dy"].t(), fmt, f) @ at.t()}
