"""Cases of the microscaled 4-bit gradient operators and of the
orthogonalised update: their plain forms in elementary torch operations, the
framework's calls, and the values the definitions give in 64 bits.

Microscaled 4-bit (MX4): blocks of 32 consecutive elements share a power of
two, 2^(floor(log2(max|g|)) - 2), and each element is one of 0, 0.5, 1, 1.5,
2, 3, 4, 6 with a sign, rounded half to even, above 6 to 6.

  quantize  one gradient or activation to MX4 (blocks along a row, or down a
            column of a matrix), and what the codes stand for
  exchange  W ranks' gradients to MX4, their sum in rank order, and the sum
            quantized again: the compute of a 4-bit AllReduce
  reduce    the same from codes that have already arrived
  product   C = A B^T of two MX4 matrices, into a new or a running C
  ortho     momentum, then the quintic Newton-Schulz iteration, for every
            matrix of a model
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5

# count x rows x cols of the weight matrices of the two networks of this
# repository's workloads (convolutions as [out, in * height * width])
RESNET152 = ("1x64x147,1x64x64,3x64x576,4x256x64,2x64x256,1x128x256,8x128x1152,8x512x128,"
             "1x512x256,7x128x512,1x256x512,36x256x2304,36x1024x256,1x1024x512,35x256x1024,"
             "1x512x1024,3x512x4608,3x2048x512,1x2048x1024,2x512x2048,1x1000x2048")
BERT_LARGE = "97x1024x1024,24x4096x1024,24x1024x4096"


def listed():
    return [
        # the smallest workload's tensor (2^20 fp32) to 4 bits: latency
        {"name": "quantize 2^20 f32", "op": "quantize", "dt": "f32", "rows": 1, "cols": 1 << 20,
         "transpose": False, "mul": 1.0},
        # activations of 8192 tokens for a weight gradient: blocks run along
        # the tokens, so the matrix is quantized down its columns
        {"name": "quantize tokens bf16", "op": "quantize", "dt": "bf16", "rows": 8192,
         "cols": 4096, "transpose": True, "mul": 1.0},
        # ResNet-152's gradients on 8 ranks
        {"name": "exchange resnet152", "op": "exchange", "dt": "f32", "W": 8, "n": 60192808,
         "mul": 1.0},
        # BERT-Large's loss-scaled fp16 gradients on 8 ranks
        {"name": "exchange bert f16", "op": "exchange", "dt": "f16", "W": 8, "n": 335141888,
         "mul": 2.0 ** -16},
        # one tensor of 2^20 from 4 ranks: latency
        {"name": "reduce 2^20", "op": "reduce", "W": 4, "n": 1 << 20},
        # one 512-token sequence's weight gradient of a 1024 x 1024 matrix,
        # added to the running fp32 gradient
        {"name": "product 512 tokens", "op": "product", "m": 1024, "n": 1024, "k": 512,
         "out": "f32", "add": True},
        # a feed-forward matrix's weight gradient over 16384 tokens, fp32
        {"name": "product ffn", "op": "product", "m": 4096, "n": 1024, "k": 16384, "out": "f32",
         "add": False},
        # the largest product
        {"name": "product 8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "add": False},
        # a few rows against a vocabulary's matrix: bound by reading it
        {"name": "product 7 rows", "op": "product", "m": 7, "n": 30522, "k": 1024, "out": "bf16",
         "add": False},
        # ResNet-152's first convolution alone: latency
        {"name": "ortho conv1", "op": "ortho", "shapes": "1x64x147", "dt": "f32", "out": "bf16",
         "mul": 1.0, "momentum": True, "nesterov": True},
        # every matrix of ResNet-152: many small and odd ones in one call
        {"name": "ortho resnet152", "op": "ortho", "shapes": RESNET152, "dt": "f32",
         "out": "bf16", "mul": 1.0, "momentum": True, "nesterov": True},
        # every matrix of BERT-Large's layers and pooler, loss-scaled fp16
        {"name": "ortho bert f16", "op": "ortho", "shapes": BERT_LARGE, "dt": "f16", "out": "f16",
         "mul": 2.0 ** -16, "momentum": True, "nesterov": False},
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("quantize", "exchange", "reduce", "product", "ortho"))
    if op == "quantize":
        rows = _size(rng, 1, 8192)
        return {"op": op, "dt": rng.choice(("f32", "f16", "bf16")), "rows": rows,
                "cols": _size(rng, 1, (1 << 25) // rows), "transpose": rng.random() < 0.5,
                "mul": rng.choice((1.0, 2.0 ** -16, 0.125))}
    if op == "exchange":
        return {"op": op, "dt": rng.choice(("f32", "f16", "bf16")), "W": rng.choice((1, 2, 3, 4, 8)),
                "n": _size(rng, 1, 1 << 26), "mul": rng.choice((1.0, 2.0 ** -16))}
    if op == "reduce":
        return {"op": op, "W": rng.choice((1, 2, 4, 5, 8, 16)), "n": _size(rng, 1, 1 << 27)}
    if op == "product":
        out = rng.choice(("f32", "f16", "bf16"))
        return {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 1, 8192),
                "k": _size(rng, 1, 8192), "out": out,
                "add": out == "f32" and rng.random() < 0.5}
    shapes = ",".join("%dx%dx%d" % (rng.randint(1, 6), _size(rng, 1, 2048), _size(rng, 1, 2048))
                      for _ in range(rng.randint(1, 3)))
    return {"op": op, "shapes": shapes, "dt": rng.choice(("f32", "f16", "bf16")),
            "out": rng.choice(("f16", "bf16")), "mul": 1.0, "momentum": rng.random() < 0.5,
            "nesterov": rng.random() < 0.5}


def _groups(text):
    """(first element, count, rows, cols) of each group of like matrices."""
    at, found = 0, []
    for part in text.split(","):
        count, rows, cols = (int(v) for v in part.split("x"))
        found.append((at, count, rows, cols))
        at += count * rows * cols
    return found


def _blocks(cols):
    return -(-cols // BLOCK)


def _gradient(n, dt, mul, gen, device):
    """n elements whose size changes every 4096 elements by up to e^4, as
    between the layers of a network, scaled for `mul`."""
    x = torch.randn(n, generator=gen, device=device)
    sigma = torch.exp(torch.rand(-(-n // 4096), generator=gen, device=device) * 4 - 9) / mul
    x *= sigma.repeat_interleave(4096)[:n]
    return x.to(dt)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(seed)
    s = dict(case)

    def bytes_(n):
        return torch.empty(n, dtype=torch.uint8, device=device)

    def codes_of(rows, cols):
        x = torch.randn(rows, cols, generator=gen, device=device)
        x *= torch.exp(torch.randn(rows, 1, generator=gen, device=device))
        return _quantize(x)

    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        s["x"] = _gradient(r * c, DTYPES[case["dt"]], case["mul"], gen, device).view(r, c)
        qr, qc = (c, r) if case["transpose"] else (r, c)
        s["q"], s["scale"] = bytes_(qr * _blocks(qc) * 16), bytes_(qr * _blocks(qc))
        s["r"] = torch.empty(qr, qc, device=device)
    elif op == "exchange":
        n, W, nb = case["n"], case["W"], _blocks(case["n"])
        s["x"] = [_gradient(n, DTYPES[case["dt"]], case["mul"], gen, device) for _ in range(W)]
        s["q"], s["scale"] = [bytes_(nb * 16) for _ in range(W)], [bytes_(nb) for _ in range(W)]
    elif op == "reduce":
        got = [_quantize(_gradient(case["n"], torch.float32, 1.0, gen, device).view(1, -1))
               for _ in range(case["W"])]
        s["q"], s["scale"] = [g[0] for g in got], [g[1] for g in got]
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = codes_of(m, k)
        s["b"], s["sb"] = codes_of(n, k)
        s["c"] = torch.randn(m, n, generator=gen, device=device).to(DTYPES[case["out"]])
        if own:
            from gradient_compression_allreduce_amd import gq
            s["ws"] = bytes_(max(1, gq.gq_mx4_product_workspace(m, n, k)))
    else:
        parts = []
        for _, count, r, c in _groups(case["shapes"]):
            # a few strong directions above noise of the same energy
            p = min(16, r, c)
            u = torch.randn(count, r, p, generator=gen, device=device)
            v = torch.randn(count, p, c, generator=gen, device=device)
            noise = torch.randn(count, r, c, generator=gen, device=device)
            parts.append((1e-3 / case["mul"] * (torch.bmm(u, v) / math.sqrt(p) + noise)).reshape(-1))
        g = torch.cat(parts)
        s["g"] = g.to(DTYPES[case["dt"]])
        n = g.numel()
        if case["momentum"]:
            s["m"] = torch.randn(n, generator=gen, device=device) * 1e-3
        s["o"] = torch.empty(n, dtype=DTYPES[case["out"]], device=device)
        if own:
            from gradient_compression_allreduce_amd import gq
            s["plan"] = gq.gq_ortho_create([(r, c) for _, count, r, c in _groups(case["shapes"])
                                            for _ in range(count)])
    if op in ("exchange", "reduce"):
        nb = _blocks(case["n"])
        s["qo"], s["so"] = bytes_(nb * 16), bytes_(nb)
        s["r"] = torch.empty(case["n"], device=device)
        s["v"] = torch.empty(case["n"], device=device)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from gradient_compression_allreduce_amd import gq
    op = s["op"]
    if op == "quantize":
        rows, cols = s["r"].shape
        gq.gq_mx4_quantize([s["x"]], [s["scale"]], [s["q"]], in_mul=s["mul"],
                           transpose=s["transpose"])
        gq.gq_mx4_reduce_dequant([s["q"]], [s["scale"]], rows, cols, s["r"])
        return s["r"]
    if op in ("exchange", "reduce"):
        n = s["n"]
        if op == "exchange":
            gq.gq_mx4_quantize(s["x"], s["scale"], s["q"], in_mul=s["mul"])
        gq.gq_mx4_reduce_requantize(s["q"], s["scale"], 1, n, s["so"], s["qo"], r_out=s["r"])
        gq.gq_mx4_reduce_dequant([s["qo"]], [s["so"]], 1, n, s["v"])
        return [s["r"], s["v"]]
    if op == "product":
        gq.gq_mx4_product(s["a"], s["sa"], s["b"], s["sb"], s["k"], s["c"], accumulate=s["add"],
                          workspace=s["ws"])
        return s["c"]
    gq.gq_ortho_step(s["plan"], s["g"], s["o"], in_mul=s["mul"], momentum=s.get("m"),
                     mu=0.95, nesterov=s["nesterov"])
    return [s["o"]] + ([s["m"]] if s["momentum"] else [])


# ---- plain forms -----------------------------------------------------------

def _quantize(x):
    """Packed codes and scale bytes of a matrix in 32 bits, blocks along the
    rows."""
    rows, cols = x.shape
    nb = _blocks(cols)
    if nb * BLOCK != cols:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - cols))
    x = x.reshape(rows * nb, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)      # floor(log2) - 2
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(x, -e)
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= torch.signbit(y).to(torch.uint8) << 3
    return (code[:, 0::2] | code[:, 1::2] << 4).reshape(-1), (e + 127).to(torch.uint8).reshape(-1)


def _values(q, scale, rows, cols):
    """What the codes stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         device=q.device)
    q = q.view(-1, 16)
    code = torch.stack((q & 15, q >> 4), 2).view(-1, BLOCK)
    two = torch.ldexp(torch.ones((), device=q.device), scale.int() - 127)
    v = table[code.int()] * two.view(-1, 1)
    return v.view(rows, -1)[:, :cols]


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].float() * s["mul"]
        if s["transpose"]:
            x = x.T.contiguous()
        q, scale = _quantize(x)
        return _values(q, scale, *x.shape).contiguous()
    if op in ("exchange", "reduce"):
        n = s["n"]
        r = torch.zeros(1, n, device=s["r"].device)
        for w in range(s["W"]):      # ranks add in order
            if op == "exchange":
                q, scale = _quantize((s["x"][w].float() * s["mul"]).view(1, n))
            else:
                q, scale = s["q"][w], s["scale"][w]
            r += _values(q, scale, 1, n)
        q, scale = _quantize(r)
        return [r.view(-1), _values(q, scale, 1, n).reshape(-1)]
    if op == "product":
        m, n = s["c"].shape
        p = _values(s["a"], s["sa"], m, s["k"]) @ _values(s["b"], s["sb"], n, s["k"]).T
        if s["add"]:
            return s["c"].add_(p)
        return s["c"].copy_(p)
    u = s["g"].float() * s["mul"]
    if s["momentum"]:
        m = s["m"].mul_(0.95).add_(u)
        u = u + 0.95 * m if s["nesterov"] else m
    a, b, c = COEF
    for at, count, rows, cols in _groups(s["shapes"]):
        x = u[at:at + count * rows * cols].view(count, rows, cols)
        if rows > cols:
            x = x.transpose(1, 2).contiguous()
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
        for _ in range(STEPS):
            g = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
        if rows > cols:
            x = x.transpose(1, 2)
        s["o"][at:at + count * rows * cols].view(count, rows, cols).copy_(x)
    return [s["o"]] + ([s["m"]] if s["momentum"] else [])


# ---- the definitions in 64 bits --------------------------------------------

def _nearest(x):
    """The MX4 values nearest to a matrix in 64 bits: round to multiples of
    the step that each magnitude's binade has."""
    rows, cols = x.shape
    y = torch.zeros(rows, _blocks(cols) * BLOCK, dtype=torch.float64, device=x.device)
    y[:, :cols] = x
    y = y.view(-1, BLOCK)
    top = y.abs().max(1, keepdim=True).values
    e = (torch.floor(torch.log2(top)) - 2).clamp(min=-127)
    two = torch.exp2(torch.where(torch.isfinite(e), e, torch.full_like(e, -127)))
    y = y / two
    step = torch.ones_like(y)
    step[y.abs() < 2] = 0.5
    step[y.abs() >= 4] = 2.0
    y = (torch.round(y / step) * step).clamp(-6, 6) * two
    return y.view(rows, -1)[:, :cols]


def _decode64(q, scale, rows, cols):
    q = q.view(-1, 16)
    code = torch.cat((q[..., None] & 15, q[..., None] >> 4), 2).view(-1, BLOCK)
    mant, expo, sign = (code & 1).double(), (code >> 1 & 3).double(), (code >> 3).double()
    v = torch.where(expo > 0, (1 + mant / 2) * torch.exp2(expo - 1), mant / 2) * (1 - 2 * sign)
    v = v * torch.exp2(scale.view(-1, 1).double() - 127)
    return v.view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double() * case["mul"]
        return _nearest(x.t() if case["transpose"] else x)
    if op in ("exchange", "reduce"):
        n = case["n"]
        r = torch.zeros(1, n, dtype=torch.float64, device=s["r"].device)
        for w in range(case["W"]):
            r += (_nearest(s["x"][w].double().mul_(case["mul"]).view(1, n)) if op == "exchange"
                  else _decode64(s["q"][w], s["scale"][w], 1, n))
        return [r.view(-1), _nearest(r).reshape(-1)]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        p = torch.mm(_decode64(s["a"], s["sa"], m, k), _decode64(s["b"], s["sb"], n, k).t())
        return p + s["c"].double() if case["add"] else p
    g = s["g"].double() * case["mul"]
    if case["momentum"]:
        m = 0.95 * s["m"].double() + g
        g = g + 0.95 * m if case["nesterov"] else m
    o = torch.empty_like(g)
    a, b, c = COEF
    for at, count, rows, cols in _groups(case["shapes"]):
        for i in range(at, at + count * rows * cols, rows * cols):
            x = g[i:i + rows * cols].view(rows, cols)
            x = x / (torch.linalg.norm(x) + 1e-7)
            eye = torch.eye(min(rows, cols), dtype=torch.float64, device=x.device)
            for _ in range(STEPS):
                if rows > cols:
                    w = x.t() @ x
                    x = x @ (a * eye + w @ (b * eye + c * w))
                else:
                    w = x @ x.t()
                    x = (a * eye + w @ (b * eye + c * w)) @ x
            o[i:i + rows * cols] = x.reshape(-1)
    return [o] + ([m] if case["momentum"] else [])


def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        nb = cols * _blocks(rows) if case["transpose"] else rows * _blocks(cols)
        # the input read, codes and scales written and read, the values written
        return {"bytes": rows * cols * (size[case["dt"]] + 4) + 2 * 17 * nb, "flops": 0}
    if op in ("exchange", "reduce"):
        n, W, nb = case["n"], case["W"], _blocks(case["n"])
        read = W * (n * size[case["dt"]] + 2 * 17 * nb) if op == "exchange" else W * 17 * nb
        return {"bytes": read + 8 * n + 2 * 17 * nb, "flops": 0}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 17 * _blocks(k) * (m + n) + m * n * size[case["out"]] * (1 + case["add"]),
                "flops": 2 * m * n * k}
    by = flops = 0
    for _, count, rows, cols in _groups(case["shapes"]):
        s, l = min(rows, cols), max(rows, cols)
        by += count * s * l * (size[case["dt"]] + 2 + 8 * case["momentum"])
        # per step: half of each symmetric product, and the whole third one
        flops += count * STEPS * (3 * s * s * l + s * s * s)
    return {"bytes": by, "flops": flops}
