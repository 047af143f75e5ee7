"""Cases of the gradient norm and clipping over a list of tensors, and of the
embedding's lookup and gradient: their plain forms in elementary torch
operations, the framework's calls, and the values the definitions give in 64
bits.

  norm   |in_mul * x| over all tensors of a model, and of each tensor
  clip   x * in_mul * min(1, max_norm / (norm + eps)), in place by a norm that
         all ranks have agreed on, or norm and clip into fp32
  embed  out[t] = mul * table[idx[t]]; an index outside the table gives zeros
  grad   the table's gradient: row v is mul times the sum of dy[t] over the
         tokens t with idx[t] = v, but for one skipped index
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
MAX_NORM = 1.0

# every tensor of the two networks of this repository's workloads, as count x
# elements; a range stands for lengths spread evenly over it
RESNET152 = ("1x9408,2x64,1x4096,3x36864,4x16384,6x64,6x64,8x256,2x16384,1x32768,2x128,"
             "8x147456,16x128,8x65536,16x512,1x131072,2x512,7x65536,14x128,1x131072,2x256,"
             "36x589824,72x256,36x262144,72x1024,1x524288,2x1024,35x262144,70x256,1x524288,2x512,"
             "3x2359296,6x512,3x1048576,6x2048,1x2097152,2x2048,2x1048576,4x512,1x2048000,1x1000")
BERT_LARGE = ("1x31254528,1x524288,1x2048,2x1024,96x1048576,96x1024,24x4194304,24x4096,"
              "24x4194304,24x1024,96x1024,1x1048576,1x1024")
VOCABULARY, WIDTH = 30522, 1024


def listed():
    return [
        # the smallest workload's tensor: latency
        {"name": "norm 2^20 f32", "op": "norm", "tensors": "1x1048576", "dt": "f32", "mul": 1.0,
         "each": False},
        # ten thousand small tensors, with the norm of each as for a log
        {"name": "norm 10000 small", "op": "norm", "tensors": "10000x1-4096", "dt": "f32",
         "mul": 0.125, "each": True},
        # BERT-Large's loss-scaled fp16 gradients
        {"name": "norm bert f16", "op": "norm", "tensors": BERT_LARGE, "dt": "f16",
         "mul": 2.0 ** -16, "each": False},
        # one tensor in place by a norm that is there: latency
        {"name": "clip 2^20 f32", "op": "clip", "tensors": "1x1048576", "dt": "f32", "mul": 1.0,
         "out": "", "ratio": 1.01},
        # ResNet-152 in place, by the norm that all ranks have agreed on
        {"name": "clip resnet152", "op": "clip", "tensors": RESNET152, "dt": "f32", "mul": 1.0,
         "out": "", "ratio": 1.01},
        # BERT-Large: norm, then unscaled and clipped into fp32
        {"name": "norm clip bert f16", "op": "clip", "tensors": BERT_LARGE, "dt": "f16",
         "mul": 2.0 ** -16, "out": "f32", "ratio": 0.0},
        # a single token: latency
        {"name": "embed 1 token", "op": "embed", "T": 1, "V": VOCABULARY, "D": WIDTH, "dt": "bf16",
         "out": "bf16", "mul": 1.0, "it": "i64", "gap": 0},
        # 8192 tokens from an fp32 table, scaled by sqrt(width)
        {"name": "embed 8192 tokens", "op": "embed", "T": 8192, "V": VOCABULARY, "D": WIDTH,
         "dt": "f32", "out": "bf16", "mul": 32.0, "it": "i64", "gap": 0},
        # the largest lookup: a wide table
        {"name": "embed 65536 tokens", "op": "embed", "T": 65536, "V": 65536, "D": 4096,
         "dt": "bf16", "out": "bf16", "mul": 1.0, "it": "i32", "gap": 0},
        # one 512-token sequence, added to the running fp32 gradient
        {"name": "grad 512 tokens", "op": "grad", "T": 512, "V": VOCABULARY, "D": WIDTH,
         "dt": "bf16", "out": "f32", "add": True, "mul": 1.0, "it": "i64", "gap": 0, "pad": 0.0,
         "skip": False},
        # a batch whose last quarter is the padding token 0, the whole gradient
        {"name": "grad 16384 padded", "op": "grad", "T": 16384, "V": VOCABULARY, "D": WIDTH,
         "dt": "f16", "out": "f32", "add": False, "mul": 2.0 ** -16, "it": "i64", "gap": 0,
         "pad": 0.25, "skip": True},
        # the largest gradient: odd vocabulary, frequent tokens thousands of times
        {"name": "grad 131072 tokens", "op": "grad", "T": 131072, "V": 100003, "D": 2048,
         "dt": "bf16", "out": "f32", "add": False, "mul": 1.0, "it": "i64", "gap": 0, "pad": 0.0,
         "skip": False},
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "clip", "embed", "grad"))
    types = ("f32", "f16", "bf16")
    if op in ("norm", "clip"):
        parts, left = [], 1 << 27
        for _ in range(rng.randint(1, 4)):
            hi = _size(rng, 1, 1 << 22)
            count = _size(rng, 1, min(5000, max(1, left // hi)))
            parts.append("%dx%d-%d" % (count, max(1, hi // rng.choice((1, 2, 1000))), hi))
            left = max(1, left - count * hi)
        case = {"op": op, "tensors": ",".join(parts), "dt": rng.choice(types + ("mixed",)),
                "mul": rng.choice((1.0, 0.125))}
        if op == "norm":
            return dict(case, each=rng.random() < 0.5)
        out = rng.choice(("", "f32", "bf16"))
        return dict(case, out=out, ratio=1.01 if not out or rng.random() < 0.5 else 0.0)
    D = _size(rng, 1, 8192)
    V = _size(rng, 1, min(1 << 18, (1 << 28) // D))
    T = _size(rng, 1, min(1 << 17, (1 << 28) // D))
    case = {"op": op, "T": T, "V": V, "D": D, "dt": rng.choice(types),
            "mul": rng.choice((1.0, 0.125, math.sqrt(D))), "it": rng.choice(("i32", "i64")),
            "gap": rng.choice((0, 0, 1, 8))}
    if op == "embed":
        return dict(case, out=rng.choice(types))
    out = rng.choice(types)
    return dict(case, out=out, add=out == "f32" and rng.random() < 0.5,
                pad=rng.choice((0.0, 0.0, 0.3)), skip=rng.random() < 0.5)


def _lengths(text):
    """The tensors' lengths."""
    found, spread = [], random.Random(1)
    for part in text.split(","):
        count, size = part.split("x")
        lo, _, hi = size.partition("-")
        lo = int(lo)
        found += [spread.randint(lo, int(hi or lo)) for _ in range(int(count))]
    return found


def _places(case):
    """(type, flat buffer, first element, length) of every tensor, and the
    buffers' types and lengths.  Of a mixed list the tensors of up to 4096
    elements (biases, norms) are fp32 and the others bf16."""
    dts = ("f32", "bf16") if case["dt"] == "mixed" else (case["dt"],)
    ends, places = [0] * len(dts), []
    for n in _lengths(case["tensors"]):
        b = 1 if len(dts) > 1 and n > 4096 else 0
        places.append((dts[b], b, ends[b], n))
        ends[b] += n
    return places, list(zip(dts, ends))


def _tokens(case, gen, device):
    """T token ids, the r-th most frequent one about 1/r as often as the
    first; the padding at the end is token 0 where that is skipped, else -1."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, generator=gen, device=device, dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)).long() - 1).clamp_(0, V - 1)
    idx = torch.randperm(V, generator=gen, device=device)[rank]
    pad = int(T * case.get("pad", 0.0))
    if pad:
        idx[T - pad:] = 0 if case["skip"] else -1
    return idx.to(torch.int32 if case["it"] == "i32" else torch.int64)


def _matrix(rows, cols, gap, dt, gen, device, mul=1.0):
    """Normal values in rows that lie `gap` elements apart."""
    x = torch.randn(rows, cols + gap, generator=gen, device=device)
    return x.mul_(mul).to(DTYPES[dt])[:, :cols]


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(seed)
    s = dict(case)
    if case["op"] in ("norm", "clip"):
        s["places"], buffers = _places(case)
        s["x"] = []
        for dt, n in buffers:
            # the size changes every 4096 elements by up to e^4, as between layers
            x = torch.randn(n, generator=gen, device=device)
            sigma = torch.rand(-(-n // 4096), generator=gen, device=device) * 4 - 9
            x *= sigma.exp_().div_(case["mul"]).repeat_interleave(4096)[:n]
            s["x"].append(x.to(DTYPES[dt]))
        s["norm"] = torch.empty(1, device=device)
        if case["op"] == "norm" and case["each"]:
            s["each_norm"] = torch.empty(len(s["places"]), device=device)
            # each buffer's tensors: their last elements and their numbers
            s["last"] = [torch.tensor([at + n - 1 for _, k, at, n in s["places"] if k == b],
                                      dtype=torch.int64, device=device) for b in range(len(buffers))]
            s["which"] = [torch.tensor([i for i, p in enumerate(s["places"]) if p[1] == b],
                                       dtype=torch.int64, device=device)
                          for b in range(len(buffers))]
        if case["op"] == "clip":
            if case["ratio"]:
                s["norm"].fill_(MAX_NORM * case["ratio"])
            if case["out"]:
                s["y"] = [torch.empty(n, dtype=DTYPES[case["out"]], device=device)
                          for _, n in buffers]
        if own:
            from gradient_compression_allreduce_amd import gq
            s["list"] = gq.gq_tensors_create([s["x"][b][at:at + n] for _, b, at, n in s["places"]])
            if case.get("out"):
                s["out_list"] = gq.gq_tensors_create([s["y"][b][at:at + n]
                                                      for _, b, at, n in s["places"]])
        return s
    T, V, D = case["T"], case["V"], case["D"]
    s["idx"] = _tokens(case, gen, device)
    if case["op"] == "embed":
        s["table"] = _matrix(V, D, case["gap"], case["dt"], gen, device, 0.02)
        s["o"] = torch.empty(T, D, dtype=DTYPES[case["out"]], device=device)
        return s
    s["dy"] = _matrix(T, D, case["gap"], case["dt"], gen, device, 1e-3 / case["mul"])
    s["o"] = torch.empty(V, D, dtype=DTYPES[case["out"]], device=device)
    if case["add"]:
        s["o"].normal_(0, 1e-3, generator=gen)
    if own:
        from gradient_compression_allreduce_amd import gq
        s["ws"] = torch.empty(gq.gq_embed_grad_workspace(T, V, D), dtype=torch.uint8,
                              device=device)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from gradient_compression_allreduce_amd import gq
    op = s["op"]
    if op == "norm":
        gq.gq_tensors_norm(s["list"], s["norm"], norms=s.get("each_norm"), in_mul=s["mul"])
        return [s["norm"]] + ([s["each_norm"]] if s["each"] else [])
    if op == "clip":
        if not s["ratio"]:
            gq.gq_tensors_norm(s["list"], s["norm"], in_mul=s["mul"])
        gq.gq_tensors_clip(s["list"], s["norm"], MAX_NORM, eps=EPS, in_mul=s["mul"],
                           out=s.get("out_list"))
        return [s["norm"]] + (s["y"] if s["out"] else s["x"])
    if op == "embed":
        gq.gq_embed(s["idx"], s["table"], s["o"], mul=s["mul"])
        return s["o"]
    gq.gq_embed_grad(s["idx"], s["dy"], s["o"], mul=s["mul"], skip=0 if s["skip"] else None,
                     accumulate=s["add"], workspace=s["ws"])
    return s["o"]


# ---- plain forms -----------------------------------------------------------

def _squares(x):
    """A buffer's sum of squares; in 64 bits, as long sums are."""
    return x.float().double().square_().sum()


def _run_plain(s):
    op = s["op"]
    if op in ("norm", "clip"):
        if op == "norm" or not s["ratio"]:
            s["norm"].copy_(torch.stack([_squares(x) for x in s["x"]]).sum().sqrt() * s["mul"])
        if op == "norm":
            if not s["each"]:
                return [s["norm"]]
            out = s["each_norm"]
            for x, last, which in zip(s["x"], s["last"], s["which"]):
                if x.numel():
                    total = x.float().double().square_().cumsum(0)[last]
                    total = torch.diff(total, prepend=torch.zeros_like(total[:1]))
                    out[which] = (total.clamp(min=0).sqrt() * s["mul"]).float()
            return [s["norm"], out]
        top = s["norm"].double() + EPS
        f = torch.where(top <= MAX_NORM, torch.ones_like(top), MAX_NORM / top) * s["mul"]
        f = f.float()
        for x, y in zip(s["x"], s["y"] if s["out"] else s["x"]):
            y.copy_(x.float() * f)
        return [s["norm"]] + (s["y"] if s["out"] else s["x"])
    V, idx = s["V"], s["idx"].long()
    inside = (idx >= 0) & (idx < V)
    if op == "embed":
        rows = s["table"][idx.clamp(0, V - 1)].float() * s["mul"]
        s["o"].copy_(torch.where(inside[:, None], rows, torch.zeros((), device=rows.device)))
        return s["o"]
    if s["skip"]:
        inside &= idx != 0
    g = torch.zeros(V + 1, s["D"], device=idx.device)      # the last row: what is left out
    g.index_add_(0, torch.where(inside, idx, torch.full_like(idx, V)), s["dy"].float())
    g = g[:V] * s["mul"]
    return s["o"].add_(g) if s["add"] else s["o"].copy_(g)


# ---- the definitions in 64 bits --------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        if case.get("ratio"):
            norm = s["norm"].double()
        else:
            each = torch.stack([torch.linalg.vector_norm(s["x"][b][at:at + n].double())
                                for _, b, at, n in s["places"]])
            norm = torch.linalg.vector_norm(each).view(1) * case["mul"]
        if op == "norm":
            return [norm] + ([each * case["mul"]] if case["each"] else [])
        f = case["mul"] * min(1.0, MAX_NORM / (float(norm) + EPS))
        return [norm] + [x.double() * f for x in s["x"]]
    V, D, idx = case["V"], case["D"], s["idx"].long()
    if op == "embed":
        o = torch.zeros(case["T"], D, dtype=torch.float64, device=idx.device)
        at = torch.nonzero((idx >= 0) & (idx < V)).view(-1)
        o[at] = torch.index_select(s["table"], 0, idx[at]).double() * case["mul"]
        return o
    # running sums over the tokens in the order of their ids, and what they
    # grow by over each id's run
    order = torch.argsort(idx, stable=True)
    key = idx[order].contiguous()
    lo = torch.searchsorted(key, torch.arange(V, device=idx.device))
    hi = torch.searchsorted(key, torch.arange(V, device=idx.device), right=True)
    if case["skip"]:
        hi[0] = lo[0]
    o = s["o"].double() if case["add"] else torch.zeros(V, D, dtype=torch.float64,
                                                        device=idx.device)
    for c in range(0, D, 512):
        part = s["dy"][:, c:c + 512]
        total = torch.zeros(case["T"] + 1, part.shape[1], dtype=torch.float64, device=idx.device)
        torch.cumsum(part[order].double(), 0, out=total[1:])
        o[:, c:c + 512] += (total[hi] - total[lo]) * case["mul"]
    return o


def _rows_met(case):
    """How many different rows the tokens name, on average."""
    T, V = case["T"] - int(case["T"] * case.get("pad", 0.0)), case["V"]
    r = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log1p(1 / r) / math.log(V + 1)
    return float((1 - (1 - p).clamp(min=0) ** T).sum())


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        places, buffers = _places(case)
        n = sum(m for _, m in buffers)
        read = sum(m * SIZE[dt] for dt, m in buffers)
        if op == "norm":
            return {"bytes": read + 4 + 4 * len(places) * case["each"], "flops": 2 * n}
        again = read if not case["ratio"] else 0
        wrote = n * SIZE[case["out"]] if case["out"] else read
        return {"bytes": read + again + wrote, "flops": n + (2 * n if again else 0)}
    T, D = case["T"], case["D"]
    ids = T * (4 if case["it"] == "i32" else 8)
    if op == "embed":
        return {"bytes": ids + D * (_rows_met(case) * SIZE[case["dt"]] + T * SIZE[case["out"]]),
                "flops": T * D}
    live = T - int(T * case["pad"])
    rows = 2 * _rows_met(case) if case["add"] else case["V"]
    return {"bytes": ids + D * (live * SIZE[case["dt"]] + rows * SIZE[case["out"]]),
            "flops": live * D}
