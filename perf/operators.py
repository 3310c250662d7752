"""Measured cases of the grouped products, the microscaled 4-bit format and
the gradient clipping: their inputs, their plain forms, the calls a program
makes of the library, and the same results from the definitions in 64 bits.

Operators
  mx_roundtrip   bf16 -> MXFP4 (E2M1 codes, one power-of-two scale per 32
                 columns) -> bf16
  mx_mm          y[p] = w[e(p)] x[p] for rows sorted by expert, x and w MXFP4
  mm             the same product with x and w in bf16
  mm_backward    its gradients with respect to x (bf16) and w (fp32 or bf16)
  clip           the norm over many gradients, and the gradients scaled by
                 min(1, max_norm / norm)

Shapes are those of the library's synthetic layers (E experts, hidden size H,
expert size I, top-k routing) or general ones.
"""

import math

import torch

own = False   # True: run() calls the library; False: the plain forms

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step's activations (16 tokens, top-4, H = 2880): latency
        dict(name="mx_roundtrip rows 64", op="mx_roundtrip", E=1, R=64, C=2880),
        # quantize-on-load of a layer's gate_up [32, 2 * 2880, 2880]: bandwidth
        dict(name="mx_roundtrip layer", op="mx_roundtrip", E=32, R=5760, C=2880),
        # decode, 16 tokens top-4 over 32 experts: two rows an expert, weight streaming
        dict(name="mx_mm decode M64", op="mx_mm", E=32, M=64, N=5760, K=2880, skew="uniform"),
        # prompt of 2048 tokens, top-4: 256 ragged rows an expert, K no multiple of a step
        dict(name="mx_mm prompt M8192", op="mx_mm", E=32, M=8192, N=5760, K=2880, skew="uniform"),
        # 16384 tokens top-2 of a large layer's gate_up: matrix rate
        dict(name="mx_mm prompt M32768", op="mx_mm", E=8, M=32768, N=28672, K=4096, skew="uniform"),
        # one token, top-8 of 64 experts: eight rows in all
        dict(name="mm decode M8", op="mm", E=64, M=8, N=2048, K=2048, skew="uniform"),
        # 512 tokens, top-2, down projection: long contraction
        dict(name="mm prompt M1024", op="mm", E=8, M=1024, N=4096, K=14336, skew="uniform"),
        # 8192 tokens, top-8 of 128 experts, popular experts first: very ragged
        dict(name="mm prompt M65536 zipf", op="mm", E=128, M=65536, N=1536, K=2048, skew="zipf"),
        # training step, 4096 tokens top-8, trainable experts
        dict(name="mm_backward M32768", op="mm_backward", E=64, M=32768, N=2048, K=2048, skew="uniform", dw="fp32"),
        # training step of rank-16 adapters on the experts
        dict(name="mm_backward rank 16", op="mm_backward", E=128, M=8192, N=16, K=2048, skew="zipf", dw="bf16"),
        # gradients of routers and adapters of 16 layers: many small tensors
        dict(name="clip adapters", op="clip", count=96, small=131072, large=1 << 21, mix="both", max_norm=1.0),
        # gradients of trainable experts of one layer: few large tensors
        dict(name="clip experts", op="clip", count=3, small=1 << 26, large=1 << 28, mix="fp32", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mx_roundtrip", "mx_mm", "mm", "mm_backward", "clip"])
    if op == "mx_roundtrip":
        return dict(op=op, E=rng.randint(1, 32), R=_log(rng, 1, 6000), C=32 * _log(rng, 1, 90))
    if op == "clip":
        small = _log(rng, 1, 1 << 16)
        return dict(op=op, count=_log(rng, 1, 300), small=small, large=small + _log(rng, 1, 1 << 20),
                    mix=rng.choice(["fp32", "bf16", "both"]), max_norm=rng.choice([0.5, 1.0, 1e9]))
    step = 32 if op == "mx_mm" else 8
    case = dict(op=op, E=_log(rng, 1, 128), M=_log(rng, 1, 20000), N=8 * _log(rng, 1, 512),
                K=step * _log(rng, 1, 4096 // step), skew=rng.choice(["uniform", "zipf"]))
    if op == "mm_backward":
        case["dw"] = rng.choice(["fp32", "bf16"])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, shape, std):
    """bf16 N(0, std), drawn in slices of the first dimension."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for s in t.split(max(1, (1 << 27) // max(1, t[0].numel()))):
        s.copy_(torch.randn(s.shape, generator=gen, device=DEV) * std)
    return t


def _sizes(case, seed):
    """Rows per expert: every row picks an expert, evenly or by Zipf's law."""
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    p = torch.ones(case["E"], dtype=torch.float64)
    if case["skew"] == "zipf":
        p /= torch.arange(1, case["E"] + 1, dtype=torch.float64) ** 1.1
    pick = torch.multinomial(p, case["M"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["E"])


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _blocks(w):
    return w.float().reshape(*w.shape[:-1], w.shape[-1] // 32, 32)


def _mx_scale_exponent(b):
    """floor(log2(largest magnitude)) - 2 of each block, at least -127."""
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    return (e - 3).clamp(min=-127)


def _mx_level_index(v):
    """Index of the E2M1 magnitude nearest to v >= 0, ties to the even index."""
    return ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))


def _mx_pack(w):
    """bf16 [..., C] -> (uint8 [..., C/2] codes, the even column in the low
    nibble; uint8 [..., C/32] scale exponents, biased by 127)."""
    b = _blocks(w)
    e = _mx_scale_exponent(b)
    code = _mx_level_index(torch.ldexp(b.abs(), -e)) | (b < 0).to(torch.uint8) * 8
    code = code.reshape(*w.shape[:-1], w.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _mx_pack_all(w):
    parts = [_mx_pack(s) for s in w.split(1)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _qweight(codes, scales):
    import bit_weight_quantization_moeq_amd as moeq
    E, R, C = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    return moeq.QWeight(moeq.FMT_MXFP4, E, R, C, codes, None, scales)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 5)
    op = case["op"]
    s = dict(case=case)
    if op == "mx_roundtrip":
        s["w"] = _randn(gen, (case["E"], case["R"], case["C"]), 0.02)
        return s
    if op == "clip":
        # lengths belong to the model, not to the step: they go by the case
        g = torch.Generator().manual_seed(case["count"] * 7919 + case["small"])
        lens = torch.randint(case["small"], case["large"] + 1, (case["count"],), generator=g).tolist()
        kind = {"fp32": [torch.float32], "bf16": [torch.bfloat16], "both": [torch.bfloat16, torch.float32]}[case["mix"]]
        s["grads"] = [(torch.randn(n, generator=gen, device=DEV) * 0.01).to(kind[i % len(kind)])
                      for i, n in enumerate(lens)]
        # the clipped gradients go to one flat buffer a type, each at a multiple of 8 elements
        s["flat"], s["out"] = [], [None] * len(lens)
        for dt in kind:
            at, spans = 0, []
            for i, t in enumerate(s["grads"]):
                if t.dtype == dt:
                    spans.append((i, at, at + t.numel()))
                    at += -(-t.numel() // 8) * 8
            if spans:
                flat = torch.zeros(at, dtype=dt, device=DEV)
                s["flat"].append(flat)
                for i, lo, hi in spans:
                    s["out"][i] = flat[lo:hi]
        return s
    E, M, N, K = (case[k] for k in "EMNK")
    sizes = _sizes(case, seed)
    s["sizes"] = sizes.tolist()
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).to(DEV)
    x, w = _randn(gen, (M, K), 1.0), _randn(gen, (E, N, K), 0.02)
    if op == "mx_mm":
        s["x"], s["w"] = _mx_pack(x[None]), _mx_pack_all(w)
        if own:
            s["xq"], s["wq"] = _qweight(*s["x"]), _qweight(*s["w"])
        return s
    s["x"], s["w"] = x, w
    if op == "mm_backward":
        s["dy"] = _randn(gen, (M, N), 1.0)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bit_weight_quantization_moeq_amd as moeq
    case = s["case"]
    op = case["op"]
    if op == "mx_roundtrip":
        return moeq.moeq_dequantize(moeq.moeq_quantize_mxfp4(s["w"]))
    if op == "mx_mm":
        return moeq.moeq_grouped_mm_mxfp4(s["xq"], s["wq"], s["offsets"])
    if op == "mm":
        return moeq.moeq_grouped_mm(s["x"], s["w"], s["offsets"])
    if op == "mm_backward":
        dt = torch.float32 if case["dw"] == "fp32" else torch.bfloat16
        return (moeq.moeq_grouped_mm_grad_input(s["dy"], s["w"], s["offsets"]),
                moeq.moeq_grouped_mm_grad_weight(s["dy"], s["x"], s["offsets"], dtype=dt))
    norm = moeq.moeq_clip_grad_norm(s["grads"], case["max_norm"], out=s["out"])
    return [norm, *s["flat"]]


def _mx_values(codes, scales):
    """The fp32 values of packed codes [..., C/2] and scales [..., C/32]."""
    level = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack([level[(codes & 15).long()], level[(codes >> 4).long()]], -1)
    v = v.reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "mx_roundtrip":
        out = torch.empty_like(s["w"])
        level = torch.tensor(E2M1, device=DEV)
        for w, o in zip(s["w"], out):
            b = _blocks(w)
            e = _mx_scale_exponent(b)
            v = torch.ldexp(level[_mx_level_index(torch.ldexp(b.abs(), -e)).long()], e)
            o.copy_(torch.where(b < 0, -v, v).reshape(w.shape))
        return out
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for g in s["grads"]:
            total += g.double().square().sum()
        norm = total.sqrt().float()
        scale = torch.where(norm > case["max_norm"], case["max_norm"] / norm, 1.0)
        for g, o in zip(s["grads"], s["out"]):
            o.copy_(g.float() * scale)
        return [norm, *s["flat"]]
    E, M, N, K = (case[k] for k in "EMNK")
    lo = 0
    if op == "mm_backward":
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        dw = torch.zeros((E, N, K), dtype=torch.float32 if case["dw"] == "fp32" else torch.bfloat16, device=DEV)
        for e, n in enumerate(s["sizes"]):
            if n:
                dy = s["dy"][lo:lo + n].float()
                dx[lo:lo + n] = dy @ s["w"][e].float()
                dw[e] = dy.t() @ s["x"][lo:lo + n].float()
            lo += n
        return dx, dw
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    for e, n in enumerate(s["sizes"]):
        if n and op == "mm":
            y[lo:lo + n] = s["x"][lo:lo + n].float() @ s["w"][e].float().t()
        elif n:
            x = _mx_values(s["x"][0][0, lo:lo + n], s["x"][1][0, lo:lo + n])
            y[lo:lo + n] = x @ _mx_values(s["w"][0][e], s["w"][1][e]).t()
        lo += n
    return y


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "mx_roundtrip":
        n = case["E"] * case["R"] * case["C"]
        packed = n // 2 + n // 32   # written by the one call, read by the other
        return dict(bytes=2 * n + 2 * packed + 2 * n, flops=4 * n)
    if op == "clip":
        n = case["count"] * (case["small"] + case["large"]) / 2
        size = {"fp32": 4, "bf16": 2, "both": 3}[case["mix"]]
        return dict(bytes=2 * size * n, flops=3 * n)
    E, M, N, K = (case[k] for k in "EMNK")
    # the weights of experts that are expected to have a row
    p = [1.0 / E] * E if case["skew"] == "uniform" else [1.0 / (i + 1) ** 1.1 for i in range(E)]
    t = sum(p)
    live = sum(1.0 - (1.0 - q / t) ** M for q in p)
    if op == "mx_mm":
        per = 17 / 32   # half a byte a value and one byte a block of 32
        return dict(bytes=per * (M + live * N) * K + 2 * M * N, flops=2 * M * N * K)
    if op == "mm":
        return dict(bytes=2 * (M + live * N) * K + 2 * M * N, flops=2 * M * N * K)
    size = 4 if case["dw"] == "fp32" else 2
    return dict(bytes=2 * (M * K + M * N + live * N * K) + 2 * M * K + size * E * N * K, flops=4 * M * N * K)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_mx(w):
    """MXFP4 values of [R, C] in 64 bits: block scale 2^(floor(log2 max) - 2),
    magnitudes rounded half to even on a grid of 1/2 below 2, 1 below 4 and 2
    above, at most 6 (E2M1)."""
    b = w.double().unflatten(-1, (-1, 32))
    top = b.abs().max(-1, keepdim=True).values
    scale = torch.where(top > 0, torch.exp2((torch.floor(torch.log2(top)) - 2).clamp(min=-127)), 1.0)
    v = b / scale
    grid = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((v / grid).round() * grid).clamp(-6, 6).mul(scale).flatten(-2)


def _exact_unpack(codes, scales):
    """Values from the bit fields of E2M1 (sign, two exponent bits, one
    fraction bit) and of the scale exponent, in 64 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    e, f = ((c >> 1) & 3).double(), (c & 1).double()
    v = torch.where(e == 0, f / 2, torch.exp2(e - 1) * (1 + f / 2)) * (1 - 2 * (c >> 3).double())
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mx_roundtrip":
        return torch.stack([_exact_mx(w).to(torch.float32) for w in s["w"]])
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
        c = min(1.0, case["max_norm"] / norm) if norm else 1.0
        out = [torch.tensor(norm, dtype=torch.float64, device=DEV)]
        for flat in s["flat"]:
            part = [torch.nn.functional.pad(g.double() * c, (0, -g.numel() % 8)) for g in s["grads"] if g.dtype == flat.dtype]
            out.append(torch.cat(part))
        return out
    E, M, N, K = (case[k] for k in "EMNK")
    off = s["offsets"].tolist()
    if op == "mm_backward":
        dx, dw = [], []
        for e in range(E):
            dy, x = s["dy"][off[e]:off[e + 1]].double(), s["x"][off[e]:off[e + 1]].double()
            dx.append(torch.matmul(dy, s["w"][e].double()))
            dw.append(torch.matmul(dy.t(), x))
        return torch.cat(dx), torch.stack(dw)
    y = []
    for e in range(E):
        if op == "mm":
            x, w = s["x"][off[e]:off[e + 1]].double(), s["w"][e].double()
        else:
            x = _exact_unpack(s["x"][0][0, off[e]:off[e + 1]], s["x"][1][0, off[e]:off[e + 1]])
            w = _exact_unpack(s["w"][0][e], s["w"][1][e])
        y.append(torch.matmul(x, w.t()))
    return torch.cat(y)
