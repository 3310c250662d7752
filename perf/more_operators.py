"""Measured cases of the experts' gated feed-forward block with its backward
pass, of the 8-bit floating-point format with a scale for each block of 128 and
the product over it, and of the orthogonalised update: their inputs, their plain
forms, the calls a program makes of the library, and the same results from the
definitions in 64 bits.

Operators
  ffn            out[p] = down[e] (silu(g) * u), (g, u) = gate_up[e] x[p], for
                 rows sorted by expert, bf16
  ffn_step       the same keeping g and u, and the gradients with respect to
                 x, gate_up and down
  fp8_roundtrip  bf16 -> E4M3 codes with an fp32 scale for each 128 columns of a
                 row ("row") or each 128 x 128 tile ("tile") -> bf16
  fp8_mm         y[p] = w[e] x[p], x with row scales and w with tile scales
  orthogonalize  five Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T,
                 from X = G / |G|, for each of a batch of matrices G

Shapes are those of the library's synthetic layers (E experts, hidden size H,
expert size I, top-k routing) or general ones.
"""

import math

import torch

own = False   # True: run() calls the library; False: the plain forms

DEV = "cuda"
FP8_MAX = 448.0
NS = (3.4445, -4.7750, 2.0315)
STEPS = 5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # decode of one token, top-8 of 64 experts: eight rows, weight streaming
        dict(name="ffn decode M8", op="ffn", E=64, M=8, H=2048, I=1024, skew="uniform"),
        # prompt of 8192 tokens, top-2 of a large layer: matrix rate
        dict(name="ffn prompt M16384", op="ffn", E=8, M=16384, H=4096, I=14336, skew="uniform"),
        # training step, 4096 tokens top-8, trainable experts
        dict(name="ffn_step M32768", op="ffn_step", E=64, M=32768, H=2048, I=1024, skew="uniform"),
        # training step, 2048 tokens top-8 of 128 experts, popular ones first: very ragged
        dict(name="ffn_step M16384 zipf", op="ffn_step", E=128, M=16384, H=2048, I=768, skew="zipf"),
        # one decode step's activations (16 tokens, top-4, H = 2880): latency
        dict(name="fp8_roundtrip rows 64", op="fp8_roundtrip", kind="row", E=1, R=64, C=2880),
        # quantize-on-load of a layer's gate_up [32, 2 * 2880, 2880]: bandwidth, ragged last tiles
        dict(name="fp8_roundtrip layer", op="fp8_roundtrip", kind="tile", E=32, R=5760, C=2880),
        # decode, 16 tokens top-4 over 32 experts: two rows an expert, weight streaming
        dict(name="fp8_mm decode M64", op="fp8_mm", E=32, M=64, N=5760, K=2880, skew="uniform"),
        # 1024 tokens, top-8 of 128 experts, popular ones first: very ragged
        dict(name="fp8_mm prompt M8192 zipf", op="fp8_mm", E=128, M=8192, N=1536, K=2048, skew="zipf"),
        # 16384 tokens top-2 of a large layer's gate_up: matrix rate
        dict(name="fp8_mm prompt M32768", op="fp8_mm", E=8, M=32768, N=28672, K=4096, skew="uniform"),
        # updates of rank-16 adapters on 64 experts: many small matrices, latency
        dict(name="orthogonalize rank 16", op="orthogonalize", E=64, N=16, K=2048, dtype="bf16"),
        # updates of 64 trainable experts' down projections, from fp32 gradients, taller than wide
        dict(name="orthogonalize experts", op="orthogonalize", E=64, N=2048, K=1024, dtype="fp32"),
        # updates of a large layer's eight down projections: matrix rate
        dict(name="orthogonalize layer", op="orthogonalize", E=8, N=4096, K=14336, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn_step", "fp8_roundtrip", "fp8_mm", "orthogonalize"])
    if op == "fp8_roundtrip":
        return dict(op=op, kind=rng.choice(["row", "tile"]), E=rng.randint(1, 32), R=_log(rng, 1, 6000),
                    C=16 * _log(rng, 1, 180))
    if op == "orthogonalize":
        return dict(op=op, E=_log(rng, 1, 64), N=_log(rng, 1, 2500), K=_log(rng, 1, 2500),
                    dtype=rng.choice(["bf16", "fp32"]))
    skew = rng.choice(["uniform", "zipf"])
    if op == "fp8_mm":
        return dict(op=op, E=_log(rng, 1, 128), M=_log(rng, 1, 20000), N=8 * _log(rng, 1, 512),
                    K=16 * _log(rng, 1, 256), skew=skew)
    return dict(op=op, E=_log(rng, 1, 128), M=_log(rng, 1, 20000), H=8 * _log(rng, 1, 400), I=8 * _log(rng, 1, 300),
                skew=skew)


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


def _tiles(w, rows):
    """[..., R, C] as [..., R / rows, rows, C / 128, 128], zeros where the last blocks stick out."""
    w = torch.nn.functional.pad(w, (0, -w.shape[-1] % 128, 0, -w.shape[-2] % rows))
    return w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, rows))


def _fp8_pack(w, rows):
    """bf16 [E, R, C] -> (E4M3 codes [E, R, C], fp32 scales, one for each `rows` rows by 128 columns)."""
    codes = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=DEV)
    scales = []
    for x, c in zip(w.split(1), codes.split(1)):
        t = _tiles(x.float(), rows)
        top = t.abs().amax((-3, -1))
        v = FP8_MAX * t / torch.where(top > 0, top, 1.0)[..., :, None, :, None]
        c.copy_(v.flatten(-4, -3).flatten(-2)[..., :x.shape[-2], :x.shape[-1]])
        scales.append(top / FP8_MAX)
    return codes, torch.cat(scales)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 5)
    op = case["op"]
    s = dict(case=case)
    if op == "fp8_roundtrip":
        s["w"] = _randn(gen, (case["E"], case["R"], case["C"]), 0.02)
        return s
    if op == "orthogonalize":
        # a gradient: some directions carry more than others
        E, N, K = (case[k] for k in "ENK")
        g = _randn(gen, (E, N, K), 0.01)
        for m in g:
            m += 0.02 * torch.randn(N, 1, generator=gen, device=DEV) * torch.randn(K, generator=gen, device=DEV)
        s["g"] = g.float() if case["dtype"] == "fp32" else g
        return s
    sizes = _sizes(case, seed)
    s["sizes"] = sizes.tolist()
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).to(DEV)
    E, M = case["E"], case["M"]
    if op == "fp8_mm":
        N, K = case["N"], case["K"]
        s["x"] = _fp8_pack(_randn(gen, (1, M, K), 1.0), 1)
        s["w"] = _fp8_pack(_randn(gen, (E, N, K), 0.02), 128)
        if own:   # the handles that a program keeps with its weights and activations
            import bit_weight_quantization_moeq_amd as moeq
            s["xq"] = moeq.QWeight(moeq.FMT_FP8_ROW, 1, M, K, *s["x"])
            s["wq"] = moeq.QWeight(moeq.FMT_FP8_TILE, E, N, K, *s["w"])
        return s
    H, I = case["H"], case["I"]
    s["x"] = _randn(gen, (M, H), 1.0)
    s["gate_up"], s["down"] = _randn(gen, (E, 2 * I, H), H ** -0.5), _randn(gen, (E, H, I), I ** -0.5)
    if op == "ffn_step":
        s["dy"] = _randn(gen, (M, H), 1.0)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bit_weight_quantization_moeq_amd as moeq
    op = s["case"]["op"]
    if op == "ffn":
        return moeq.moeq_grouped_ffn(s["x"], s["gate_up"], s["down"], s["offsets"])
    if op == "ffn_step":
        y, gu = moeq.moeq_grouped_ffn(s["x"], s["gate_up"], s["down"], s["offsets"], save=True)
        return (y, *moeq.moeq_grouped_ffn_backward(s["dy"], s["x"], s["gate_up"], s["down"], s["offsets"], gu,
                                                   dtype=torch.bfloat16))
    if op == "fp8_roundtrip":
        q = moeq.moeq_quantize_fp8(s["w"], moeq.FMT_FP8_ROW if s["case"]["kind"] == "row" else moeq.FMT_FP8_TILE)
        return moeq.moeq_dequantize(q), q.scales
    if op == "fp8_mm":
        return moeq.moeq_grouped_mm_fp8(s["xq"], s["wq"], s["offsets"])
    return moeq.moeq_orthogonalize(s["g"], steps=STEPS, coefficients=NS)


def _fp8_values(codes, scales, rows):
    """fp32 values of codes [R, C] with scales of `rows` rows by 128 columns."""
    v = _tiles(codes.float(), rows) * scales[:, None, :, None]
    return v.flatten(0, 1).flatten(1)[:codes.shape[0], :codes.shape[1]]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "fp8_roundtrip":
        rows = 1 if case["kind"] == "row" else 128
        t = _tiles(s["w"].float(), rows)
        top = t.abs().amax((-3, -1))
        scale = top / FP8_MAX
        v = FP8_MAX * t / torch.where(top > 0, top, 1.0)[..., :, None, :, None]
        v = v.to(torch.float8_e4m3fn).float() * scale[..., :, None, :, None]
        return v.flatten(-4, -3).flatten(-2)[..., :case["R"], :case["C"]].to(torch.bfloat16).contiguous(), scale
    if op == "orthogonalize":
        a, b, c = NS
        g = s["g"]
        tall = g.shape[1] > g.shape[2]
        x = g.float()
        norm = g.double().square().sum((1, 2)).sqrt().float()[:, None, None]
        x = x / torch.where(norm > 0, norm, 1.0)
        x = x.mT.contiguous() if tall else x
        for _ in range(STEPS):
            m = x @ x.mT
            x = a * x + (b * m + c * (m @ m)) @ x
        return (x.mT if tall else x).to(torch.bfloat16).contiguous()
    out = torch.empty((case["M"], case["N"] if op == "fp8_mm" else case["H"]), dtype=torch.bfloat16, device=DEV)
    if op == "ffn_step":
        dx, dgu, dd = torch.empty_like(s["x"]), torch.zeros_like(s["gate_up"]), torch.zeros_like(s["down"])
    lo = 0
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        p = slice(lo, lo + n)
        lo += n
        if op == "fp8_mm":
            x = _fp8_values(s["x"][0][0, p], s["x"][1][0, p], 1)
            out[p] = x @ _fp8_values(s["w"][0][e], s["w"][1][e], 128).t()
            continue
        x, gate_up, down = s["x"][p].float(), s["gate_up"][e].float(), s["down"][e].float()
        g, u = (x @ gate_up.t()).chunk(2, 1)
        sig = torch.sigmoid(g)
        h = g * sig * u
        out[p] = h @ down.t()
        if op == "ffn_step":
            dy = s["dy"][p].float()
            dh = dy @ down
            d = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
            dx[p], dgu[e], dd[e] = d @ gate_up, d.t() @ x, dy.t() @ h
    return (out, dx, dgu, dd) if op == "ffn_step" else out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "fp8_roundtrip":
        n = case["E"] * case["R"] * case["C"]
        blocks = case["E"] * -(-case["C"] // 128) * (case["R"] if case["kind"] == "row" else -(-case["R"] // 128))
        # the codes and scales are written by the one call and read by the other
        return dict(bytes=2 * n + 2 * (n + 4 * blocks) + 2 * n, flops=4 * n)
    if op == "orthogonalize":
        E, n, m = case["E"], min(case["N"], case["K"]), max(case["N"], case["K"])
        # A and b A + c A A are symmetric: half of them is enough
        return dict(bytes=(4 if case["dtype"] == "fp32" else 2) * E * n * m + 2 * E * n * m,
                    flops=STEPS * E * (3 * n * n * m + n * n * n))
    E, M = case["E"], case["M"]
    # the weights of experts that are expected to have a row
    p = [1.0 / E] * E if case["skew"] == "uniform" else [1.0 / (i + 1) ** 1.1 for i in range(E)]
    t = sum(p)
    live = sum(1.0 - (1.0 - q / t) ** M for q in p)
    if op == "fp8_mm":
        N, K = case["N"], case["K"]
        kb = -(-K // 128)
        return dict(bytes=M * (K + 4 * kb) + live * (N * K + 4 * kb * -(-N // 128)) + 2 * M * N, flops=2 * M * N * K)
    H, I = case["H"], case["I"]
    if op == "ffn":
        return dict(bytes=2 * (2 * M * H + live * 3 * H * I), flops=6 * M * H * I)
    return dict(bytes=2 * (4 * M * H + (live + E) * 3 * H * I), flops=18 * M * H * I)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_e4m3(v):
    """v (|v| <= 448 and a little) rounded half to even to E4M3: three fraction
    bits, steps of 2^-9 at the bottom."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return ((v / step).round() * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_roundtrip(w, rows):
    R, C = w.shape
    out, scales = torch.empty((R, C), dtype=torch.float64, device=DEV), []
    top = w.double().abs()
    # the largest of each 128 columns, then of each `rows` rows
    top = torch.stack([c.amax(1) for c in top.split(128, 1)], 1)
    top = torch.stack([r.amax(0) for r in top.split(rows, 0)], 0) if rows > 1 else top
    each = top.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :C]
    code = _exact_e4m3(FP8_MAX * w.double() / torch.where(each > 0, each, 1.0))
    return code * (each / FP8_MAX), top / FP8_MAX


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8_roundtrip":
        parts = [_exact_roundtrip(w, 1 if case["kind"] == "row" else 128) for w in s["w"]]
        return torch.stack([p[0].float() for p in parts]), torch.stack([p[1] for p in parts])
    if op == "orthogonalize":
        a, b, c = NS
        out = []
        for g in s["g"]:
            x = g.double()
            norm = torch.linalg.vector_norm(x)
            x = x / norm if norm > 0 else x
            eye = torch.eye(min(x.shape), dtype=torch.float64, device=DEV)
            for _ in range(STEPS):
                if x.shape[0] > x.shape[1]:
                    m = x.t().contiguous() @ x
                    x = x @ (a * eye + b * m + c * (m @ m))
                else:
                    m = x @ x.t().contiguous()
                    x = (a * eye + b * m + c * (m @ m)) @ x
            out.append(x.float())
        return torch.stack(out)
    off = s["offsets"].tolist()
    y, dx, dgu, dd = [], [], [], []
    for e in range(case["E"]):
        p = slice(off[e], off[e + 1])
        if op == "fp8_mm":
            x = s["x"][0][0, p].double() * s["x"][1][0, p].double().repeat_interleave(128, 1)[:, :case["K"]]
            each = s["w"][1][e].double().repeat_interleave(128, 0)[:case["N"]].repeat_interleave(128, 1)[:, :case["K"]]
            y.append(torch.matmul(x, (s["w"][0][e].double() * each).t()))
            continue
        I = case["I"]
        x, wg, wu = s["x"][p].double(), s["gate_up"][e, :I].double(), s["gate_up"][e, I:].double()
        wd = s["down"][e].double()
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
        act = g / (1 + torch.exp(-g))
        y.append(torch.matmul(act * u, wd.t()))
        if op == "ffn_step":
            dy = s["dy"][p].double()
            dh = torch.matmul(dy, wd)
            # d silu = silu / g + silu (1 - silu / g), with sigmoid = 1 / (1 + exp(-g))
            sig = 1 / (1 + torch.exp(-g))
            dg, du = dh * u * (sig + act * (1 - sig)), dh * act
            dx.append(torch.matmul(dg, wg) + torch.matmul(du, wu))
            dgu.append(torch.cat([torch.matmul(dg.t(), x), torch.matmul(du.t(), x)]).float())
            dd.append(torch.matmul(dy.t(), act * u).float())
    if op == "ffn_step":
        return torch.cat(y), torch.cat(dx), torch.stack(dgu), torch.stack(dd)
    return torch.cat(y)
