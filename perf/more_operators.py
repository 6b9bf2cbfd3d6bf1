"""Cases of the 4-bit block-scaled (MXFP4) product and its quantiser, of the
router's losses and gradient, and of the orthogonalised update: inputs, plain
forms and the library's calls.

A case is a dict of plain values; its "op" says which operator it runs:

  quantize  a matrix to 4-bit floats (e2m1) with a power of two for each block
            of 32 values of a row, as it lies ("rows"), transposed ("cols"), or
            both from one read ("both"), and each read back as the values that
            it stands for
  gemm      C = bias + sum over blocks b of 32 k of
            2^(sa[b, m] + sb[b, n]) * sum_k A[m, k] * B[n, k]
  balance   how often the router chose each expert, the loss that balances
            them, and the loss that keeps the logits small
  grad      the gradient of the chosen experts' weights and of both losses by
            the logits
  ortho     an update's matrix brought near the nearest orthogonal one by
            Newton-Schulz steps, X <- a X + (b X X^T + c (X X^T)^2) X

`run` computes the plain form in 32 bits with elementary torch operations, or,
with `own`, calls the library.  Four scales of a row's consecutive blocks lie
in one 32-bit word, the words block-major: [k / 128][row].
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # the activations of 16 decoding tokens, before a layer's product: a call bound by its latency
        dict(name="quant_rows_16", op="quantize", rows=16, cols=4096, x="bf16", out="rows"),
        # a training step's activations, an odd number of them: the forward operand and, transposed, the weight gradient's
        dict(name="quant_both_8003", op="quantize", rows=8003, cols=8192, x="bf16", out="both"),
        # one decoding token through a square layer
        dict(name="gemm_m1", op="gemm", M=1, N=4096, K=4096, c="bf16", bias=False),
        # a decoding batch of odd size through a wider layer
        dict(name="gemm_m37", op="gemm", M=37, N=5120, K=8192, c="f16", bias=True),
        # weight gradient: both operands transposed, summed over an odd number of tokens
        dict(name="gemm_wgrad", op="gemm", M=4096, N=4096, K=5003, c="f32", bias=False),
        # forward product of a large batch, the headline size of the dense products
        dict(name="gemm_8192", op="gemm", M=8192, N=8192, K=8192, c="bf16", bias=True),
        # losses of a small batch's routing
        dict(name="balance_64", op="balance", tokens=64, experts=64, topk=6, x="f32", scoring="softmax", mask=False),
        # losses of a training batch of packed sequences, padded at their ends, over many experts
        dict(name="balance_16384", op="balance", tokens=16384, experts=256, topk=8, x="bf16", scoring="sigmoid", mask=True),
        # the router's gradient for a small batch
        dict(name="grad_64", op="grad", tokens=64, experts=64, topk=6, x="f32", scoring="softmax", norm=True, mask=False, d="f32"),
        # the router's gradient of the training batch above
        dict(name="grad_16384", op="grad", tokens=16384, experts=256, topk=8, x="bf16", scoring="sigmoid", norm=True, mask=True, d="bf16"),
        # the update of one tall projection
        dict(name="ortho_4096x1024", op="ortho", batch=1, rows=4096, cols=1024, x="bf16", o="bf16", steps=5),
        # the updates of a layer's experts in one call, momentum and update held in 32 bits
        dict(name="ortho_experts", op="ortho", batch=8, rows=768, cols=2048, x="f32", o="f32", steps=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "balance", "grad", "ortho"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 32, 8192), x=rng.choice(["f32", "f16", "bf16"]),
                    out=rng.choice(["rows", "cols", "both"]))
    if op == "gemm":
        # layers' sizes come in steps, token counts do not; the weight gradient sums over tokens
        n, k, m = 16 * _log(rng, 8, 512), 16 * _log(rng, 8, 512), _log(rng, 1, 8192)
        if rng.random() < 0.3:
            m, k = k, m
        return dict(op=op, M=m, N=n, K=k, c=rng.choice(["f32", "f16", "bf16"]), bias=rng.random() < 0.5)
    if op in ("balance", "grad"):
        experts = _log(rng, 4, 384)
        case = dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, topk=rng.randint(1, min(10, experts)),
                    x=rng.choice(["f32", "f16", "bf16"]), scoring=rng.choice(["softmax", "sigmoid"]), mask=rng.random() < 0.5)
        if op == "grad":
            case.update(norm=rng.random() < 0.5, d=rng.choice(["f32", case["x"]]))
        return case
    rows, cols = _log(rng, 32, 4096), _log(rng, 32, 4096)
    n, m, steps = min(rows, cols), max(rows, cols), rng.randint(4, 6)
    most = int(4e11 / (steps * n * n * (3 * m + n)))
    x = rng.choice(["f32", "f16", "bf16"])
    return dict(op=op, batch=_log(rng, 1, max(1, min(16, most))), rows=rows, cols=cols, x=x, o=rng.choice(["f32", x]), steps=steps)


# ------------------------------------------------------------------ inputs

def _blocks(n, size=128):
    return -(-n // size)


def _pitch(cols):
    """Bytes of a row of 4-bit values, at a multiple of 16."""
    return -(-cols // 32) * 16


def _matrix(gen, rows, cols, t, row_spread):
    """Normal values whose rows differ in size, as activations' and gradients' do."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    if row_spread:
        x *= torch.exp(0.7 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x.to(t)


def _in_blocks(x):
    """float32 (rows, cols): its 4-bit values times their scales, (rows, blocks, 32), and the scales' exponents + 127."""
    rows, cols = x.shape
    p = torch.zeros(rows, _blocks(cols) * 128, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, -1, 32)
    top = p.abs().amax(2).contiguous().view(torch.int32) >> 23  # floor(log2) + 127
    e = (top - 2).clamp_min(0)
    v = p.double() * torch.exp2((127 - e).double())[:, :, None]
    a = v.abs().clamp_max(6.0)
    step = 0.5 + 0.5 * (a >= 2) + (a >= 4)
    a = a / step
    low = a - a % 1
    up = (a - low > 0.5) | ((a - low == 0.5) & (low % 2 == 1))
    v = torch.where(v < 0, -1.0, 1.0) * (low + up) * step
    e[_blocks(cols, 32) * torch.ones_like(e) <= torch.arange(e.shape[1], device=e.device)] = 0  # blocks past the last column
    return v, e


def _words(e):
    """Exponents (rows, blocks) as scale words [block / 4][row]."""
    return e.to(torch.uint8).view(torch.int32).t().contiguous()


def _packed(v, cols):
    """e2m1 values (rows, blocks, 32) in 4 bits, the even column's lower; rows at a multiple of 16 bytes."""
    a = v.abs()
    code = (2 * a * (a < 2) + (a + 2) * ((a >= 2) & (a < 4)) + (a / 2 + 4) * (a >= 4)).to(torch.uint8) | (v < 0).to(torch.uint8) * 8
    code = code.view(v.shape[0], -1, 2)
    return (code[:, :, 0] | code[:, :, 1] << 4)[:, :_pitch(cols)].contiguous()


def _quantized(x):
    v, e = _in_blocks(x)
    return _packed(v, x.shape[1]), _words(e)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        rows, cols, t = case["rows"], case["cols"], TYPES[case["x"]]
        s["x"] = _matrix(gen, rows, cols, t, True)
        for name, r, c in (("rows", rows, cols), ("cols", cols, rows)):
            if case["out"] in (name, "both"):
                s[name] = (torch.zeros(r, _pitch(c), dtype=torch.uint8, device=dev),
                           torch.zeros(_blocks(c), r, dtype=torch.int32, device=dev), torch.zeros(r, c, dtype=t, device=dev))
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["sa"] = _quantized(_matrix(gen, M, K, torch.float32, True))
        s["B"], s["sb"] = _quantized(_matrix(gen, N, K, torch.float32, False) * K ** -0.5)
        s["bias"] = torch.randn(N, generator=gen, device=dev) if case["bias"] else None
        s["C"] = torch.zeros(M, N, dtype=TYPES[case["c"]], device=dev)
    elif op in ("balance", "grad"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        lean = 0.5 * torch.randn(E, generator=gen, device=dev)  # some experts are chosen more often
        s["logits"] = (2 * torch.randn(T, E, generator=gen, device=dev) + lean).to(TYPES[case["x"]])
        s["ids"] = torch.topk(s["logits"].float(), k, dim=1)[1].to(torch.int32).contiguous()
        s["mask"] = (torch.rand(T, generator=gen, device=dev) > 0.1).to(torch.uint8) if case["mask"] else None
        if op == "balance":
            s["counts"] = torch.zeros(E + 1, dtype=torch.int32, device=dev)
            s["losses"] = torch.zeros(2, device=dev)
        else:
            s["counts"] = _counts(s)
            # (of a loss scaled by the number of tokens, as 16-bit gradients need)
            s["dweights"] = torch.randn(T, k, generator=gen, device=dev)
            s["dlosses"] = torch.tensor([0.01 * T, 0.001 * T], device=dev)
            s["D"] = torch.zeros(T, E, dtype=TYPES[case["d"]], device=dev)
    else:
        b, r, c = case["batch"], case["rows"], case["cols"]
        # a few strong directions over noise, as a gradient's momentum has
        g = torch.randn(b, r, c, generator=gen, device=dev)
        strong = torch.randn(b, r, 8, generator=gen, device=dev) @ torch.randn(b, 8, c, generator=gen, device=dev)
        s["G"] = (1e-3 * (g + strong)).to(TYPES[case["x"]])
        s["O"] = torch.zeros(b, r, c, dtype=TYPES[case["o"]], device=dev)
        s["scale"] = 0.2 * math.sqrt(max(r, c))
    return s


# ------------------------------------------------------- the library's calls

CODES = {"f16": "TCM_F16_F32", "bf16": "TCM_BF16_F32", "f32": "TCM_F32_F32"}


def _out_flag(T, name):
    return {"f32": 0, "f16": T.TCM_C_F16, "bf16": T.TCM_C_BF16}[name]


def _scales(words):
    """The values that scale words hold, [block / 4][row][block % 4]."""
    return words.view(torch.uint8).view(torch.float8_e8m0fnu)


def _own_quantize(T, s, stream):
    case, x = s["case"], s["x"]
    rows, cols, code = case["rows"], case["cols"], getattr(T, CODES[case["x"]])
    a, b = s.get("rows"), s.get("cols")
    pa = (a[0].data_ptr(), a[0].stride(0), a[1].data_ptr(), rows) if a else (None, 0, None, 0)
    pb = (b[0].data_ptr(), b[0].stride(0), b[1].data_ptr(), cols) if b else (None, 0, None, 0)
    st = T.tcm_quantize_mxfp4(rows, cols, x.data_ptr(), cols, code, *pa, *pb, stream)
    out = []
    if a and st == T.TCM_OK:
        st = T.tcm_dequantize_mxfp4(rows, cols, *pa, a[2].data_ptr(), cols, code, stream)
        out += [a[2], _scales(a[1])]
    if b and st == T.TCM_OK:
        st = T.tcm_dequantize_mxfp4(cols, rows, *pb, b[2].data_ptr(), rows, code, stream)
        out += [b[2], _scales(b[1])]
    return st, out


def _own_gemm(T, s, stream):
    case, A, B, bias = s["case"], s["A"], s["B"], s["bias"]
    st = T.tcm_gemm_mxfp4(case["M"], case["N"], case["K"], A.data_ptr(), A.stride(0), s["sa"].data_ptr(), case["M"], B.data_ptr(),
                          B.stride(0), s["sb"].data_ptr(), case["N"], s["C"].data_ptr(), case["N"],
                          T.TCM_MXFP4_F32 | _out_flag(T, case["c"]), bias.data_ptr() if bias is not None else None,
                          T.TCM_EPI_BIAS if bias is not None else T.TCM_EPI_NONE, stream)
    return st, s["C"]


def _own_balance(T, s, stream):
    case, mask = s["case"], s["mask"]
    code = getattr(T, CODES[case["x"]]) | (T.TCM_ROUTE_SIGMOID if case["scoring"] == "sigmoid" else 0)
    st = T.tcm_moe_balance(case["tokens"], case["experts"], case["topk"], s["logits"].data_ptr(), case["experts"], code,
                           s["ids"].data_ptr(), mask.data_ptr() if mask is not None else None, s["counts"].data_ptr(),
                           s["losses"].data_ptr(), stream)
    return st, [s["counts"], s["losses"]]


def _own_grad(T, s, stream):
    case, mask = s["case"], s["mask"]
    code = getattr(T, CODES[case["x"]]) | (T.TCM_ROUTE_SIGMOID if case["scoring"] == "sigmoid" else 0)
    code |= (T.TCM_ROUTE_NORM if case["norm"] else 0) | _out_flag(T, case["d"])
    st = T.tcm_moe_route_grad(case["tokens"], case["experts"], case["topk"], s["logits"].data_ptr(), case["experts"], code, 1.0,
                              s["ids"].data_ptr(), mask.data_ptr() if mask is not None else None, s["dweights"].data_ptr(),
                              s["counts"].data_ptr(), s["dlosses"].data_ptr(), s["D"].data_ptr(), case["experts"], stream)
    return st, s["D"]


def _own_ortho(T, s, stream):
    case, r, c = s["case"], s["case"]["rows"], s["case"]["cols"]
    st = T.tcm_orthogonalize(case["batch"], r, c, s["G"].data_ptr(), c, r * c, s["O"].data_ptr(), c, r * c,
                             getattr(T, CODES[case["x"]]) | _out_flag(T, case["o"]), COEFFICIENTS * case["steps"], EPS, s["scale"],
                             stream)
    return st, s["O"]


OWN = {"quantize": _own_quantize, "gemm": _own_gemm, "balance": _own_balance, "grad": _own_grad, "ortho": _own_ortho}


# ----------------------------------------------------------- the plain forms

def _plain_quantize(s):
    def one(x):
        v, e = _in_blocks(x.float())
        y = v * torch.exp2((e - 127).double())[:, :, None]
        return [y.view(x.shape[0], -1)[:, :x.shape[1]].to(x.dtype), _scales(_words(e))]
    return (one(s["x"]) if "rows" in s else []) + (one(s["x"].t()) if "cols" in s else [])


def _values(q, words, cols):
    """What 4-bit codes and their scale words stand for, float32 (rows, cols)."""
    rows = q.shape[0]
    codes = torch.stack((q & 15, q >> 4), 2).view(rows, -1, 32)
    at = codes.new_tensor([0, 1, 2, 3, 4, 6, 8, 12] * 2).float() * 0.5
    at[8:] *= -1
    e = words.t().contiguous().view(torch.uint8)[:, :codes.shape[1]]
    return (at[codes.int()] * torch.exp2(e.float() - 127)[:, :, None]).view(rows, -1)[:, :cols]


def _plain_gemm(s):
    case = s["case"]
    c = _values(s["A"], s["sa"], case["K"]) @ _values(s["B"], s["sb"], case["K"]).t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return c.to(TYPES[case["c"]])


def _valid(s):
    return torch.ones(len(s["logits"]), device="cuda") if s["mask"] is None else s["mask"].float()


def _counts(s):
    """How often each expert is chosen by the tokens that count, and the number of these."""
    E, v = s["case"]["experts"], _valid(s)
    here = (s["ids"][:, :, None] == torch.arange(E, device="cuda", dtype=torch.int32)).sum(1) * v[:, None]
    return torch.cat((here.sum(0), v.sum()[None])).to(torch.int32)


def _softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_balance(s):
    case, x, v = s["case"], s["logits"].float(), _valid(s)
    top = x.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(x - top).sum(1, keepdim=True)))[:, 0]
    score = _softmax(x) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-x))
    p = score / score.sum(1, keepdim=True)
    counts, n = _counts(s), v.sum().clamp_min(1)
    share = counts[:-1].float() / (n * case["topk"])
    mean = (p * v[:, None]).sum(0) / n
    return [counts, torch.stack((case["experts"] * (share * mean).sum(), (lse * lse * v).sum() / n))]


def _plain_grad(s):
    case, x, v = s["case"], s["logits"].double(), _valid(s)  # differences of near values: 64 bits
    E, k = case["experts"], case["topk"]
    ids = s["ids"].long()
    soft = _softmax(x)
    score = soft if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-x))
    # by the scores: of the weights, then of the balance loss
    chosen, g = torch.gather(score, 1, ids), s["dweights"].double()
    if case["norm"]:
        total = chosen.sum(1, keepdim=True)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(x).scatter(1, ids, g)
    n = v.sum().clamp_min(1)
    share = s["counts"][:-1].double() / (n * k)
    total = score.sum(1, keepdim=True)
    dp = s["dlosses"][0] * E / n * share
    ds = ds + (dp - (dp * score).sum(1, keepdim=True) / total) / total
    # by the logits
    d = score * (ds - (ds * score).sum(1, keepdim=True)) if case["scoring"] == "softmax" else ds * score * (1 - score)
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    d = d + s["dlosses"][1] * 2 / n * lse * soft
    return (d * v[:, None]).to(TYPES[case["d"]])


def _plain_ortho(s):
    case, a, b, c = s["case"], *COEFFICIENTS
    x = s["G"].float()
    tall = case["rows"] > case["cols"]
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(case["steps"]):  # each step needs the one before
        g = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
    x = x.transpose(1, 2) if tall else x
    return (s["scale"] * x).to(TYPES[case["o"]]).contiguous()


PLAIN = {"quantize": _plain_quantize, "gemm": _plain_gemm, "balance": _plain_balance, "grad": _plain_grad, "ortho": _plain_ortho}


def run(state):
    op = state["case"]["op"]
    if own:
        import tensor_core_mixed_amd as T
        st, out = OWN[op](T, state, torch.cuda.current_stream().cuda_stream)
        if st != T.TCM_OK:
            raise T.TcmError(st, op)
        return out
    return PLAIN[op](state)


# --------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; the products' multiplications and additions."""
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op = case["op"]
    if op == "quantize":  # X to 4 bits, and 4 bits to their values
        r, c, z = case["rows"], case["cols"], size[case["x"]]
        n, outs = r * c, 2 if case["out"] == "both" else 1
        q = (r * _pitch(c) + 4 * r * _blocks(c)) * (case["out"] != "cols") + (c * _pitch(r) + 4 * c * _blocks(r)) * (case["out"] != "rows")
        return {"bytes": n * z + 2 * q + outs * n * z, "flops": 3 * n * outs}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (_pitch(K) + 4 * _blocks(K)) + M * N * size[case["c"]] + 4 * N * case["bias"], "flops": 2 * M * N * K}
    if op in ("balance", "grad"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        n = T * E * size[case["x"]] + 4 * T * k + T * case["mask"]
        if op == "balance":
            return {"bytes": n + 4 * E + 12, "flops": 6 * T * E}
        return {"bytes": n + T * E * size[case["d"]] + 4 * T * k + 4 * E + 12, "flops": 12 * T * E}
    b, r, c = case["batch"], case["rows"], case["cols"]
    n, m = min(r, c), max(r, c)  # X X^T and its square are symmetric: half of each
    return {"bytes": b * r * c * (size[case["x"]] + size[case["o"]]), "flops": case["steps"] * b * n * n * (3 * m + n)}


# -------------------------------------------------------------------- exact

def _exact_quantized(x):
    rows, cols = x.shape
    p = torch.nn.functional.pad(x, (0, -cols % 128)).unflatten(1, (-1, 32))
    top = p.abs().max(2).values
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    # the nearest of the type's values by its table, an even code where two are as near
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    middles, v = (table[1:] + table[:-1]) / 2, torch.ldexp(p, -e[:, :, None])
    low, high = torch.searchsorted(middles, v.abs()), torch.searchsorted(middles, v.abs(), right=True)
    q = table[torch.where(low % 2 == 0, low, high)] * torch.sign(v)
    y = torch.ldexp(q, e[:, :, None]).flatten(1)[:, :cols]
    e[:, -(-cols // 32):] = -127
    scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=x.device), e)
    return [y, scale.unflatten(1, (-1, 4)).transpose(0, 1).reshape(-1, 4 * rows)]


def _exact_values(q, words, cols):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=q.device)
    table = torch.cat((table, -table))
    v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = table[(q % 16).long()], table[(q // 16).long()]
    e = torch.stack([(words >> (8 * i)) & 255 for i in range(4)], 2).transpose(0, 1).flatten(1)
    e = e.repeat_interleave(32, 1)[:, :cols]
    return torch.ldexp(v[:, :cols], e - 127)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x = s["x"].double()
        return (_exact_quantized(x) if "rows" in s else []) + (_exact_quantized(x.t().contiguous()) if "cols" in s else [])
    if op == "gemm":
        K = case["K"]
        c = torch.matmul(_exact_values(s["A"], s["sa"], K), _exact_values(s["B"], s["sb"], K).t())
        return c if s["bias"] is None else c + s["bias"].double()
    if op in ("balance", "grad"):
        x = s["logits"].double().requires_grad_(op == "grad")
        keep = torch.ones(len(x), dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
        E, k, n = case["experts"], case["topk"], max(1, int(keep.sum()))
        score = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
        p = torch.nn.functional.normalize(score, p=1, dim=1)
        counts = torch.bincount(s["ids"][keep].long().flatten(), minlength=E)
        loss = E * torch.dot(counts.double() / (n * k), p[keep].sum(0) / n)
        z = torch.logsumexp(x, 1)[keep].square().sum() / n
        if op == "balance":
            return [torch.cat((counts, keep.sum()[None])).to(torch.int32), torch.stack((loss, z))]
        w = score.gather(1, s["ids"].long())
        if case["norm"]:
            w = w / w.sum(1, keepdim=True)
        dl = s["dlosses"].double()
        return torch.autograd.grad((w * s["dweights"].double())[keep].sum() + dl[0] * loss + dl[1] * z, x)[0]
    a, b, c = COEFFICIENTS
    x = s["G"].double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + EPS)
    if case["rows"] < case["cols"]:
        x = x.mT
    eye = torch.eye(x.shape[2], dtype=torch.float64, device="cuda")
    x = x.contiguous()
    for _ in range(case["steps"]):  # with the smaller side's products on the right
        g = torch.matmul(x.mT.contiguous(), x)
        x = torch.matmul(x, a * eye + torch.matmul(g, b * eye + c * g))
    return s["scale"] * (x.mT if case["rows"] < case["cols"] else x).contiguous()
