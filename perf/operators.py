"""Cases of the 8-bit block-scaled product, its quantiser, the expert router
and the mixture-of-experts layer: inputs, plain forms and the library's calls.

A case is a dict of plain values; its "op" says which operator it runs:

  quantize  a matrix to 8-bit floats with one float32 scale for each block of
            128 values of a row ("row") or each 128 x 128 tile ("tile"), as it
            lies ("rows"), transposed ("cols"), or both from one read ("both")
  gemm      C = bias + sum over blocks b of 128 k of
            a_scale[b, m] * b_scale[..] * sum_k A[m, k] * B[n, k]
  route     the topk experts of every token and their weights, from logits
  moe       sum over a token's experts of
            weight * W2 (silu(W1_gate x) * (W1_up x))

`run` computes the plain form in 32 bits with elementary torch operations, or,
with `own`, calls the library.  Scales of 1 x 128 blocks lie block-major,
[block][row]; scales of 128 x 128 tiles lie [row tile][column tile].
"""
import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": E4M3, "e5m2": E5M2}
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
TINY = 2.0 ** -126  # the least scale: a block of zeros keeps a normal, finite one


def listed():
    return [
        # the activations of 16 decoding tokens, before a layer's product: a call bound by its latency
        dict(name="quant_rows_16", op="quantize", rows=16, cols=4096, x="bf16", q="e4m3", block="row", out="rows"),
        # a training step's activations: one read gives the forward operand and, transposed, the weight gradient's
        dict(name="quant_both_8192", op="quantize", rows=8192, cols=8192, x="bf16", q="e4m3", block="row", out="both"),
        # a layer's master weights after an optimizer step, for the forward product and (transposed) the input gradient
        dict(name="quant_weight", op="quantize", rows=4096, cols=11008, x="f32", q="e4m3", block="tile", out="both"),
        # one decoding token through a square layer
        dict(name="gemm_m1", op="gemm", M=1, N=4096, K=4096, a="e4m3", b="e4m3", c="bf16", b_block="tile", bias=False),
        # a decoding batch of odd size through a wider layer
        dict(name="gemm_m37", op="gemm", M=37, N=5120, K=8192, a="e4m3", b="e4m3", c="f16", b_block="tile", bias=True),
        # input gradient of a ragged batch: gradients in e5m2 times the transposed weight
        dict(name="gemm_dgrad", op="gemm", M=1999, N=4096, K=11008, a="e5m2", b="e4m3", c="bf16", b_block="tile", bias=False),
        # weight gradient: both operands transposed, summed over an odd number of tokens
        dict(name="gemm_wgrad", op="gemm", M=4096, N=4096, K=5003, a="e5m2", b="e4m3", c="f32", b_block="row", bias=False),
        # forward product of a large batch, the headline size of the dense products
        dict(name="gemm_8192", op="gemm", M=8192, N=8192, K=8192, a="e4m3", b="e4m3", c="bf16", b_block="tile", bias=True),
        # routing of a small decoding batch
        dict(name="route_16", op="route", tokens=16, experts=64, topk=6, x="f32", scoring="softmax", norm=True, bias=False),
        # routing of a prompt over many experts, with the selection bias that balances their load
        dict(name="route_8192", op="route", tokens=8192, experts=256, topk=8, x="f32", scoring="sigmoid", norm=True, bias=True),
        # one decoding token through a layer of 64 experts held in 8 bits
        dict(name="moe_1_e4m3", op="moe", tokens=1, hidden=2048, inter=1024, experts=64, topk=8, x="bf16", w="e4m3"),
        # a decoding batch through 16-bit experts, most of them with a token or two
        dict(name="moe_24_bf16", op="moe", tokens=24, hidden=4096, inter=1536, experts=32, topk=4, x="bf16", w="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "route", "moe"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), x=rng.choice(["f32", "f16", "bf16"]),
                    q=rng.choice(["e4m3", "e5m2"]), block=rng.choice(["row", "tile"]),
                    out=rng.choice(["rows", "cols", "both"]))
    if op == "gemm":
        # layers' sizes come in steps, token counts do not; the weight gradient sums over tokens
        grad = rng.random() < 0.3
        n, k, m = 16 * _log(rng, 8, 512), 16 * _log(rng, 8, 512), _log(rng, 1, 8192)
        if grad:
            m, k = k, m
        return dict(op=op, M=m, N=n, K=k, a=rng.choice(["e4m3", "e5m2"]), b=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    c=rng.choice(["f32", "f16", "bf16"]), b_block="row" if grad else rng.choice(["tile", "tile", "row"]),
                    bias=rng.random() < 0.5)
    if op == "route":
        experts = _log(rng, 4, 384)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, topk=rng.randint(1, min(10, experts)),
                    x=rng.choice(["f32", "f16", "bf16"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    norm=rng.random() < 0.5, bias=rng.random() < 0.5)
    experts = _log(rng, 4, 64)
    x = rng.choice(["f16", "bf16"])
    return dict(op=op, tokens=_log(rng, 1, 64), hidden=8 * _log(rng, 64, 512), inter=8 * _log(rng, 32, 192),
                experts=experts, topk=rng.randint(1, min(8, experts)), x=x, w=rng.choice([x, "e4m3"]))


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // 128)


def _pad16(n):
    return -(-n // 16) * 16


def _matrix(gen, rows, cols, t, row_spread):
    """Normal values whose rows differ in size, as activations' and gradients' do."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    if row_spread:
        x *= torch.exp(0.7 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x.to(t)


def _eight_bits(v, t):
    """v (rows, cols) with |v| at most the type's largest, in 8 bits; rows lie at a multiple of 16 bytes."""
    rows, cols = v.shape
    q = torch.zeros(rows, _pad16(cols), dtype=t, device=v.device)
    q[:, :cols] = v.to(t)
    return q[:, :cols]


def _in_row_blocks(x, t):
    """(q, scale [block][row]) of a float32 matrix."""
    rows, cols = x.shape
    nb = _blocks(cols)
    p = torch.zeros(rows, nb * 128, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, nb, 128)
    s = (p.abs().amax(2) / LARGEST[t]).clamp_min(TINY)
    return _eight_bits((p / s[:, :, None]).view(rows, -1)[:, :cols], t), s.t().contiguous()


def _in_tiles(x, t):
    """(q, scale [row tile][column tile]) of float32 matrices (..., rows, cols)."""
    rows, cols = x.shape[-2:]
    rb, cb = _blocks(rows), _blocks(cols)
    p = torch.zeros(*x.shape[:-2], rb * 128, cb * 128, device=x.device)
    p[..., :rows, :cols] = x
    p = p.view(*x.shape[:-2], rb, 128, cb, 128)
    s = (p.abs().amax((-3, -1)) / LARGEST[t]).clamp_min(TINY)
    q = (p / s[..., :, None, :, None]).view(*x.shape[:-2], rb * 128, cb * 128)[..., :rows, :cols]
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        rows, cols, q = case["rows"], case["cols"], TYPES[case["q"]]
        s["x"] = _matrix(gen, rows, cols, TYPES[case["x"]], case["block"] == "row")
        tile = case["block"] == "tile"
        if case["out"] in ("rows", "both"):
            s["q"] = _eight_bits(torch.zeros(rows, cols, device=dev), q)
            s["s"] = torch.zeros(*((_blocks(rows), _blocks(cols)) if tile else (_blocks(cols), rows)), device=dev)
        if case["out"] in ("cols", "both"):
            s["qt"] = _eight_bits(torch.zeros(cols, rows, device=dev), q)
            s["st"] = torch.zeros(*((_blocks(cols), _blocks(rows)) if tile else (_blocks(rows), cols)), device=dev)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["sa"] = _in_row_blocks(_matrix(gen, M, K, torch.float32, True), TYPES[case["a"]])
        w = _matrix(gen, N, K, torch.float32, False) * K ** -0.5
        if case["b_block"] == "row":
            s["B"], s["sb"] = _in_row_blocks(w, TYPES[case["b"]])
        else:
            q, s["sb"] = _in_tiles(w, TYPES[case["b"]])
            s["B"] = _eight_bits(q, TYPES[case["b"]])
        s["bias"] = torch.randn(N, generator=gen, device=dev) if case["bias"] else None
        s["C"] = torch.zeros(M, N, dtype=TYPES[case["c"]], device=dev)
    elif op == "route":
        T, E, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = (2 * torch.randn(T, E, generator=gen, device=dev)).to(TYPES[case["x"]])
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device=dev) if case["bias"] else None
        s["ids"] = torch.zeros(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.zeros(T, k, device=dev)
    else:
        T, H, I, E, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
        t = TYPES[case["x"]]
        s["x"] = torch.randn(T, H, generator=gen, device=dev).to(t)
        w1 = torch.randn(E, 2, I, H, generator=gen, device=dev) * H ** -0.5
        w2 = torch.randn(E, H, I, generator=gen, device=dev) * I ** -0.5
        s["s1"] = s["s2"] = None
        if case["w"] == "e4m3":
            (w1, s["s1"]), (w2, s["s2"]) = _in_tiles(w1, E4M3), _in_tiles(w2, E4M3)
        s["w1"], s["w2"] = w1.to(TYPES[case["w"]]).contiguous(), w2.to(TYPES[case["w"]]).contiguous()
        score = torch.softmax(torch.randn(T, E, generator=gen, device=dev), 1)
        weights, ids = torch.topk(score, k, dim=1)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["weights"] = (weights / weights.sum(1, keepdim=True)).contiguous()
        s["out"] = torch.zeros(T, H, dtype=t, device=dev)
    return s


# ------------------------------------------------------- the library's calls

def _own_quantize(T, s, stream):
    case, x = s["case"], s["x"]
    dtype = {"f16": T.TCM_F16_F32, "bf16": T.TCM_BF16_F32, "f32": T.TCM_F32_F32}[case["x"]]
    dtype |= (T.TCM_Q_E5M2 if case["q"] == "e5m2" else 0) | (T.TCM_BLOCK_TILE if case["block"] == "tile" else 0)
    q, qt = s.get("q"), s.get("qt")
    a = (q.data_ptr(), q.stride(0), s["s"].data_ptr(), s["s"].shape[1]) if q is not None else (None, 0, None, 0)
    b = (qt.data_ptr(), qt.stride(0), s["st"].data_ptr(), s["st"].shape[1]) if qt is not None else (None, 0, None, 0)
    st = T.tcm_quantize_fp8(case["rows"], case["cols"], x.data_ptr(), case["cols"], dtype, *a, *b, stream)
    return st, [s[n] for n in ("q", "s", "qt", "st") if n in s]


def _own_gemm(T, s, stream):
    case, A, B, sa, sb, C, bias = s["case"], s["A"], s["B"], s["sa"], s["sb"], s["C"], s["bias"]
    dtype = T.TCM_E4M3_F32 | (T.TCM_A_E5M2 if case["a"] == "e5m2" else 0) | (T.TCM_B_E5M2 if case["b"] == "e5m2" else 0)
    dtype |= {"f32": 0, "f16": T.TCM_C_F16, "bf16": T.TCM_C_BF16}[case["c"]]
    dtype |= T.TCM_B_ROW_SCALES if case["b_block"] == "row" else 0
    st = T.tcm_gemm_fp8(case["M"], case["N"], case["K"], A.data_ptr(), A.stride(0), sa.data_ptr(), sa.shape[1],
                        B.data_ptr(), B.stride(0), sb.data_ptr(), sb.shape[1], C.data_ptr(), case["N"], dtype,
                        bias.data_ptr() if bias is not None else None,
                        T.TCM_EPI_BIAS if bias is not None else T.TCM_EPI_NONE, stream)
    return st, C


def _own_route(T, s, stream):
    case, bias = s["case"], s["bias"]
    dtype = {"f16": T.TCM_F16_F32, "bf16": T.TCM_BF16_F32, "f32": T.TCM_F32_F32}[case["x"]]
    dtype |= (T.TCM_ROUTE_SIGMOID if case["scoring"] == "sigmoid" else 0) | (T.TCM_ROUTE_NORM if case["norm"] else 0)
    st = T.tcm_moe_route(case["tokens"], case["experts"], case["topk"], s["logits"].data_ptr(), case["experts"], dtype,
                         bias.data_ptr() if bias is not None else None, 1.0, s["ids"].data_ptr(),
                         s["weights"].data_ptr(), stream)
    return st, [s["ids"], s["weights"]]


def _own_moe(T, s, stream):
    case, s1, s2 = s["case"], s["s1"], s["s2"]
    dtype = (T.TCM_F16_F32 | T.TCM_C_F16) if case["x"] == "f16" else (T.TCM_BF16_F32 | T.TCM_C_BF16)
    dtype |= T.TCM_W_E4M3 if case["w"] == "e4m3" else 0
    st = T.tcm_moe(case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"], s["x"].data_ptr(),
                   case["hidden"], s["ids"].data_ptr(), s["weights"].data_ptr(), s["w1"].data_ptr(),
                   s1.data_ptr() if s1 is not None else None, s["w2"].data_ptr(),
                   s2.data_ptr() if s2 is not None else None, s["out"].data_ptr(), case["hidden"], dtype, stream)
    return st, s["out"]


OWN = {"quantize": _own_quantize, "gemm": _own_gemm, "route": _own_route, "moe": _own_moe}


# ----------------------------------------------------------- the plain forms

def _spread_tiles(s, rows, cols):
    """Tile scales (..., row tiles, column tiles) as one scale a value."""
    return s.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def _spread_rows(s, cols):
    """Row-block scales [block][row] as one scale a value, (rows, cols)."""
    return s.t().repeat_interleave(128, 1)[:, :cols]


def _round_to(v, t):
    """float64 values to the nearest of an 8-bit type's, ties to even.  (A conversion would round to 32 bits on its
    way, onto ties that the values only lie next to.)"""
    bits, least = (3, -6) if t == E4M3 else (2, -14)
    power = (v.view(torch.int64) & (0x7FF << 52)).view(torch.float64).clamp_min(2.0 ** least)  # 2^floor(log2 |v|)
    big = power * (1.5 * 2.0 ** (52 - bits))  # a sum with it keeps the type's bits of v and no more
    return (v + big - big).float()


def _plain_quantize(s):
    case, t = s["case"], TYPES[s["case"]["q"]]
    out = []
    for x in ([s["x"]] if case["out"] != "cols" else []) + ([s["x"].t()] if case["out"] != "rows" else []):
        rows, cols = x.shape
        br, rb, cb = (128, _blocks(rows), _blocks(cols)) if case["block"] == "tile" else (1, rows, _blocks(cols))
        p = torch.zeros(rb * br, cb * 128, dtype=torch.float64, device=x.device)  # quotients next to a tie: 64 bits
        p[:rows, :cols] = x
        p = p.view(rb, br, cb, 128)
        scale = (p.abs().amax((1, 3)) / LARGEST[t]).float().clamp_min(TINY)
        q = _round_to((p / scale.double()[:, None, :, None]).view(rb * br, -1)[:rows, :cols], t)
        out += [_eight_bits(q, t), scale if case["block"] == "tile" else scale.t().contiguous()]
    return out


def _plain_gemm(s):
    case, M, N, K = s["case"], s["case"]["M"], s["case"]["N"], s["case"]["K"]
    a = s["A"].float() * _spread_rows(s["sa"], K)
    b = s["B"].float() * (_spread_rows(s["sb"], K) if case["b_block"] == "row" else _spread_tiles(s["sb"], N, K))
    c = a @ b.t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return c.to(TYPES[case["c"]])


def _plain_route(s):
    case, k = s["case"], s["case"]["topk"]
    x = s["logits"].double()  # the choice among near scores: 64 bits
    if case["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    key = score + s["bias"].double() if s["bias"] is not None else x  # both scores rise with x
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(score, 1, ids)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True)
    return [ids.to(torch.int32), w.float()]


def _plain_moe(s):
    case, T, E = s["case"], s["case"]["tokens"], s["case"]["experts"]
    H, I = case["hidden"], case["inter"]
    w1, w2 = s["w1"].float(), s["w2"].float()
    if s["s1"] is not None:
        w1, w2 = w1 * _spread_tiles(s["s1"], I, H), w2 * _spread_tiles(s["s2"], H, I)
    g = (s["x"].float() @ w1.view(E * 2 * I, H).t()).view(T, E, 2, I)
    h = g[:, :, 0] / (1 + torch.exp(-g[:, :, 0])) * g[:, :, 1]
    here = (s["ids"].long()[:, :, None] == torch.arange(E, device=w1.device)).float() * s["weights"][:, :, None]
    h = h * here.sum(1)[:, :, None]  # every expert's share of every token, zero where it has none
    y = torch.bmm(h.transpose(0, 1).contiguous(), w2.transpose(1, 2).contiguous())
    return y.sum(0).to(TYPES[case["x"]])


PLAIN = {"quantize": _plain_quantize, "gemm": _plain_gemm, "route": _plain_route, "moe": _plain_moe}


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
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
    op = case["op"]
    if op == "quantize":
        n, r, c = case["rows"] * case["cols"], case["rows"], case["cols"]
        one = _blocks(r) * _blocks(c)
        outs = (["rows"] if case["out"] != "cols" else []) + (["cols"] if case["out"] != "rows" else [])
        scales = sum(one if case["block"] == "tile" else (r * _blocks(c) if o == "rows" else c * _blocks(r)) for o in outs)
        return {"bytes": n * size[case["x"]] + len(outs) * n + 4 * scales, "flops": 2 * n * len(outs)}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = M * _blocks(K) + (N if case["b_block"] == "row" else _blocks(N)) * _blocks(K)
        return {"bytes": M * K + N * K + M * N * size[case["c"]] + 4 * scales + 4 * N * case["bias"], "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": T * E * size[case["x"]] + 8 * T * k + 4 * E * case["bias"], "flops": 5 * T * E}
    T, H, I, E, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
    weights = used * 3 * I * H * size[case["w"]]
    scales = used * 4 * 3 * _blocks(I) * _blocks(H) if case["w"] == "e4m3" else 0
    return {"bytes": weights + scales + 2 * 2 * T * H + 8 * T * k, "flops": 2 * T * k * 3 * I * H}


# -------------------------------------------------------------------- exact

def _exact_scaled(x, t, block):
    """Every value's scale and quotient in 64 bits; the scale is held in 32."""
    rows, cols = x.shape
    br = 128 if block == "tile" else 1
    mag = torch.nn.functional.pad(x.abs(), (0, -cols % 128, 0, -rows % br))
    s = mag.reshape(-(-rows // br), br, -(-cols // 128), 128).permute(0, 2, 1, 3).flatten(2).max(2).values
    s = torch.clamp((s / LARGEST[t]).float(), min=TINY)
    each = torch.kron(s.double(), torch.ones(br, 128, dtype=torch.float64, device=x.device))[:rows, :cols]
    # the nearest of the type's values by its table, an even code where two are as near
    codes = torch.arange(127 if t == E4M3 else 124, dtype=torch.uint8, device=x.device)
    values = codes.view(t).double()
    middles, v = (values[1:] + values[:-1]) / 2, x / each
    low, high = torch.searchsorted(middles, v.abs()), torch.searchsorted(middles, v.abs(), right=True)
    q = values[torch.where(low % 2 == 0, low, high)] * torch.where(v < 0, -1.0, 1.0)
    return q.to(t), s if block == "tile" else s.t().contiguous()


def _exact_dequantized(q, s, block):
    rows, cols = q.shape
    s = s.double() if block == "tile" else s.double().t()
    ones = torch.ones(128 if block == "tile" else 1, 128, dtype=torch.float64, device=q.device)
    return q.double() * torch.kron(s.contiguous(), ones)[:rows, :cols]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x, t = s["x"].double(), TYPES[case["q"]]
        out = []
        if case["out"] in ("rows", "both"):
            out += _exact_scaled(x, t, case["block"])
        if case["out"] in ("cols", "both"):
            out += _exact_scaled(x.t().contiguous(), t, case["block"])
        return out
    if op == "gemm":
        c = torch.matmul(_exact_dequantized(s["A"], s["sa"], "row"), _exact_dequantized(s["B"], s["sb"], case["b_block"]).t())
        return c if s["bias"] is None else c + s["bias"].double()
    if op == "route":
        x, k = s["logits"].double(), case["topk"]
        score = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
        key = x if s["bias"] is None else score + s["bias"].double()
        ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
        w = score.gather(1, ids)
        return [ids.to(torch.int32), w / w.sum(1, keepdim=True) if case["norm"] else w]
    out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not len(token):
            continue
        gate, up, down = s["w1"][e, 0].double(), s["w1"][e, 1].double(), s["w2"][e].double()
        if s["s1"] is not None:
            gate, up = (_exact_dequantized(w, s["s1"][e, i], "tile") for i, w in enumerate((s["w1"][e, 0], s["w1"][e, 1])))
            down = _exact_dequantized(s["w2"][e], s["s2"][e], "tile")
        x = s["x"][token].double()
        h = torch.nn.functional.silu(x @ gate.t()) * (x @ up.t())
        out.index_add_(0, token, s["weights"][token, slot].double()[:, None] * (h @ down.t()))
    return out
