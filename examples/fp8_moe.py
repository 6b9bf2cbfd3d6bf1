"""8-bit training step of a linear layer and a mixture-of-experts decoding step.

    python examples/fp8_moe.py [--tokens 512] [--hidden 2048] [--inter 1024] [--experts 32] [--topk 4] [--batch 8]

The training step quantises x, W and dy once each (tcm_quantize_fp8, both
ways from one read) and multiplies them three times (tcm_gemm_fp8): y = x W^T,
dx = dy W, dW += dy^T x.  The decoding step routes a batch of tokens
(tcm_moe_route) and runs the layer of experts held in 8 bits (tcm_moe).  Both
print how far they are from the same in float32 without the 8-bit rounding.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_core_mixed_amd as T  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def blocks(n):
    return -(-n // 128)


def check(status, what):
    if status != T.TCM_OK:
        raise T.TcmError(status, what)


def stream():
    return torch.cuda.current_stream().cuda_stream


class Quantised:
    """A bf16 matrix in 8 bits as it lies (q, s) and transposed (qt, st), rows at multiples of 16 bytes."""

    def __init__(self, x, t, tile):
        r, c = x.shape
        pad = lambda n: -(-n // 16) * 16
        self.rows, self.cols = r, c
        self.q, self.qt = torch.empty(r, pad(c), dtype=t, device=x.device), torch.empty(c, pad(r), dtype=t, device=x.device)
        self.s = torch.empty((blocks(r), blocks(c)) if tile else (blocks(c), r), device=x.device)
        self.st = torch.empty((blocks(c), blocks(r)) if tile else (blocks(r), c), device=x.device)
        code = T.TCM_BF16_F32 | (T.TCM_Q_E5M2 if t == E5M2 else 0) | (T.TCM_BLOCK_TILE if tile else 0)
        check(T.tcm_quantize_fp8(r, c, x.data_ptr(), x.stride(0), code, self.q.data_ptr(), self.q.stride(0), self.s.data_ptr(),
                                 self.s.shape[1], self.qt.data_ptr(), self.qt.stride(0), self.st.data_ptr(), self.st.shape[1], stream()),
              "quantize")


def product(M, N, K, a, sa, b, sb, C, flags, epilogue=T.TCM_EPI_NONE, bias=None):
    check(T.tcm_gemm_fp8(M, N, K, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.shape[1], b.data_ptr(), b.stride(0), sb.data_ptr(),
                         sb.shape[1], C.data_ptr(), C.stride(0), T.TCM_E4M3_F32 | flags, bias.data_ptr() if bias is not None else None,
                         epilogue, stream()), "gemm_fp8")
    return C


def training_step(x, w, dy, grad):
    """y, dx (bf16) and the weight gradient, added to `grad` (float32)."""
    tok, din, dout = x.shape[0], w.shape[1], w.shape[0]
    X, W, G = Quantised(x, E4M3, False), Quantised(w, E4M3, True), Quantised(dy, E5M2, False)
    y = product(tok, dout, din, X.q, X.s, W.q, W.s, torch.empty_like(dy), T.TCM_C_BF16)
    dx = product(tok, din, dout, G.q, G.s, W.qt, W.st, torch.empty_like(x), T.TCM_A_E5M2 | T.TCM_C_BF16)
    product(dout, din, tok, G.qt, G.st, X.qt, X.st, grad, T.TCM_A_E5M2 | T.TCM_B_ROW_SCALES, T.TCM_EPI_ACCUM)
    return y, dx, grad


def quantise_experts(w):
    """(..., rows, cols) bf16 expert weights in e4m3 with tile scales, as tcm_moe takes them."""
    rows, cols = w.shape[-2:]
    q = torch.empty(w.shape, dtype=E4M3, device=w.device)
    s = torch.empty(*w.shape[:-2], blocks(rows), blocks(cols), device=w.device)
    for m, qm, sm in zip(w.reshape(-1, rows, cols), q.view(-1, rows, cols), s.view(-1, blocks(rows), blocks(cols))):
        check(T.tcm_quantize_fp8(rows, cols, m.data_ptr(), cols, T.TCM_BF16_F32 | T.TCM_BLOCK_TILE, qm.data_ptr(), cols, sm.data_ptr(),
                                 sm.shape[1], None, 0, None, 0, stream()), "quantize")
    return q, s


def decoding_step(x, gate, w1, s1, w2, s2, topk):
    """The expert layer of a batch of tokens; `gate` is the router's matrix."""
    tok, hidden = x.shape
    experts, _, inter, _ = w1.shape
    logits = (x.float() @ gate.float().t()).contiguous()
    ids = torch.empty(tok, topk, dtype=torch.int32, device=x.device)
    weights = torch.empty(tok, topk, device=x.device)
    check(T.tcm_moe_route(tok, experts, topk, logits.data_ptr(), experts, T.TCM_F32_F32 | T.TCM_ROUTE_NORM, None, 1.0, ids.data_ptr(),
                          weights.data_ptr(), stream()), "moe_route")
    out = torch.empty_like(x)
    check(T.tcm_moe(tok, hidden, inter, experts, topk, x.data_ptr(), x.stride(0), ids.data_ptr(), weights.data_ptr(), w1.data_ptr(),
                    s1.data_ptr(), w2.data_ptr(), s2.data_ptr(), out.data_ptr(), out.stride(0),
                    T.TCM_BF16_F32 | T.TCM_C_BF16 | T.TCM_W_E4M3, stream()), "moe")
    return out, ids, weights


def relative(got, ref):
    return float((got.float() - ref).norm() / ref.norm())


def main(argv=None):
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 512), ("hidden", 2048), ("inter", 1024), ("experts", 32), ("topk", 4), ("batch", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")

    x, w, dy = randn(a.tokens, a.hidden).bfloat16(), (randn(a.inter, a.hidden) * a.hidden ** -0.5).bfloat16(), randn(a.tokens, a.inter).bfloat16()
    y, dx, dw = training_step(x, w, dy, torch.zeros(a.inter, a.hidden, device="cuda"))
    errors = {"y": relative(y, x.float() @ w.float().t()), "dx": relative(dx, dy.float() @ w.float()),
              "dW": relative(dw, dy.float().t() @ x.float())}

    x = randn(a.batch, a.hidden).bfloat16()
    gate = randn(a.experts, a.hidden) * a.hidden ** -0.5
    e1 = (randn(a.experts, 2, a.inter, a.hidden) * a.hidden ** -0.5).bfloat16()
    e2 = (randn(a.experts, a.hidden, a.inter) * a.inter ** -0.5).bfloat16()
    (w1, s1), (w2, s2) = quantise_experts(e1), quantise_experts(e2)
    out, ids, weights = decoding_step(x, gate, w1, s1, w2, s2, a.topk)
    ref = torch.zeros(a.batch, a.hidden, device="cuda")
    for t in range(a.batch):
        for j in range(a.topk):
            e = int(ids[t, j])
            g, u = e1[e, 0].float() @ x[t].float(), e1[e, 1].float() @ x[t].float()
            ref[t] += weights[t, j] * (e2[e].float() @ (g / (1 + torch.exp(-g)) * u))
    errors["experts"] = relative(out, ref)
    for name, e in errors.items():
        print(f"{name:8s} relative difference from float32 {e:.4f}", flush=True)
    return errors


if __name__ == "__main__":
    main()
