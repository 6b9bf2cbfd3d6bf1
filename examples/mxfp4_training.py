"""Training step of a routed layer in 4-bit products.

    python examples/mxfp4_training.py [--tokens 512] [--hidden 1024] [--inter 768] [--experts 16] [--topk 2]

The router's logits choose the experts (tcm_moe_route); their losses
(tcm_moe_balance) and the gradient of the weights that the layer used come back
to the logits (tcm_moe_route_grad).  One expert's matrix W then takes a step on
its tokens: x, W and dy are quantised once each, both ways from one read
(tcm_quantize_mxfp4), and multiplied three times (tcm_gemm_mxfp4): y = x W^T,
dx = dy W, dW = dy^T x.  dW goes into the momentum, and the momentum brought
near an orthogonal matrix is the update (tcm_orthogonalize).  Everything runs on
torch's current stream without a synchronisation; at the end it prints how far
each result is from the same in float32 or float64 without the 4-bit rounding.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_core_mixed_amd as T  # noqa: E402

COEFFICIENTS = (3.4445, -4.7750, 2.0315) * 5


def check(status, what):
    if status != T.TCM_OK:
        raise T.TcmError(status, what)


def stream():
    return torch.cuda.current_stream().cuda_stream


class Quantised:
    """A bf16 matrix in 4 bits as it lies (q, s) and transposed (qt, st), rows at multiples of 16 bytes."""

    def __init__(self, x):
        r, c = x.shape
        words, pitch = (lambda n: -(-n // 128)), (lambda n: -(-n // 32) * 16)
        new = lambda *s, t: torch.empty(*s, dtype=t, device=x.device)
        self.q, self.s = new(r, pitch(c), t=torch.uint8), new(words(c), r, t=torch.int32)
        self.qt, self.st = new(c, pitch(r), t=torch.uint8), new(words(r), c, t=torch.int32)
        check(T.tcm_quantize_mxfp4(r, c, x.data_ptr(), x.stride(0), T.TCM_BF16_F32, self.q.data_ptr(), self.q.stride(0), self.s.data_ptr(), r,
                                   self.qt.data_ptr(), self.qt.stride(0), self.st.data_ptr(), c, stream()), "quantize")


def product(M, N, K, a, sa, b, sb, C, flags=0, epilogue=T.TCM_EPI_NONE):
    check(T.tcm_gemm_mxfp4(M, N, K, a.data_ptr(), a.stride(0), sa.data_ptr(), M, b.data_ptr(), b.stride(0), sb.data_ptr(), N, C.data_ptr(),
                           C.stride(0), T.TCM_MXFP4_F32 | flags, None, epilogue, stream()), "gemm_mxfp4")
    return C


def layer_step(x, w, dy, grad):
    """y, dx (bf16) and the weight gradient, added to `grad` (float32)."""
    tok, din, dout = x.shape[0], w.shape[1], w.shape[0]
    X, W, G = Quantised(x), Quantised(w), Quantised(dy)
    y = product(tok, dout, din, X.q, X.s, W.q, W.s, torch.empty_like(dy), T.TCM_C_BF16)
    dx = product(tok, din, dout, G.q, G.s, W.qt, W.st, torch.empty_like(x), T.TCM_C_BF16)
    product(dout, din, tok, G.qt, G.st, X.qt, X.st, grad, 0, T.TCM_EPI_ACCUM)
    return y, dx, grad


def update(momentum, scale):
    """The momentum (float32) brought near an orthogonal matrix, bf16."""
    rows, cols = momentum.shape
    o = torch.empty(rows, cols, dtype=torch.bfloat16, device=momentum.device)
    check(T.tcm_orthogonalize(1, rows, cols, momentum.data_ptr(), momentum.stride(0), 0, o.data_ptr(), cols, 0, T.TCM_F32_F32 | T.TCM_C_BF16,
                              COEFFICIENTS, 1e-7, scale, stream()), "orthogonalize")
    return o


class Router:
    """The choice of a batch's experts, its losses, and the gradient by its logits."""

    def __init__(self, logits, topk, mask):
        self.x, self.topk, self.mask = logits, topk, mask
        tok, experts = logits.shape
        new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=logits.device)
        self.ids, self.weights = new(tok, topk, t=torch.int32), new(tok, topk)
        self.counts, self.losses = new(experts + 1, t=torch.int32), new(2)
        check(T.tcm_moe_route(tok, experts, topk, logits.data_ptr(), experts, T.TCM_F32_F32 | T.TCM_ROUTE_NORM, None, 1.0, self.ids.data_ptr(),
                              self.weights.data_ptr(), stream()), "moe_route")
        check(T.tcm_moe_balance(tok, experts, topk, logits.data_ptr(), experts, T.TCM_F32_F32, self.ids.data_ptr(), mask.data_ptr(),
                                self.counts.data_ptr(), self.losses.data_ptr(), stream()), "moe_balance")

    def gradient(self, dweights, dlosses):
        tok, experts = self.x.shape
        d = torch.empty_like(self.x)
        check(T.tcm_moe_route_grad(tok, experts, self.topk, self.x.data_ptr(), experts, T.TCM_F32_F32 | T.TCM_ROUTE_NORM, 1.0,
                                   self.ids.data_ptr(), self.mask.data_ptr(), dweights.data_ptr(), self.counts.data_ptr(), dlosses.data_ptr(),
                                   d.data_ptr(), experts, stream()), "moe_route_grad")
        return d


def relative(got, ref):
    return float((got.double() - ref.double()).norm() / ref.double().norm())


def main(argv=None):
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 512), ("hidden", 1024), ("inter", 768), ("experts", 16), ("topk", 2)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")

    logits = 2 * randn(a.tokens, a.experts)
    mask = (torch.rand(a.tokens, generator=gen, device="cuda") > 0.1).to(torch.uint8)  # (padding at 0)
    dweights, dlosses = randn(a.tokens, a.topk), torch.tensor([0.01, 0.001], device="cuda") * a.tokens
    router = Router(logits, a.topk, mask)
    dlogits = router.gradient(dweights, dlosses)

    x, w, dy = randn(a.tokens, a.hidden).bfloat16(), (randn(a.inter, a.hidden) * a.hidden ** -0.5).bfloat16(), randn(a.tokens, a.inter).bfloat16()
    momentum = randn(a.inter, a.hidden)
    before = momentum.clone()
    y, dx, momentum = layer_step(x, w, dy, momentum)
    o = update(momentum, 0.2 * max(a.inter, a.hidden) ** 0.5)
    w_new = w - 0.02 * o

    # the same in plain torch
    keep, v = mask != 0, logits.double().requires_grad_()
    share = torch.softmax(v, 1)
    chosen = share.gather(1, router.ids.long())
    n = int(keep.sum())
    counts = torch.bincount(router.ids[keep].long().flatten(), minlength=a.experts)
    balance = a.experts * (counts / (n * a.topk) * share[keep].sum(0) / n).sum()
    z = torch.logsumexp(v, 1)[keep].square().sum() / n
    total = ((chosen / chosen.sum(1, keepdim=True)) * dweights)[keep].sum() + dlosses[0] * balance + dlosses[1] * z
    m = momentum.double()
    m = m / m.norm()
    for _ in range(5):
        s = m @ m.t()
        m = COEFFICIENTS[0] * m + (COEFFICIENTS[1] * s + COEFFICIENTS[2] * (s @ s)) @ m
    errors = {"losses": relative(router.losses, torch.stack((balance, z)).detach()), "dlogits": relative(dlogits, torch.autograd.grad(total, v)[0]),
              "y": relative(y, x.float() @ w.float().t()), "dx": relative(dx, dy.float() @ w.float()),
              "dW": relative(momentum - before, dy.float().t() @ x.float()), "update": relative(o, 0.2 * max(a.inter, a.hidden) ** 0.5 * m)}
    for name, e in errors.items():
        print(f"{name:8s} relative difference from plain torch {e:.2e}", flush=True)
    assert torch.isfinite(w_new.float()).all()
    return errors


if __name__ == "__main__":
    main()
