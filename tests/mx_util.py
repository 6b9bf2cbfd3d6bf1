"""References in 64 bits and error bounds for the 4-bit product and its quantiser."""
import torch

import tensor_core_mixed_amd as T

X_CODE = {torch.float16: T.TCM_F16_F32, torch.bfloat16: T.TCM_BF16_F32, torch.float32: T.TCM_F32_F32}
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def words(n):
    return -(-n // 128)


def nbytes(n):
    return -(-n // 2)


def quantize(x):
    """(codes uint8 (rows, cols), scale bytes int64 (rows, 4 words)) of a CPU matrix."""
    rows, cols = x.shape
    p = torch.zeros(rows, words(cols) * 128, dtype=torch.float64)
    p[:, :cols] = x.double()
    p = p.view(rows, -1, 32)
    amax = p.abs().amax(2)  # (a NaN passes)
    bad = ~torch.isfinite(amax)
    e = torch.where(bad | (amax == 0), torch.tensor(-127), torch.frexp(torch.where(bad, 0.0, amax)).exponent - 3).clamp(-127, 127)
    v = torch.where(bad[:, :, None], 0.0, p) * torch.exp2(-e.double())[:, :, None]
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    a = v.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    code = torch.where(lo % 2 == 0, lo, hi) + 8 * torch.signbit(v)
    e = torch.where(bad, 255, e + 127)
    e[:, -(-cols // 32):] = 0  # blocks past the last column
    return code.view(rows, -1)[:, :cols].to(torch.uint8), e


def pack(codes, ld, fill=0xAA):
    """Codes (rows, cols) two a byte in a (rows, ld) buffer of `fill`; an odd row's last half byte is zero."""
    rows, cols = codes.shape
    p = torch.zeros(rows, 2 * nbytes(cols), dtype=torch.uint8)
    p[:, :cols] = codes
    buf = torch.full((rows, ld), fill, dtype=torch.uint8)
    buf[:, :nbytes(cols)] = p[:, 0::2] | p[:, 1::2] << 4
    return buf


def scale_words(e, ld, fill=-1):
    """Scale bytes (rows, 4 words) as words [word][row], in rows of ld."""
    rows = e.shape[0]
    buf = torch.full((max(e.shape[1] // 4, 1), ld), fill, dtype=torch.int32)
    if e.shape[1]:
        buf[:, :rows] = e.to(torch.uint8).contiguous().view(torch.int32).t()
    return buf


def values(codes, e):
    """What codes (rows, cols) and scale bytes stand for, float64; NaN under a scale of 255."""
    cols = codes.shape[1]
    v = torch.cat((VALUES, -VALUES))[codes.long()]
    s = torch.where(e == 255, torch.nan, torch.exp2((e - 127).double()))
    return v * s.repeat_interleave(32, 1)[:, :cols]


def operand(gen, rows, K, spread):
    """(codes, scale bytes) of a matrix with every code, and scales of 2^-spread .. 2^spread."""
    codes = torch.randint(0, 16, (rows, K), generator=gen, dtype=torch.uint8)
    e = 127 + torch.randint(-spread, spread + 1, (rows, 4 * words(K)), generator=gen)
    return codes, e


def gemm_ref(a, ea, b, eb, bias=None, c_in=None, relu=False):
    """(C, error bound of binary32 accumulation) in float64, CPU.

    The bound: a block's products are summed exactly; each scaled block, the bias and C_in lose at most one unit of
    2^-23 of the sum of magnitudes as they are added."""
    x, y = values(a, ea), values(b, eb)
    c, m = x @ y.t(), x.abs() @ y.abs().t()
    init = torch.zeros_like(c)
    mag = m
    for t in (bias, c_in):
        if t is not None:
            init = init + t.double()
            mag = mag + t.double().abs()
    c = c + init
    return (c.clamp_min(0) if relu else c), (-(-a.shape[1] // 32) + 3) * 2.0 ** -23 * mag
