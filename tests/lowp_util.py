"""References in 64 bits and error bounds for the 8-bit product, its quantiser, the router and the expert layer."""
import torch

import tensor_core_mixed_amd as T

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
X_CODE = {torch.float16: T.TCM_F16_F32, torch.bfloat16: T.TCM_BF16_F32, torch.float32: T.TCM_F32_F32}


def blocks(n):
    return -(-n // 128)


def values(t):
    """The finite non-negative values of an 8-bit type in the order of their codes."""
    codes = torch.arange(127 if t == E4M3 else 124, dtype=torch.uint8)
    return codes.view(t).double()


def nearest(v, t):
    """float64 values to the nearest of the type's, ties to the even code; NaN stays."""
    tab = values(t)
    mid = (tab[1:] + tab[:-1]) / 2
    a = v.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    q = tab[torch.where(lo % 2 == 0, lo, hi).clamp(max=len(tab) - 1)] * torch.where(v < 0, -1.0, 1.0).double()
    return torch.where(v.isnan(), v, q)


def quantize(x, t, tile):
    """(values q in float64, scales as the library lays them) of a CPU matrix."""
    rows, cols = x.shape
    br = 128 if tile else 1
    p = torch.zeros(-(-rows // br) * br, blocks(cols) * 128, dtype=torch.float64)
    p[:rows, :cols] = x.double()
    amax = p.view(-1, br, blocks(cols), 128).abs().amax((1, 3))  # (a NaN passes)
    s = (amax / LARGEST[t]).float()
    s = torch.where(s < 2.0 ** -126, torch.tensor(2.0 ** -126), s)
    each = s.double().repeat_interleave(br, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return nearest(x.double() / each, t), s if tile else s.t().contiguous()


def spread(s, rows, cols, tile):
    """Scales as laid out -> one per value of the (rows, cols) matrix."""
    if tile:
        return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return s.t().repeat_interleave(128, 1)[:, :cols]


def gemm_ref(A, sa, B, sb, b_row, bias=None, c_in=None, relu=False):
    """(C, error bound of binary32 accumulation) in float64, CPU.

    The bound: a block's 128 products are exact and their sum loses at most one unit of 2^-23 of the sum of magnitudes
    an addition; the scales' product, its multiplication and each block's addition to the accumulator lose one more each."""
    M, K = A.shape
    N = B.shape[0]
    a = A.double() * spread(sa, M, K, False).double()
    b = B.double() * spread(sb, N, K, not b_row).double()
    c, m = a @ b.t(), a.abs() @ b.abs().t()
    init = torch.zeros(M, N, dtype=torch.float64)
    if bias is not None:
        init = init + bias.double()
    if c_in is not None:
        init = init + c_in.double()
    bound = (min(K, 128) + blocks(K) + 4) * 2.0 ** -23 * (m + init.abs())
    c = c + init
    return (c.clamp_min(0) if relu else c), bound


def half_step(ref, t):
    """Half a step of a rounding to type t, also below its normal range."""
    if t == torch.float32:
        return torch.zeros_like(ref)
    f = torch.finfo(t)
    return ref.abs().clamp_min(f.smallest_normal) * f.eps / 2


def check_close(got, ref, bound):
    got = got.double()
    # a value may round across to the next step: the bound itself scales the half step
    bad = (got - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off; worst {((got - ref).abs() / bound.clamp_min(1e-300)).max():.3f} of the bound"


def padded(q, ld, t):
    """q (rows, cols) in type t inside a (rows, ld) buffer whose other bytes are NaN codes."""
    rows, cols = q.shape
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8)
    buf[:, :cols] = q.to(t).contiguous().view(torch.uint8)
    return buf


def moe_ref(x, ids, weights, w1, s1, w2, s2):
    """(out, bound) in float64 on the CPU.

    The bound: g and u are binary32 sums of `hidden` terms, silu changes by at most 1.1 of its argument's error, the
    product and its weighting lose eight units of 2^-24 and the 16-bit parts 2^-16; the second sum has `inter` terms a
    slot, and topk slots."""
    T_, H = x.shape
    E, _, I, _ = w1.shape
    out = torch.zeros(T_, H, dtype=torch.float64)
    bound = torch.zeros(T_, H, dtype=torch.float64)
    x = x.double()
    for t in range(T_):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            g_w, u_w, d_w = w1[e, 0].double(), w1[e, 1].double(), w2[e].double()
            if s1 is not None:
                g_w, u_w = g_w * spread(s1[e, 0].double(), I, H, True), u_w * spread(s1[e, 1].double(), I, H, True)
                d_w = d_w * spread(s2[e].double(), H, I, True)
            g, u = g_w @ x[t], u_w @ x[t]
            dg = (H + 8) * 2.0 ** -23 * (g_w.abs() @ x[t].abs())
            du = (H + 8) * 2.0 ** -23 * (u_w.abs() @ x[t].abs())
            silu = g / (1 + torch.exp(-g))
            w = float(weights[t, j])
            h = w * silu * u
            dh = abs(w) * (1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du) + h.abs() * (2.0 ** -16 + 8 * 2.0 ** -24)
            out[t] += d_w @ h
            bound[t] += d_w.abs() @ dh + (I + 8 + ids.shape[1]) * 2.0 ** -23 * (d_w.abs() @ h.abs())
    return out, bound
