"""Rows longer than one launch of the quantiser takes (2^30 columns)."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, blocks, quantize

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", [False, True])
def test_columns_past_one_launch(tile):
    rows, cols = 3, (1 << 30) + 131
    near = slice((1 << 30) - 256, cols)  # both sides of the launches' border and the row's end
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(rows, cols - near.start, generator=gen).half()
    X = torch.zeros(rows, cols, dtype=torch.float16, device="cuda")
    X[:, near] = x.cuda()
    Q, QT = (torch.full(s, 0x55, dtype=torch.uint8, device="cuda") for s in ((rows, cols), (cols, rows)))
    S = torch.zeros((1, blocks(cols)) if tile else (blocks(cols), rows), device="cuda")
    ST = torch.zeros((blocks(cols), 1) if tile else (1, cols), device="cuda")
    args = lambda q, s, qt, st: (q.data_ptr(), cols, s.data_ptr(), s.shape[1]) + \
        ((qt.data_ptr(), rows, st.data_ptr(), st.shape[1]) if qt is not None else (None, 0, None, 0))
    code = T.TCM_F16_F32 | (T.TCM_BLOCK_TILE if tile else 0)
    stream = torch.cuda.current_stream().cuda_stream
    ref, rs = quantize(x, E4M3, tile)
    rt, rst = quantize(x.t().contiguous(), E4M3, tile)
    first = near.start // 128
    for transposed in (True, False):
        Q.fill_(0x55), S.zero_()
        assert T.tcm_quantize_fp8(rows, cols, X.data_ptr(), cols, code, *args(Q, S, QT if transposed else None, ST), stream) == T.TCM_OK
        assert torch.equal(Q[:, near].cpu().view(E4M3).double(), ref) and not Q[:, :near.start].any()
        s = S[:, first:] if tile else S[first:]
        assert torch.equal(s.cpu(), rs) and (S[:, :first] if tile else S[:first]).eq(2.0 ** -126).all()
    assert torch.equal(QT[near].cpu().view(E4M3).double(), rt) and not QT[:near.start].any()
    st = ST[first:] if tile else ST[:, near]
    assert torch.equal(st.cpu(), rst)
