"""Grids of the largest sizes that the 8-bit product, its quantiser, the router and the expert layer take: a launch counts
its threads in 32 bits along x and its workgroups in 16 along y."""
import pytest

import host_util

CHECK = """
        assert launches()
        for l in launches():
            assert 0 < l.grid.x and l.grid.x * l.block.x < 1 << 32, (l.grid.x, l.block.x, T.tcm_last_plan())
            assert 0 < l.grid.y < 1 << 16 and l.grid.z == 1 and l.block.x <= 1024 and l.block.y == l.block.z == 1
"""


@pytest.mark.parametrize("tokens", [(1 << 26) - 1, 1 << 26, (1 << 26) + 5, 1 << 28, (1 << 35) + 3])
def test_router(tmp_path, tokens):
    out = host_util.run(tmp_path, f"""
        assert T.tcm_moe_route({tokens}, 4, 1, 1 << 44, 4, T.TCM_F16_F32, None, 1.0, 1 << 45, 1 << 46, None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x for l in launches()))
    """)
    assert int(out) == -(-tokens // 4)


@pytest.mark.parametrize("cols", [(1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1])
@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("tile", [0, 1])
def test_quantiser_of_long_rows(tmp_path, cols, rows, tile):
    blocks, row_blocks = -(-cols // 128), -(-rows // 128)
    out = host_util.run(tmp_path, f"""
        tile, cols, rows, blocks, row_blocks = {tile}, {cols}, {rows}, {blocks}, {row_blocks}
        dtype = T.TCM_F16_F32 | (T.TCM_BLOCK_TILE if tile else 0)
        lds, ldst = (blocks, row_blocks) if tile else (rows, cols)
        assert T.tcm_quantize_fp8(rows, cols, at(10), cols, dtype, at(11), cols, at(12), lds, at(13), rows, at(14), ldst, None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x * l.grid.y for l in launches()))
        hip.stub_clear()
        assert T.tcm_quantize_fp8(rows, cols, at(10), cols, dtype, at(11), cols, at(12), lds, None, 0, None, 0, None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x * l.grid.y for l in launches()))
    """)
    assert [int(x) for x in out.split()] == [blocks * row_blocks, blocks * (row_blocks if tile else -(-rows // 16))]


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(1024, 1 << 22, 2, 1, 1), (1024, (1 << 26) - 2, 2, 1, 1), (700, 1 << 23, 4, 7, 1),
                                                              (5000, 1 << 20, 2, 1, 1)])
def test_expert_layer_of_wide_rows(tmp_path, tokens, hidden, inter, experts, topk):
    host_util.run(tmp_path, f"""
        assert T.tcm_moe({tokens}, {hidden}, {inter}, {experts}, {topk}, at(10), {hidden}, at(11), at(12), at(13), None, at(14), None, at(15),
                         {hidden}, T.TCM_BF16_F32 | T.TCM_C_BF16, None) == T.TCM_OK
        assert "moe_tile" in T.tcm_last_plan()
        {CHECK}
        sums = launches()[2::3]
        assert sum(l.grid.x for l in sums) * 256 >= {tokens} * {hidden}
    """)


@pytest.mark.parametrize("config", [-1, 0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("split", [0, 2, 64])
@pytest.mark.parametrize("M,N", [(1 << 17, 1 << 17), ((1 << 18) - 3, 1 << 16), (1 << 12, (1 << 21) - 16), (60, (1 << 27) - 16), (1 << 20, 1 << 16)])
def test_product_of_many_tiles(tmp_path, config, split, M, N):
    host_util.run(tmp_path, f"""
        assert T.tcm_set_option("fp8_config", {config}) == T.tcm_set_option("fp8_split", {split}) == T.TCM_OK
        st = T.tcm_gemm_fp8({M}, {N}, 8192, at(10), 8192, at(11), {M}, at(12), 8192, at(13), 64, at(14), {N}, T.TCM_E4M3_F32 | T.TCM_C_BF16,
                            None, 0, None)
        assert st == T.TCM_OK or st == T.TCM_ERR_NOT_SUPPORTED and not launches(), st
        if st == T.TCM_OK:
            {CHECK.strip().replace(chr(10), chr(10) + "    ")}
    """)
