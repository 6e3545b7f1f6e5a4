"""Sizes of microscaled matrices, on the host alone."""
import pytest


@pytest.fixture(scope="module")
def B():
    from eagle_feature_level_gb300.build import build
    build()
    from eagle_feature_level_gb300 import _binding
    return _binding


@pytest.mark.parametrize("fmt,block,bits", [("MX_FP8", 32, 8), ("MX_FP4", 32, 4), ("NV_FP4", 16, 4)])
def test_layout(B, fmt, block, bits):
    for rows in (1, 127, 128, 129, 1000, 1 << 20):
        for cols in (32, 64, 96, 128, 160, 4096, 11008):
            data, scale = B.eagle_mx_layout(getattr(B, fmt), rows, cols)
            groups = -(-rows // 128) * -(-(cols // block) // 4)
            assert (data, scale) == (rows * cols * bits // 8, groups * 512)
    data, scale = B.eagle_mx_layout(getattr(B, fmt), B.EAGLE_MAX_EXTENT, B.EAGLE_MAX_EXTENT)   # 64 bits throughout
    assert data == (1 << 60) * bits // 8 and scale == (1 << 60) // block


def test_layout_refuses(B):
    most = B.EAGLE_MAX_EXTENT
    for bad in ((0, 4, 64), (4, 4, 64), (1, 0, 64), (1, 4, 0), (1, 4, 40), (1, -1, 64), (1, 4, -32), (1, most + 1, 64),
                (1, 4, most + 32)):
        with pytest.raises(B.EagleError):
            B.eagle_mx_layout(*bad)
