"""The most rows the experts' calls take: row numbers are 32-bit and pass the
last row by up to a block of row tiles, so the calls refuse the last 2^16 of
the 31-bit range.  Host checks alone: nothing is launched."""
import pytest

from test_experts_abi import B, backward_args, change, product_args  # noqa: F401  (B is a fixture)

LIMIT = (1 << 31) - (1 << 16)


@pytest.mark.parametrize("rows", [LIMIT + 1, (1 << 31) - 256, (1 << 31) - 64, (1 << 31) - 1])
def test_rows_at_the_end_of_the_32_bit_range_are_refused(B, rows):  # noqa: F811
    lib = B.library()
    for dtype in (0, 1):
        fp8 = dict(dtype=1, K=128, N=128, x_sf=product_args()["x"], w_sf=product_args()["w"]) if dtype else {}
        assert lib.ep_expert_gemm(*change(product_args(), rows=rows, **fp8)) == B.EP_ERR_UNSUPPORTED
    for act in (0, 4):
        assert lib.ep_expert_gemm_backward(*change(backward_args(), rows=rows, act=act,
                                                   ws_bytes=1 << 50)) == B.EP_ERR_UNSUPPORTED


def split(count, tile_rows, step):
    """Rows of each tile of an expert with `count` rows, as the kernels share them, and the largest number met."""
    n = (count + tile_rows - 1) // tile_rows
    even = ((count - 1) // n + step) // step * step
    per = even if (n - 1) * even < count else tile_rows
    return n, per, max(count + tile_rows - 1, (count - 1) // n + step, (n - 1) * even, (n - 1) * per + tile_rows,
                       n * per)


@pytest.mark.parametrize("tile_rows,step", [(64, 16), (128, 16), (256, 32)])
def test_the_split_into_tiles_stays_within_32_bits(tile_rows, step):
    for count in list(range(1, 3000)) + [LIMIT - i for i in range(600)] + [LIMIT // 3, 1 << 30, (1 << 30) + 1]:
        n, per, largest = split(count, tile_rows, step)
        assert largest < 1 << 31
        assert per <= tile_rows and (n - 1) * per < count <= n * per
        # what it has always been
        even = ((count + n - 1) // n + step - 1) // step * step
        assert per == (even if (n - 1) * even < count else tile_rows)
