"""Sizes and strides whose products do not fit 64 bits are refused by the C
entry points, not wrapped around. No GPU needed."""
from test_ops_host import INVALID, P, Q, R, S, W, dg, fn, gemm      # noqa: F401

BIG = (1 << 31) - 5000
FAR = 1 << 36


def test_scales_beyond_the_addresses(fn):
    for bad in (dict(sr=1 << 62), dict(sk=1 << 62), dict(sr=(1 << 63) - 1), dict(sr=1 << 60, sk=1 << 60), dict(M=BIG, sr=1 << 40)):
        assert gemm(fn, **bad) == INVALID, bad


def test_rows_beyond_the_addresses(fn):
    gather = fn("det_moe_gather")
    assert gather(P, Q, R, BIG, 8, 64, 1, FAR, 64, None) == INVALID
    assert gather(P, Q, R, 4, BIG, 64, 1, 64, FAR, None) == INVALID
    rows = fn("det_fp8_quantize_rows")
    assert rows(P, None, Q, R, BIG, BIG, 256, 1, FAR, 256, BIG, None) == INVALID
    tiles = fn("det_fp8_quantize_tiles")
    assert tiles(P, Q, R, None, None, 1 << 30, 64, 64, 64, 1 << 40, 64, 4096, 64, 4096, None) == INVALID
    assert tiles(P, Q, R, None, None, 1 << 30, 64, 64, 64, 4096, 64, 1 << 40, 64, 4096, None) == INVALID


def test_blocks_of_any_bounds_are_counted(fn):
    wgrad = fn("det_fp8_gemm_wgrad")
    M, nb = 1 << 30, (1 << 23) + 512
    ld = nb * 128
    assert wgrad(P, Q, R, S, W, 2 * W, 0, 512, M, 16, 16, nb, ld, 16, ld, 16, 16, 256, None) == INVALID
