"""CPU-only: the pitches that products with an epilogue take."""
from test_act_host import STRIDE, mx


def test_gated_results_at_any_pitch_that_plain_ones_may_have():
    for gated, ld_pre in ((0, 128), (1, 256)):
        empty = dict(gated=gated, M=0, res=None, pre=None, ld_pre=ld_pre)
        for ldc in (128, 129, 256, 1 << 20, (1 << 24) - 128, (1 << 24) - 127, 1 << 24):
            assert mx(ldc=ldc, **empty) == 0, (gated, ldc)
        for ldc in (-1, 0, 127, (1 << 24) + 1, 1 << 40, (1 << 63) - 1):
            assert mx(ldc=ldc, **empty) == STRIDE, (gated, ldc)
