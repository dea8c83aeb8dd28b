"""Which tiling of the W4A4 product each shape of the GPU tests takes (no GPU needed): the cost table and the rule are read
from the source and worked out here, so that a change of either that leaves a tiling untested is seen."""
import math
import re
from pathlib import Path

import pytest

from test_gpu_mx4 import SHAPES, WIDE_SHAPES

SOURCE = (Path(__file__).resolve().parent.parent / "gemm_w4a16_amd" / "csrc" / "w4a4.hip").read_text()
TILES = {m[1]: tuple(int(v) for v in m[2].split(",")) for m in re.finditer(r"using (T\d+x\d+) = Tiling<([\d, ]+)>;", SOURCE)}
COSTS = [(m[1], *(float(v) for v in m[2].split(","))) for m in re.finditer(r"f\(\d, (T\d+x\d+)\{\}, Cost\{([\d., ]+)\}\);", SOURCE)]


def tiling(M, N, K):
    """The name of the tiling that M > 16 rows take."""
    best = None
    for name, us_ktile, us_first, next_ktile, us_next, blocks in COSTS:
        WM, WN, WK, TM, TN, _ = TILES[name]
        BM, BN = 16 * TM * WM, 16 * TN * WN
        tiles = -(-N // BN) * -(-M // BM)
        if tiles >= 2 ** 31 // (64 * WM * WN * WK):
            continue
        waves, ktiles, slots = tiles / 256, -(-K // 256), 256 * blocks
        up = math.ceil(waves)
        rounds = up if blocks == 1 else 1.0 if waves <= 1 else max(waves, 0.9 * up)
        work = ktiles * us_ktile + us_first + (rounds - 1) * (ktiles * next_ktile + us_next)
        stream = N * K * 17 / 32 / 5.6e6 * (1 + 0.2 * slots / tiles if tiles > slots else 1)
        us = math.hypot(work, stream)
        if best is None or us < best[0]:
            best = us, name
    return best[1]


def test_the_table_is_read():
    assert len(TILES) == 7 and {c[0] for c in COSTS} == set(TILES) and all(len(c) == 6 for c in COSTS)


@pytest.mark.parametrize("name", sorted(TILES))
def test_every_tiling_is_tested(name):
    """... with K of whole k-tiles of 256, and with the last one up to and past its first half."""
    mine = [s for s in SHAPES + WIDE_SHAPES if s[0] > 16 and tiling(*s) == name]
    assert any(0 < K % 256 <= 128 for _, _, K in mine) and any(K % 256 > 128 for _, _, K in mine)
    assert any(K % 256 == 0 for _, _, K in mine)
    assert any(M % 16 for M, _, _ in mine) and any(N % 16 for _, N, _ in mine)
