"""The rule that chooses the e4m3 product's tile, read from its source, against the sizes that the
tests on a GPU give it: every tile in every output type is among them, cut short and whole."""
import os
import re

import pytest

pytest.importorskip("torch")
from test_gpu_fp8_exact import EXACT, TILES  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_offloaded_ffn_moe_amd", "csrc")
GEMM = open(os.path.join(CSRC, "k_fp8_gemm.hip")).read()
COSTS = [(int(t), int(c), float(v)) for t, c, v in
         re.findall(r"\{(\d+), (\d+), ([\d.]+)f\}", re.search(r"kTiles\[\] = \{(.*?)\};", GEMM, re.S).group(1))]
FEW = int(re.search(r"kSkinnyRows = (\d+);", open(os.path.join(CSRC, "k_fp8.hip")).read()).group(1))


def tile_of(T, N, bf16):
    assert T > FEW
    rounds = lambda t, c: (-(-T // t) * -(-N // c) - 1) // 256 + 1  # noqa: E731
    return min((rounds(t, c) * v, i) for i, (t, c, v) in enumerate(COSTS) if i >= (0 if bf16 else 1))[1]


def test_the_source_has_the_tiles():
    """The forms that the source builds, one for each case of its choice, are those of the table."""
    forms = re.findall(r"gemm_tile<BF16, (\d+), (\d+), (\d+), (\d+), \d+, \d+>", GEMM)
    assert [(32 * int(tm) * int(wm), 32 * int(tn) * int(wn)) for wm, wn, tm, tn in forms] == [c[:2] for c in COSTS]
    assert sorted(t[0] for t in TILES) == sorted(c[:2] for c in COSTS)


@pytest.mark.parametrize("tile,cut,whole,K", TILES)
def test_sizes_choose_the_tile(tile, cut, whole, K):
    for bf16 in (True, False):
        if bf16 or tile != COSTS[0][:2]:
            assert COSTS[tile_of(*cut, bf16)][:2] == tile and COSTS[tile_of(*whole, bf16)][:2] == tile
    assert cut[0] % tile[0] and cut[1] % tile[1] and whole[0] % tile[0] == 0 and whole[1] % tile[1] == 0
    groups = {(64, 64): 2, (64, 32): 4, (32, 32): 4}.get(tile, 1)  # of waves that take the blocks of K in turn
    assert K % 128 and (-(-K // 128)) // groups > 8


def test_every_form_is_run():
    want = {(t[0], o) for t in TILES for o in ("bf16", "f32")} - {(COSTS[0][:2], "f32")}
    for add in (True, False):
        assert {(t, o) for t, T, N, K, o, a in EXACT if a == add} == want
    for t, T, N, K, o, a in EXACT:
        assert COSTS[tile_of(T, N, o == "bf16")][:2] == t
