"""The layer on e4m3 blocks at the borders of the rules that choose its second half's form, each form
with more assignments than LDS has places for among them."""
import pytest

import test_gpu_fp8 as base
from test_gpu_fp8 import moe  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [
    # T, H, I, E, k, act, pad, wide
    (2, 2048, 512, 8, 2, "bf16", 0, False), (2, 2064, 512, 8, 2, "bf16", 0, False), (16, 2048, 400, 20, 5, "f32", 1, True),
    (16, 2064, 384, 20, 5, "f32", 0, True), (1, 2032, 256, 9, 3, "bf16", 0, False), (3, 2080, 272, 9, 3, "bf16", 3, False),
    (64, 1040, 512, 40, 32, "bf16", 0, True), (64, 2048, 640, 33, 32, "f32", 0, False), (40, 2048, 2048, 36, 32, "f32", 0, False),
    (64, 2064, 512, 40, 32, "bf16", 0, False), (33, 2064, 2048, 12, 8, "bf16", 0, True), (48, 400, 1920, 34, 32, "bf16", 0, False),
    (1, 1024, 4096, 8, 1, "bf16", 0, False), (64, 512, 272, 1, 1, "bf16", 0, False), (64, 4112, 144, 2, 2, "f32", 0, False),
]


@pytest.mark.parametrize("T,H,I,E,k,act,pad,wide", FORMS)
def test_layer_forms(moe, T, H, I, E, k, act, pad, wide):  # noqa: E741, F811
    base.test_layer(moe, T, H, I, E, k, act, pad, wide)
