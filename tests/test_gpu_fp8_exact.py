"""The product of e4m3 codes on numbers whose sums are exact in fp32 in any order: every output is
the definition's, rounded once. A piece of K, a row's scale or an addend that is lost, taken twice or
taken for another's shows in every output that it belongs to."""
import pytest

from test_gpu_fp8 import ACT, B, D, F8, _full, _gen, _say, _up, moe  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [1, 2, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("N,out", [(100, "bf16"), (6128, "bf16"), (6129, "f32"), (6200, "bf16"), (14336, "bf16")])
def test_few_tokens_are_summed_exactly(moe, T, N, out):
    """Small products beside two large ones that cancel: up to 8 tokens, whatever N is, keep them.
    (Adding eight neighbouring products cut to 2^-13 of the largest loses every one of them.)"""
    _say("exact:", T, N, out)
    K, g = 272, _gen(T + N)
    x, w = torch.zeros(T, K, device="cuda"), torch.zeros(N, K, device="cuda")
    draw = lambda *n: torch.randint(-7, 8, n, device="cuda", generator=g).float() / 8  # noqa: E731
    for at in (8, 136, 264):  # in each block two large products and six small ones beside them
        x[:, at:at + 2] = 448.0
        w[:, at], w[:, at + 1] = 448.0, -448.0
        x[:, at + 2:at + 8], w[:, at + 2:at + 8] = draw(T, 6), draw(N, 6)
    sx, sw = torch.full((T, 3), 0.5, device="cuda"), torch.full((_up(N), 3), 2.0, device="cuda")
    sx[:, 1], sw[:, 2] = 2.0, 0.25
    got = torch.empty(T, N, device="cuda", dtype=ACT[out])
    moe.fp8_matmul(x.to(F8), sx, w.to(F8), sw, got)
    # multiples of 2^-9 under 2^18 + 2^6 in every partial sum
    want = _full(x.to(F8), sx) @ _full(w.to(F8), sw, B).T
    assert torch.equal(got, want.to(ACT[out])) and bool((got != 0).any())
