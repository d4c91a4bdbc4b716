"""The product of e4m3 codes on numbers whose sums are exact in fp32 in any order: every output is
the definition's, rounded once. A piece of K, a row's scale or an addend that is lost, taken twice or
taken for another's shows in every output that it belongs to."""
import pytest

from test_gpu_fp8 import ACT, B, D, F8, R32, Padded, _codes, _full, _gen, _normal, _product_tolerance, _rn, _say, _up, moe  # noqa: F401

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


# Every tile in both output types: cut short in tokens, channels and the last block of K, and whole; as
# many steps as leave the loop at each of its exits, and several rounds of scales in each group
# of waves. test_fp8_tiles_cpu.py holds the list to the rule that chooses the tile.
# tile (tokens, channels), cut short T, N, whole T, N, K of many steps
TILES = [((32, 32), (27, 4001), (32, 4096), 4624), ((64, 32), (61, 5003), (64, 5120), 4624), ((64, 64), (125, 5003), (128, 5120), 4112),
         ((64, 128), (253, 5003), (256, 5120), 2064), ((128, 128), (509, 5003), (512, 5120), 2064), ((128, 256), (1021, 5003), (1024, 5120), 2064)]
EXACT = []
for _tile, _cut, _whole, _K in TILES:
    for _out in ("bf16", "f32"):
        if _tile != (128, 256) or _out == "bf16":  # fp32 outputs have no such tile
            EXACT += [(_tile, *_cut, _K, _out, True), (_tile, *_whole, _K // B * B, _out, False), (_tile, *_cut, 16, _out, False)]
            EXACT += [(_tile, *(_whole if k % 2 else _cut), k * B - 16 * (k % 3), _out, k % 2 == 0) for k in (2, 3, 4, 5, 9, 13)]


@pytest.mark.parametrize("tile,T,N,K,out,add", EXACT)
def test_tiles_of_whole_numbers(moe, tile, T, N, K, out, add):
    """Codes are whole numbers and scales powers of two, so that every sum is a multiple of 1/4 under
    2^22. With addends that leave a few bits of it, no output's rounding hides anything."""
    _say("tile:", tile, T, N, K, out, add)
    g, KB, pad = _gen(T + N + K), _up(K), 16 if add else 0
    whole = lambda most, *n: torch.randint(-most, most + 1, n, device="cuda", generator=g)  # noqa: E731
    power = lambda *n: 2.0 ** torch.randint(-1, 2, n, device="cuda", generator=g).float()  # noqa: E731
    qx, qw = Padded(T, K, K + pad, F8, whole(7, T, K).float()), Padded(N, K, K + 2 * pad, F8, whole(7, N, K).float())
    sx, sw = Padded(T, KB, KB + pad // 16, torch.float32, power(T, KB)), Padded(_up(N), KB, KB + pad // 8, torch.float32, power(_up(N), KB))
    o = Padded(T, N, N + pad // 2, ACT[out])
    want, bias, y, res = _full(qx.m, sx.m) @ _full(qw.m, sw.m, B).T, None, None, None
    assert float(want.abs().max()) * 4 < 2.0 ** 22
    if add:
        bias, left = whole(9, N).float(), whole(127, T, N).to(D) / 4
        res = Padded(T, N, N + pad, ACT[out], whole(100, T, N).float())
        y = Padded(T, N, N + 3 * pad, torch.float32, left - want - bias - res.m.to(D))
        want = left
    moe.fp8_matmul(qx.m, sx.m, qw.m, sw.m, o.m, bias=bias, y_in=y.m if add else None, res=res.m if add else None)
    assert torch.equal(o.m, want.to(ACT[out]))
    assert all(m is None or m.untouched() for m in (qx, qw, sx, sw, y, res, o))


@pytest.mark.parametrize("tile,T,N,K", [(t, *n, k) for t, n, _, k in TILES])
@pytest.mark.parametrize("wide", [False, True])
def test_tiles_are_cut_as_documented(moe, tile, T, N, K, wide):
    """What the 8-bit matrix instruction may cut, product by product: of eight neighbours each to a
    multiple of 2^-13 of the largest one's binade. The addend takes the sum's fp32 value away, so
    that the output is what the sums are off by."""
    _say("cut:", tile, T, N, K, wide)
    g, KB = _gen(T * 3 + N + K), _up(K)
    make = _codes if wide else _normal
    qx, qw = make(g, T, K), make(g, N, K)
    sx, sw = torch.exp(_rn(g, T, KB)) / 100, torch.exp(_rn(g, _up(N), KB)) / 100
    x, w = _full(qx, sx), _full(qw, sw, B)
    exact = x @ w.T
    y, out = (-exact).float(), torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    moe.fp8_matmul(qx, sx, qw, sw, out, y_in=y)
    want = exact + y.to(D)
    t, n = torch.arange(0, T, max(1, T // 24), device="cuda"), torch.arange(0, N, N // 40, device="cuda")
    off = _product_tolerance(x[t], w[n], True) + exact[t][:, n].abs() * 2 * R32
    for j in range(0, K, B):  # a block: its products' sizes before the scales, in eights
        p = (qx[t, None, j:j + B].to(D) * qw[None, n, j:j + B].to(D)).abs().unflatten(2, (-1, 8))
        unit = 2.0 ** (torch.frexp(p.amax(3, keepdim=True))[1].to(D) - 14)
        lost = torch.where(torch.remainder(p, unit) != 0, unit, 0.0).sum((2, 3))
        off += lost * sx[t, None, j // B].to(D) * sw[None, n // B, j // B].to(D)
    got = out[t][:, n].to(D)
    err = (got - want[t][:, n]).abs() - got.abs() * 2 * 2.0 ** -8  # its own rounding, of a value of got's binade
    assert bool((err <= off).all()), float((err / off).max())


@pytest.mark.parametrize("T,N,K,out", [(1, 4096, 2064, "bf16"), (8, 6200, 2064, "f32"), (61, 5003, 4624, "bf16"), (509, 5003, 2064, "f32"),
                                       (1021, 5003, 2064, "bf16")])
def test_products_repeat(moe, T, N, K, out):
    g, KB = _gen(T), _up(K)
    qx, qw, sx, sw = _normal(g, T, K), _normal(g, N, K), torch.exp(_rn(g, T, KB)), torch.exp(_rn(g, _up(N), KB))
    first = moe.fp8_matmul(qx, sx, qw, sw, torch.empty(T, N, device="cuda", dtype=ACT[out])).clone()
    for _ in range(8):
        assert torch.equal(moe.fp8_matmul(qx, sx, qw, sw, torch.empty_like(first)), first)
