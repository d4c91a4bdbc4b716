"""The layer on e4m3 blocks at the ends of fp32's range, and logits of tokens that are not finite.

What a power of two moves from a factor of a product to the other changes no bit of the product, as
long as each is a normal number: many of these tests hold two calls that differ by such a move to
the same bits."""
import pytest

from test_gpu_fp8 import ACT, B, D, F8, R32, _gen, _layer_inputs, _normal, _outputs, _rn, _say, _up, _workspace, moe  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [1, 11])
@pytest.mark.parametrize("act,by", [("bf16", 110), ("f32", 110)])
def test_sizes_between_activations_and_scales(moe, T, act, by):
    """Activations of 2^by times the size on scales of 2^-by times theirs, and an intermediate so on
    down's: the same bits, also where a block's sum of codes times activations alone leaves fp32's
    range or the activations come near its end."""
    _say("sizes:", T, act, by)
    H, I, E, k = 528, 272, 6, 3  # noqa: E741
    s = _layer_inputs(T, H, I, E, k, act, 41 + T, wide=True)
    s["logits_in"], f, one = _rn(_gen(3), T, E), 2.0 ** by, dict(workspace=_workspace(moe, T, H, I, E, k))
    run = lambda **c: moe.fp8_layer(**{**s, **c}, y=torch.empty(T, H, device="cuda"), **one).clone()  # noqa: E731
    # gate and up of some hundreds: at 2^110 the blocks' sums of codes times activations pass 2^128
    x0 = s["x"] * 512
    want = run(x=x0)
    assert bool(torch.isfinite(want).all())
    x, gu = x0 * f, s["s_gu"] / f
    assert torch.equal(x / f, x0) and torch.equal(gu * f, s["s_gu"])  # nothing is lost on the way
    assert torch.equal(run(x=x, s_gu=gu), want)
    s["s_gu"][:, 1] *= 128  # so an intermediate's
    want, gu, dn = run(), s["s_gu"].clone(), s["s_dn"] / f
    assert bool(torch.isfinite(want).all())
    gu[:, 1] *= f
    assert torch.equal(gu[:, 1] / f, s["s_gu"][:, 1]) and torch.equal(dn * f, s["s_dn"])
    assert torch.equal(run(s_gu=gu, s_dn=dn), want)


def test_scales_of_every_kind(moe):
    """Scales below fp32's normal range, of its largest binade, negative, 0: a weight is its code
    times its scale. Infinite and NaN ones stay with the rows that they scale."""
    H, I, n = 144, 16, 8  # noqa: E741
    kinds = [2.0 ** -149, 3 * 2.0 ** -140, 1.5 * 2.0 ** -126, 1.25 * 2.0 ** 127, -0.75, 0.0, -1.5 * 2.0 ** -101, 1.75 * 2.0 ** 101]
    q_gu = torch.zeros(n, 2 * I, H, device="cuda")
    q_gu[:, 0, 0], q_gu[:, I, 0] = 64.0, 1.0
    q_dn = torch.zeros(n, H, I, device="cuda")
    q_dn[:, :, 0] = torch.arange(H, device="cuda") % 15 - 7.0
    s_gu, s_dn = torch.ones(n, 2, 1, 2, device="cuda"), torch.ones(n, 2, 1, device="cuda")
    x = torch.ones(n, H, device="cuda")
    logits = torch.full((n, n), float("-inf"), device="cuda")
    logits.fill_diagonal_(0.0)
    for i, v in enumerate(kinds):
        if 0 < abs(v) < 1e-20 or abs(v) > 1e20:
            up = 2.0 ** (100 if abs(v) < 1 else -100)
            s_gu[i, 1, 0, 0] = up  # the intermediate is 64 times that
        s_dn[i] = v
    want = torch.stack([q_dn[i, :, 0].to(D) * 64 * float(s_gu[i, 1, 0, 0]) * v for i, v in enumerate(kinds)])
    s = dict(router_w=None, q_gu=q_gu.to(F8), q_dn=q_dn.to(F8), k=1, logits_in=logits)
    run = lambda **c: moe.fp8_layer(**{**s, **c}, y=torch.empty(n, H, device="cuda"), workspace=_workspace(moe, n, H, I, n, 1))  # noqa: E731
    y = run(x=x, s_gu=s_gu, s_dn=s_dn)
    assert torch.equal(y.to(D), want)  # few bits everywhere: each product is exact
    # the same scales on gate and up, x having the other size
    s_gu2, s_dn2, x2 = torch.ones_like(s_gu), torch.ones_like(s_dn), x.clone()
    for i, v in enumerate(kinds):
        s_gu2[i, 1, 0, 0] = v
        if float(s_gu[i, 1, 0, 0]) != 1:
            x2[i, 0] = float(s_gu[i, 1, 0, 0])
            s_gu2[i, 0, 0, 0] = 1 / float(s_gu[i, 1, 0, 0])
    assert torch.equal(run(x=x2, s_gu=s_gu2, s_dn=s_dn2).to(D), want)
    # not finite: 0 times it is NaN, so every row of the block that it scales is hit, and no other
    for v in (float("inf"), float("nan")):
        bad = torch.ones_like(s_dn)
        bad[2, 1] = v
        y = run(x=x, s_gu=torch.ones_like(s_gu), s_dn=bad)
        hit = torch.zeros(n, H, dtype=torch.bool, device="cuda")
        hit[2, B:] = True
        assert bool((~torch.isfinite(y[hit])).all()) and bool(torch.isfinite(y[~hit]).all())
