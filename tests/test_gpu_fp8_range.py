"""The layer on e4m3 blocks at the ends of fp32's range, and logits of tokens that are not finite.

What a power of two moves from a factor of a product to the other changes no bit of the product, as
long as each is a normal number: many of these tests hold two calls that differ by such a move to
the same bits."""
import pytest

from test_gpu_fp8 import ACT, B, D, F8, R32, _gen, _layer_inputs, _normal, _outputs, _rn, _say, _up, _workspace, moe  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


TOP = torch.finfo(torch.float32).max
BF_TOP = 255.0 * 2.0 ** 120  # bfloat16's largest; from half a step above it on, rounding gives infinity


@pytest.mark.parametrize("value", [TOP, -TOP, BF_TOP + 2.0 ** 119, -BF_TOP - 2.0 ** 119, BF_TOP + 2.0 ** 119 - 2.0 ** 104, BF_TOP,
                                   1.0 + 2.0 ** -23, -1.7182819, 2.0 ** -100 * (2 - 2.0 ** -23), 2.0 ** -112 * 1.2345678,
                                   -(2.0 ** -118) * (1 + 2.0 ** -23), 2.0 ** -126, 2.0 ** -126 * (2 - 2.0 ** -23), 2.0 ** -130 * 1.171875,
                                   2.0 ** -149])
def test_any_size_of_activation_and_intermediate(moe, value):
    """One activation of that size, one intermediate of 64 (or 1) times it, and an output of that
    times a code and a scale. The other products are of zeros."""
    _say("size:", value)
    v = torch.tensor(value, device="cuda").item()
    H, I = 288, 144  # noqa: E741
    s = dict(x=torch.zeros(1, H, device="cuda"), router_w=None, k=1)
    s["q_gu"], s["q_dn"] = torch.zeros(1, 2 * I, H, device="cuda"), torch.zeros(1, H, I, device="cuda")
    s["s_gu"], s["s_dn"] = torch.ones(1, 2, _up(I), _up(H), device="cuda"), torch.ones(1, _up(H), _up(I), device="cuda")
    # gate of the intermediate's element 130: 64 from x's element 0, whose silu is 64 in fp32; up: v from element 200
    s["x"][0, 0], s["x"][0, 200] = 1.0, v
    s["q_gu"][0, 130, 0], s["q_gu"][0, I + 130, 200] = 64.0, 1.0
    large = abs(v) > 1
    if large:
        s["s_gu"][0, 1, 1, 1] = 2.0 ** -6
    codes = torch.arange(H, device="cuda") % 15 - 7.0
    s["q_dn"][0, :, 130] = codes
    s["s_dn"][:] = 2.0 ** (-100 if large else 100)
    s["q_gu"], s["q_dn"] = s["q_gu"].to(F8), s["q_dn"].to(F8)
    y = moe.fp8_layer(**s, y=torch.empty(1, H, device="cuda"), workspace=_workspace(moe, 1, H, I, 1, 1),
                      logits_in=torch.zeros(1, 1, device="cuda"))
    h = v if large else 64.0 * v
    want = codes.to(D) * h * (2.0 ** -100 if large else 2.0 ** 100)
    # u and h are exact; a code times h in three parts: two additions that may cut (2^-23 each)
    err = (y[0].to(D) - want).abs()
    assert bool((err <= want.abs() * 4 * R32).all()), (v, y[0, :15].tolist(), want[:15].tolist())
    # x of that size where every weight is 0: as if it were not there
    codes = torch.zeros(1, 2 * I, H, device="cuda")
    codes[0, 130, 0], codes[0, I + 130, 0] = 64.0, 1.0
    s["q_gu"] = codes.to(F8)
    ys = []
    for at in (v, 0.0):
        s["x"][0, 200] = at
        ys.append(moe.fp8_layer(**s, y=torch.empty(1, H, device="cuda"), workspace=_workspace(moe, 1, H, I, 1, 1),
                                logits_in=torch.zeros(1, 1, device="cuda")))
    assert bool(torch.isfinite(ys[0]).all()) and torch.equal(*ys)


@pytest.mark.parametrize("low", [2.0 ** -7 - 2.0 ** -23, 2.0 ** -8 - 2.0 ** -23, 2.0 ** -8, 2.0 ** -9 + 2.0 ** -17])
def test_sums_next_to_the_range_s_end(moe, low):
    """1.5 times a value of fp32's last binade, as the up product and as an output: finite, whatever
    parts the value goes in."""
    v = torch.tensor(2.0 ** 127 * (1.3125 + low), device="cuda").item()
    H, I = 144, 16  # noqa: E741
    q_gu, q_dn, x = torch.zeros(1, 2 * I, H, device="cuda"), torch.zeros(1, H, I, device="cuda"), torch.zeros(1, H, device="cuda")
    s_gu, s_dn = torch.ones(1, 2, 1, 2, device="cuda"), torch.ones(1, 2, 1, device="cuda")
    x[0, 3], x[0, 130] = 64.0, v
    q_gu[0, 2, 3], q_gu[0, I + 2, 130] = 1.0, 1.5  # gate 64, up 1.5 v, the intermediate 64 times that times the scale
    q_dn[0, :, 2] = 1.0
    run = lambda **c: moe.fp8_layer(x, None, q_gu.to(F8), c["s_gu"], q_dn.to(F8), c["s_dn"], 1, torch.empty(1, H, device="cuda"),  # noqa: E731
                                    _workspace(moe, 1, H, I, 1, 1), logits_in=torch.zeros(1, 1, device="cuda"))
    s_gu[0, 0], s_dn[:] = 2.0 ** -12, 2.0 ** 5  # gate 2^-6, whose silu is 2^-7 (1 + 2^-7 + ...)
    silu = 2.0 ** -6 / (1 + torch.exp(torch.tensor(-(2.0 ** -6), dtype=D))).item()
    y = run(s_gu=s_gu, s_dn=s_dn)
    want = 1.5 * v * silu * 2.0 ** 5
    # u three additions that may cut; exp, 1 +, the quotient and the product; the output three again
    assert bool(((y.to(D) - want).abs() <= abs(want) * (6 + 8 + 6) * R32).all()), (y[0, :3].tolist(), want)
    q_dn[0, :, 2], q_gu[0, I + 2, 130] = 1.5, 1.0
    s_gu[0, 0], s_gu[0, 1] = 1.0, 2.0 ** -6
    y = run(s_gu=s_gu, s_dn=torch.ones_like(s_dn))
    assert bool(((y.to(D) - 1.5 * v).abs() <= 1.5 * v * 6 * R32).all()), (y[0, :3].tolist(), 1.5 * v)


@pytest.mark.parametrize("T", [1, 11])
@pytest.mark.parametrize("act,by", [("bf16", 110), ("bf16", -110), ("f32", 110), ("f32", -105)])
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


def test_masked_experts_of_tokens_that_are_not_finite(moe):
    """A logit of -infinity gives weight 0, and its expert is not read, also where another logit of
    the token is NaN or infinite."""
    T, H, I, E, k = 6, 144, 32, 70, 4  # noqa: E741
    s = _layer_inputs(T, H, I, E, k, "bf16", 71)
    inf, nan = float("inf"), float("nan")
    li = torch.full((T, E), -inf, device="cuda")
    li[0, 33], li[1, 69], li[2, [5, 66]] = nan, inf, torch.tensor([inf, 2.0], device="cuda")
    li[3, [7, 8, 9]] = torch.tensor([nan, 1.0, inf], device="cuda")
    li[4, 0], li[5, 12] = 1.0, torch.finfo(torch.float32).min
    for some in (list(range(T)), [0], [1], [2], [3], [4]):
        n = len(some)
        o, flat = _outputs(n, H, E, k, torch.bfloat16)
        moe.fp8_layer(**{**s, "x": s["x"][some].contiguous()}, y=o["y"].m, x_out=o["x_out"].m, workspace=_workspace(moe, n, H, I, E, k),
                      logits_in=li[some].contiguous(), **flat)
        chosen = li[some].gather(1, flat["topk_ids"].long())
        masked = chosen == -inf
        assert bool((flat["topk_w"][masked] == 0).all()), flat["topk_w"]
        for t, i in enumerate(some):
            w = flat["topk_w"][t][~masked[t]]
            if i in (0, 1, 3):
                assert bool(torch.isnan(w).all())
            if i in (0, 1, 2, 3):
                assert bool(torch.isnan(o["y"].m[t]).all())
            else:
                assert w.tolist() == [1.0] and bool(torch.isfinite(o["y"].m[t]).all())
    # what is masked may hold NaN codes
    want = moe.fp8_layer(**s, y=torch.empty(T, H, device="cuda"), workspace=_workspace(moe, T, H, I, E, k), logits_in=li).clone()
    for name in ("q_gu", "q_dn"):
        s[name] = s[name].clone()
        s[name].view(torch.uint8)[torch.isinf(li).logical_and(li < 0).all(0)] = 0x7F
    y = moe.fp8_layer(**s, y=torch.empty(T, H, device="cuda"), workspace=_workspace(moe, T, H, I, E, k), logits_in=li)
    assert torch.equal(y.nan_to_num(), want.nan_to_num())
