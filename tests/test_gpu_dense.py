"""The dense operators beside the routed layer against their definitions in 64 bits: norm
with the residual's addition and 8-bit output, codes of rows, the 8-bit product, the gated
block, and a run of them with the routed layer.

Tolerances count roundings. One to fp32 is off by at most 2^-24 of its value, one to bf16 by
2^-8 (half of finfo.eps); sums and products in fp32 are counted where they stand."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import layer_cases as LC  # noqa: E402

R32, RBF = 2.0 ** -24, 2.0 ** -8
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
D = torch.float64


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def moe():
    import expert_offloaded_ffn_moe_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.load_library()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rn(g, *n):
    return torch.randn(*n, device="cuda", generator=g)


def _codes(g, rows, cols, low=-128):
    return torch.randint(low, 128, (rows, cols), device="cuda", dtype=torch.int8, generator=g)


class Padded:
    """A matrix inside a larger buffer: a row stride of its own, rows behind the last one,
    and a fill whose bytes must survive."""

    def __init__(self, rows, cols, ld, dtype, value=None):
        self.buf = torch.full((rows + 2, ld), 77, device="cuda", dtype=dtype)
        self.m = self.buf[:rows, :cols]
        if value is not None:
            self.m.copy_(value)

    def untouched(self):
        rows, cols = self.m.shape
        return bool((self.buf[rows:] == 77).all()) and bool((self.buf[:, cols:] == 77).all())


def _special_rows(v):
    """Rows of unlike kinds at the front: nothing, next to nothing, huge, halves everywhere."""
    T, H = v.shape
    kinds = [torch.zeros(H), torch.full((H,), 2.0 ** -110), torch.full((H,), 2.0 ** 110), torch.linspace(-1, 1, H) * 2 ** -60]
    ties = torch.arange(H, dtype=torch.float32) % 254 / 2 - 63.25 + 0.25
    ties[0] = 127.0
    kinds.append(ties)
    for i, k in enumerate(kinds):
        if i + 1 < T:
            v[i + 1] = k.to(v.dtype).to(v.device)
    return v


def _check_codes(q, s, p, rstd):
    """q, s: what the operator wrote; p [T][H] in fp64, whose codes they are; rstd [T] or 1."""
    top = p.abs().amax(1)
    none = top < 2.0 ** -100
    want = torch.round(127.0 * p / torch.where(none, torch.ones_like(top), top)[:, None])
    want[none] = 0
    assert torch.equal(q.to(D), want)
    scale = torch.where(none, torch.zeros_like(top), top * rstd / 127.0)
    assert bool(((s.to(D) - scale).abs() <= scale * R32 * 1.01).all())


NORM = [
    # T, H, act, add, extra stride
    (1, 1, "bf16", "none", 0), (3, 7, "bf16", "act", 1), (2, 8, "f32", "f32", 0), (9, 9, "f32", "none", 3),
    (5, 64, "bf16", "f32", 0), (6, 512, "bf16", "act", 5), (7, 513, "f32", "act", 0), (300, 2047, "bf16", "f32", 1),
    (8, 2048, "f32", "act", 4), (1, 7168, "bf16", "f32", 0), (17, 7168, "bf16", "none", 8), (7, 4101, "bf16", "f32", 3),
    (6, 8192, "f32", "none", 0), (7, 8193, "bf16", "act", 7), (6, 16384, "bf16", "f32", 0), (3, 16383, "f32", "act", 1),
    (1025, 256, "bf16", "f32", 0), (261, 4096, "bf16", "f32", 0),
    # more rows than workgroups: each goes on to further ones
    (1300, 4100, "bf16", "f32", 1), (5000, 300, "bf16", "act", 0), (3000, 1030, "f32", "act", 2), (1500, 3000, "bf16", "act", 0),
    (7, 2561, "f32", "f32", 1), (5, 4096, "f32", "act", 0), (700, 9000, "bf16", "none", 0),
    (4101, 512, "f32", "f32", 0),
]


@pytest.mark.parametrize("T,H,act,add,pad", NORM)
def test_rms_norm(moe, T, H, act, add, pad):
    _say("norm:", T, H, act, add, pad)
    g, dt, eps = _gen(T * 100003 + H), ACT[act], float(np.float32(1e-5))  # the ABI's eps is a float
    x = Padded(T, H, H + pad, dt, _special_rows((_rn(g, T, H) * torch.exp(_rn(g, H))).to(dt)))
    w = (1 + 0.3 * _rn(g, H)).to(dt)
    adt = {"none": None, "act": dt, "f32": torch.float32}[add]
    r = None
    if adt is not None:
        r = Padded(T, H, H + 2 * pad, adt, _rn(g, T, H).to(adt))
        r.m[1:6] = 0
    xo, out = Padded(T, H, H + pad, dt), Padded(T, H, H + 3 * pad, dt)
    q, s = Padded(T, H, H + 5 * pad, torch.int8), torch.full((T + 1,), 77.0, device="cuda")
    x0 = x.buf.clone()
    moe.rms_norm(x.m, w, eps, add=None if r is None else r.m, x_out=None if r is None else xo.m, out=out.m, q_out=q.m,
                 s_out=s[:T])
    torch.cuda.synchronize()
    assert torch.equal(x.buf, x0)
    for m in (xo, out, q):
        assert m.untouched()
    assert float(s[T]) == 77.0
    st = x.m
    if r is not None:
        st = (x.m.float() + r.m.float()).to(dt)
        assert torch.equal(xo.m, st)
    p = st.to(D) * w.to(D)
    rstd = 1 / (st.to(D).square().mean(1) + eps).sqrt()
    n = p * rstd[:, None]
    # bf16: rstd and the product rounded to fp32, then to bf16; fp32: the fp64 product rounded once
    tol = (RBF + 2.02 * R32 if act == "bf16" else 1.01 * R32) * n.abs() + 2.0 ** -140
    assert bool(((out.m.to(D) - n).abs() <= tol).all())
    _check_codes(q.m, s[:T], p, rstd)
    # each output alone gives the same bits
    out2, q2, s2 = torch.empty_like(out.m), torch.empty_like(q.m), torch.empty_like(s[:T])
    moe.rms_norm(x.m, w, eps, add=None if r is None else r.m, out=out2)
    moe.rms_norm(x.m, w, eps, add=None if r is None else r.m, q_out=q2, s_out=s2)
    torch.cuda.synchronize()
    assert torch.equal(out2, out.m) and torch.equal(q2, q.m) and torch.equal(s2, s[:T])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_rms_norm_in_place(moe, act):
    """x_out over x, out over add."""
    g, dt = _gen(5), ACT[act]
    for T, H in [(33, 1000), (1301, 2100), (5001, 200)]:
        x, r, w = _rn(g, T, H).to(dt), _rn(g, T, H).to(dt), _rn(g, H).to(dt)
        xo, out = torch.empty_like(x), torch.empty_like(x)
        moe.rms_norm(x, w, 1e-6, add=r, x_out=xo, out=out)
        moe.rms_norm(x, w, 1e-6, add=r, x_out=x, out=r)
        torch.cuda.synchronize()
        assert torch.equal(x, xo) and torch.equal(r, out)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [40, 1500, 7000, 16000])
def test_norm_of_rows_that_are_not_finite(moe, act, H):
    """NaN and infinity in x, in the weight's product, and squares beyond fp32."""
    g, dt, T = _gen(H), ACT[act], 6
    x, w = _rn(g, T, H).to(dt), (1 + 0.1 * _rn(g, H)).to(dt)
    x[1, H // 2] = float("nan")
    x[2, H - 1] = float("inf")
    x[3] *= 2.0 ** 80  # finite, with squares of 2^160
    x[4, 3] = -float("inf")
    out = torch.empty_like(x)
    q, s = torch.full((T, H), 5, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.rms_norm(x, w, 1e-6, out=out, q_out=q, s_out=s)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    moe.quantize_rows(x, q2, s2)
    torch.cuda.synchronize()
    for k in (q, q2):
        assert not k[[1, 2, 4]].any() and k[[0, 3, 5]].any(1).all()
    for k in (s, s2):
        assert k[[1, 2, 4]].isnan().all() and k[[0, 3, 5]].isfinite().all()
    assert out[1].isnan().all() and out[2, H - 1].isnan() and not out[2, : H - 1].any()
    ok = [0, 3, 5]
    n = x.to(D)[ok] / (x.to(D)[ok].square().mean(1, keepdim=True) + 1e-6).sqrt() * w.to(D)
    assert bool(((out[ok].to(D) - n).abs() <= (RBF if act == "bf16" else 0) * n.abs() + 2.1 * R32 * n.abs()).all())
    _check_codes(q[ok], s[ok], x.to(D)[ok] * w.to(D), 1 / (x.to(D)[ok].square().mean(1) + 1e-6).sqrt())


@pytest.mark.parametrize("T,H,act,pad", [(1, 1, "f32", 0), (5, 7168, "bf16", 0), (6, 33, "bf16", 2), (2000, 2048, "bf16", 0),
                                         (7, 1029, "f32", 1), (6, 16384, "f32", 0), (8, 511, "f32", 0), (6, 5001, "bf16", 1)])
def test_quantize_rows(moe, T, H, act, pad):
    _say("quantize:", T, H, act, pad)
    g, dt = _gen(T + H), ACT[act]
    x = Padded(T, H, H + pad, dt, _special_rows((_rn(g, T, H) * torch.exp(_rn(g, H))).to(dt)))
    q, s = Padded(T, H, H + 3 * pad, torch.int8), torch.full((T + 1,), 77.0, device="cuda")
    moe.quantize_rows(x.m, q.m, s[:T])
    torch.cuda.synchronize()
    assert q.untouched() and float(s[T]) == 77.0
    _check_codes(q.m, s[:T], x.m.to(D), 1.0)


def _product_tol(v, others, out_act):
    """Roundings of act(acc sx sw + b + y + r) in fp32: the sum's conversion and two products
    (of v), then up to three additions of partial sums of at most |v| + |b| + |y| + |r|."""
    size = v.abs() + sum(o.abs() for o in others)
    total = v + sum(others)
    return 1.01 * R32 * (3 * v.abs() + 3 * size) + (RBF if out_act == "bf16" else 0) * total.abs() * 1.01 + 2.0 ** -140


MATMUL = [
    # T, N, K, out, extra bytes of the code rows
    (1, 1, 16, "f32", 0), (1, 7168, 2048, "bf16", 0), (2, 7, 48, "f32", 16), (15, 100, 64, "bf16", 32), (16, 257, 80, "f32", 0),
    (17, 33, 1040, "bf16", 0), (31, 768, 2064, "f32", 16), (33, 130, 256, "bf16", 0), (64, 1001, 528, "f32", 0),
    (65, 64, 7168, "bf16", 0), (100, 129, 144, "f32", 48), (129, 1000, 2048, "bf16", 0), (333, 1001, 2064, "f32", 0),
    (513, 515, 1008, "bf16", 16), (260, 2048, 128, "f32", 0), (1024, 768, 384, "bf16", 0), (70, 5, 4096, "f32", 0),
    (255, 256, 112, "f32", 0), (640, 2300, 640, "bf16", 0),
    # enough tiles for each of the larger ones, ragged at both ends
    (2050, 6500, 144, "f32", 0), (2047, 7168, 1168, "bf16", 0), (1000, 6700, 272, "bf16", 16), (1023, 6401, 48, "f32", 0),
    (3, 6200, 208, "f32", 0), (16, 7165, 96, "bf16", 0), (29, 6163, 1040, "f32", 16), (32, 100, 64, "bf16", 0),
    (20000, 50, 64, "f32", 0), (520, 6401, 400, "bf16", 0), (520, 6401, 400, "f32", 0), (250, 7001, 784, "bf16", 0), (127, 7165, 320, "f32", 0),
    # at the rule that takes a few tokens to tiles
    (12, 6129, 4096, "bf16", 0), (13, 6129, 4096, "f32", 16), (13, 6128, 4096, "bf16", 0), (13, 6129, 4080, "f32", 0),
    (16, 7165, 4112, "bf16", 0),
]


@pytest.mark.parametrize("T,N,K,out_act,pad", MATMUL)
def test_int8_matmul(moe, T, N, K, out_act, pad):
    _say("matmul:", T, N, K, out_act, pad)
    g, dt = _gen(T * 7 + N * 3 + K), ACT[out_act]
    x, w = Padded(T, K, K + pad, torch.int8, _codes(g, T, K)), Padded(N, K, K + 2 * pad, torch.int8, _codes(g, N, K))
    acc = x.m.to(D) @ w.m.to(D).t()
    # scales of 1: the sums themselves, exact in fp32 under 2^24 and rounded once above
    out = Padded(T, N, N + pad // 4, torch.float32)
    moe.int8_matmul(x.m, torch.ones(T, device="cuda"), w.m, torch.ones(N, device="cuda"), out.m)
    torch.cuda.synchronize()
    assert torch.equal(out.m, acc.float()) and out.untouched()
    sx, sw = torch.rand(T, device="cuda", generator=g) * 0.01, torch.rand(N, device="cuda", generator=g) * 0.01
    bias, y, res = _rn(g, N), Padded(T, N, N + 3, torch.float32, _rn(g, T, N)), Padded(T, N, N + 1, dt, _rn(g, T, N).to(dt))
    v = acc * sx.to(D)[:, None] * sw.to(D)
    for b_, y_, r_ in [(None, None, None), (bias, None, None), (None, y, None), (None, None, res), (bias, y, res)]:
        others = ([b_.to(D).expand(T, N)] if b_ is not None else []) + [m.m.to(D) for m in (y_, r_) if m is not None]
        out = Padded(T, N, N + pad // 4, dt)
        moe.int8_matmul(x.m, sx, w.m, sw, out.m, bias=b_, y_in=y_ and y_.m, res=r_ and r_.m)
        torch.cuda.synchronize()
        assert out.untouched()
        err = (out.m.to(D) - (v + sum(others))).abs()
        assert bool((err <= _product_tol(v, others, out_act)).all()), float((err / _product_tol(v, others, out_act)).max())


def test_int8_matmul_over_its_inputs(moe):
    """out over res, and over y_in."""
    g, T, N, K = _gen(3), 37, 200, 128
    for T in (5, 37, 300):
        q, w, sx, sw = _codes(g, T, K), _codes(g, N, K), torch.rand(T, device="cuda"), torch.rand(N, device="cuda")
        y, res = _rn(g, T, N), _rn(g, T, N).bfloat16()
        a, b = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
        moe.int8_matmul(q, sx, w, sw, a, y_in=y)
        moe.int8_matmul(q, sx, w, sw, b, y_in=y, res=res)
        moe.int8_matmul(q, sx, w, sw, res, y_in=y, res=res)
        moe.int8_matmul(q, sx, w, sw, y, y_in=y)
        torch.cuda.synchronize()
        assert torch.equal(y, a) and torch.equal(res, b)


@pytest.mark.parametrize("T", [2, 70, 300])
def test_int8_matmul_largest_sums(moe, T):
    """K of 131056 codes of -128: the sum 2147221504 is within int32."""
    K = 131056
    q, w = torch.full((T, K), -128, dtype=torch.int8, device="cuda"), torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    out = torch.empty(T, 3, device="cuda")
    moe.int8_matmul(q, torch.ones(T, device="cuda"), w, torch.ones(3, device="cuda"), out)
    want = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K, 128.0 * 128 * K], dtype=D).float()
    assert torch.equal(out.cpu(), want.expand(T, 3))


def test_int8_matmul_row_of_nan(moe):
    """A row with a NaN, quantised, gives NaN in its own row of the product alone."""
    g, T, N, K = _gen(4), 20, 40, 64
    x, w = _rn(g, T, K).bfloat16(), _codes(g, N, K)
    x[7, 3] = float("nan")
    q, s = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.quantize_rows(x, q, s)
    out = torch.empty(T, N, device="cuda")
    moe.int8_matmul(q, s, w, torch.ones(N, device="cuda"), out)
    nan = out.isnan()
    assert nan[7].all() and int(nan.sum()) == N


def _ffn_ref(qx, sx, qgu, sgu, qdn, sdn):
    """(product, tolerance): the block in fp64, and how far fp32 may take it.

    g and u carry 3 roundings each; silu passes g's on (1 + |g|)-fold; exp(-g) adds
    2 |g| + 2 (its argument's product and constant, its own result), then a sum, a quotient and
    a product: (5 |g| + 12) R32 in all, taken as (6 |g| + 16) R32. Where 127 h / max|h| lies
    within twice that (h's and the largest's) of a half, a code may be the next one: one
    scale times the weight there."""
    gu = (qx.to(D) @ qgu.to(D).t()) * sx.to(D)[:, None] * sgu.to(D)
    g, u = gu.chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    off = (6 * g.abs() + 16) * R32
    top = h.abs().amax(1, keepdim=True)
    top = torch.where(top > 0, top, torch.ones_like(top))
    v = 127 * h / top
    reach = v.abs() * (off + off.amax(1, keepdim=True)) + 2.0 ** -100
    near = ((v - torch.floor(v)) - 0.5).abs() <= reach
    code, scale = torch.round(v), top / 127
    p = (code * scale) @ (qdn.to(D) * sdn.to(D)[:, None]).t()
    size = (code.abs() * scale) @ (qdn.to(D).abs() * sdn.to(D)[:, None]).t()
    turn = (near.to(D) * scale) @ (qdn.to(D).abs() * sdn.to(D)[:, None]).t()
    # the scale's error takes the whole sum along; turned codes come on top
    return p, size * off.amax(1, keepdim=True) + turn, int(near.sum())


FFN = [
    # T, H, I, out, pad
    (1, 16, 16, "f32", 0), (1, 7168, 2048, "bf16", 0), (2, 256, 128, "f32", 16), (4, 2048, 768, "bf16", 0), (5, 80, 16, "f32", 0),
    (16, 2048, 768, "f32", 0), (17, 400, 240, "bf16", 16), (61, 1040, 496, "f32", 0), (65, 256, 128, "bf16", 0),
    (130, 528, 80, "f32", 0), (300, 2048, 768, "bf16", 0), (1025, 512, 272, "f32", 32), (3, 64, 16384, "f32", 0),
    (257, 1024, 1040, "f32", 0), (96, 2064, 304, "bf16", 0),
    # the second product on codes formed beside it, at the ends of that
    (1, 64, 16384, "f32", 0), (2, 48, 8192, "f32", 0), (4, 80, 4096, "bf16", 0), (3, 96, 4112, "f32", 0), (16, 256, 1024, "f32", 16),
    (16, 6160, 16, "bf16", 0), (7, 128, 2048, "f32", 0), (9, 6145 + 15, 96, "f32", 0), (16, 128, 1040, "f32", 0),
    (5, 96, 3280, "f32", 0), (19, 80, 3104, "bf16", 16), (31, 256, 96, "f32", 0),
    (300, 64, 3584, "f32", 0), (2050, 96, 3264, "f32", 0), (1001, 272, 3360, "bf16", 0), (515, 144, 3280, "f32", 16), (251, 80, 3504, "bf16", 0),
]


def _ffn_case(T, H, I, pad, seed):
    g = _gen(seed)
    qx, sx = Padded(T, H, H + pad, torch.int8, _codes(g, T, H, -127)), torch.rand(T, device="cuda", generator=g) * 0.02 + 0.01
    qgu, qdn = Padded(2 * I, H, H + pad, torch.int8, _codes(g, 2 * I, H)), Padded(H, I, I + 2 * pad, torch.int8, _codes(g, H, I))
    sgu = (torch.rand(2 * I, device="cuda", generator=g) + 0.5) / (50 * H ** 0.5)
    sdn = (torch.rand(H, device="cuda", generator=g) + 0.5) / (74 * I ** 0.5)
    return qx, sx, qgu, sgu, qdn, sdn


@pytest.mark.parametrize("T,H,I,out_act,pad", FFN)
def test_int8_ffn(moe, T, H, I, out_act, pad):
    _say("ffn:", T, H, I, out_act, pad)
    dt = ACT[out_act]
    qx, sx, qgu, sgu, qdn, sdn = _ffn_case(T, H, I, pad, T * 31 + H * 17 + I)
    g = _gen(1)
    y, res = Padded(T, H, H + 1, torch.float32, _rn(g, T, H)), Padded(T, H, H + 2, dt, _rn(g, T, H).to(dt))
    n = moe.int8_ffn_workspace(T, H, I)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every float
    p, tol, near = _ffn_ref(qx.m, sx, qgu.m, sgu, qdn.m, sdn)
    for y_, r_ in [(None, None), (y, None), (None, res), (y, res)]:
        out = Padded(T, H, H + pad, dt)
        moe.int8_ffn(qx.m, sx, qgu.m, sgu, qdn.m, sdn, out.m, ws[:n], y_in=y_ and y_.m, res=r_ and r_.m)
        torch.cuda.synchronize()
        assert out.untouched() and bool((ws[n:] == 0xFF).all())
        others = [m.m.to(D) for m in (y_, r_) if m is not None]
        # the product's sum moves by at most `tol` before its own roundings
        bound = tol * 1.01 + _product_tol(p.abs() + tol, [o.abs() for o in others], out_act)
        err = (out.m.to(D) - (p + sum(others))).abs()
        assert bool((err <= bound).all()), (near, float((err / bound).max()))


def test_int8_ffn_zero_and_nan_tokens(moe):
    """A token of zeros gives zeros (and so the residual alone); a token of NaN gives NaN."""
    T, H, I = 6, 256, 128
    for T in (6, 70, 300):
        qx, sx, qgu, sgu, qdn, sdn = _ffn_case(T, H, I, 0, 9)
        sx[2] = 0.0
        sx[4] = float("nan")
        qx.m[5] = 0
        res = _rn(_gen(2), T, H).bfloat16()
        out = torch.empty_like(res)
        ws = torch.empty(moe.int8_ffn_workspace(T, H, I), dtype=torch.uint8, device="cuda")
        moe.int8_ffn(qx.m, sx, qgu.m, sgu, qdn.m, sdn, out, ws, res=res)
        torch.cuda.synchronize()
        nan = out.isnan()
        assert nan[4].all() and int(nan.sum()) == H
        assert torch.equal(out[2], res[2]) and torch.equal(out[5], res[5])


@pytest.mark.parametrize("H,I", [(512, 272), (2048, 768)])
def test_a_token_alone_or_among_others(moe, H, I):
    """A token's output does not depend on the call's other tokens: bit for bit the same in
    batches that take different kernels and tiles."""
    T = 700
    qx, sx, qgu, sgu, qdn, sdn = _ffn_case(T, H, I, 0, 5)
    g = _gen(6)
    y, res, bias = _rn(g, T, H), _rn(g, T, H).bfloat16(), _rn(g, 2 * I)

    def ffn(a, b):
        out = torch.empty(b - a, H, device="cuda", dtype=torch.bfloat16)
        ws = torch.empty(moe.int8_ffn_workspace(b - a, H, I), dtype=torch.uint8, device="cuda")
        return moe.int8_ffn(qx.m[a:b], sx[a:b], qgu.m, sgu, qdn.m, sdn, out, ws, y_in=y[a:b], res=res[a:b])

    def matmul(a, b):
        out = torch.empty(b - a, 2 * I, device="cuda")
        return moe.int8_matmul(qx.m[a:b], sx[a:b], qgu.m, sgu, out, bias=bias)

    for f in (ffn, matmul):
        whole = f(0, T)
        for n in (1, 2, 5, 16, 24, 33, 100, 260):
            for a in (0, 333, T - n):
                assert torch.equal(f(a, a + n), whole[a:a + n]), n


def test_binding_refuses_on_the_gpu(moe):
    z = lambda *n, dt=torch.bfloat16: torch.zeros(*n, device="cuda", dtype=dt)  # noqa: E731
    i8 = torch.int8
    ok = dict(q_x=z(4, 32, dt=i8), s_x=z(4, dt=torch.float32), q_w=z(8, 32, dt=i8), s_w=z(8, dt=torch.float32), out=z(4, 8))
    moe.int8_matmul(**ok)
    for change in [dict(s_x=z(5, dt=torch.float32)), dict(s_x=z(4)), dict(out=z(8, 4)), dict(out=z(8, 4).t()),
                   dict(q_w=z(8, 48, dt=i8)), dict(res=z(4, 8, dt=torch.float32)), dict(y_in=z(4, 8)), dict(bias=z(8)),
                   dict(s_w=torch.zeros(8)), dict(q_x=z(4, 64, dt=i8)[:, ::2]), dict(s_x=z(8, dt=torch.float32)[::2]),
                   dict(q_x=z(4, 33, dt=i8)[:, 1:]), dict(out=ok["s_x"].expand(4, 4)[:, :4])]:
        with pytest.raises(moe.MoeError) as e:
            moe.int8_matmul(**{**ok, **change})
        assert e.value.status == moe.MOE_E_INVALID
    # one row, whose stride says nothing
    moe.int8_matmul(z(4, 64, dt=i8)[:1, :32], z(1, dt=torch.float32), ok["q_w"], ok["s_w"], z(1, 8))
    # no rows
    moe.int8_matmul(z(0, 32, dt=i8), z(0, dt=torch.float32), ok["q_w"], ok["s_w"], z(0, 8))
    moe.rms_norm(z(0, 32), z(32), out=z(0, 32))


class Block:
    """One transformer layer's dense and routed halves, as a user strings them together: the
    projection of attention's output onto the residual stream, the norm, the routed
    experts, and the shared expert added to both."""

    def __init__(self, moe, T, seed=11):
        H, I, E, k, G = 2048, 768, 16, 4, 128
        self.moe, self.T = moe, T
        c = LC.make_case(H, I, E, k, G, "bf16", T, seed, 0.5)
        self.plan = moe.Plan(moe.make_config(H, I, E, k, G, "bf16", max_tokens=T))
        self.plan.load_layer(0, c.Wr_store, c.b, c.blobs)
        g = _gen(seed)
        wp = (_rn(g, H, H) * 0.02).bfloat16()
        new = lambda *n, dt=torch.bfloat16: torch.empty(*n, device="cuda", dtype=dt)  # noqa: E731
        i8, f32 = torch.int8, torch.float32
        self.w_proj, self.s_proj = new(H, H, dt=i8), new(H, dt=f32)
        moe.quantize_rows(wp, self.w_proj, self.s_proj)
        _, _, gu, self.s_gu, dn, self.s_dn = _ffn_case(T, H, I, 0, seed)
        self.gu, self.dn = gu.m, dn.m
        self.weight = (1 + 0.1 * _rn(g, H)).bfloat16()
        self.x, self.attn = _rn(g, T, H).bfloat16(), _rn(g, T, H).bfloat16()
        self.qa, self.sa, self.x1, self.n = new(T, H, dt=i8), new(T, dt=f32), new(T, H), new(T, H)
        self.o = new(T, H, dt=f32)
        self.qn, self.sn, self.y, self.out = new(T, H, dt=i8), new(T, dt=f32), new(T, H, dt=f32), new(T, H)
        self.ws = new(moe.int8_ffn_workspace(T, H, I), dt=torch.uint8)

    def run(self):
        m = self.moe
        m.quantize_rows(self.attn, self.qa, self.sa)
        m.int8_matmul(self.qa, self.sa, self.w_proj, self.s_proj, self.o)
        m.rms_norm(self.x, self.weight, 1e-6, add=self.o, x_out=self.x1, out=self.n, q_out=self.qn, s_out=self.sn)
        self.plan.forward(0, self.n, self.y)
        m.int8_ffn(self.qn, self.sn, self.gu, self.s_gu, self.dn, self.s_dn, self.out, self.ws, y_in=self.y, res=self.x1)

    def outputs(self):
        return [t.clone() for t in (self.qa, self.sa, self.o, self.x1, self.n, self.qn, self.sn, self.y, self.out)]


@pytest.mark.parametrize("T", [1, 4, 40, 200])
def test_run_of_them(moe, T):
    """The layer's steps against 64 bits, each from what the step before it left."""
    b = Block(moe, T)
    b.run()
    torch.cuda.synchronize()
    _check_codes(b.qa, b.sa, b.attn.to(D), 1.0)
    v = (b.qa.to(D) @ b.w_proj.to(D).t()) * b.sa.to(D)[:, None] * b.s_proj.to(D)
    assert bool(((b.o.to(D) - v).abs() <= _product_tol(v, [], "f32")).all())
    assert torch.equal(b.x1, (b.x.float() + b.o).bfloat16())
    p = b.x1.to(D) * b.weight.to(D)
    rstd = 1 / (b.x1.to(D).square().mean(1) + 1e-6).sqrt()
    assert bool(((b.n.to(D) - p * rstd[:, None]).abs() <= (RBF + 2.02 * R32) * (p * rstd[:, None]).abs()).all())
    _check_codes(b.qn, b.sn, p, rstd)
    y = torch.empty_like(b.y)
    b.plan.forward(0, b.n, y)
    assert torch.equal(y, b.y)
    f, tol, _ = _ffn_ref(b.qn, b.sn, b.gu, b.s_gu, b.dn, b.s_dn)
    others = [b.y.to(D), b.x1.to(D)]
    bound = tol * 1.01 + _product_tol(f.abs() + tol, [o.abs() for o in others], "bf16")
    assert bool(((b.out.to(D) - (f + sum(others))).abs() <= bound).all())
    b.plan.destroy()


@pytest.mark.parametrize("T", [1, 40])
def test_run_captured_and_replayed(moe, T):
    """The run in a HIP graph: several replays on changed inputs, the program's own eager runs
    between them, each replay bit for bit the eager run."""
    b = Block(moe, T)
    b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            b.run()
    torch.cuda.synchronize()
    for i in range(4):
        g = _gen(100 + i)
        b.x.copy_(_rn(g, *b.x.shape))
        b.attn.copy_(_rn(g, *b.attn.shape))
        b.run()
        torch.cuda.synchronize()
        want = b.outputs()
        for t in (b.o, b.x1, b.n, b.y, b.out, b.ws, b.qa, b.qn):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, b.outputs()):
            assert torch.equal(w, o)
    b.plan.destroy()


def test_two_streams_at_once(moe):
    """Calls on two streams, each with buffers and a workspace of its own, give what they give alone."""
    cases = []
    for k in range(2):
        T, H, I = (48, 1024, 512) if k else (3, 2048, 768)
        case = _ffn_case(T, H, I, 0, 21 + k)
        out = torch.empty(T, H, device="cuda")
        ws = torch.empty(moe.int8_ffn_workspace(T, H, I), dtype=torch.uint8, device="cuda")
        cases.append((case, out, ws))

    def run(k, stream=None):
        (qx, sx, qgu, sgu, qdn, sdn), out, ws = cases[k]
        moe.int8_ffn(qx.m, sx, qgu.m, sgu, qdn.m, sdn, out, ws, stream=stream)

    alone = []
    for k in range(2):
        run(k)
        torch.cuda.synchronize()
        alone.append(cases[k][1].clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for k in range(2):
            run(k, streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(cases[k][1], alone[k])


def test_long_strides(moe):
    """Offsets past 32 bits: rows 2^28 bytes apart, the last one 2^32 bytes from the first."""
    T, H, ld = 17, 64, 1 << 28
    g = _gen(8)
    buf = torch.empty((T - 1) * ld + H, dtype=torch.int8, device="cuda")
    q = buf.as_strided((T, H), (ld, 1))
    x = _rn(g, T, H).bfloat16()
    s, s2, q2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, H, dtype=torch.int8, device="cuda")
    moe.quantize_rows(x, q, s)
    moe.quantize_rows(x, q2, s2)
    w, one = _codes(g, 24, H), torch.ones(24, device="cuda")
    a, b = torch.empty(T, 24, device="cuda"), torch.empty(T, 24, device="cuda")
    moe.int8_matmul(q, s, w, one, a)
    moe.int8_matmul(q2, s2, w, one, b)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(a, b)
    # the same matrix as weights: 17 channels
    moe.int8_matmul(w, one, q, s, out := torch.empty(24, T, device="cuda"))
    moe.int8_matmul(w, one, q2, s2, out2 := torch.empty(24, T, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out, out2)
    assert np.isfinite(out.cpu().numpy()).all()
