"""The dense operators at the ends of their ranges: values whose intermediate products leave
fp32, and arguments that are refused.

Tolerances count roundings: one to fp32 is off by at most 2^-24 of its value, one to bf16 by
2^-8; a bf16 result under 2^-126 is a multiple of 2^-133 and off by half of that."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

R32, RBF = 2.0 ** -24, 2.0 ** -8
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
D = torch.float64


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


def _codes(g, rows, cols):
    return torch.randint(-127, 128, (rows, cols), device="cuda", dtype=torch.int8, generator=g)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-6, 2e-38])
@pytest.mark.parametrize("H", [40, 1500, 7000, 16000])
def test_norm_whose_products_leave_fp32(moe, act, eps, H):
    """s * weight beyond fp32's range, or among its subnormals, where the norm itself is
    ordinary: `out` follows the formula."""
    g, dt, eps = _gen(H), ACT[act], float(np.float32(eps))
    sizes = [126, 120, 70, 0, -60, -75, -110]
    x = _rn(g, len(sizes), H).clamp(-2, 2)
    x = (x.to(D) * (2.0 ** torch.tensor(sizes, device="cuda", dtype=D))[:, None]).to(dt)
    powers = torch.tensor([0, 10, -10, 100, -65, 0, -100, 61], device="cuda", dtype=D)
    w = ((1 + 0.1 * _rn(g, H)).to(D) * 2.0 ** powers[torch.arange(H, device="cuda") % 8]).to(dt)
    out = torch.empty_like(x)
    moe.rms_norm(x, w, eps, out=out)
    torch.cuda.synchronize()
    n = x.to(D) / (x.to(D).square().mean(1, keepdim=True) + eps).sqrt() * w.to(D)
    # fp32: the fp64 product rounded once; bf16: rstd and the product to fp32, then to bf16, where a
    # product among fp32's subnormals is off by 2^-150 and rstd, at most 2^10 then, takes that to 2^-140
    tol = (RBF + 2.02 * R32) * n.abs() + 1.02 * 2.0 ** -134 if act == "bf16" else 1.01 * R32 * n.abs() + 1.01 * 2.0 ** -150
    assert bool((n.abs() < 3e38).all())
    err = (out.to(D) - n).abs()
    assert bool((err <= tol).all()), [(sizes[i], int((~(err <= tol))[i].sum())) for i in range(len(sizes))]


def test_broadcast_rows_are_refused(moe):
    g, T, H, N = _gen(2), 4, 32, 8
    q, s, w, sw = _codes(g, T, H), torch.ones(T, device="cuda"), _codes(g, N, H), torch.ones(N, device="cuda")
    out = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    row, row32 = out.new_zeros(1, N).expand(T, N), s.new_zeros(N).expand(T, N)
    for change in (dict(res=row), dict(y_in=row32), dict(out=row), dict(q_x=q[:1].expand(T, H)), dict(q_w=w[0].expand(N, H))):
        with pytest.raises(moe.MoeError, match="its rows overlap"):
            moe.int8_matmul(**{**dict(q_x=q, s_x=s, q_w=w, s_w=sw, out=out), **change})
    x, weight = _rn(g, T, H).bfloat16(), _rn(g, H).bfloat16()
    for change in (dict(add=s.new_zeros(H).expand(T, H)), dict(x=x[:1].expand(T, H)), dict(out=x[0].expand(T, H))):
        with pytest.raises(moe.MoeError, match="its rows overlap"):
            moe.rms_norm(**{**dict(x=x, weight=weight, out=torch.empty_like(x)), **change})
    # the same values as rows of their own
    v = _rn(g, N)
    a = moe.int8_matmul(q, s, w, sw, torch.empty(T, N, device="cuda"), y_in=v.expand(T, N).contiguous())
    b = moe.int8_matmul(q, s, w, sw, torch.empty(T, N, device="cuda"), bias=v)
    assert torch.equal(a, b)
