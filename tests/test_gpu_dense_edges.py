"""The dense operators at the ends of what their arguments may be."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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
