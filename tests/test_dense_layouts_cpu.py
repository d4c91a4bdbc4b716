"""The layouts of the dense operators' arguments, on the CPU: every call here is turned down
before any GPU work, for the reason that its message names."""
import ctypes

import pytest

import expert_offloaded_ffn_moe_amd as moe

torch = pytest.importorskip("torch")
BF, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8
T, H, N, I = 4, 32, 8, 16  # noqa: E741


def _z(*n, dt=BF):
    return torch.zeros(*n, dtype=dt)


# an entry point, its tensors, and which of them are matrices
CALLS = {
    "norm": (lambda **a: moe.rms_norm(a.pop("x"), a.pop("weight"), 1e-6, **a),
             lambda: dict(x=_z(T, H), weight=_z(H), add=_z(T, H, dt=F32), x_out=_z(T, H), out=_z(T, H), q_out=_z(T, H, dt=I8),
                          s_out=_z(T, dt=F32)), ["x", "add", "x_out", "out", "q_out"]),
    "quantize": (lambda **a: moe.quantize_rows(**a), lambda: dict(x=_z(T, H), q_out=_z(T, H, dt=I8), s_out=_z(T, dt=F32)),
                 ["x", "q_out"]),
    "matmul": (lambda **a: moe.int8_matmul(**a),
               lambda: dict(q_x=_z(T, H, dt=I8), s_x=_z(T, dt=F32), q_w=_z(N, H, dt=I8), s_w=_z(N, dt=F32), out=_z(T, N),
                            y_in=_z(T, N, dt=F32), res=_z(T, N)), ["q_x", "q_w", "out", "y_in", "res"]),
    "ffn": (lambda **a: moe.int8_ffn(**a),
            lambda: dict(q_x=_z(T, H, dt=I8), s_x=_z(T, dt=F32), q_gu=_z(2 * I, H, dt=I8), s_gu=_z(2 * I, dt=F32),
                         q_dn=_z(H, I, dt=I8), s_dn=_z(H, dt=F32), out=_z(T, H), workspace=_z(moe.int8_ffn_workspace(T, H, I), dt=U8),
                         y_in=_z(T, H, dt=F32), res=_z(T, H)), ["q_x", "q_gu", "q_dn", "out", "y_in", "res"]),
}
MATRICES = [(op, name) for op, (_, _, names) in CALLS.items() for name in names]


def _refusal(op, **change):
    call, args, _ = CALLS[op]
    with pytest.raises(moe.MoeError) as e:
        call(**{**args(), **change})
    assert e.value.status == moe.MOE_E_INVALID
    return str(e.value)


@pytest.mark.parametrize("op", list(CALLS))
def test_sound_layouts_reach_the_device_check(op):
    """What the changes below start from is turned down for being on the CPU alone."""
    assert "not on a GPU" in _refusal(op)


@pytest.mark.parametrize("op,name", MATRICES)
def test_row_of_a_broadcast_matrix(op, name):
    """One row for all: the ABI's stride of 0 stands for packed rows, which such a tensor does not hold."""
    m = CALLS[op][1]()[name]
    for rows in (m[:1].expand(*m.shape), m[0].expand(*m.shape)):
        assert rows.shape == m.shape and rows.stride(0) == 0
        msg = _refusal(op, **{name: rows})
        assert msg.startswith("moe_") and name + ": its rows overlap" in msg, msg


@pytest.mark.parametrize("op,name", MATRICES)
def test_rows_that_overlap(op, name):
    m = CALLS[op][1]()[name]
    rows = m.reshape(-1).as_strided(m.shape, (m.shape[1] - 1, 1))
    assert name + ": its rows overlap" in _refusal(op, **{name: rows})


def test_broadcast_single_element_rows():
    one = torch.zeros(1, 1, dtype=F32).expand(T, 1)
    args = dict(q_x=_z(T, H, dt=I8), s_x=_z(T, dt=F32), q_w=_z(1, H, dt=I8), s_w=_z(1, dt=F32), out=_z(T, 1, dt=F32))
    for name in ("y_in", "res", "out"):
        assert name + ": its rows overlap" in _refusal("matmul", **{**args, "y_in": None, "res": None, name: one})


def test_a_single_row_may_have_any_stride():
    m = torch.zeros(1, H, dtype=BF)
    for rows in (m.expand(1, H), m.as_strided((1, H), (0, 1)), m.as_strided((1, H), (5, 1))):
        assert moe._mat("moe_rms_norm", "x", rows, 1, H, BF, -1) == (rows.data_ptr(), H)


MB = 1 << 20


def _c_refusal(fn, args):
    """The message of a refused call of the C interface (its made-up addresses are never looked at)."""
    lib = moe.load_library()
    assert getattr(lib, fn)(ctypes.byref(args), None) == moe.MOE_E_INVALID
    return lib.moe_last_error().decode()


def test_largest_workspace_of_the_block():
    """2^20 tokens of 16384 intermediate channels, 80 GiB of workspace, within the documented
    sizes: the call gets past the workspace, to an output that overlaps it."""
    n, G = ctypes.c_size_t(), 1 << 30
    assert moe.load_library().moe_int8_ffn_workspace(1 << 20, 16, 16384, ctypes.byref(n)) == moe.MOE_OK
    assert n.value >= (1 << 20) * 16384 * 5
    a = dict(T=1 << 20, H=16, I=16384, out_dtype=1, q_x=MB, s_x=64 * MB, q_gu=96 * MB, s_gu=97 * MB, q_dn=98 * MB, s_dn=99 * MB,
             out=G, workspace=2 * G, workspace_bytes=n.value)
    assert _c_refusal("moe_int8_ffn", moe.Int8FfnArgs(**{**a, "out": 3 * G})) == "workspace overlaps out"
    assert "are needed" in _c_refusal("moe_int8_ffn", moe.Int8FfnArgs(**{**a, "workspace_bytes": n.value - 1}))
    assert _c_refusal("moe_int8_ffn", moe.Int8FfnArgs(**{**a, "workspace": 2 * G + 16})) == "workspace must be 256-byte aligned"
