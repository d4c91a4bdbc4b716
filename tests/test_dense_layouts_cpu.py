"""The layouts of the dense operators' arguments, on the CPU: every call here is turned down
before any GPU work, for the reason that its message names."""
import ctypes
import random

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


def _bytes(at, rows, cols, ld, size):
    return {at + r * ld * size + c for r in range(rows) for c in range(cols * size)}


def test_overlap_is_of_elements():
    """Codes at every kind of place beside their rows: refused where they share a byte, let by
    where the strides are equal and they do not (two unlike strides that interleave are refused
    as well). Calls that get by the check are turned down for the scales, which stand in the codes."""
    rng, seen = random.Random(5), [0, 0, 0]
    for _ in range(4000):
        rows, cols, f32 = rng.randint(1, 4), rng.randint(1, 6), rng.random() < 0.5
        size = 4 if f32 else 2
        ld_x = cols + rng.randint(0, 8)
        ld_q = ld_x * size if rng.random() < 0.7 else cols + rng.randint(0, 30)
        at = MB + rng.randint(-2 * ld_x * size - 8, (rows + 1) * ld_x * size)
        args = moe.QuantizeArgs(T=rows, H=cols, act_dtype=0 if f32 else 1, x=MB, ld_x=ld_x, q_out=at, ld_q=max(ld_q, cols),
                                s_out=at // 4 * 4)
        x, q = _bytes(MB, rows, cols, ld_x, size), _bytes(at, rows, cols, max(ld_q, cols), 1)
        if x & _bytes(args.s_out, 1, rows, rows, 4) and not x & q:
            continue  # the scales stand in x as well
        msg = _c_refusal("moe_quantize_rows", args)
        if x & q:
            assert msg == "q_out overlaps x", (rows, cols, size, ld_x, ld_q, at - MB)
            seen[0] += 1
        elif rows == 1 or ld_q == ld_x * size:
            assert msg != "q_out overlaps x", (rows, cols, size, ld_x, ld_q, at - MB)
            seen[1] += 1
        else:
            assert msg in ("q_out overlaps x", "s_out overlaps x", "s_out overlaps q_out")
            seen[2] += 1
    assert min(seen) > 200, seen


def test_columns_of_one_buffer_get_by():
    """Every operator's matrices side by side in one buffer; the scales (the bias, the
    workspace) stand in an output, for which the call is turned down in the end."""
    H, ld = 256, 1024
    a = dict(T=4, H=H, act_dtype=1, add_dtype=1, eps=1e-6, x=MB, ld_x=ld, add=MB + 2 * H, ld_add=ld, weight=3 * MB,
             x_out=MB + 4 * H, ld_x_out=ld, out=MB + 6 * H, ld_out=ld, q_out=6 * MB, s_out=6 * MB)
    assert _c_refusal("moe_rms_norm", moe.RmsNormArgs(**a)) == "s_out overlaps q_out"
    assert _c_refusal("moe_rms_norm", moe.RmsNormArgs(**{**a, "out": MB + 6 * H - 2})) == "out overlaps x_out"
    assert _c_refusal("moe_rms_norm", moe.RmsNormArgs(**{**a, "out": MB + 6 * H + 2})) == "out overlaps x"
    assert _c_refusal("moe_rms_norm", moe.RmsNormArgs(**{**a, "weight": MB + 4 * H})) == "x_out overlaps weight"
    a = dict(T=4, N=100, K=256, out_dtype=1, q_x=MB, s_x=2 * MB, q_w=3 * MB, s_w=4 * MB, res=8 * MB, ld_res=250, out=8 * MB + 200,
             ld_out=250, y_in=8 * MB + 400, ld_y=125, bias=8 * MB + 200)
    assert _c_refusal("moe_int8_matmul", moe.Int8MatmulArgs(**a)) == "out overlaps y_in"
    a["ld_res"], a["ld_out"], a["ld_y"] = 400, 400, 200
    assert _c_refusal("moe_int8_matmul", moe.Int8MatmulArgs(**a)) == "out overlaps bias"
    a = dict(T=4, H=256, I=64, out_dtype=1, q_x=MB, s_x=2 * MB, q_gu=3 * MB, s_gu=4 * MB, q_dn=5 * MB, s_dn=6 * MB, res=8 * MB,
             ld_res=512, out=8 * MB + 512, ld_out=512, workspace=8 * MB + 512, workspace_bytes=MB)
    assert _c_refusal("moe_int8_ffn", moe.Int8FfnArgs(**a)).startswith("workspace overlaps")
    assert _c_refusal("moe_int8_ffn", moe.Int8FfnArgs(**{**a, "out": 8 * MB + 2})) == "out overlaps res"


def test_sizes_beyond_the_abi():
    """Sizes and numbers that the C structs cannot hold are refused like others out of range."""
    for sizes in [((1 << 32) + 3, 256, 64), (3, (1 << 32) + 256, 64), (3, 256, (1 << 32) + 64), (-(1 << 32) + 3, 256, 64)]:
        with pytest.raises(moe.MoeError) as e:
            moe.int8_ffn_workspace(*sizes)
        assert e.value.status == moe.MOE_E_INVALID
    rows = (1 << 31) + 16
    far = lambda *n, dt=I8: torch.empty(*n, dtype=dt, device="meta")  # noqa: E731
    many = dict(T=far(rows, 16), v=far(rows, dt=F32), out=far(rows, 16, dt=BF))
    calls = [
        lambda: moe.rms_norm(many["out"], far(16, dt=BF), out=many["out"]),
        lambda: moe.quantize_rows(many["out"], many["T"], many["v"]),
        lambda: moe.int8_matmul(many["T"], many["v"], far(16, 16), far(16, dt=F32), many["out"]),
        lambda: moe.int8_matmul(far(16, 16), far(16, dt=F32), many["T"], many["v"], far(16, rows, dt=BF)),
        lambda: moe.int8_ffn(many["T"], many["v"], far(32, 16), far(32, dt=F32), far(16, 16), far(16, dt=F32), many["out"],
                             far(256, dt=U8)),
    ]
    for f in calls:
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.status == moe.MOE_E_INVALID
