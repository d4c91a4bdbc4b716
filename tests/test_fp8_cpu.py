"""Refusals, struct layouts and workspace sizes of the operators on e4m3 codes, on the CPU:
every call here is turned down before any GPU work (made-up addresses are never looked at)."""
import ctypes
import os
import re

import pytest

import expert_offloaded_ffn_moe_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MB = 1 << 20
INVALID = moe.MOE_E_INVALID


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail("library not built: run __graft_entry__.build()")
    return moe.load_library(with_torch=False)


@pytest.mark.parametrize("cname,pyname,size", [("moe_fp8_quantize_args", "Fp8QuantizeArgs", 64),
                                               ("moe_fp8_matmul_args", "Fp8MatmulArgs", 136),
                                               ("moe_fp8_layer_args", "Fp8LayerArgs", 176)])
def test_structs_match_header(cname, pyname, size):
    txt = open(os.path.join(ROOT, "include", "moe_offload.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % cname, txt).group(1)
    want = re.findall(r"([\w ]+?\*?)\s*(\w+)\s*;", body)
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t}
    fields = getattr(moe, pyname)._fields_
    assert [n for n, _ in fields] == [n for _, n in want]
    for (_, t), (c, n) in zip(fields, want):
        assert t is (ctypes.c_void_p if c.endswith("*") else kinds[c.strip()]), n
    assert ctypes.sizeof(getattr(moe, pyname)) == size


def quant(**kw):
    return moe.Fp8QuantizeArgs(**{**dict(T=4, H=256, act_dtype=1, block_rows=1, x=MB, q_out=2 * MB, s_out=3 * MB), **kw})


def matmul(**kw):
    a = dict(T=4, N=100, K=256, out_dtype=1, q_x=MB, s_x=2 * MB, q_w=3 * MB, s_w=4 * MB, bias=5 * MB, y_in=6 * MB,
             res=7 * MB, out=8 * MB)
    return moe.Fp8MatmulArgs(**{**a, **kw})


def layer(**kw):
    a = dict(T=4, H=256, I=64, E=8, k=2, act_dtype=1, x=MB, router_w=2 * MB, router_b=3 * MB, q_gu=4 * MB, s_gu=5 * MB,
             q_dn=6 * MB, s_dn=7 * MB, y=8 * MB, x_out=9 * MB, logits=10 * MB, topk_ids=11 * MB, topk_w=12 * MB,
             workspace=13 * MB, workspace_bytes=MB)
    return moe.Fp8LayerArgs(**{**a, **kw})


BAD_QUANT = [dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0), dict(H=(1 << 20) + 1), dict(act_dtype=2), dict(block_rows=0),
             dict(block_rows=2), dict(block_rows=-1), dict(x=None), dict(q_out=None), dict(s_out=None), dict(ld_x=255),
             dict(ld_q=-1), dict(ld_s=1), dict(x=MB + 1), dict(s_out=3 * MB + 2), dict(q_out=MB + 64), dict(s_out=MB),
             dict(s_out=2 * MB)]
BAD_MATMUL = [dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=8), dict(K=24),
              dict(K=131072), dict(out_dtype=3), dict(q_x=None), dict(s_x=None), dict(q_w=None), dict(s_w=None), dict(out=None),
              dict(q_x=MB + 8), dict(q_w=3 * MB + 4), dict(ld_x=264), dict(ld_w=248), dict(ld_sx=1), dict(ld_sw=-2),
              dict(s_x=2 * MB + 2), dict(ld_out=99), dict(out=MB), dict(out=2 * MB), dict(out=3 * MB), dict(out=4 * MB),
              dict(out=5 * MB), dict(out=6 * MB), dict(out=7 * MB, ld_out=128), dict(out=8 * MB + 1), dict(bias=5 * MB + 2)]
BAD_LAYER = [dict(T=-1), dict(T=65), dict(H=0), dict(H=8), dict(H=264), dict(H=131072), dict(I=8), dict(I=72), dict(I=16400),
             dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(act_dtype=2), dict(x=None),
             dict(router_w=None), dict(q_gu=None), dict(s_gu=None), dict(q_dn=None), dict(s_dn=None), dict(y=None),
             dict(workspace=None), dict(workspace_bytes=511), dict(workspace=13 * MB + 128), dict(x=MB + 1), dict(ld_x=100),
             dict(ld_router=255), dict(ld_y=1), dict(ld_x_out=8), dict(q_gu=4 * MB + 8), dict(q_dn=6 * MB + 4),
             dict(s_gu=5 * MB + 1), dict(router_b=3 * MB + 2), dict(logits_in=14 * MB + 2), dict(x_out=MB + 2),
             dict(x_out=MB, ld_x_out=512), dict(x_out=8 * MB), dict(y=MB), dict(y=2 * MB), dict(y=4 * MB), dict(y=5 * MB),
             dict(y=6 * MB), dict(logits=MB), dict(logits=14 * MB, logits_in=14 * MB), dict(topk_ids=8 * MB),
             dict(topk_w=11 * MB), dict(workspace=MB), dict(workspace=6 * MB), dict(workspace=8 * MB), dict(topk_ids=13 * MB)]


@pytest.mark.parametrize("kw", BAD_QUANT)
def test_quantize_refusals(lib, kw):
    assert lib.moe_fp8_quantize(ctypes.byref(quant(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


@pytest.mark.parametrize("kw", BAD_MATMUL)
def test_matmul_refusals(lib, kw):
    assert lib.moe_fp8_matmul(ctypes.byref(matmul(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


@pytest.mark.parametrize("kw", BAD_LAYER)
def test_layer_refusals(lib, kw):
    assert lib.moe_fp8_layer(ctypes.byref(layer(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


def test_null_args_and_no_rows(lib):
    for fn in (lib.moe_fp8_quantize, lib.moe_fp8_matmul, lib.moe_fp8_layer):
        assert fn(None, None) == INVALID
    # no rows: nothing is looked at but the sizes
    assert lib.moe_fp8_quantize(ctypes.byref(moe.Fp8QuantizeArgs(T=0, H=8, block_rows=1)), None) == moe.MOE_OK
    assert lib.moe_fp8_matmul(ctypes.byref(moe.Fp8MatmulArgs(T=0, N=5, K=16)), None) == moe.MOE_OK
    assert lib.moe_fp8_layer(ctypes.byref(moe.Fp8LayerArgs(T=0, H=16, I=16, E=1, k=1)), None) == moe.MOE_OK
    assert lib.moe_fp8_layer(ctypes.byref(moe.Fp8LayerArgs(T=0, H=16, I=16, E=1, k=2)), None) == INVALID


def test_workspace_size(lib):
    n = ctypes.c_size_t(7)
    assert lib.moe_fp8_layer_workspace(0, 256, 64, 8, 2, ctypes.byref(n)) == moe.MOE_OK
    assert lib.moe_fp8_layer_workspace(3, 256, 64, 8, 2, ctypes.byref(n)) == moe.MOE_OK
    assert n.value >= 3 * 8 * 4 + 3 * 2 * 64 * 4 and n.value % 256 == 0
    for bad in [(-1, 256, 64, 8, 2), (65, 256, 64, 8, 2), (1, 250, 64, 8, 2), (1, 256, 60, 8, 2), (1, 256, 64, 0, 1),
                (1, 256, 64, 8, 9), (1, 256, 64, 1025, 1)]:
        assert lib.moe_fp8_layer_workspace(*bad, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.moe_fp8_layer_workspace(1, 256, 64, 8, 2, None) == INVALID
    with pytest.raises(moe.MoeError):
        moe.fp8_layer_workspace(1 << 32, 256, 64, 8, 2)


# ---- the binding's own checks, by tensor

torch = pytest.importorskip("torch")
BF, F32, F8, U8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.int32
T, H, N, I, E, K = 4, 144, 136, 32, 3, 2  # noqa: E741


def _z(*n, dt=F32):
    return torch.zeros(*n, dtype=dt)


CALLS = {
    "quantize": (lambda **a: moe.fp8_quantize(**a), lambda: dict(x=_z(T, H, dt=BF), q_out=_z(T, H, dt=F8), s_out=_z(T, 2)),
                 ["x", "q_out", "s_out"], []),
    "matmul": (lambda **a: moe.fp8_matmul(**a),
               lambda: dict(q_x=_z(T, H, dt=F8), s_x=_z(T, 2), q_w=_z(N, H, dt=F8), s_w=_z(2, 2), out=_z(T, N, dt=BF), bias=_z(N),
                            y_in=_z(T, N), res=_z(T, N, dt=BF)), ["q_x", "s_x", "q_w", "s_w", "out", "y_in", "res"], ["bias"]),
    "layer": (lambda **a: moe.fp8_layer(**a),
              lambda: dict(x=_z(T, H, dt=BF), router_w=_z(E, H, dt=BF), q_gu=_z(E, 2 * I, H, dt=F8), s_gu=_z(E, 2, 1, 2),
                           q_dn=_z(E, H, I, dt=F8), s_dn=_z(E, 2, 1), k=K, y=_z(T, H),
                           workspace=_z(moe.fp8_layer_workspace(T, H, I, E, K), dt=U8), router_b=_z(E), logits_in=_z(T, E),
                           x_out=_z(T, H, dt=BF), logits=_z(T, E), topk_ids=_z(T, K, dt=I32), topk_w=_z(T, K)),
              ["x", "router_w", "y", "x_out"],
              ["q_gu", "s_gu", "q_dn", "s_dn", "workspace", "router_b", "logits_in", "logits", "topk_ids", "topk_w"]),
}
MATRICES = [(op, name) for op, c in CALLS.items() for name in c[2]]
PACKED = [(op, name) for op, c in CALLS.items() for name in c[3]]


def _refusal(op, **change):
    with pytest.raises(moe.MoeError) as e:
        CALLS[op][0](**{**CALLS[op][1](), **change})
    assert e.value.status == INVALID
    return str(e.value)


@pytest.mark.parametrize("op", list(CALLS))
def test_sound_tensors_reach_the_device_check(op):
    """What the changes below start from is turned down for being on the CPU alone."""
    assert "not on a GPU" in _refusal(op)


@pytest.mark.parametrize("op,name", MATRICES)
def test_matrix_layouts(op, name):
    m = CALLS[op][1]()[name]
    assert name + ": its rows overlap" in _refusal(op, **{name: m[:1].expand(*m.shape)})
    wide = torch.zeros(m.shape[0], 2 * m.shape[1], dtype=m.dtype)
    assert "not on a GPU" in _refusal(op, **{name: wide[:, :m.shape[1]]})  # a row stride of its own is sound
    if name not in ("x", "q_x"):  # whose shape the others are measured by
        _refusal(op, **{name: wide[:, ::2]})
        _refusal(op, **{name: wide})
        if name != "out":
            assert name + " has dtype" in _refusal(op, **{name: m.to(torch.float64)})


@pytest.mark.parametrize("op,name", PACKED)
def test_packed_layouts(op, name):
    m = CALLS[op][1]()[name]
    wide = torch.zeros(*m.shape[:-1], 2 * m.shape[-1], dtype=m.dtype)
    _refusal(op, **{name: wide[..., ::2]})
    _refusal(op, **{name: wide})
    assert name + " has dtype" in _refusal(op, **{name: m.to(torch.float64)})


def test_types_and_numbers():
    assert "block_rows" in _refusal("quantize", block_rows=64)
    assert "float64" in _refusal("quantize", x=_z(T, H, dt=torch.float64))
    assert "q_out has dtype" in _refusal("quantize", q_out=_z(T, H, dt=torch.float8_e5m2))
    _refusal("quantize", block_rows=128)
    assert "q_dn has 2 dimensions" in _refusal("layer", q_dn=_z(H, I, dt=F8))
    _refusal("layer", k=3)
    assert "out of range" in _refusal("layer", k=1 << 40, topk_ids=None, topk_w=None)
    assert "float16" in _refusal("layer", x=_z(T, H, dt=torch.float16))
