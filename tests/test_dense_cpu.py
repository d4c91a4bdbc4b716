"""The dense operators' refusals and struct layouts, on the CPU: every call here is turned
down before any GPU work (made-up addresses are never looked at)."""
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


@pytest.mark.parametrize("cname,pyname,size", [("moe_rms_norm_args", "RmsNormArgs", 120),
                                               ("moe_quantize_args", "QuantizeArgs", 56),
                                               ("moe_int8_matmul_args", "Int8MatmulArgs", 120),
                                               ("moe_int8_ffn_args", "Int8FfnArgs", 152)])
def test_structs_match_header(cname, pyname, size):
    txt = open(os.path.join(ROOT, "include", "moe_offload.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % cname, txt).group(1)
    want = re.findall(r"([\w ]+?\*?)\s*(\w+)\s*;", body)
    kinds = {"int32_t": ctypes.c_int32, "float": ctypes.c_float, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t}
    fields = getattr(moe, pyname)._fields_
    assert [n for n, _ in fields] == [n for _, n in want]
    for (_, t), (c, n) in zip(fields, want):
        assert t is (ctypes.c_void_p if c.endswith("*") else kinds[c.strip()]), n
    assert ctypes.sizeof(getattr(moe, pyname)) == size


def norm(**kw):
    a = dict(T=4, H=256, act_dtype=1, add_dtype=0, eps=1e-6, x=MB, add=2 * MB, weight=3 * MB, x_out=4 * MB,
             out=5 * MB, q_out=6 * MB, s_out=7 * MB)
    a.update(kw)
    return moe.RmsNormArgs(**a)


def quant(**kw):
    a = dict(T=4, H=256, act_dtype=1, x=MB, q_out=2 * MB, s_out=3 * MB)
    a.update(kw)
    return moe.QuantizeArgs(**a)


def matmul(**kw):
    a = dict(T=4, N=100, K=256, out_dtype=1, q_x=MB, s_x=2 * MB, q_w=3 * MB, s_w=4 * MB, bias=5 * MB, y_in=6 * MB,
             res=7 * MB, out=8 * MB)
    a.update(kw)
    return moe.Int8MatmulArgs(**a)


def ffn(**kw):
    a = dict(T=4, H=256, I=64, out_dtype=1, q_x=MB, s_x=2 * MB, q_gu=3 * MB, s_gu=4 * MB, q_dn=5 * MB, s_dn=6 * MB,
             y_in=7 * MB, res=8 * MB, out=9 * MB, workspace=10 * MB, workspace_bytes=MB)
    a.update(kw)
    return moe.Int8FfnArgs(**a)


BAD_NORM = [dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0), dict(H=16385), dict(act_dtype=2), dict(add_dtype=7),
            dict(act_dtype=0, add_dtype=1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
            dict(eps=float("inf")), dict(x=None), dict(weight=None), dict(x=MB + 1), dict(add=2 * MB + 2),
            dict(x_out=None, out=None, q_out=None, s_out=None), dict(q_out=None), dict(s_out=None), dict(add=None),
            dict(ld_x=255), dict(ld_q=-1), dict(ld_out=(1 << 36) + 1), dict(x_out=5 * MB + 16), dict(out=MB + 64), dict(out=MB, ld_out=512),
            dict(q_out=MB), dict(s_out=MB), dict(weight=5 * MB), dict(out=2 * MB), dict(s_out=6 * MB + 256),
            # scales at the place of fp32 activations of the same stride
            dict(T=256, act_dtype=0, s_out=MB)]
BAD_QUANT = [dict(T=-1), dict(H=0), dict(H=16385), dict(act_dtype=-1), dict(x=None), dict(q_out=None), dict(s_out=None),
             dict(ld_x=10), dict(q_out=MB + 128), dict(s_out=2 * MB), dict(x=MB + 1), dict(s_out=3 * MB + 2)]
BAD_MATMUL = [dict(T=-1), dict(N=0), dict(K=0), dict(K=8), dict(K=24), dict(K=131072), dict(out_dtype=3), dict(q_x=None),
              dict(s_x=None), dict(q_w=None), dict(s_w=None), dict(out=None), dict(q_x=MB + 8), dict(q_w=3 * MB + 4),
              dict(ld_x=264), dict(ld_w=248), dict(ld_w=264), dict(ld_out=99), dict(out=MB), dict(out=3 * MB + 2),
              dict(out=7 * MB, ld_out=128), dict(out=6 * MB), dict(out=2 * MB), dict(out=4 * MB), dict(out=5 * MB),
              dict(bias=5 * MB + 2), dict(N=(1 << 24) + 1)]
BAD_FFN = [dict(T=-1), dict(H=8), dict(I=8), dict(I=16400), dict(H=264), dict(out_dtype=2), dict(q_x=None), dict(q_gu=None),
           dict(q_dn=None), dict(s_x=None), dict(s_gu=None), dict(s_dn=None), dict(out=None), dict(workspace=None),
           dict(workspace_bytes=1023), dict(workspace=10 * MB + 16), dict(workspace=9 * MB), dict(workspace=MB),
           dict(out=MB), dict(out=5 * MB), dict(res=10 * MB), dict(y_in=10 * MB), dict(ld_gu=100), dict(q_dn=5 * MB + 8)]


@pytest.mark.parametrize("kw", BAD_NORM)
def test_norm_refusals(lib, kw):
    assert lib.moe_rms_norm(ctypes.byref(norm(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


@pytest.mark.parametrize("kw", BAD_QUANT)
def test_quantize_refusals(lib, kw):
    assert lib.moe_quantize_rows(ctypes.byref(quant(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


@pytest.mark.parametrize("kw", BAD_MATMUL)
def test_matmul_refusals(lib, kw):
    assert lib.moe_int8_matmul(ctypes.byref(matmul(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


@pytest.mark.parametrize("kw", BAD_FFN)
def test_ffn_refusals(lib, kw):
    assert lib.moe_int8_ffn(ctypes.byref(ffn(**kw)), None) == INVALID
    assert len(lib.moe_last_error()) > 0


def test_null_args_and_no_rows(lib):
    for fn in (lib.moe_rms_norm, lib.moe_quantize_rows, lib.moe_int8_matmul, lib.moe_int8_ffn):
        assert fn(None, None) == INVALID
    # no rows: nothing is looked at but the sizes
    assert lib.moe_rms_norm(ctypes.byref(moe.RmsNormArgs(T=0, H=8, act_dtype=1, eps=1e-6)), None) == moe.MOE_OK
    assert lib.moe_quantize_rows(ctypes.byref(moe.QuantizeArgs(T=0, H=8)), None) == moe.MOE_OK
    assert lib.moe_int8_matmul(ctypes.byref(moe.Int8MatmulArgs(T=0, N=5, K=16)), None) == moe.MOE_OK
    assert lib.moe_int8_ffn(ctypes.byref(moe.Int8FfnArgs(T=0, H=16, I=16)), None) == moe.MOE_OK
    assert lib.moe_rms_norm(ctypes.byref(moe.RmsNormArgs(T=0, H=0, act_dtype=1, eps=1e-6)), None) == INVALID


def test_workspace_size(lib):
    n = ctypes.c_size_t(7)
    assert lib.moe_int8_ffn_workspace(0, 256, 64, ctypes.byref(n)) == moe.MOE_OK and n.value >= 0
    assert lib.moe_int8_ffn_workspace(3, 256, 64, ctypes.byref(n)) == moe.MOE_OK and n.value >= 3 * 64
    assert n.value % 256 == 0
    for bad in [(-1, 256, 64), (1, 250, 64), (1, 256, 60), (1, 256, 0), (1, 0, 64), (1, 256, 16400)]:
        assert lib.moe_int8_ffn_workspace(*bad, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.moe_int8_ffn_workspace(1, 256, 64, None) == INVALID


def test_binding_refuses_by_tensor():
    """The binding's own checks: shapes, types, strides and CPU tensors."""
    torch = pytest.importorskip("torch")
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    x = torch.zeros(4, 32, dtype=bf)
    calls = [
        lambda: moe.rms_norm(x, torch.zeros(32, dtype=bf), out=torch.zeros(4, 32, dtype=bf)),  # on the CPU
        lambda: moe.rms_norm(x.half(), torch.zeros(32, dtype=bf), out=x),
        lambda: moe.rms_norm(x[0], torch.zeros(32, dtype=bf), out=x),
        lambda: moe.quantize_rows(x.double(), torch.zeros(4, 32, dtype=i8), torch.zeros(4)),
        lambda: moe.int8_matmul(torch.zeros(4, 32), torch.zeros(4), torch.zeros(8, 32, dtype=i8), torch.zeros(8), torch.zeros(4, 8)),
        lambda: moe.int8_matmul(torch.zeros(4, 32, dtype=i8), torch.zeros(4), torch.zeros(8, dtype=i8), torch.zeros(8), torch.zeros(4, 8)),
        lambda: moe.int8_matmul(torch.zeros(4, 32, dtype=i8), torch.zeros(4), torch.zeros(8, 32, dtype=i8), torch.zeros(8), torch.zeros(4, 8, dtype=i8)),
    ]
    for f in calls:
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.status == INVALID
