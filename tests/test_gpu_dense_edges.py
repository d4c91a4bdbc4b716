"""The dense operators at the ends of their ranges: values whose intermediate products leave
fp32, layouts that share a buffer, and calls after an error of the caller's own.

Tolerances count roundings: one to fp32 is off by at most 2^-24 of its value, one to bf16 by
2^-8; a bf16 result under 2^-126 is a multiple of 2^-133 and off by half of that."""
import ctypes

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


def _out(moe, T, N, dt):
    return torch.full((T, N), 77, device="cuda", dtype=dt)


@pytest.mark.parametrize("out_act", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(1, 100, 256), (5, 33, 7168), (16, 6200, 256), (40, 100, 256), (300, 130, 512)])
def test_matmul_whose_scaled_sums_leave_fp32(moe, T, N, K, out_act):
    """Powers of two moved from a channel's scale to a token's change no bit, also where the
    sum times the token's scale alone is beyond fp32."""
    g, dt = _gen(T + N), ACT[out_act]
    q, w = _codes(g, T, K), _codes(g, N, K)
    q[0], w[0] = 127, 127  # a sum of 127 127 K
    sx, sw = torch.rand(T, device="cuda", generator=g) + 0.5, torch.rand(N, device="cuda", generator=g) + 0.5
    bias, y, res = _rn(g, N), _rn(g, T, N), _rn(g, T, N).to(dt)
    for more in ({}, dict(bias=bias, y_in=y, res=res)):
        want = moe.int8_matmul(q, sx, w, sw, _out(moe, T, N, dt), **more)
        for k in (64, 95, 96, 97, 110, 125):
            got = moe.int8_matmul(q, sx * 2.0 ** k, w, sw * 2.0 ** -k, _out(moe, T, N, dt), **more)
            torch.cuda.synchronize()
            assert torch.equal(got, want), k
    # and as it should be: what is finite comes out finite, what is not does not
    got = moe.int8_matmul(q, sx * 2.0 ** 110, w, sw * 2.0 ** -60, _out(moe, T, N, dt))
    v = (q.to(D) @ w.to(D).t()) * sx.to(D)[:, None] * sw.to(D) * 2.0 ** 50
    assert bool(((got.to(D) - v).abs() <= (3.03 * R32 + (RBF if out_act == "bf16" else 0)) * v.abs()).all())
    got = moe.int8_matmul(q, sx * 2.0 ** 110, w, sw * 2.0 ** 60, _out(moe, T, N, dt))
    acc = q.to(D) @ w.to(D).t()
    assert torch.equal(got, torch.where(acc == 0, acc, acc.sign() * float("inf")).to(dt))
    sx[0] = float("nan")
    sx[T - 1] = float("inf") if T > 1 else sx[0]
    got = moe.int8_matmul(q, sx, w, sw, _out(moe, T, N, dt))
    assert got[0].isnan().all() and int(got.isnan().sum()) == N + int((T > 1) * (acc[T - 1] == 0).sum())


@pytest.mark.parametrize("T,H,I", [(1, 2048, 128), (16, 2048, 768), (16, 96, 2048), (40, 2048, 272), (300, 2048, 128)])
def test_ffn_whose_scaled_sums_leave_fp32(moe, T, H, I):
    """As above for the block: between the token's scale and the gate and up channels', and
    between the up channels' (and so h, and the scales of its codes) and the down channels'."""
    g = _gen(T + I)
    q, gu, dn = _codes(g, T, H), _codes(g, 2 * I, H), _codes(g, H, I)
    q[0], gu[I] = 127, 127
    sx = torch.rand(T, device="cuda", generator=g) + 0.5
    sgu = (torch.rand(2 * I, device="cuda", generator=g) + 0.5) / (5000 * H ** 0.5)
    sdn = torch.rand(H, device="cuda", generator=g) + 0.5
    ws = torch.empty(moe.int8_ffn_workspace(T, H, I), dtype=torch.uint8, device="cuda")
    want = moe.int8_ffn(q, sx, gu, sgu, dn, sdn, _out(moe, T, H, torch.float32), ws)
    assert bool(want.isfinite().all()) and bool(want.any())
    for k in (64, 105):  # sgu stays above 2^-126
        got = moe.int8_ffn(q, sx * 2.0 ** k, gu, sgu * 2.0 ** -k, dn, sdn, _out(moe, T, H, torch.float32), ws)
        assert torch.equal(got, want), k
    up = sgu.clone()
    up[I:] *= 2.0 ** 114  # h under 2^126
    got = moe.int8_ffn(q, sx, gu, up, dn, sdn * 2.0 ** -114, _out(moe, T, H, torch.float32), ws)
    assert torch.equal(got, want)


def _hip():
    """The HIP runtime that this process runs on."""
    for line in open("/proc/self/maps"):
        if "libamdhip64" in line:
            return ctypes.CDLL(line.split()[-1])
    raise AssertionError("no HIP runtime is loaded")


def test_an_error_of_the_callers_own(moe):
    """A failed HIP call of the caller's (a device that there is not), its error not yet asked
    for: the operators report their own launches alone."""
    g, hip = _gen(1), _hip()
    x, w = _rn(g, 20, 256).bfloat16(), _rn(g, 256).bfloat16()
    q, s, out = torch.empty(20, 256, dtype=torch.int8, device="cuda"), torch.empty(20, device="cuda"), torch.empty_like(x)
    wq, ws = _codes(g, 256, 256), torch.ones(256, device="cuda")
    block = torch.empty(moe.int8_ffn_workspace(20, 256, 128), dtype=torch.uint8, device="cuda")
    calls = [lambda: moe.rms_norm(x, w, out=out), lambda: moe.quantize_rows(x, q, s),
             lambda: moe.int8_matmul(q, s, wq, ws, out),
             lambda: moe.int8_ffn(q, s, wq, ws, wq[:, :128], ws, out, block)]
    side = torch.cuda.Stream()
    for f in calls:
        f()
    torch.cuda.synchronize()
    for f in calls:
        for stream in (None, side):
            with torch.cuda.stream(stream):
                assert hip.hipSetDevice(1 << 20) != 0
                f()
                assert hip.hipGetLastError() == 0  # and leave nothing behind
            torch.cuda.synchronize()


def test_on_the_per_thread_stream(moe):
    """HIP's handle of the thread's own default stream."""
    g, per_thread = _gen(4), 2
    x, w = _rn(g, 20, 256).bfloat16(), _rn(g, 256).bfloat16()
    out, want = torch.empty_like(x), torch.empty_like(x)
    moe.rms_norm(x, w, out=want)
    torch.cuda.synchronize()
    moe.rms_norm(x, w, out=out, stream=per_thread)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


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


@pytest.mark.parametrize("T", [1, 5, 37, 300])
def test_columns_of_one_buffer(moe, T):
    """Matrices side by side in one buffer, as a fused projection leaves them."""
    g, H, N = _gen(T), 128, 256
    both = torch.full((T, 2 * H + 3), 77, device="cuda", dtype=torch.bfloat16)
    x, n = both[:, :H], both[:, H: 2 * H]
    x.copy_(_rn(g, T, H))
    w, one = _rn(g, H).bfloat16(), torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    moe.rms_norm(x, w, out=one)
    moe.rms_norm(x, w, out=n)
    torch.cuda.synchronize()
    assert torch.equal(n, one) and bool((both[:, 2 * H:] == 77).all())
    # codes of both halves into one buffer, and a product from one half over a part of the other
    codes = torch.full((T, 2 * H), 77, device="cuda", dtype=torch.int8)
    s, s2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.rms_norm(x, w, x_out=None, q_out=codes[:, H:], s_out=s)
    assert bool((codes[:, :H] == 77).all())
    moe.quantize_rows(x, codes[:, :H], s2)
    q, sw = _codes(g, N, H), torch.rand(N, device="cuda", generator=g)
    outs = torch.full((T, 3 * N), 77.0, device="cuda")
    outs[:, N: 2 * N] = _rn(g, T, N)
    want = moe.int8_matmul(codes[:, :H].contiguous(), s2, q, sw, torch.empty(T, N, device="cuda"), y_in=outs[:, N: 2 * N])
    moe.int8_matmul(codes[:, :H], s2, q, sw, outs[:, 2 * N:], y_in=outs[:, N: 2 * N])
    torch.cuda.synchronize()
    assert torch.equal(outs[:, 2 * N:], want) and bool((outs[:, :N] == 77).all())


def test_block_of_the_largest_workspace(moe):
    """2^20 tokens of 16384 intermediate channels: 80 GiB of workspace, offsets past 2^36 bytes.
    Tokens from all over are bit for bit what they are in small calls."""
    T, H, I = 1 << 20, 16, 16384  # noqa: E741
    n = moe.int8_ffn_workspace(T, H, I)
    if torch.cuda.mem_get_info()[0] < n + (4 << 30):
        pytest.skip("needs %d GiB of device memory" % ((n >> 30) + 4))
    g = _gen(3)
    q, gu, dn = _codes(g, T, H), _codes(g, 2 * I, H), _codes(g, H, I)
    sx, sgu, sdn = (torch.rand(k, device="cuda", generator=g) * 0.01 + 0.01 for k in (T, 2 * I, H))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = moe.int8_ffn(q, sx, gu, sgu, dn, sdn, _out(moe, T, H, torch.float32), ws)
    torch.cuda.synchronize()
    assert bool(out.isfinite().all())
    for a, b in [(0, 300), (T // 2 - 9, T // 2 + 7), (T * 13 // 16, T * 13 // 16 + 1), (T - 40, T)]:
        part = moe.int8_ffn(q[a:b], sx[a:b], gu, sgu, dn, sdn, _out(moe, b - a, H, torch.float32), ws)
        assert torch.equal(part, out[a:b]), (a, b)
    del ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,N,K", [(1, 1 << 24, 16), (17, 1 << 24, 16), (1 << 20, 1, 16), (1 << 20, 33, 32), (5, 1 << 24, 32)])
def test_matmul_of_the_largest_sizes(moe, T, N, K):
    g = _gen(6)
    q, w = _codes(g, T, K), _codes(g, N, K)
    out = moe.int8_matmul(q, torch.ones(T, device="cuda"), w, torch.ones(N, device="cuda"), _out(moe, T, N, torch.float32))
    # sums under 2^24, exact in fp32
    assert torch.equal(out, q.float() @ w.float().t())


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_norm_and_codes_of_the_most_rows(moe, act):
    T, H, g, dt = 1 << 20, 5, _gen(7), ACT[act]
    x, w = _rn(g, T, H).to(dt), (1 + 0.1 * _rn(g, H)).to(dt)
    out, q, s = torch.empty_like(x), torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.rms_norm(x, w, 1e-6, out=out, q_out=q, s_out=s)
    n = x.to(D) / (x.to(D).square().mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt() * w.to(D)
    assert bool(((out.to(D) - n).abs() <= (RBF + 2.02 * R32 if act == "bf16" else 1.01 * R32) * n.abs() + 2.0 ** -134).all())
    p = x.to(D) * w.to(D)
    assert torch.equal(q.to(D), torch.round(127 * p / p.abs().amax(1, keepdim=True)))
    moe.quantize_rows(x, q, s)
    top = x.to(D).abs().amax(1)
    assert torch.equal(q.to(D), torch.round(127 * x.to(D) / top[:, None]))
    assert bool(((s.to(D) - top / 127).abs() <= 1.01 * R32 * top / 127).all())


def test_block_of_the_longest_rows(moe):
    """131056 channels, the most: a sum of K for the gated product, channels for the second."""
    T, H, I = 20, 131056, 32  # noqa: E741
    g = _gen(8)
    q, gu, dn = _codes(g, T, H), _codes(g, 2 * I, H), _codes(g, H, I)
    sx, sgu, sdn = (torch.rand(k, device="cuda", generator=g) + 0.5 for k in (T, 2 * I, H))
    sgu /= 5000 * H ** 0.5
    run = lambda a, b: moe.int8_ffn(q[a:b], sx[a:b], gu, sgu, dn, sdn, _out(moe, b - a, H, torch.float32),  # noqa: E731
                                    torch.empty(moe.int8_ffn_workspace(b - a, H, I), dtype=torch.uint8, device="cuda"))
    whole = run(0, T)
    for a, b in [(0, 1), (3, 19), (7, 9)]:
        assert torch.equal(run(a, b), whole[a:b])
    import test_gpu_dense as TD
    p, tol, _ = TD._ffn_ref(q, sx, gu, sgu, dn, sdn)
    assert bool(((whole.to(D) - p).abs() <= tol * 1.01 + TD._product_tol(p.abs() + tol, [], "f32")).all())


def test_over_every_input_that_may_be(moe):
    """The norm over its x (the sum over its addend), a product over y_in and res at once."""
    g, H = _gen(9), 900
    for T in (1, 6, 700):
        x, r, w = _rn(g, T, H), _rn(g, T, H), _rn(g, H)
        xo, out = torch.empty_like(x), torch.empty_like(x)
        moe.rms_norm(x, w, add=r, x_out=xo, out=out)
        moe.rms_norm(x, w, add=r, x_out=r, out=x)
        assert torch.equal(x, out) and torch.equal(r, xo)
        moe.rms_norm(x, w, out=out)
        moe.rms_norm(x, w, out=x)
        assert torch.equal(x, out)
        moe.rms_norm(x, w, add=x, out=out)
        moe.rms_norm(x, w, add=x, out=x)
        assert torch.equal(x, out)
        q, wq, y = _codes(g, T, 64), _codes(g, H, 64), _rn(g, T, H)
        sx, sw = torch.rand(T, device="cuda", generator=g), torch.rand(H, device="cuda", generator=g)
        want = moe.int8_matmul(q, sx, wq, sw, torch.empty_like(y), y_in=y, res=y)
        assert torch.equal(moe.int8_matmul(q, sx, wq, sw, y, y_in=y, res=y), want)


def test_two_threads_at_once(moe):
    """Calls from two threads, refused ones among them, each with its own stream and buffers."""
    import threading
    cases, wants, faults = [], [], []
    for k, (T, H, I) in enumerate([(2, 1024, 256), (90, 512, 768)]):  # noqa: E741
        g = _gen(30 + k)
        q, gu, dn = _codes(g, T, H), _codes(g, 2 * I, H), _codes(g, H, I)
        sx, sgu, sdn = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (T, 2 * I, H))
        ws = torch.empty(moe.int8_ffn_workspace(T, H, I), dtype=torch.uint8, device="cuda")
        cases.append((q, sx, gu, sgu, dn, sdn, _out(moe, T, H, torch.float32), ws))
        wants.append(moe.int8_ffn(*cases[k]).clone())
    torch.cuda.synchronize()

    def work(k):
        stream = torch.cuda.Stream()
        for _ in range(200):
            moe.int8_ffn(*cases[k], stream=stream)
            try:
                moe.int8_ffn(*cases[k][:6], cases[k][6][:, : 16 * (k + 1)], cases[k][7], stream=stream)
                faults.append("not refused")
            except moe.MoeError as e:
                if "%d)" % (16 * (k + 1)) not in str(e):
                    faults.append(str(e))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults
    for k in range(2):
        assert torch.equal(cases[k][6], wants[k])


def test_tiles_captured_twice_on_one_workspace(moe):
    """Two graphs that share a workspace and a stream, replayed in turn with eager calls between."""
    T, H, I = 300, 512, 256  # noqa: E741
    g = _gen(40)
    gu, dn, q, sx = _codes(g, 2 * I, H), _codes(g, H, I), _codes(g, 2 * T, H), torch.rand(2 * T, device="cuda", generator=g) * 0.01
    sgu, sdn = torch.rand(2 * I, device="cuda", generator=g) * 0.01, torch.rand(H, device="cuda", generator=g)
    ws = torch.empty(moe.int8_ffn_workspace(T, H, I), dtype=torch.uint8, device="cuda")
    x, w = _rn(g, T, H), _rn(g, H)
    codes, scales, side = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.cuda.Stream()
    outs = [_out(moe, T, H, torch.float32) for _ in range(2)]
    calls = [lambda: moe.int8_ffn(q[:T], sx[:T], gu, sgu, dn, sdn, outs[0], ws),
             lambda: (moe.rms_norm(x, w, q_out=codes, s_out=scales),
                      moe.int8_ffn(codes, scales, gu, sgu, dn, sdn, outs[1], ws, res=x))]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    with torch.cuda.stream(side):
        for graph, call in zip(graphs, calls):
            call()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                call()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(_rn(g, T, H))
        q.copy_(_codes(g, 2 * T, H))
        wants = []
        for call, out in zip(calls, outs):
            call()
            torch.cuda.synchronize()
            wants.append(out.clone())
            out.zero_()
        ws.fill_(255)
        with torch.cuda.stream(side):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for out, want in zip(outs, wants):
            assert torch.equal(out, want), i
