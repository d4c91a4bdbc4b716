"""Operators on 8-bit floating-point codes (e4m3) with a scale for each block of 128: codes of
activations and weights, the matrix product, and a whole routed layer for a few tokens on
experts held so. Cases, inputs, plain forms and 64-bit values.

Codes of a block v: amax = max |v|, scale = amax / 448, code = the e4m3 number nearest to
448 v / amax, ties to even. A block is 128 neighbours of a row (activations) or 128 x 128
(weights); blocks at a matrix's edge are cut short.
"""
import torch

own = False

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
B = 128


def listed():
    return [
        # attention's output of one token, before its projection
        {"name": "quantize token", "op": "quant", "T": 1, "H": 7168, "act": "bf16", "rows": 1},
        # fp32 activations, a ragged batch whose last block is short
        {"name": "quantize ragged", "op": "quant", "T": 1023, "H": 2000, "act": "f32", "rows": 1},
        # a projection's weight matrix, once when a model is loaded
        {"name": "quantize weight", "op": "quant", "T": 7168, "H": 2048, "act": "bf16", "rows": 128},
        # a square projection of one token, onto the residual stream
        {"name": "matmul decode", "op": "matmul", "T": 1, "N": 7168, "K": 7168, "out": "bf16", "bias": False, "add": "res"},
        # a decode batch of 64 sequences
        {"name": "matmul batch", "op": "matmul", "T": 64, "N": 4096, "K": 7168, "out": "bf16", "bias": False, "add": "both"},
        # ragged in every direction, with bias, fp32 out
        {"name": "matmul ragged", "op": "matmul", "T": 333, "N": 1001, "K": 2064, "out": "f32", "bias": True, "add": "none"},
        # the square projection of a prefill micro-batch
        {"name": "matmul prefill", "op": "matmul", "T": 2048, "N": 7168, "K": 7168, "out": "bf16", "bias": False, "add": "none"},
        # a small layer whose sizes fit no block, fp32 activations
        {"name": "layer ragged", "op": "layer", "T": 7, "H": 400, "I": 208, "E": 24, "k": 3, "act": "f32"},
        # one token through the 2048-wide layer
        {"name": "layer narrow token", "op": "layer", "T": 1, "H": 2048, "I": 768, "E": 128, "k": 8, "act": "bf16"},
        # a decode batch through it: the hot experts take several tokens each
        {"name": "layer narrow batch", "op": "layer", "T": 16, "H": 2048, "I": 768, "E": 128, "k": 8, "act": "bf16"},
        # one token through the 7168-wide layer of 384 experts
        {"name": "layer wide token", "op": "layer", "T": 1, "H": 7168, "I": 2048, "E": 384, "k": 6, "act": "bf16"},
        # a decode batch through it
        {"name": "layer wide batch", "op": "layer", "T": 16, "H": 7168, "I": 2048, "E": 384, "k": 6, "act": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "layer", "layer", "layer"])
    if op == "quant":
        return {"op": op, "T": _log(rng, 1, 7168), "H": _log(rng, 100, 7168), "act": rng.choice(["bf16", "bf16", "f32"]),
                "rows": rng.choice([1, 1, 128])}
    if op == "matmul":
        return {"op": op, "T": _log(rng, 1, 2048), "N": _log(rng, 64, 7168), "K": 16 * _log(rng, 8, 448),
                "out": rng.choice(["bf16", "bf16", "f32"]), "bias": rng.random() < 0.5, "add": rng.choice(["none", "res", "both"])}
    k, H, I = rng.randint(1, 8), 16 * _log(rng, 16, 448), 16 * _log(rng, 8, 128)  # noqa: E741
    most = min(64, max(1, 16 * 6 * 7168 * 2048 // (k * H * I)))  # the listed batch's products
    return {"op": op, "T": _log(rng, 1, most), "H": H, "I": I, "E": _log(rng, 8, 384), "k": k,
            "act": rng.choice(["bf16", "bf16", "f32"])}


def _up(n):
    return -(-n // B)


def _spread(s, rows, cols, by=B):
    """The scales of blocks at each of the matrix's elements."""
    return s.repeat_interleave(by, -2)[..., :rows, :].repeat_interleave(B, -1)[..., :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rn = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
    new = lambda *n, dt: torch.empty(*n, device="cuda", dtype=dt)  # noqa: E731

    def codes(*n):  # codes of normal values, whose blocks reach 448 at about four standard deviations
        return rn(*n).mul_(108.0).clamp_(-448.0, 448.0).to(F8)

    def scales(*n, width):  # of weights that keep an activation's size
        return torch.exp(0.2 * rn(*n)) / (108.0 * width ** 0.5)

    s, T = {"case": case, "op": case["op"]}, case["T"]
    if case["op"] == "quant":
        H, r = case["H"], case["rows"]
        s["x"] = (rn(T, H) * torch.exp(0.3 * rn(H))).to(ACT[case["act"]])
        s["codes"], s["scale"] = new(T, H, dt=F8), new(-(-T // r), _up(H), dt=torch.float32)
        s["values"] = new(T, H, dt=torch.float32)
        return s
    if case["op"] == "matmul":
        N, K, act = case["N"], case["K"], ACT[case["out"]]
        s["w"], s["sw"] = codes(N, K), scales(_up(N), _up(K), width=K)
        s["q"], s["sx"] = codes(T, K), torch.exp(0.3 * rn(T, _up(K))) / 108.0
        s["bias"] = rn(N) if case["bias"] else None
        s["y"] = rn(T, N) if case["add"] == "both" else None
        s["res"] = rn(T, N).to(act) if case["add"] in ("res", "both") else None
        s["out"] = new(T, N, dt=act)
        return s
    H, I, E, k, act = case["H"], case["I"], case["E"], case["k"], ACT[case["act"]]
    s["w_gu"], s["w_dn"] = new(E, 2 * I, H, dt=F8), new(E, H, I, dt=F8)
    for e in range(E):
        s["w_gu"][e], s["w_dn"][e] = codes(2 * I, H), codes(H, I)
    s["s_gu"] = scales(E, 2, _up(I), _up(H), width=H)
    s["s_dn"] = scales(E, _up(H), _up(I), width=I)
    s["x"] = (rn(T, H) * torch.exp(0.3 * rn(H))).to(act)
    s["wr"] = (rn(E, H) / H ** 0.5).to(act)
    rank = torch.randperm(E, device="cuda", generator=g) + 1
    s["br"] = -0.8 * torch.log(rank.float())  # some experts are asked for more often than others
    s["y"], s["x_out"] = new(T, H, dt=torch.float32), new(T, H, dt=act)
    s["ids"], s["gate"] = new(T, k, dt=torch.int32), new(T, k, dt=torch.float32)
    return s


def _run_own(s):
    import expert_offloaded_ffn_moe_amd as moe

    if s["op"] == "quant":
        moe.fp8_quantize(s["x"], s["codes"], s["scale"], block_rows=s["case"]["rows"])
        return {"codes": s["values"].copy_(s["codes"]), "scale": s["scale"]}
    if s["op"] == "matmul":
        moe.fp8_matmul(s["q"], s["sx"], s["w"], s["sw"], s["out"], bias=s["bias"], y_in=s["y"], res=s["res"])
        return {"out": s["out"]}
    case = s["case"]
    if "workspace" not in s:  # a program keeps it
        n = moe.fp8_layer_workspace(case["T"], case["H"], case["I"], case["E"], case["k"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.fp8_layer(s["x"], s["wr"], s["w_gu"], s["s_gu"], s["w_dn"], s["s_dn"], case["k"], s["y"], s["workspace"],
                  router_b=s["br"], x_out=s["x_out"], topk_ids=s["ids"], topk_w=s["gate"])
    return {"y": s["y"], "x_out": s["x_out"], "ids": s["ids"], "gate": s["gate"]}


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quant":
        r, (T, H) = s["case"]["rows"], s["x"].shape
        v = torch.zeros(-(-T // r) * r, _up(H) * B, dtype=torch.float64, device="cuda")  # quotients lie next to borders
        v[:T, :H] = s["x"]
        v = v.view(-1, r, _up(H), B)
        amax = v.abs().amax((1, 3), keepdim=True)
        q = v * 448.0 / amax
        e = torch.frexp(q)[1].clamp(min=-5)  # |q| < 2^e, the numbers under 2^-6 in the steps of those above it
        step = (e.long() + (1023 - 4) << 52).view(torch.float64)  # 2^(e - 4): three bits behind the first
        return {"codes": (torch.round(q / step) * step).view(-1, _up(H) * B)[:T, :H].float(),
                "scale": (amax / 448.0).view(-1, _up(H)).float()}
    if s["op"] == "matmul":
        (T, K), N = s["q"].shape, s["w"].shape[0]
        y = (s["q"].float() * _spread(s["sx"], T, K, 1)) @ (s["w"].float() * _spread(s["sw"], N, K)).t()
        for more in (s["bias"], s["y"], s["res"]):
            if more is not None:
                y = y + more.float()
        return {"out": y.to(s["out"].dtype)}
    (T, H), I, k = s["x"].shape, s["w_dn"].shape[2], s["case"]["k"]  # noqa: E741
    # sums of the router in 64 bits: which expert is chosen turns on values next to each other
    logits = (s["x"].double() @ s["wr"].double().t() + s["br"].double()).float()
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)  # ties to the lower expert
    best, ids = best[:, :k], ids[:, :k]
    p = torch.exp(best - best[:, :1])
    gate = p / p.sum(1, keepdim=True)
    e = ids.reshape(-1)
    held = lambda w: w.view(torch.uint8)[e].view(F8).float()  # noqa: E731
    gu = held(s["w_gu"]).view(-1, 2, I, H) * _spread(s["s_gu"][e], I, H)
    x = s["x"].float().repeat_interleave(k, 0).view(-1, 1, H, 1)
    h = torch.matmul(gu, x).view(-1, 2, I)
    del gu
    h = h[:, 0] / (1.0 + torch.exp(-h[:, 0])) * h[:, 1]
    d = torch.matmul(held(s["w_dn"]) * _spread(s["s_dn"][e], H, I), h.unsqueeze(-1)).view(T, k, H)
    y = (d * gate.unsqueeze(-1)).sum(1)
    return {"y": y, "x_out": (s["x"].float() + y).to(s["x"].dtype), "ids": ids.to(torch.int32), "gate": gate}


def _numbers():
    """The finite e4m3 numbers from 0 up, by their bits."""
    c = torch.arange(127)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m / 512, (8 + m) * 2.0 ** (e - 10).double())


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64

    def blockwise(q, sc, rows):
        out = q.to(D)
        for i in range(sc.shape[-2]):
            for j in range(sc.shape[-1]):
                out[..., i * rows:(i + 1) * rows, j * B:(j + 1) * B] *= sc[..., i, j, None, None].to(D)
        return out

    if case["op"] == "quant":
        x, r, table = s["x"].to(D), case["rows"], _numbers().cuda()
        T, H = x.shape
        columns = [x[:, j:j + B] for j in range(0, H, B)]
        tops = torch.stack([c.abs().max(1).values for c in columns], 1)
        tops = torch.stack([t.max(0).values for t in tops.split(r)])
        codes = torch.empty_like(x)
        for j, c in enumerate(columns):
            a = c.abs() * 448 / tops[:, j].repeat_interleave(r)[:T, None]
            lo = (torch.searchsorted(table, a, right=True) - 1).clamp(max=125)
            up, down = table[lo + 1] - a, a - table[lo]
            best = torch.where((up < down) | ((up == down) & (lo % 2 == 1)), lo + 1, lo)
            codes[:, j * B:j * B + B] = torch.copysign(table[best], c)
        return {"codes": codes, "scale": tops / 448}
    if case["op"] == "matmul":
        if case["T"] == 1:
            x = s["q"].to(D) * s["sx"].to(D).repeat_interleave(B, 1)[:, :case["K"]]
        else:
            x = torch.cat([s["q"][:, j * B:j * B + B].to(D) * s["sx"][:, j, None].to(D) for j in range(s["sx"].shape[1])], 1)
        y = torch.matmul(x, blockwise(s["w"], s["sw"], B).T)
        for more in (s["bias"], s["y"], s["res"]):
            y += 0 if more is None else more.to(D)
        return {"out": y}
    x, k, I = s["x"].to(D), case["k"], case["I"]  # noqa: E741
    logits = (x @ s["wr"].to(D).T + s["br"].to(D)).to(torch.float32).cpu()
    chosen = [sorted(range(case["E"]), key=lambda e, row=row: (-row[e], e))[:k] for row in logits.tolist()]
    gate = torch.softmax(torch.stack([logits[t][c] for t, c in enumerate(chosen)]).to(D), 1).cuda()
    y = torch.zeros(case["T"], case["H"], dtype=D, device="cuda")
    for e in sorted({e for c in chosen for e in c}):
        t, j = zip(*[(t, c.index(e)) for t, c in enumerate(chosen) if e in c])
        t, j = torch.tensor(t).cuda(), torch.tensor(j).cuda()
        g = x[t] @ blockwise(s["w_gu"][e, :I], s["s_gu"][e, 0], B).T
        u = x[t] @ blockwise(s["w_gu"][e, I:], s["s_gu"][e, 1], B).T
        y[t] += (g * torch.sigmoid(g) * u) @ blockwise(s["w_dn"][e], s["s_dn"][e], B).T * gate[t, j, None]
    return {"y": y, "x_out": x + y, "ids": torch.tensor(chosen, dtype=torch.int32).cuda(), "gate": gate}


def _experts(case):
    """How many experts the tokens ask for together, expected of the bias that prepare gives them."""
    p = [(e + 1) ** -0.8 for e in range(case["E"])]
    each = [1 - (1 - v / sum(p)) ** min(case["k"], case["E"]) for v in p]
    return max(case["k"], round(sum(1 - (1 - v) ** case["T"] for v in each)))


def work(case):
    T, size = case["T"], {"bf16": 2, "f32": 4}
    if case["op"] == "quant":
        H = case["H"]
        return {"bytes": T * H * (size[case["act"]] + 1) + 4 * -(-T // case["rows"]) * _up(H), "flops": 3 * T * H}
    if case["op"] == "matmul":
        N, K, b = case["N"], case["K"], size[case["out"]]
        add = {"none": 0, "res": b, "both": 4 + b}[case["add"]]
        return {"bytes": N * K + T * K + 4 * _up(K) * (T + _up(N)) + 4 * N * case["bias"] + T * N * (b + add),
                "flops": 2 * T * N * K}
    H, I, E, k, b = case["H"], case["I"], case["E"], case["k"], size[case["act"]]  # noqa: E741
    expert = 3 * H * I + 12 * _up(H) * _up(I)
    return {"bytes": _experts(case) * expert + E * (H * b + 4) + T * H * (b + 4 + b) + 8 * T * k,
            "flops": 6 * T * k * H * I + 2 * T * E * H}
