"""Cases of the 16-bit expert products, of SwiGLU and of low-rank adapters, with their gradients.

A case's ``op`` names the operator and ``backward`` its direction; ``run`` computes it in plain torch operations
in 32 bits, or, where ``own`` is true, by the calls a user of the library makes.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # 8 sequences' next tokens, top-8 of 64 experts: the stream of the experts' weights
        {"name": "gemm_decode", "op": "gemm", "backward": False, "R": 64, "E": 64, "N": 768, "K": 2048,
         "dtype": "bf16", "out": "bf16"},
        # a long prompt's rows through a few large experts: the matrix rate
        {"name": "gemm_prefill", "op": "gemm", "backward": False, "R": 8192, "E": 8, "N": 11008, "K": 4096,
         "dtype": "bf16", "out": "bf16"},
        # odd sizes, rows kept in fp32 for the weighted sum behind
        {"name": "gemm_odd", "op": "gemm", "backward": False, "R": 2331, "E": 7, "N": 520, "K": 1032,
         "dtype": "f16", "out": "f32"},
        # a training batch of 4096 tokens, top-8 of 64 experts: both gradients, the weights' in fp32
        {"name": "gemm_backward_train", "op": "gemm", "backward": True, "R": 32768, "E": 64, "N": 768, "K": 2048,
         "dtype": "bf16", "out": "f32"},
        # a small fine-tuning batch, odd sizes
        {"name": "gemm_backward_odd", "op": "gemm", "backward": True, "R": 1111, "E": 7, "N": 520, "K": 1032,
         "dtype": "f16", "out": "f16"},
        # the expert rows of a training batch
        {"name": "swiglu_rows", "op": "swiglu", "backward": False, "R": 32768, "C": 768, "dtype": "bf16"},
        # a dense layer's gradient over a long batch
        {"name": "swiglu_backward", "op": "swiglu", "backward": True, "R": 8192, "C": 11008, "dtype": "bf16"},
        # a decode step of 32 requests, each with one of 64 adapters: latency, and the adapters' stream
        {"name": "lora_decode", "op": "lora", "backward": False, "M": 32, "E": 64, "r": 16, "K": 4096, "N": 11008,
         "dtype": "f16"},
        # prompts of several requests in one batch, of wide adapters
        {"name": "lora_prefill", "op": "lora", "backward": False, "M": 8192, "E": 8, "r": 64, "K": 4096, "N": 11008,
         "dtype": "bf16"},
        # several adapters trained beside one frozen projection
        {"name": "lora_backward_train", "op": "lora", "backward": True, "M": 4096, "E": 4, "r": 16, "K": 4096,
         "N": 4096, "dtype": "bf16"},
        # the same on a small batch of odd sizes
        {"name": "lora_backward_odd", "op": "lora", "backward": True, "M": 777, "E": 7, "r": 24, "K": 2056,
         "N": 1032, "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "swiglu", "lora", "lora"])
    c = {"op": op, "backward": rng.random() < 0.5}
    if op == "swiglu":
        c.update(R=_log_int(rng, 1, 20000), C=8 * _log_int(rng, 16, 1400), dtype=rng.choice(["f16", "bf16", "f32"]))
        while c["R"] * c["C"] > 8192 * 11008:
            c["R"] = c["R"] // 2 + 1
        return c
    if op == "gemm":
        c.update(R=_log_int(rng, 1, 30000), E=rng.choice([1, 2, 4, 8, 16, 37, 64, 64, 128, 256]),
                 N=8 * _log_int(rng, 16, 1000), K=8 * _log_int(rng, 16, 1000), dtype=rng.choice(["f16", "bf16"]))
        c["out"] = rng.choice([c["dtype"], "f32"])
        while c["E"] * c["N"] * c["K"] > 8 * 11008 * 4096:
            c["N"] = 8 * (c["N"] // 16 + 1)
        while c["R"] * c["N"] * c["K"] * (2 if c["backward"] else 1) > 8192 * 11008 * 4096:
            c["R"] = c["R"] // 2 + 1
        return c
    c.update(M=_log_int(rng, 1, 8000), E=rng.choice([1, 2, 4, 8, 16, 64]), r=rng.choice([8, 16, 16, 24, 32, 64, 128]),
             K=8 * _log_int(rng, 64, 1000), N=8 * _log_int(rng, 64, 1400), dtype=rng.choice(["f16", "bf16"]))
    while c["M"] * (c["K"] + c["N"]) > 8192 * 15104 // (2 if c["backward"] else 1):
        c["M"] = c["M"] // 2 + 1
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype, size=1.0):
    return (size * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _activations(g, rows, cols, dtype):
    """Normal values with a per-row size and a few columns that are much larger, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= 1.0 + 7.0 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01).float()
    return x.to(dtype)


def _ids(g, rows, E):
    """One group per row, some groups more popular than others."""
    logits = 0.7 * torch.randn(E, generator=g, device="cuda")
    return torch.multinomial(torch.softmax(logits, 0), rows, replacement=True, generator=g)


def _request_ids(g, M, E):
    """The adapter of each row: runs of rows of one request, a tenth of the requests without one (-1)."""
    requests = max(1, min(M, 4 * E))
    request = torch.arange(M, device="cuda") * requests // M
    ids = _ids(g, requests, E)
    ids[torch.rand(requests, generator=g, device="cuda") < 0.1] = -1
    return ids[request]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "swiglu":
        R, C = case["R"], case["C"]
        s["gate"], s["up"] = _activations(g, R, C, dtype), _activations(g, R, C, dtype)
        if case["backward"]:
            s["dh"] = _randn(g, R, C, dtype=dtype, size=0.1)
    elif op == "gemm":
        R, E, N, K = (case[n] for n in "RENK")
        s["a"] = _activations(g, R, K, dtype)
        s["w"] = _randn(g, E, N, K, dtype=dtype, size=0.02)
        if case["backward"]:
            s["dc"] = _randn(g, R, N, dtype=dtype, size=0.1)
        s["offsets"], _, _ = _sort(_ids(g, R, E), E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        M, E, r, K, N = (case[n] for n in ("M", "E", "r", "K", "N"))
        s["x"] = _activations(g, M, K, dtype)
        s["a"] = _randn(g, E, r, K, dtype=dtype, size=K ** -0.5)
        s["b"] = _randn(g, E, N, r, dtype=dtype, size=r ** -0.5)
        s["scales"] = 0.5 + torch.rand(E, generator=g, device="cuda")
        # the plan of a batch, made once and used by every projection of every layer
        s["offsets"], s["slot_row"], s["row_slot"] = _sort(_request_ids(g, M, E), E)
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        if case["backward"]:
            s["dy"] = _randn(g, M, N, dtype=dtype, size=0.1)
            s["base"] = _randn(g, M, K, dtype=dtype, size=0.1)      # the frozen projection's gradient of x
        else:
            s["base"] = _randn(g, M, N, dtype=dtype)                # the shared projection's output
    return s


def _sort(ids, E):
    """(offsets, row of each slot, slot of each row), ids outside 0 .. E - 1 left out: the slots by group, equal ones
    in their order."""
    n = ids.numel()
    key = torch.where((ids >= 0) & (ids < E), ids, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    is_in = torch.arange(n, device=ids.device) < offsets[-1]
    row_slot = torch.where(is_in, order, -1)
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.where(is_in, torch.arange(n, device=ids.device), -1)
    return offsets.to(torch.int32), slot_row.reshape(n, 1).to(torch.int32), row_slot.to(torch.int32)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _padded(offsets, most, rows):
    """Row numbers [E, most] of each group's rows; past its end the row behind all others."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return torch.where(at < offsets[1:, None], at, rows)


def _take(x, at):
    """x's rows at `at` in 32 bits, a row of zeros behind the last."""
    return torch.cat([x.float(), x.new_zeros(1, x.shape[1], dtype=torch.float32)])[at]


def _put(c, at, rows):
    out = c.new_zeros(rows + 1, c.shape[-1])
    out[at] = c
    return out[:rows]


def _plain_gemm(s):
    case, a, w = s["case"], s["a"], s["w"].float()
    out, R = DTYPES[case["out"]], case["R"]
    at = _padded(s["offsets"], s["most"], R)
    rows = _take(a, at)
    if not case["backward"]:
        return [_put(torch.bmm(rows, w.transpose(1, 2).contiguous()), at, R).to(out)]
    dc = _take(s["dc"], at)
    da = _put(torch.bmm(dc, w), at, R).to(a.dtype)
    return [da, torch.bmm(dc.transpose(1, 2).contiguous(), rows).to(out)]


def _plain_swiglu(s):
    dtype, g, u = s["gate"].dtype, s["gate"].float(), s["up"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    if not s["case"]["backward"]:
        return [(g * sig * u).to(dtype)]
    dh = s["dh"].float()
    return [(dh * u * sig * (1.0 + g * (1.0 - sig))).to(dtype), (dh * g * sig).to(dtype)]


def _plain_lora(s):
    case, x = s["case"], s["x"]
    dtype, M = x.dtype, case["M"]
    a, b, scale = s["a"].float(), s["b"].float(), s["scales"][:, None, None]
    row_slot = torch.cat([s["row_slot"], s["row_slot"].new_full((1,), -1)]).long()
    at = _padded(s["offsets"], s["most"], M)
    at = row_slot[at]
    at = torch.where(at < 0, M, at)
    rows = _take(x, at)
    h = torch.bmm(rows, a.transpose(1, 2).contiguous())
    if not case["backward"]:
        y = scale * torch.bmm(h, b.transpose(1, 2).contiguous())
        return [(s["base"].float() + _put(y, at, M)).to(dtype)]
    dy = scale * _take(s["dy"], at)
    dh = torch.bmm(dy, b)
    dx = s["base"].float() + _put(torch.bmm(dh, a), at, M)
    da = torch.bmm(dh.transpose(1, 2).contiguous(), rows)
    db = torch.bmm(dy.transpose(1, 2).contiguous(), h)
    return [dx.to(dtype), da.to(dtype), db.to(dtype)]


def _plain(s):
    return {"gemm": _plain_gemm, "swiglu": _plain_swiglu, "lora": _plain_lora}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import q4_swiglu_mlp_amd as Z

    case = s["case"]
    op = case["op"]
    if op == "swiglu":
        if case["backward"]:
            return list(Z.zinc_swiglu_backward(s["dh"], s["gate"], s["up"]))
        return [Z.zinc_swiglu(s["gate"], s["up"])]
    if op == "gemm":
        if case["backward"]:
            return list(Z.zinc_moe_gemm_backward(s["dc"], s["a"], s["w"], s["offsets"], dw_dtype=DTYPES[case["out"]]))
        return [Z.zinc_moe_gemm(s["a"], s["w"], s["offsets"], DTYPES[case["out"]])]
    plan = s["offsets"], s["slot_row"], s["row_slot"]
    if case["backward"]:
        return list(Z.zinc_lora_backward(s["dy"], s["x"], s["a"], s["b"], s["scales"], *plan, base=s["base"]))
    return [Z.zinc_lora(s["x"], s["a"], s["b"], s["scales"], *plan, base=s["base"])]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def _used(rows, E):
    """Groups of E that `rows` even picks meet, on average."""
    return int(round(E * (1.0 - (1.0 - 1.0 / E) ** rows)))


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "swiglu":
        n = case["R"] * case["C"]
        return {"bytes": (5 if case["backward"] else 3) * n * b, "flops": (12 if case["backward"] else 5) * n}
    if op == "gemm":
        R, E, N, K = (case[n] for n in "RENK")
        weights, used, o = N * K, _used(R, E), BYTES[case["out"]]
        if not case["backward"]:
            return {"bytes": R * K * b + used * weights * b + R * N * o + 4 * (E + 1), "flops": 2 * R * N * K}
        return {"bytes": R * (2 * K + N) * b + used * weights * b + E * weights * o + 4 * (E + 1),
                "flops": 4 * R * N * K}
    M, E, r, K, N = (case[n] for n in ("M", "E", "r", "K", "N"))
    adapters = _used(min(M, 4 * E), E) * r * (K + N) * b + 4 * E
    plan = 8 * M + 4 * (E + 1)
    if not case["backward"]:
        return {"bytes": M * (K + 2 * N) * b + adapters + plan, "flops": 2 * M * r * (K + N)}
    return {"bytes": M * (3 * K + N) * b + adapters + E * r * (K + N) * b + plan,
            "flops": 2 * M * r * (3 * K + 2 * N)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_swiglu(s):
    outs = []
    for i in range(0, s["case"]["R"], 1024):            # in parts, for the memory
        g, u = s["gate"][i:i + 1024].double(), s["up"][i:i + 1024].double()
        p = torch.sigmoid(g)
        if s["case"]["backward"]:
            dh = s["dh"][i:i + 1024].double()
            outs.append([dh * u * (p + g * p * torch.sigmoid(-g)), dh * g * p])
        else:
            outs.append([g * p * u])
    return [torch.cat(parts) for parts in zip(*outs)]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "swiglu":
        return _exact_swiglu(s)
    ends = s["offsets"].tolist()
    zeros = lambda *shape: torch.zeros(*shape, device="cuda", dtype=torch.float64)  # noqa: E731
    if op == "gemm":
        R, E, N, K = (case[n] for n in "RENK")
        c, da, dw = zeros(R, N), zeros(R, K), zeros(E, N, K) if case["backward"] else None
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            if ends[e] == ends[e + 1]:
                continue
            rows, w = s["a"][at].double(), s["w"][e].double()
            if case["backward"]:
                dc = s["dc"][at].double()
                da[at], dw[e] = dc @ w, dc.t() @ rows
            else:
                c[at] = rows @ w.t()
        return [da, dw] if case["backward"] else [c]
    y, da, db = s["base"].double(), zeros(s["a"].shape), zeros(s["b"].shape)
    for e in range(case["E"]):
        at = s["row_slot"][ends[e]:ends[e + 1]].long()
        if not at.numel():
            continue
        x, a, b, scale = s["x"][at].double(), s["a"][e].double(), s["b"][e].double(), s["scales"][e].double()
        if case["backward"]:
            dy = s["dy"][at].double()
            dh = scale * (dy @ b)
            y[at] += dh @ a
            da[e] = dh.t() @ x
            db[e] = scale * (dy.t() @ (x @ a.t()))
        else:
            y[at] += scale * ((x @ a.t()) @ b.t())
    return [y, da, db] if case["backward"] else [y]
