"""Cases of the expert layer's FP8 operators: dispatch (sort and gather), combine, quantise, product, experts.

A case's ``op`` names the operator; ``run`` computes it in plain torch operations in 32 bits, or, where ``own``
is true, by the calls a user of the library makes.  FP8 values are e4m3 (torch.float8_e4m3fn) with one fp32
scale per block of 128: activations per row and 128 columns, weights per 128 x 128 tile.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 sequences: the index is pure latency, rows leave as FP8
        {"name": "dispatch_decode", "op": "dispatch", "M": 16, "k": 8, "E": 64, "H": 2048, "dtype": "f16", "fp8": True},
        # a long prompt (or a training batch) sorted whole
        {"name": "dispatch_prefill", "op": "dispatch", "M": 8192, "k": 8, "E": 64, "H": 2048, "dtype": "bf16",
         "fp8": False},
        # the way back of a prompt's chunk
        {"name": "combine_prefill", "op": "combine", "M": 2048, "k": 8, "E": 64, "H": 4096, "dtype": "f16",
         "weighted": True},
        # the gather's gradient in fp32, few experts, odd sizes
        {"name": "gather_backward_odd", "op": "combine", "M": 777, "k": 3, "E": 7, "H": 2056, "dtype": "f32",
         "weighted": False},
        # the combine's gradient over a training batch
        {"name": "combine_backward", "op": "combine_backward", "M": 4096, "k": 8, "E": 64, "H": 2048,
         "dtype": "bf16"},
        # activations of a small batch, the last block of each row cut short
        {"name": "quantize_rows", "op": "quantize", "R": 333, "C": 2064, "block_rows": 1, "dtype": "f16"},
        # a weight matrix brought to FP8 when it is loaded
        {"name": "quantize_weight", "op": "quantize", "R": 11008, "C": 4096, "block_rows": 128, "dtype": "bf16"},
        # one token through a projection: the weight's stream
        {"name": "product_decode", "op": "product", "M": 1, "N": 11008, "K": 4096, "E": 0, "dtype": "f16"},
        # a long prompt through a projection: the matrix rate
        {"name": "product_prefill", "op": "product", "M": 8192, "N": 11008, "K": 4096, "E": 0, "dtype": "bf16"},
        # 512 tokens' top-8 rows through the experts' gate projection, with skewed group sizes
        {"name": "product_grouped", "op": "product", "M": 4096, "N": 768, "K": 2048, "E": 64, "dtype": "f16"},
        # the whole expert layer for 8 sequences' next tokens
        {"name": "experts_decode", "op": "experts", "M": 8, "k": 8, "E": 64, "H": 2048, "I": 768, "dtype": "f16"},
        # and for a prompt of odd length
        {"name": "experts_prefill", "op": "experts", "M": 4001, "k": 8, "E": 64, "H": 2048, "I": 768,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_backward", "quantize", "product", "experts"])
    E = rng.choice([4, 8, 16, 37, 64, 64, 128, 256])
    k = min(E, rng.choice([1, 2, 3, 4, 6, 8, 8]))
    if op in ("dispatch", "combine", "combine_backward"):
        c = {"op": op, "M": _log_int(rng, 1, 5000), "k": k, "E": E, "H": 16 * _log_int(rng, 16, 300),
             "dtype": rng.choice(["f16", "bf16", "bf16", "f32"])}
        if op == "dispatch":
            c["fp8"] = rng.random() < 0.5
        if op == "combine":
            c["weighted"] = rng.random() < 0.7
        while c["M"] * c["k"] * c["H"] * BYTES[c["dtype"]] > 1 << 28:
            c["M"] = c["M"] // 2 + 1
        return c
    if op == "quantize":
        return {"op": op, "R": _log_int(rng, 1, 8000), "C": 16 * _log_int(rng, 16, 320),
                "block_rows": rng.choice([1, 1, 128]), "dtype": rng.choice(["f16", "bf16", "f32"])}
    if op == "product":
        grouped = rng.random() < 0.5
        c = {"op": op, "M": _log_int(rng, 1, 8000), "N": _log_int(rng, 100, 6000), "K": 16 * _log_int(rng, 16, 500),
             "E": E if grouped else 0, "dtype": rng.choice(["f16", "bf16", "bf16"])}
        while max(c["E"], 1) * c["N"] * c["K"] > 1 << 29:
            c["N"] = c["N"] // 2 + 1
        return c
    c = {"op": op, "M": _log_int(rng, 1, 4000), "k": k, "E": E, "H": 128 * rng.randint(2, 24),
         "I": 128 * rng.randint(2, 14), "dtype": rng.choice(["f16", "bf16"])}
    while c["E"] * c["H"] * c["I"] > 1 << 28:
        c["I"] = 128 * max(1, c["I"] // 256)
        c["E"] = max(c["k"], c["E"] // 2)
    while c["M"] * c["k"] * c["H"] * c["I"] > 4001 * 8 * 2048 * 768:
        c["M"] = c["M"] // 2 + 1
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype):
    """Normal values with a per-row size and a few columns that are much larger, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= 1.0 + 15.0 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01).float()
    return x.to(dtype)


def _routing(g, M, E, k):
    """Distinct experts per token, some of them more popular, and softmax weights of the chosen logits."""
    logits = torch.randn(M, E, generator=g, device="cuda") + 0.7 * torch.randn(1, E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _fp8_weight(g, *shape):
    """A checkpoint's weights: e4m3 values and one fp32 scale, amax / 448, per 128 x 128 tile."""
    *lead, N, K = shape
    nb, kb = -(-N // 128), -(-K // 128)
    w = 0.02 * torch.randn(*lead, N, K, generator=g, device="cuda")
    size = torch.exp(0.4 * torch.randn(*lead, nb, kb, generator=g, device="cuda"))
    w = torch.clamp(w / (0.02 * 4.5) * E4M3_MAX, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return w, (size * (0.02 * 4.5 / E4M3_MAX)).contiguous()


def _fp8_rows(g, rows, cols):
    return _quantize(_activations(g, rows, cols, torch.float32), 1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "quantize":
        s["x"] = _activations(g, case["R"], case["C"], dtype)
    elif op == "product":
        s["a"], s["a_scales"] = _fp8_rows(g, case["M"], case["K"])
        if case["E"]:
            s["w"], s["w_scales"] = _fp8_weight(g, case["E"], case["N"], case["K"])
            ids, _ = _routing(g, case["M"], case["E"], 1)
            s["offsets"] = _sort(ids, case["E"])[0]
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        else:
            s["w"], s["w_scales"] = _fp8_weight(g, case["N"], case["K"])
    else:
        s["ids"], s["p"] = _routing(g, case["M"], case["E"], case["k"])
        if op in ("dispatch", "experts"):
            s["x"] = _activations(g, case["M"], case["H"], dtype)
        if op == "experts":
            s["gate"] = _fp8_weight(g, case["E"], case["I"], case["H"])
            s["up"] = _fp8_weight(g, case["E"], case["I"], case["H"])
            s["down"] = _fp8_weight(g, case["E"], case["H"], case["I"])
            s["most"] = int(torch.bincount(s["ids"].reshape(-1).long()).max())
        if op in ("combine", "combine_backward"):
            s["slot_row"] = _sort(s["ids"], case["E"])[1]
            s["ys"] = _activations(g, case["M"] * case["k"], case["H"], dtype)
        if op == "combine_backward":
            s["dy"] = _activations(g, case["M"], case["H"], dtype)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _sort(ids, E):
    """(offsets, row of each slot, slot of each row): slots ordered by expert, equal experts by slot."""
    flat = ids.reshape(-1)
    row_slot = torch.sort(flat, stable=True).indices
    slot_row = torch.empty_like(row_slot)
    slot_row[row_slot] = torch.arange(flat.numel(), device=flat.device)
    counts = (flat[None, :] == torch.arange(E, device=flat.device, dtype=flat.dtype)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets.to(torch.int32), slot_row.reshape(ids.shape).to(torch.int32), row_slot.to(torch.int32)


def _quantize(x, block_rows):
    """Per block the smallest power-of-two scale that brings the largest value to at most 448."""
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // 128)
    p = torch.zeros(rb * block_rows, cb * 128, device=x.device, dtype=torch.float32)
    p[:R, :C] = x.float()
    p = p.reshape(rb, block_rows, cb, 128)
    amax = p.abs().amax(dim=(1, 3))
    m, e = torch.frexp(amax)                      # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    scales = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    q = (p / scales[:, None, :, None]).reshape(rb * block_rows, cb * 128)[:R, :C]
    return q.to(torch.float8_e4m3fn).contiguous(), scales


def _rows32(q, scales):
    return q.float() * scales.repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _weight32(w, scales):
    s = scales.repeat_interleave(128, dim=-1)[..., :w.shape[-1]].repeat_interleave(128, dim=-2)[..., :w.shape[-2], :]
    return w.float() * s


def _padded(offsets, most, rows):
    """Row numbers [E, most] of each expert's rows; past its end the row behind all others."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return torch.where(at < offsets[1:, None], at, rows)


def _grouped(a32, offsets, most, *weights):
    """a32's rows times their expert's weights, as batched products over experts padded to one size."""
    rows = a32.shape[0]
    at = _padded(offsets, most, rows)
    a = torch.cat([a32, a32.new_zeros(1, a32.shape[1])])[at]
    outs = []
    for w32 in weights:
        c = a32.new_zeros(rows + 1, w32.shape[1])
        c[at] = torch.bmm(a, w32.transpose(1, 2).contiguous())
        outs.append(c[:rows])
    return outs


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        return list(_quantize(s["x"], case["block_rows"]))
    if op == "dispatch":
        offsets, slot_row, row_slot = _sort(s["ids"], case["E"])
        xs = s["x"][(row_slot // case["k"]).long()]
        return [offsets, slot_row, row_slot] + (list(_quantize(xs, 1)) if case["fp8"] else [xs])
    if op == "combine":
        y = s["ys"].float()[s["slot_row"].long()]
        return [(y * s["p"][:, :, None] if case["weighted"] else y).sum(1).to(dtype)]
    if op == "combine_backward":
        at, dy = s["slot_row"].long(), s["dy"].float()
        dys = torch.empty_like(s["ys"])
        dys[at] = (s["p"][:, :, None] * dy[:, None, :]).to(dtype)
        return [dys, (s["ys"].float()[at] * dy[:, None, :]).sum(2)]
    if op == "product":
        a32, w32 = _rows32(s["a"], s["a_scales"]), _weight32(s["w"], s["w_scales"])
        if case["E"]:
            return [_grouped(a32, s["offsets"], s["most"], w32)[0].to(dtype)]
        return [(a32 @ w32.t()).to(dtype)]
    offsets, slot_row, row_slot = _sort(s["ids"], case["E"])
    xq = _rows32(*_quantize(s["x"][(row_slot // case["k"]).long()], 1))
    gate, up = _grouped(xq, offsets, s["most"], _weight32(*s["gate"]), _weight32(*s["up"]))
    hq = _rows32(*_quantize(gate / (1.0 + torch.exp(-gate)) * up, 1))
    ys = _grouped(hq, offsets, s["most"], _weight32(*s["down"]))[0]
    return [(ys[slot_row.long()] * s["p"][:, :, None]).sum(1).to(dtype)]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import q4_swiglu_mlp_amd as Z

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return list(Z.zinc_fp8_quantize(s["x"], case["block_rows"]))
    if op == "dispatch":
        offsets, slot_row, row_slot = Z.zinc_moe_sort(s["ids"], case["E"])
        if case["fp8"]:
            return [offsets, slot_row, row_slot, *Z.zinc_moe_gather_fp8(s["x"], slot_row)]
        return [offsets, slot_row, row_slot, Z.zinc_moe_gather(s["x"], slot_row)]
    if op == "combine":
        if case["weighted"]:
            return [Z.zinc_moe_combine(s["ys"], s["slot_row"], s["p"])]
        return [Z.zinc_moe_gather_backward(s["ys"], s["slot_row"])]
    if op == "combine_backward":
        return list(Z.zinc_moe_combine_backward(s["dy"], s["ys"], s["slot_row"], s["p"]))
    if op == "product":
        dtype = DTYPES[case["dtype"]]
        if case["E"]:
            return [Z.zinc_moe_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"], dtype)]
        return [Z.zinc_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], dtype)]
    return [Z.zinc_moe_fp8_experts(*s["gate"], *s["up"], *s["down"], s["x"], s["ids"], s["p"])]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def _fp8_bytes(rows, cols, block_rows):
    return rows * cols + 4 * -(-rows // block_rows) * -(-cols // 128)


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "quantize":
        n = case["R"] * case["C"]
        return {"bytes": n * b + _fp8_bytes(case["R"], case["C"], case["block_rows"]), "flops": 2 * n}
    if op == "product":
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        used = min(max(E, 1), M)
        return {"bytes": _fp8_bytes(M, K, 1) + used * _fp8_bytes(N, K, 128) + 4 * (E + 1) * (E > 0) + M * N * b,
                "flops": 2 * M * N * K}
    M, k, E, H = case["M"], case["k"], case["E"], case["H"]
    rows = M * k
    if op == "dispatch":
        out = _fp8_bytes(rows, H, 1) if case["fp8"] else rows * H * b
        return {"bytes": 4 * rows + 4 * (E + 1) + 8 * rows + M * H * b + out, "flops": 0}
    if op == "combine":
        return {"bytes": rows * H * b + (8 if case["weighted"] else 4) * rows + M * H * b, "flops": 2 * rows * H}
    if op == "combine_backward":
        return {"bytes": M * H * b + 2 * rows * H * b + 12 * rows, "flops": 3 * rows * H}
    weights = min(E, rows) * (2 * _fp8_bytes(case["I"], H, 128) + _fp8_bytes(H, case["I"], 128))
    return {"bytes": 2 * M * H * b + 8 * rows + weights, "flops": 6 * rows * H * case["I"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(v):
    """v (|v| <= 448) rounded to e4m3: three bits behind the leading one, steps of 2^-9 below 2^-6; ties to even."""
    a = v.abs().clamp_min(2.0 ** -60)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp_min(-6.0) - 3.0)
    return torch.round(v / step) * step


def _blocks_64(x, block_rows):
    """(e4m3 values, scales) of x in 64 bits, the scale by comparison with 448 times powers of two."""
    R, C = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -C % 128, 0, -R % block_rows))
    x = x.reshape(x.shape[0] // block_rows, block_rows, x.shape[1] // 128, 128)
    amax = x.abs().amax(dim=(1, 3))
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448.0))
    e = e + (amax > 448.0 * torch.exp2(e)).double()
    e = e - ((amax > 0) & (amax <= 448.0 * torch.exp2(e - 1))).double()
    scales = torch.exp2(e)
    q = _e4m3_64(x / scales[:, None, :, None])
    return q.reshape(q.shape[0] * block_rows, -1)[:R, :C], scales


def _times_64(q, scales, rows_each):
    K = q.shape[-1]
    s = scales.double()
    if rows_each > 1:
        s = s.repeat_interleave(rows_each, dim=-2)[..., :q.shape[-2], :]
    return q.double() * s.repeat_interleave(128, dim=-1)[..., :K]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return list(_blocks_64(s["x"], case["block_rows"]))
    if op == "product":
        a = _times_64(s["a"], s["a_scales"], 1)
        if not case["E"]:
            return [a @ _times_64(s["w"], s["w_scales"], 128).t()]
        c, at = a.new_zeros(case["M"], case["N"]), s["offsets"].tolist()
        for e in range(case["E"]):
            c[at[e]:at[e + 1]] = a[at[e]:at[e + 1]] @ _times_64(s["w"][e], s["w_scales"][e], 128).t()
        return [c]
    if op == "combine":
        y = torch.zeros(case["M"], case["H"], device="cuda", dtype=torch.float64)
        for j in range(case["k"]):
            part = s["ys"].double()[s["slot_row"][:, j].long()]
            y += part * s["p"][:, j, None].double() if case["weighted"] else part
        return [y]
    if op == "combine_backward":
        dy, dys, dp = s["dy"].double(), torch.zeros(s["ys"].shape, device="cuda", dtype=torch.float64), []
        for j in range(case["k"]):
            at = s["slot_row"][:, j].long()
            dys[at] = s["p"][:, j, None].double() * dy
            dp.append((dy * s["ys"][at].double()).sum(1))
        return [dys, torch.stack(dp, 1)]
    # the order by expert, as the key expert * slots + slot, which no two slots share
    flat = s["ids"].reshape(-1).long()
    order = torch.argsort(flat * flat.numel() + torch.arange(flat.numel(), device="cuda"))
    token = order // case["k"]
    if op == "dispatch":
        xs = s["x"].double()[token]
        return [None, None, None] + (list(_blocks_64(xs, 1)) if case["fp8"] else [xs])
    y = torch.zeros(case["M"], case["H"], device="cuda", dtype=torch.float64)
    for e in range(case["E"]):
        slots = order[flat[order] == e]
        if slots.numel():
            q, qs = _blocks_64(s["x"][slots // case["k"]], 1)
            x = _times_64(q, qs, 1)
            g = x @ _times_64(s["gate"][0][e], s["gate"][1][e], 128).t()
            u = x @ _times_64(s["up"][0][e], s["up"][1][e], 128).t()
            q, qs = _blocks_64(g * torch.sigmoid(g) * u, 1)
            out = _times_64(q, qs, 1) @ _times_64(s["down"][0][e], s["down"][1][e], 128).t()
            y.index_add_(0, slots // case["k"], out * s["p"].reshape(-1)[slots, None].double())
    return [y]
