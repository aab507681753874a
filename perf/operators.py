"""The expert-layer operators, measured: products with 4-bit weights, the codec of those
weights, expert products on sorted rows, and tokens sorted by expert and back with gradients.

``run`` computes an operator in plain torch where ``own`` is false, and with the library's
calls where it is true; ``exact`` computes it in 64 bits.

Formats.  A 4-bit matrix of N rows and K columns holds codes 0..15, two to a byte (even
column in the low nibble), and one scale (the type of the activations) and optionally one
zero point per group of G columns: W = (code - zero) * scale, zero 8 where there is none.
A slot is one (token, choice) pair; sorted rows are the slots ordered by expert, equal
experts in slot order, slots without a valid expert last.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_DEV = "cuda"


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # One token through a small projection (a head, a low-rank or router-side matrix of one
        # tensor-parallel rank): the latency of the call counts.  Odd row count, zero points.
        {"name": "mm_1x1001x1024_f16_g32z", "op": "mm", "tokens": 1, "rows": 1001, "cols": 1024,
         "group": 32, "zeros": True, "type": "f16"},
        # One token of decode through the 7168-wide projection: the bytes of the weights count.
        {"name": "mm_1x7168x7168_bf16_g128", "op": "mm", "tokens": 1, "rows": 7168, "cols": 7168,
         "group": 128, "zeros": False, "type": "bf16"},
        # A batch of 16 decoding sequences through the library's widest staged projection.
        {"name": "mm_16x7168x43008_bf16_g64z", "op": "mm", "tokens": 16, "rows": 7168,
         "cols": 43008, "group": 64, "zeros": True, "type": "bf16"},
        # Decode through an expert layer: 24 tokens, 8 choices each, over 64 experts of 7168
        # columns.  Nearly every expert gets a few rows, and all weights have to be read.
        {"name": "experts_24t8_64x4096x7168_bf16_g128", "op": "experts", "tokens": 24, "topk": 8,
         "experts": 64, "rows": 4096, "cols": 7168, "group": 128, "zeros": False, "type": "bf16"},
        # Prefill through an expert layer: hundreds of rows for each expert, so that the matrix
        # units count.  The token count is ragged, as chunks of a prompt are.
        {"name": "experts_4099t6_32x2048x7168_f16_g64z", "op": "experts", "tokens": 4099, "topk": 6,
         "experts": 32, "rows": 2048, "cols": 7168, "group": 64, "zeros": True, "type": "f16"},
        # Dispatch of a decode step to 256 experts: sort and row copies of 32 tokens.
        {"name": "dispatch_32t8_e256_h7168_bf16", "op": "dispatch", "tokens": 32, "topk": 8,
         "experts": 256, "hidden": 7168, "drop": 0.0, "type": "bf16"},
        # Dispatch of a prefill of 16384 tokens, an eighth of the slots dropped (experts of
        # other ranks, or over capacity).
        {"name": "dispatch_16384t4_e64_h7168_bf16", "op": "dispatch", "tokens": 16384, "topk": 4,
         "experts": 64, "hidden": 7168, "drop": 0.125, "type": "bf16"},
        # The gradient of dispatch in training: a ragged batch, binary16, an odd width.
        {"name": "dispatch_grad_4093t6_h2055_f16", "op": "dispatch_grad", "tokens": 4093, "topk": 6,
         "experts": 48, "hidden": 2055, "drop": 0.0, "type": "f16"},
        # The way back of a prefill: the experts' rows weighted and summed per token.
        {"name": "combine_16384t8_h7168_bf16", "op": "combine", "tokens": 16384, "topk": 8,
         "experts": 256, "hidden": 7168, "drop": 0.0, "type": "bf16"},
        # The gradient of the way back in training: rows and weights, with dropped slots.
        {"name": "combine_grad_8192t8_h4096_bf16", "op": "combine_grad", "tokens": 8192, "topk": 8,
         "experts": 64, "hidden": 4096, "drop": 0.125, "type": "bf16"},
        # The codec's round trip on a small matrix (an adapter, one expert's part): latency counts.
        {"name": "codec_1001x1024_f16_g32", "op": "codec", "rows": 1001, "cols": 1024, "group": 32,
         "type": "f16"},
        # The codec's round trip on the widest staged projection: what is kept of its weights.
        {"name": "codec_7168x43008_bf16_g128", "op": "codec", "rows": 7168, "cols": 43008,
         "group": 128, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mm", "mm", "experts", "experts", "dispatch", "dispatch_grad", "combine",
                     "combine_grad", "codec"])
    if op in ("mm", "experts", "codec"):
        group = rng.choice([32, 64, 128])
        case = {"op": op, "group": group, "type": rng.choice(["bf16", "f16"])}
        rows, cols = _log(rng, 256, 8192), group * _log(rng, max(1, 512 // group), 43008 // group)
        if op == "codec":
            return {**case, "rows": rows, "cols": cols}
        case["zeros"] = rng.random() < 0.5
        if op == "mm":
            while rows * cols > 7168 * 43008:
                rows, cols = rows // 2 + 1, cols
            return {**case, "tokens": _log(rng, 1, 512), "rows": rows, "cols": cols}
        experts = _log(rng, 4, 64)
        cols = min(cols, 14336)
        while experts * rows * cols > 64 * 4096 * 7168:
            rows = rows // 2 + 1
        topk = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 4096)
        while tokens * topk * rows * cols > 4099 * 6 * 2048 * 7168:
            tokens = tokens // 2 + 1
        return {**case, "tokens": tokens, "topk": topk, "experts": experts, "rows": rows,
                "cols": cols}
    topk = rng.randint(1, 8)
    hidden = 8 * _log(rng, 32, 1024) if rng.random() < 0.75 else _log(rng, 257, 8191)
    types = ["bf16", "f16", "f32"]
    tokens = _log(rng, 1, 16384)
    case = {"op": op, "topk": topk, "experts": _log(rng, max(2, topk), 256), "hidden": hidden,
            "drop": rng.choice([0.0, 0.125, 0.5]), "type": rng.choice(types)}
    while tokens * topk * hidden > 8192 * 8 * 4096:
        tokens = tokens // 2 + 1
    return {**case, "tokens": tokens}


# ---- inputs ---------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32).to(dtype)


def _matrix(g, case, lead=()):
    """Codes, scales and zero points of one 4-bit matrix, or of one per expert."""
    n, k, group = case["rows"], case["cols"], case["group"]
    shape = lead + (n, k // group)
    codes = torch.randint(0, 256, lead + (n, -(-k // 32) * 16), generator=g, device=_DEV,
                          dtype=torch.uint8)
    # row strides of scales and zero points are multiples of four groups, as the library asks
    wide = lead + (n, -(-(k // group) // 4) * 4)
    spread = torch.rand(shape, generator=g, device=_DEV) * 1.5 + 0.25
    scale = torch.zeros(wide, dtype=_TYPES[case["type"]], device=_DEV)
    scale[..., : k // group] = (spread / (4.0 * math.sqrt(k))).to(scale.dtype)
    zero = None
    if case["zeros"]:
        zero = torch.zeros(wide, dtype=torch.uint8, device=_DEV)
        zero[..., : k // group] = torch.randint(4, 12, shape, generator=g, device=_DEV,
                                                dtype=torch.uint8)
    return codes, scale, zero


def _choices(g, case):
    """Every token's distinct experts: a router with noise on uneven expert popularity.  A
    share of the slots has no expert here (-1)."""
    t, e = case["tokens"], case["experts"]
    liking = torch.randn((e,), generator=g, device=_DEV) * 0.5
    noise = -torch.log(-torch.log(torch.rand((t, e), generator=g, device=_DEV).clamp(1e-9, 1 - 1e-6)))
    logits, ids = torch.topk(liking + noise, case["topk"], dim=1)
    ids = ids.to(torch.int32)
    if case.get("drop"):
        gone = torch.rand(ids.shape, generator=g, device=_DEV) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(logits, 1).contiguous()


def _order(ids, experts):
    """The sorted order in plain torch: offsets, the slot in each row, the row of each slot."""
    flat = ids.reshape(-1)
    key = torch.where((flat < 0) | (flat >= experts), experts, flat).to(torch.int64)
    src = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(src)
    pos[src] = torch.arange(src.numel(), device=src.device)
    bounds = torch.arange(experts, device=key.device)
    off = torch.zeros(experts + 1, dtype=torch.int64, device=key.device)
    off[1:] = torch.searchsorted(key[src], bounds, right=True)
    return off.to(torch.int32), src.to(torch.int32), pos.to(torch.int32)


def prepare(case, seed):
    g, op, dtype = _generator(seed), case["op"], _TYPES[case["type"]]
    state = {"case": case}
    if op == "codec":
        n, k, group = case["rows"], case["cols"], case["group"]
        gain = torch.exp(torch.rand((n, 1), generator=g, device=_DEV) * 3 - 1.5)
        state["x"] = (torch.randn((n, k), generator=g, device=_DEV) * gain * 0.02).to(dtype)
        state["codes"] = torch.zeros((n, -(-k // 32) * 16), dtype=torch.uint8, device=_DEV)
        state["scale"] = torch.zeros((n, -(-(k // group) // 4) * 4), dtype=dtype, device=_DEV)
        state["y"] = torch.empty((n, k), dtype=dtype, device=_DEV)
        return state
    if op == "mm":
        state["x"] = _normal(g, (case["tokens"], case["cols"]), dtype)
        state["codes"], state["scale"], state["zero"] = _matrix(g, case)
        state["y"] = torch.empty((case["tokens"], case["rows"]), dtype=dtype, device=_DEV)
        return state
    ids, weight = _choices(g, case)
    slots = ids.numel()
    if op == "experts":
        off, src, _ = _order(ids, case["experts"])
        state.update(off=off, src=src, x=_normal(g, (case["tokens"], case["cols"]), dtype),
                     most=int((off[1:] - off[:-1]).max()))
        state["codes"], state["scale"], state["zero"] = _matrix(g, case, (case["experts"],))
        state["y"] = torch.empty((slots, case["rows"]), dtype=dtype, device=_DEV)
        return state
    h, t = case["hidden"], case["tokens"]
    if op == "dispatch":
        state.update(ids=ids, x=_normal(g, (t, h), dtype),
                     out=torch.empty((slots, h), dtype=dtype, device=_DEV))
        # the sort's scratch: 256 counts for each expert and for the dropped
        state["work"] = torch.empty(256 * (case["experts"] + 1), dtype=torch.int32, device=_DEV)
        for name, size in (("off", case["experts"] + 1), ("src", slots), ("pos", slots)):
            state[name] = torch.empty(size, dtype=torch.int32, device=_DEV)
        return state
    state["off"], _, state["pos"] = _order(ids, case["experts"])
    state["rows"] = _normal(g, (slots, h), dtype)
    if op != "dispatch_grad":
        state["weight"] = weight
    if op == "combine_grad":
        state.update(dy=_normal(g, (t, h), dtype), drows=torch.empty((slots, h), dtype=dtype, device=_DEV),
                     dweight=torch.empty((t, case["topk"]), dtype=torch.float32, device=_DEV))
    else:
        state["y"] = torch.empty((t, h), dtype=dtype, device=_DEV)
    return state


# ---- the plain forms ------------------------------------------------------------------------

def _weights(state, dtype):
    """The matrix that codes, scales and zero points stand for."""
    k, group = state["case"]["cols"], state["case"]["group"]
    codes = state["codes"][..., : k // 2]
    c = torch.stack((codes & 15, codes >> 4), -1).to(dtype)
    c = c.reshape(codes.shape[:-1] + (k // group, group))
    z = 8.0 if state["zero"] is None else state["zero"][..., : k // group, None].to(dtype)
    w = (c - z) * state["scale"][..., : k // group, None].to(dtype)
    return w.reshape(codes.shape[:-1] + (k,))


def _plain_mm(state):
    return (state["x"].float() @ _weights(state, torch.float32).t()).to(state["x"].dtype)


def _plain_experts(state):
    case, off, most = state["case"], state["off"].long(), state["most"]
    x = state["x"].float()[state["src"].long() // case["topk"]]
    row = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(off[1:], row, right=True)
    place = row - off[expert]
    # one product for each expert on its rows, padded to the longest expert
    padded = torch.zeros((case["experts"], case["cols"], most), device=x.device)
    padded[expert, :, place] = x
    y = torch.bmm(_weights(state, torch.float32), padded)
    return y[expert, :, place].to(state["x"].dtype)


def _plain_dispatch(state):
    case = state["case"]
    off, src, pos = _order(state["ids"], case["experts"])
    rows = state["x"][src.long() // case["topk"]]
    kept = torch.arange(src.numel(), device=src.device) < off[-1]
    return off, src, pos, torch.where(kept[:, None], rows, torch.zeros_like(rows[:1]))


def _slots(state):
    """Every slot's row in 32 bits, zero for the dropped, and which are kept."""
    pos = state["pos"].long()
    kept = pos < state["off"][-1]
    rows = torch.where(kept[:, None], state["rows"][pos].float(), 0.0)
    t, k = state["case"]["tokens"], state["case"]["topk"]
    return rows.view(t, k, -1), kept.view(t, k), pos


def _plain_combine(state):
    rows, _, _ = _slots(state)
    if "weight" in state:
        rows = rows * state["weight"][:, :, None]
    return rows.sum(1).to(state["rows"].dtype)


def _plain_combine_grad(state):
    rows, kept, pos = _slots(state)
    dy = state["dy"].float()
    dweight = torch.where(kept, (rows * dy[:, None, :]).sum(2), 0.0)
    weight = torch.where(kept, state["weight"], 0.0)
    each = weight[:, :, None] * dy[:, None, :]
    drows = torch.empty_like(state["rows"])
    drows[pos] = each.view(drows.shape).to(drows.dtype)
    return drows, dweight


def _plain_codec(state):
    case, x = state["case"], state["x"].float()
    g = x.view(case["rows"], -1, case["group"])
    amax = g.abs().amax(2)
    # divided by a tensor: a number's reciprocal would be multiplied, which rounds twice
    scale = (amax / torch.full_like(amax, 7.0)).to(state["x"].dtype)
    s = scale.float()[:, :, None]
    q = torch.where(s > 0, torch.round(g / s), 0.0).clamp(-7, 7)
    c = (q + 8).to(torch.uint8).view(case["rows"], -1)
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    back = torch.stack((codes & 15, codes >> 4), -1).float().view(g.shape) - 8
    return (back * s).to(state["x"].dtype).view(case["rows"], -1), scale


def _plain(state):
    return {"mm": _plain_mm, "experts": _plain_experts, "dispatch": _plain_dispatch,
            "dispatch_grad": _plain_combine, "combine": _plain_combine,
            "combine_grad": _plain_combine_grad, "codec": _plain_codec}[state["case"]["op"]](state)


# ---- the library's calls --------------------------------------------------------------------

def _own(state):
    import block_quantized_wire_amd as bq
    case, s = state["case"], state
    op, f16 = case["op"], case["type"] == "f16"
    if op == "mm":
        call = bq.bq_mm_i4_f16 if f16 else bq.bq_mm_i4
        call(s["x"], s["codes"], s["scale"], s["y"], zero=s["zero"], group=case["group"])
        return s["y"]
    if op == "experts":
        call = bq.bq_moe_mm_i4_f16 if f16 else bq.bq_moe_mm_i4
        call(s["x"], s["off"], s["codes"], s["scale"], s["y"], zero=s["zero"],
             group=case["group"], src=s["src"], topk=case["topk"])
        return s["y"]
    if op == "dispatch":
        bq.bq_moe_sort(s["ids"], case["experts"], s["off"], s["src"], s["pos"], s["work"])
        bq.bq_moe_gather(s["x"], s["pos"], s["off"], s["out"], topk=case["topk"])
        return s["off"], s["src"], s["pos"], s["out"]
    if op in ("combine", "dispatch_grad"):
        call = {"bf16": bq.bq_moe_combine, "f16": bq.bq_moe_combine_f16,
                "f32": bq.bq_moe_combine_f32}[case["type"]]
        call(s["rows"], s["pos"], s["off"], s["y"], weight=s.get("weight"), topk=case["topk"])
        return s["y"]
    if op == "combine_grad":
        call = {"bf16": bq.bq_moe_combine_bwd, "f16": bq.bq_moe_combine_bwd_f16,
                "f32": bq.bq_moe_combine_bwd_f32}[case["type"]]
        call(s["dy"], s["rows"], s["pos"], s["off"], s["weight"], s["drows"], s["dweight"])
        return s["drows"], s["dweight"]
    quant, dequant = (bq.bq_quant_i4_f16, bq.bq_dequant_i4_f16) if f16 else (bq.bq_quant_i4, bq.bq_dequant_i4)
    quant(s["x"], s["codes"], s["scale"], group=case["group"])
    dequant(s["codes"], s["scale"], s["y"], group=case["group"])
    return s["y"], s["scale"][:, : case["cols"] // case["group"]]


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    size = 4 if case["type"] == "f32" else 2
    if op in ("mm", "experts", "codec"):
        n, k = case["rows"], case["cols"]
        groups = n * (k // case["group"])
        if op == "codec":
            # the values in and out; the codes written and read between the two calls
            return {"bytes": 4 * n * k + n * k + 4 * groups, "flops": 5 * n * k}
        matrix = n * k // 2 + groups * (3 if case["zeros"] else 2)
        if op == "mm":
            return {"bytes": matrix + 2 * case["tokens"] * (n + k),
                    "flops": 2 * case["tokens"] * n * k}
        slots, e = case["tokens"] * case["topk"], case["experts"]
        read = e * (1 - (1 - case["topk"] / e) ** case["tokens"])   # experts that get a row
        return {"bytes": matrix * read + 2 * case["tokens"] * k + 2 * slots * n + 4 * slots,
                "flops": 2 * slots * n * k}
    t, h, slots = case["tokens"], case["hidden"], case["tokens"] * case["topk"]
    kept = slots * (1 - case["drop"])
    if op == "dispatch":
        return {"bytes": size * h * (t + slots) + 4 * 3 * slots, "flops": 0}
    if op == "combine_grad":
        return {"bytes": size * h * (t + kept + slots) + 4 * 3 * slots, "flops": 3 * kept * h}
    return {"bytes": size * h * (t + kept) + 4 * 2 * slots, "flops": 2 * kept * h}


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_weight(codes, scale, zero, k, group):
    """One matrix (N, K) in 64 bits, column by column of its nibbles."""
    w = torch.empty((codes.shape[0], k), dtype=torch.float64, device=codes.device)
    w[:, 0::2] = (codes[:, : k // 2] % 16).double()
    w[:, 1::2] = torch.div(codes[:, : k // 2], 16, rounding_mode="floor").double()
    blocks = w.view(codes.shape[0], k // group, group)
    blocks -= 8.0 if zero is None else zero[:, : k // group].double().unsqueeze(2)
    blocks *= scale[:, : k // group].double().unsqueeze(2)
    return w


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "codec":
        x = s["x"].double().reshape(case["rows"], -1, case["group"])
        unit = x.abs().max(2)[0] / 7
        held = unit.to(s["x"].dtype).double().unsqueeze(2)   # the format holds it in x's type
        steps = torch.round(x / held.clamp(min=1e-300)).clamp(-7, 7)
        return (steps * held).reshape(case["rows"], -1), unit
    if op == "mm":
        w = _exact_weight(s["codes"], s["scale"], s["zero"], case["cols"], case["group"])
        return torch.mm(s["x"].double(), w.t())
    if op == "experts":
        y = torch.empty(s["y"].shape, dtype=torch.float64, device=s["y"].device)
        edge, token = s["off"].tolist(), torch.div(s["src"].long(), case["topk"], rounding_mode="floor")
        for e in range(case["experts"]):
            lo, hi = edge[e], edge[e + 1]
            if hi > lo:
                w = _exact_weight(s["codes"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e],
                                  case["cols"], case["group"])
                y[lo:hi] = torch.mm(s["x"][token[lo:hi]].double(), w.t())
        return y
    topk = case["topk"]
    if op == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(case["experts"] + 1)]
        for slot, e in enumerate(ids):
            lists[e if 0 <= e < case["experts"] else -1].append(slot)
        order = [slot for slots in lists for slot in slots]
        kept = len(order) - len(lists[-1])
        rows = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
        token = torch.tensor([slot // topk for slot in order[:kept]], dtype=torch.int64, device=_DEV)
        rows[:kept] = s["x"].double()[token]
        return None, None, None, rows
    kept = s["off"][-1].item()
    pos = s["pos"].long().view(-1, topk)
    live = pos < kept
    if op in ("combine", "dispatch_grad"):
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=_DEV)
        for j in range(topk):
            part = s["rows"][pos[:, j]].double()
            if op == "combine":
                part *= s["weight"][:, j].double().unsqueeze(1)
            y += part * live[:, j].double().unsqueeze(1)
        return y
    drows = torch.zeros(s["drows"].shape, dtype=torch.float64, device=_DEV)
    dweight = torch.zeros(s["dweight"].shape, dtype=torch.float64, device=_DEV)
    dy = s["dy"].double()
    for j in range(topk):
        on = live[:, j]
        at = pos[on, j]
        drows[at] = dy[on] * s["weight"][on, j].double().unsqueeze(1)
        dweight[on, j] = (s["rows"][at].double() * dy[on]).sum(1)
    return drows, dweight
