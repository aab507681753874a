"""The 4-bit cache of keys and values, measured: rows quantised into it and read back, and
attention over it for one token, a few and many.

``run`` computes an operator in plain torch where ``own`` is false, and with the library's
calls where it is true; ``exact`` computes it in 64 bits.

Formats.  A pool of pages, each with page_size tokens (a multiple of 8) for every key-value head.
A token's vector of D values of one head holds a 4-bit code a value, and for every group of G
values a scale and a least value (two 16-bit numbers of the type of the activations): value =
code * scale + least.  A slot is page * page_size + the token's place in the page.

  k codes  u8 [pages, heads, page_size, D/2]: 32-bit word (g*(D/32) + i) of a token's row holds
           values 32i + 8g .. +7, the first in the lowest nibble.
  v codes  the same shape, by blocks of 8 tokens: value d = 16j + r of token t of a block is
           nibble j%4 of half-word t%2 of the block's word (r*4 + t/2)*(D/64) + j/4.
  scales   16-bit [pages, heads, D/G, page_size, 2]: scale and least value, for k and for v.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_DEV = "cuda"


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # A decode step of 32 sequences writes its tokens and reads them back: latency counts.
        {"name": "store_32_8x128_bf16_g128", "op": "store", "tokens": 32, "kv_heads": 8, "dim": 128,
         "group": 128, "page": 16, "drop": 0.0, "type": "bf16"},
        # A ragged prefill chunk with padding, out of a fused projection, into small groups.
        {"name": "store_16379_8x128_bf16_g32", "op": "store", "tokens": 16379, "kv_heads": 8,
         "dim": 128, "group": 32, "page": 64, "drop": 0.03, "type": "bf16"},
        # One sequence's cache read back to be moved or attended to in 16 bits: short, narrow heads.
        {"name": "fetch_1001_5x64_f16_g64", "op": "fetch", "tokens": 1001, "kv_heads": 5, "dim": 64,
         "group": 64, "page": 16, "drop": 0.0, "type": "f16"},
        # A long shared prefix read back.
        {"name": "fetch_65536_8x128_f16_g128", "op": "fetch", "tokens": 65536, "kv_heads": 8,
         "dim": 128, "group": 128, "page": 64, "drop": 0.0, "type": "f16"},
        # One token of one short sequence: the latency of a call.
        {"name": "decode_1x1001_32of8x128_f16_g32", "op": "attend", "seqs": 1, "new": 1,
         "shortest": 1001, "longest": 1001, "heads": 32, "kv_heads": 8, "dim": 128, "group": 32,
         "page": 16, "causal": True, "window": 0, "empty": 0, "type": "f16"},
        # A decode step of a batch: ragged lengths, bytes of the cache count.
        {"name": "decode_32x8192_64of8x128_bf16_g128", "op": "attend", "seqs": 32, "new": 1,
         "shortest": 701, "longest": 8192, "heads": 64, "kv_heads": 8, "dim": 128, "group": 128,
         "page": 64, "causal": True, "window": 0, "empty": 0, "type": "bf16"},
        # One token of one long sequence: the work has to be split over the tokens.
        {"name": "decode_1x131071_64of8x128_bf16_g64", "op": "attend", "seqs": 1, "new": 1,
         "shortest": 131071, "longest": 131071, "heads": 64, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 64, "causal": True, "window": 0, "empty": 0, "type": "bf16"},
        # Many short sequences whose heads share nothing, two of the batch's places empty.
        {"name": "decode_128x2048_16of16x64_f16_g64", "op": "attend", "seqs": 128, "new": 1,
         "shortest": 17, "longest": 2048, "heads": 16, "kv_heads": 16, "dim": 64, "group": 64,
         "page": 16, "causal": True, "window": 0, "empty": 2, "type": "f16"},
        # Five drafted tokens a sequence are verified at once; pages that are no power of two.
        {"name": "verify_16x5x4099_32of4x128_bf16_g32", "op": "attend", "seqs": 16, "new": 5,
         "shortest": 900, "longest": 4099, "heads": 32, "kv_heads": 4, "dim": 128, "group": 32,
         "page": 24, "causal": True, "window": 0, "empty": 0, "type": "bf16"},
        # Chunks of four prompts over what is cached of each.
        {"name": "chunk_4x1021x4096_32of8x128_bf16_g128", "op": "attend", "seqs": 4, "new": 1021,
         "shortest": 1500, "longest": 4096, "heads": 32, "kv_heads": 8, "dim": 128, "group": 128,
         "page": 64, "causal": True, "window": 0, "empty": 0, "type": "bf16"},
        # A whole prompt under a sliding window, wide heads.
        {"name": "window_1x4096x4096_16of2x256_f16_g128", "op": "attend", "seqs": 1, "new": 4096,
         "shortest": 4096, "longest": 4096, "heads": 16, "kv_heads": 2, "dim": 256, "group": 128,
         "page": 64, "causal": True, "window": 1000, "empty": 0, "type": "f16"},
        # A whole prompt of a long document.
        {"name": "prompt_1x8192x8192_32of8x128_bf16_g64", "op": "attend", "seqs": 1, "new": 8192,
         "shortest": 8192, "longest": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 64, "causal": True, "window": 0, "empty": 0, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "fetch", "decode", "decode", "few", "chunk", "chunk"])
    dim = rng.choice([64, 128, 128, 256])
    case = {"op": op, "dim": dim, "group": rng.choice([g for g in (32, 64, 128) if g <= dim]),
            "page": rng.choice([8, 16, 24, 64, 200, 256]), "type": rng.choice(["bf16", "f16"])}
    kv = rng.choice([1, 2, 3, 4, 8])
    if op in ("store", "fetch"):
        tokens = _log(rng, 1, 65536)
        while tokens * kv * dim > (16379 if op == "store" else 65536) * 8 * 128:
            tokens = tokens // 2 + 1
        return {**case, "tokens": tokens, "kv_heads": kv, "drop": rng.choice([0.0, 0.0, 0.1])}
    share = rng.choice([1, 3, 4, 8, 8, 16])
    case.update(op="attend", kv_heads=kv, heads=kv * share, empty=rng.choice([0, 0, 1]),
                causal=rng.random() < 0.8, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    if op == "decode":
        longest, seqs, new = _log(rng, 1, 131071), _log(rng, 1, 256), 1
        while seqs * longest * kv * dim > 131071 * 8 * 128:
            seqs, longest = (seqs // 2, longest) if seqs > 1 else (1, longest // 2)
    elif op == "few":
        longest, seqs, new = _log(rng, 16, 16384), _log(rng, 1, 32), rng.randint(2, 16)
        while seqs * longest * kv * dim * new > 8 * 131071 * 8 * 128:
            seqs, longest = (seqs // 2, longest) if seqs > 1 else (1, longest // 2 + 16)
    else:
        new, seqs = _log(rng, 17, 4096), _log(rng, 1, 8)
        longest = new + _log(rng, 1, 4096)
        while seqs * new * longest * case["heads"] * dim > 8192 * 4096 * 32 * 128:
            seqs, new = (seqs // 2, new) if seqs > 1 else (1, new // 2 + 1)
    case.update(seqs=seqs, new=new, longest=longest, shortest=max(1, min(longest, longest // rng.randint(1, 8))))
    return case


def _counts(case):
    """Every sequence's length and its number of new tokens: uneven, the same for a case."""
    rng = random.Random(7)
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    lens = [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]
    rng.shuffle(lens)
    for i in range(min(case["empty"], n - 1)):
        lens[(5 * i + 1) % n] = 0
    new = [case["new"] if case["new"] < 17 else rng.randint((case["new"] + 1) // 2, case["new"])
           for _ in range(n)]
    new[0] = case["new"]
    return lens, new


# ---- inputs ---------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _pool(g, case, pages):
    """Codes and scales of a filled cache: codes as of rows near a normal distribution."""
    h, d, s = case["kv_heads"], case["dim"], case["page"]
    dtype, out = _TYPES[case["type"]], {}
    for name in ("k", "v"):
        codes = torch.empty((pages, h, s, d // 2), dtype=torch.uint8, device=_DEV)
        flat = codes.view(-1)
        for at in range(0, flat.numel(), 1 << 26):      # in parts, to keep what it takes small
            n = min(1 << 26, flat.numel() - at)
            two = (torch.randn((2, n), generator=g, device=_DEV, dtype=torch.float16) * 2.6 + 7.5)
            two = two.round_().clamp_(0, 15).to(torch.uint8)
            flat[at:at + n] = two[0] + (two[1] << 4)
        shape = (pages, h, d // case["group"], s)
        scale = torch.rand(shape, generator=g, device=_DEV) * 0.3 + 0.2
        least = scale * (torch.randn(shape, generator=g, device=_DEV) * 0.7 - 7.5)
        out[name] = codes
        out[name + "s"] = torch.stack((scale, least), -1).to(dtype)
    return out


def _empty_pool(case, pages):
    h, d, s = case["kv_heads"], case["dim"], case["page"]
    out = {}
    for name in ("k", "v"):
        out[name] = torch.zeros((pages, h, s, d // 2), dtype=torch.uint8, device=_DEV)
        out[name + "s"] = torch.zeros((pages, h, d // case["group"], s, 2),
                                      dtype=_TYPES[case["type"]], device=_DEV)
    return out


def _slots(g, case, pages):
    """Slots of `tokens` consecutive tokens of a sequence on pages in any order; some are padding."""
    t, s = case["tokens"], case["page"]
    order = torch.randperm(pages, generator=g, device=_DEV)
    at = torch.arange(t, device=_DEV) + 3 % s
    slots = (order[at // s] * s + at % s).to(torch.int32)
    if case["drop"]:
        gone = torch.rand((t,), generator=g, device=_DEV) < case["drop"]
        slots = torch.where(gone, torch.full_like(slots, -1), slots)
    return slots


def prepare(case, seed):
    g, dtype, op = _generator(seed), _TYPES[case["type"]], case["op"]
    h, d, s = case["kv_heads"], case["dim"], case["page"]
    state = {"case": case}
    if op in ("store", "fetch"):
        t = case["tokens"]
        pages = -(-(t + s) // s) + 2
        state["slots"] = _slots(g, case, pages)
        state.update(_empty_pool(case, pages) if op == "store" else _pool(g, case, pages))
        if op == "store":
            # keys and values lie in the rows of a fused projection, which holds the queries too;
            # keys have channels that stand out
            x = torch.randn((t, 3 * h * d), generator=g, device=_DEV)
            lift = torch.randn((h * d,), generator=g, device=_DEV)
            x[:, h * d:2 * h * d] += 4.0 * lift * (lift.abs() > 2.0)
            x = x.to(dtype)
            state["k_rows"] = x[:, h * d:2 * h * d].view(t, h, d)
            state["v_rows"] = x[:, 2 * h * d:].view(t, h, d)
        state["k_back"] = torch.empty((t, h, d), dtype=dtype, device=_DEV)
        state["v_back"] = torch.empty((t, h, d), dtype=dtype, device=_DEV)
        return state
    lens, new = _counts(case)
    each = [-(-n // s) for n in lens]
    pages = sum(each) + 3
    state.update(_pool(g, case, pages))
    order = torch.randperm(pages, generator=g, device=_DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(each))), dtype=torch.int32, device=_DEV)
    used, starts = 0, [0]
    for i, n in enumerate(each):
        table[i, :n] = order[used:used + n]
        used += n
        starts.append(starts[-1] + new[i])
    rows, heads = starts[-1], case["heads"]
    x = (torch.randn((rows, (heads + 2 * h) * d), generator=g, device=_DEV) * 2.0).to(dtype)
    state.update(
        q=x[:, :heads * d].view(rows, heads, d), table=table, most=max(new), longest=max(1, max(lens)),
        lens=torch.tensor(lens, dtype=torch.int32, device=_DEV),
        starts=torch.tensor(starts, dtype=torch.int32, device=_DEV) if case["new"] > 1 else None,
        out=torch.empty((rows, heads, d), dtype=dtype, device=_DEV),
        lse=torch.empty((rows, heads), dtype=torch.float32, device=_DEV),
        # the workspace that a program keeps for all its calls
        work=torch.empty(64 << 20, dtype=torch.uint8, device=_DEV))
    return state


# ---- the plain forms ------------------------------------------------------------------------

def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1)


def _values(codes, scales, case, is_v):
    """32-bit values [..., heads, tokens, D] of whole pages [..., heads, page, D/2]."""
    d, group, s = case["dim"], case["group"], case["page"]
    lead = codes.shape[:-2]
    if is_v:
        c = _nibbles(codes.reshape(lead + (s // 8, 16, 4, d // 64, 2, 2)))
        # (block, r, pair, word, parity, byte, nibble) -> (block, pair, parity, word, byte, nibble, r)
        n = len(lead)
        c = c.permute(*range(n), n, n + 2, n + 4, n + 3, n + 5, n + 6, n + 1)
    else:
        c = _nibbles(codes.reshape(lead + (s, 4, d // 32, 4))).transpose(-4, -3)
    c = c.reshape(lead + (s, d // group, group)).float()
    both = scales.float().transpose(-3, -2)[..., None]       # (..., token, group, 2, 1)
    return (c * both[..., 0, :] + both[..., 1, :]).reshape(lead + (s, d))


def _rows_at(state, name):
    """The rows [tokens, heads, D] that the cache holds at the state's slots."""
    case, slots = state["case"], state["slots"].long()
    page = slots.clamp(min=0) // case["page"]
    first = torch.unique_consecutive(page, return_inverse=True)
    whole = _values(state[name][first[0]], state[name + "s"][first[0]], case, name == "v")
    rows = whole.transpose(1, 2)[first[1], slots.clamp(min=0) % case["page"]]
    return torch.where((slots >= 0)[:, None, None], rows, 0.0).to(state[name + "_back"].dtype)


def _quantised(x, group):
    """The values that rows come back as: codes 0..15 between a group's least and largest."""
    g = x.double().reshape(x.shape[:-1] + (-1, group))
    least, most = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((most - least) / 15).float().to(x.dtype).double()
    c = torch.where(scale > 0, torch.round(((g - least) / scale).float()).double(), 0.0).clamp(0, 15)
    return (c * scale + least).float().to(x.dtype).reshape(x.shape)


def _plain_store(state):
    kept = (state["slots"] >= 0)[:, None, None]
    zero = torch.zeros((), dtype=state["k_back"].dtype, device=_DEV)
    return [torch.where(kept, _quantised(state[n], state["case"]["group"]), zero)
            for n in ("k_rows", "v_rows")]


def _plain_attend(state):
    case, q = state["case"], state["q"]
    d, h, heads, most = case["dim"], case["kv_heads"], case["heads"], state["most"]
    lens = state["lens"].long()
    n, rows = lens.numel(), q.shape[0]
    table = state["table"].long()
    k, v = [_values(state[m][table], state[m + "s"][table], case, m == "v").transpose(1, 2)
            .reshape(n, h, -1, d) for m in ("k", "v")]
    # the sequences' new rows, padded to the longest
    starts = torch.arange(n + 1, device=_DEV) if state["starts"] is None else state["starts"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(most, device=_DEV)
    at = (starts[:-1, None] + i).clamp(max=rows - 1)
    x = q[at].float().view(n, most, h, heads // h, d).permute(0, 2, 1, 3, 4).reshape(n, h, -1, d)
    score = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    # what a new row sees: tokens [last - window, last]
    token = torch.arange(k.shape[2], device=_DEV)
    last = (lens - count)[:, None] + i if case["causal"] else (lens - 1)[:, None] + 0 * i
    sees = (token <= last[..., None]) & (token < lens[:, None, None])
    if case["window"]:
        sees &= token > (lens - count)[:, None, None] + i[:, None] - case["window"]
    sees = sees[:, None, :, None, :].expand(n, 1, most, heads // h, token.numel())
    sees = sees.reshape(n, 1, -1, token.numel())
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p, v) / total.clamp(min=1e-30)
    lse = torch.log(total) + top
    y = y.view(n, h, most, heads // h, d).permute(0, 2, 1, 3, 4).reshape(n, most, heads, d)
    lse = lse.view(n, h, most, heads // h).permute(0, 2, 1, 3).reshape(n, most, heads)
    lse = torch.where(lse < -1e29, -math.inf, lse)
    mine = i < count[:, None]
    return y[mine].to(q.dtype), lse[mine]


def _plain(state):
    op = state["case"]["op"]
    return (_plain_attend(state) if op == "attend" else _plain_store(state) if op == "store"
            else [_rows_at(state, "k"), _rows_at(state, "v")])


# ---- the library's calls --------------------------------------------------------------------

def _own(state):
    import block_quantized_wire_amd as bq
    case, s = state["case"], state
    f16 = case["type"] == "f16"
    if "cache" not in s:        # the description of its cache, which a program makes once
        s["cache"] = bq.KvI4(s["k"], s["v"], s["ks"], s["vs"], group=case["group"])
    if case["op"] == "attend":
        call = bq.bq_attn_i4_f16 if f16 else bq.bq_attn_i4
        call(s["q"], s["cache"], s["table"], s["lens"], s["out"], starts=s["starts"], max_q=s["most"],
             max_len=s["longest"], causal=case["causal"], window=case["window"], lse=s["lse"], ws=s["work"])
        return s["out"], s["lse"]
    if case["op"] == "store":
        call = bq.bq_kv_write_i4_f16 if f16 else bq.bq_kv_write_i4
        call(s["k_rows"], s["v_rows"], s["slots"], s["cache"])
    call = bq.bq_kv_read_i4_f16 if f16 else bq.bq_kv_read_i4
    call(s["cache"], s["slots"], s["k_back"], s["v_back"])
    return [s["k_back"], s["v_back"]]


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------

def _seen(case):
    """(tokens of the cache that some row sees, pairs of a row and a token that it sees)."""
    tokens = pairs = 0
    for n, new in zip(*_counts(case)):
        first, past = n, 0
        for i in range(new):
            hi = min(n, n - new + i + 1) if case["causal"] else n
            lo = max(0, n - new + i + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, hi - lo)
            if hi > lo:
                first, past = min(first, lo), max(past, hi)
        tokens += max(0, past - first)
    return tokens, pairs


def work(case):
    h, d = case["kv_heads"], case["dim"]
    row = d // 2 + 4 * (d // case["group"])         # a cached row of keys or of values
    if case["op"] in ("store", "fetch"):
        t = case["tokens"]
        kept = t * h * (1 - case["drop"])
        if case["op"] == "fetch":
            return {"bytes": 2 * kept * row + 4 * t * h * d + 4 * t, "flops": 4 * kept * d}
        # rows in, their codes written and read between the two calls, rows out
        return {"bytes": 4 * kept * d + 4 * kept * row + 4 * t * h * d + 8 * t, "flops": 12 * kept * d}
    tokens, pairs = _seen(case)
    rows = sum(_counts(case)[1])
    return {"bytes": 2 * tokens * h * row + 4 * rows * case["heads"] * d + 4 * rows * case["heads"],
            "flops": 4 * pairs * case["heads"] * d}


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_rows(codes, scales, slot, case, is_v):
    """Rows [tokens, D] in 64 bits of one head's codes [pages, page, D/2], value by value."""
    d, group, s = case["dim"], case["group"], case["page"]
    page, place = slot // s, slot % s
    i = torch.arange(d, device=slot.device)
    if is_v:
        j, r = torch.div(i, 16, rounding_mode="floor"), i % 16
        t = (place % 8)[:, None]
        word = (r * 4 + torch.div(t, 2, rounding_mode="floor")) * (d // 64) + torch.div(j, 4, rounding_mode="floor")
        byte = word * 4 + (t % 2) * 2 + torch.div(j % 4, 2, rounding_mode="floor")
        byte, odd = byte + (place - place % 8)[:, None] * (d // 2), j % 2
    else:
        word = torch.div(i % 32, 8, rounding_mode="floor") * (d // 32) + torch.div(i, 32, rounding_mode="floor")
        byte, odd = (word * 4 + torch.div(i % 8, 2, rounding_mode="floor"))[None], i % 2
        byte = byte + place[:, None] * (d // 2)
    two = codes.reshape(codes.shape[0], -1)[page[:, None], byte].long()
    c = torch.where(odd == 1, torch.div(two, 16, rounding_mode="floor"), two % 16).double()
    of = torch.div(i, group, rounding_mode="floor")
    both = scales[page[:, None], of[None], place[:, None]].double()
    return c * both[..., 0] + both[..., 1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        back = []
        for name in ("k_rows", "v_rows"):
            x = s[name].double()
            y = torch.zeros_like(x)
            for at in range(0, case["dim"], case["group"]):
                part = x[:, :, at:at + case["group"]]
                low = part.min(2, keepdim=True)[0]
                unit = (part.max(2, keepdim=True)[0] - low) / 15
                held = unit.to(s[name].dtype).double()       # the format holds it in 16 bits
                steps = torch.round((part - low) / held.clamp(min=1e-300)).clamp(0, 15)
                y[:, :, at:at + case["group"]] = steps * held + low
            y[s["slots"] < 0] = 0
            back.append(y)
        return back
    if case["op"] == "fetch":
        slots = s["slots"].long()
        back = []
        for name in ("k", "v"):
            heads = [_exact_rows(s[name][:, h], s[name + "s"][:, h], slots.clamp(min=0), case, name == "v")
                     for h in range(case["kv_heads"])]
            y = torch.stack(heads, 1)
            y[slots < 0] = 0
            back.append(y)
        return back
    lens, new = _counts(case)
    share, d = case["heads"] // case["kv_heads"], case["dim"]
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=_DEV)
    row = 0
    for b, n in enumerate(lens):
        rows, row = slice(row, row + new[b]), row + new[b]
        if n == 0:
            continue
        token = torch.arange(n, device=_DEV)
        slot = s["table"][b].long()[torch.div(token, case["page"], rounding_mode="floor")] * case["page"] + token % case["page"]
        at = torch.arange(n - new[b], n, device=_DEV)[:, None]      # the new rows' places
        hidden = (token > at) if case["causal"] else (token < 0)[None].expand(new[b], n)
        if case["window"]:
            hidden = hidden | (token <= at - case["window"])
        blind = hidden.all(1)
        for h in range(case["kv_heads"]):
            k, v = (_exact_rows(s[m][:, h], s[m + "s"][:, h], slot, case, m == "v") for m in ("k", "v"))
            for i in range(h * share, (h + 1) * share):
                score = torch.mm(s["q"][rows, i].double(), k.t()) / math.sqrt(d)
                score.masked_fill_(hidden, -math.inf)
                score[blind] = 0.0
                total = torch.logsumexp(score, 1)
                part = torch.mm(torch.exp(score - total[:, None]), v)
                part[blind], total[blind] = 0.0, -math.inf
                y[rows, i], lse[rows, i] = part, total
    return y, lse
