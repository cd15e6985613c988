"""The products whose stored operand is held in few bits, case by case.

Four operators of a model that is served with this library:

* ``w4``      C = A W^T with the N x K matrix W held in 4 bits, a scale (and
              with ``zeros`` a zero point) for each group of k of a row.
* ``w4pack``  a matrix quantised to that form and read back.
* ``kv8``     new keys and values quantised into a paged cache of 8-bit
              floats (e4m3) with one power-of-two scale for each page and
              head, and the end of every sequence read back.
* ``attend``  softmax attention of new queries over such a cache.

With ``own`` false a pass is made of elementary torch operations in float32;
with ``own`` true it is made of this package's calls.

Every sequence's length and its number of new rows follow from the case
alone (``_lengths``), everything else that is random from the seed.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # One token through a square layer: the shortest call, bound by its latency.
        {"name": "w4 1x1024x1024 f16", "op": "w4", "M": 1, "N": 1024, "K": 1024, "group": 64, "zeros": False,
         "dtype": "f16", "stype": "f16"},
        # One token through the wide layer of a block or its output layer: bound by the reading of the weights.
        {"name": "w4 1x16384x4096 bf16 zeros", "op": "w4", "M": 1, "N": 16384, "K": 4096, "group": 128, "zeros": True,
         "dtype": "bf16", "stype": "bf16"},
        # A small batch of tokens in float32 (what the library's own products return), no size a multiple of a tile.
        {"name": "w4 13x2047x4093 f32 zeros", "op": "w4", "M": 13, "N": 2047, "K": 4093, "group": 32, "zeros": True,
         "dtype": "f32", "stype": "f32"},
        # A prompt: many rows, bound by the matrix cores.
        {"name": "w4 2048x4096x4096 bf16", "op": "w4", "M": 2048, "N": 4096, "K": 4096, "group": 128, "zeros": False,
         "dtype": "bf16", "stype": "f16"},
        # A layer's weights quantised and read back, as a program does once per layer when it loads a model.
        {"name": "w4pack 4096x4096 bf16", "op": "w4pack", "N": 4096, "K": 4096, "group": 128, "zeros": False,
         "dtype": "bf16", "stype": "f16", "out": "bf16"},
        {"name": "w4pack 2047x4093 f32 zeros", "op": "w4pack", "N": 2047, "K": 4093, "group": 32, "zeros": True,
         "dtype": "f32", "stype": "f32", "out": "f32"},
        # One new token of one short conversation.
        {"name": "kv8 1 sequence 1 new f32", "op": "kv8", "seqs": 1, "length": 77, "new": 1, "back": 13, "heads": 2,
         "dim": 64, "block": 16, "dtype": "f32", "out": "f32"},
        # A batch that is being answered: one new token each, the last tokens read back.
        {"name": "kv8 64 sequences 1 new bf16", "op": "kv8", "seqs": 64, "length": 2000, "new": 1, "back": 128,
         "heads": 8, "dim": 128, "block": 32, "dtype": "bf16", "out": "f32"},
        # Prompts written whole and read back whole, to be used by a dense product.
        {"name": "kv8 4 prompts bf16", "op": "kv8", "seqs": 4, "length": 4096, "new": 4096, "back": 4096, "heads": 8,
         "dim": 128, "block": 64, "dtype": "bf16", "out": "bf16"},
        # The next token of one short conversation: bound by latency.
        {"name": "attend 1 sequence 200 tokens f32", "op": "attend", "seqs": 1, "length": 200, "new": 1, "heads": 2,
         "ratio": 4, "dim": 64, "block": 16, "window": 0, "causal": True, "dtype": "f32"},
        # The next token of a batch of long conversations: bound by the reading of the cache.
        {"name": "attend 32 sequences 8192 tokens bf16", "op": "attend", "seqs": 32, "length": 8192, "new": 1,
         "heads": 8, "ratio": 4, "dim": 128, "block": 64, "window": 0, "causal": True, "dtype": "bf16"},
        # A piece of two prompts behind what the cache already holds: bound by the matrix cores.
        {"name": "attend 2 prompts of 1024 behind 4096 f16", "op": "attend", "seqs": 2, "length": 5120, "new": 1024,
         "heads": 8, "ratio": 4, "dim": 128, "block": 32, "window": 0, "causal": True, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w4", "w4", "w4pack", "kv8", "attend", "attend"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("w4", "w4pack"):
        c = {"op": op, "N": _log(rng, 64, 16384), "K": _log(rng, 64, 16384), "group": rng.choice([32, 64, 128, 256]),
             "zeros": rng.random() < 0.5, "dtype": dtype, "stype": rng.choice(["f32", "bf16", "f16"])}
        if rng.random() < 0.6:  # most layers are multiples of 64
            c["N"], c["K"] = (c["N"] + 63) // 64 * 64, (c["K"] + 63) // 64 * 64
        if op == "w4":
            most = 2048 * 4096 * 4096 // (c["N"] * c["K"])
            if dtype == "f32":
                most //= 2
            c["M"] = _log(rng, 1, max(1, min(2048, most)))
            if c["N"] * c["K"] > 1 << 26:
                c["N"] = (1 << 26) // c["K"]
        else:
            c["out"] = rng.choice(["f32", dtype])
            if c["N"] * c["K"] > 1 << 24:
                c["N"] = (1 << 24) // c["K"]
        return c
    c = {"op": op, "seqs": _log(rng, 1, 64), "heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([32, 64, 80, 96, 128, 128, 256]),
         "block": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    per_token = c["heads"] * c["dim"]
    if op == "kv8":
        c["out"] = rng.choice(["f32", dtype])
        c["length"] = _log(rng, 1, max(1, min(8192, 4 * 4096 * 8 * 128 // (per_token * c["seqs"]))))
        c["new"] = 1 if rng.random() < 0.3 else _log(rng, 1, c["length"])
        c["back"] = _log(rng, 1, c["length"])
        return c
    c["ratio"] = rng.choice([1, 2, 4, 7, 8])
    c["length"] = _log(rng, 1, max(1, min(16384, 32 * 8192 * 8 * 128 // (2 * per_token * c["seqs"]))))
    most = 2 * 1024 * 5120 * 32 * 128 // (4 * c["seqs"] * c["length"] * per_token * c["ratio"])
    c["new"] = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, min(c["length"], 1024, most)))
    c["causal"] = rng.random() < 0.8
    c["window"] = _log(rng, 1, c["length"]) if c["causal"] and rng.random() < 0.25 else 0
    return c


def _lengths(case):
    """Tokens and new rows of each sequence: from half to all of the case's, spread by fixed irrational steps."""
    length, new = [], []
    for b in range(case["seqs"]):
        l = case["length"] - int(case["length"] / 2 * ((b * 0.6180339887) % 1.0))
        n = case["new"] - int(case["new"] / 2 * ((b * 0.4142135624) % 1.0))
        length.append(l)
        new.append(min(n, l))
    return length, new


def _visible(case, length, new):
    """Tokens of the cache that some new row of a sequence sees, and (row, token) pairs, over all sequences."""
    tokens = pairs = 0
    for l, n in zip(length, new):
        if not case["causal"]:
            tokens, pairs = tokens + l, pairs + n * l
            continue
        w = case["window"] or l
        pairs += sum(min(p + 1, w) for p in range(l - n, l))
        tokens += min(l, n - 1 + w)
    return tokens, pairs


def work(case):
    op, a = case["op"], SIZE[case["dtype"]]
    if op in ("w4", "w4pack"):
        N, K = case["N"], case["K"]
        groups = -(-K // case["group"])
        held = N * -(-K // 2) + N * groups * (SIZE[case["stype"]] + (1 if case["zeros"] else 0))
        if op == "w4":
            return {"bytes": held + case["M"] * (K * a + N * 4), "flops": 2 * case["M"] * N * K}
        return {"bytes": 2 * held + N * K * (a + SIZE[case["out"]]), "flops": 4 * N * K}
    length, new = _lengths(case)
    H, D = case["heads"], case["dim"]
    if op == "kv8":
        back = sum(min(case["back"], l) for l in length)
        return {"bytes": 2 * H * D * (sum(new) * (a + 1) + back * (1 + SIZE[case["out"]])),
                "flops": 2 * H * D * (2 * sum(new) + back)}
    tokens, pairs = _visible(case, length, new)
    return {"bytes": 2 * H * D * tokens + sum(new) * H * case["ratio"] * D * (a + 4),
            "flops": 4 * H * case["ratio"] * D * pairs}


# --------------------------------------------------------------- the inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _scale_of(amax):
    """The smallest power of two s with amax / s <= 448, e4m3's largest value; 0 for 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    power = ((e + 127) << 23).view(torch.float32)  # by its bits: a power function may miss the last one
    return torch.where(amax > 0, power, torch.zeros_like(amax))


def _inputs(case, seed):
    """The operands that a program has in hand, as plain tensors, and the host's knowledge of the sequences."""
    g, op, dtype = _generator(seed), case["op"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = {}
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        groups = -(-K // case["group"])
        x["A"] = normal(M, K).to(dtype)
        x["codes"] = torch.randint(0, 256, (N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8)
        if K % 2:
            x["codes"][:, -1] &= 15
        x["scales"] = (torch.rand(N, groups, generator=g, device="cuda") * 0.9 + 0.1).mul_(1 / 128).to(TYPES[case["stype"]])
        x["zeros"] = None
        if case["zeros"]:
            x["zeros"] = torch.randint(5, 11, (N, groups), generator=g, device="cuda", dtype=torch.uint8)
        return x
    if op == "w4pack":
        x["W"] = (normal(case["N"], case["K"]) * (normal(case["N"], 1).exp() / 32)).to(dtype)
        return x
    length, new = _lengths(case)
    B, H, D, T = case["seqs"], case["heads"], case["dim"], case["block"]
    per_seq = -(-max(length) // T)
    used = [-(-l // T) for l in length]
    pages = sum(used)
    x["length"], x["new"] = length, new
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, per_seq), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    x["table"] = table
    x["lens"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    x["rows"] = starts[-1]
    x["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for name in ("K", "V"):
        values = normal(pages, H, T, D) * (0.25 + torch.rand(1, H, 1, 1, generator=g, device="cuda"))
        s = _scale_of(values.abs().amax(dim=(2, 3)))
        x["cache" + name] = (values / s[:, :, None, None]).to(torch.float8_e4m3fn)
        x["scale" + name] = s
    if op == "kv8":
        grow = 4 * torch.rand(x["rows"], 1, 1, generator=g, device="cuda")
        x["newK"] = (normal(x["rows"], H, D) * grow).to(dtype)
        x["newV"] = (normal(x["rows"], H, D) * grow.flip(0)).to(dtype)
    else:
        x["Q"] = normal(x["rows"], H * case["ratio"], D).to(dtype)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    state = {"case": case, "x": x}
    op = case["op"]
    if op == "kv8":
        # Rows to read back: the last `back` tokens of every sequence.
        back = [min(case["back"], l) for l in x["length"]]
        ends = [0]
        for n in back:
            ends.append(ends[-1] + n)
        state["back"], state["back_rows"] = torch.tensor(ends, dtype=torch.int32, device="cuda"), ends[-1]
        # Pages that receive new rows, and whether they hold older ones.
        touched, kept = [], []
        T = case["block"]
        for b, (l, n) in enumerate(zip(x["length"], x["new"])):
            for p in range((l - n) // T, -(-l // T)):
                touched.append(b * x["table"].shape[1] + p)
                kept.append(max(0, l - n - p * T))
        state["touched"] = torch.tensor(touched, device="cuda")
        state["kept"] = torch.tensor(kept, device="cuda")
    if own:
        import dense_fp32_matrix_sgemm_amd as sg

        state["sg"] = sg
        if op == "w4":
            state["W"] = sg.W4(x["codes"], x["scales"], x["zeros"], case["K"], case["group"])
        elif op in ("kv8", "attend"):
            state["cache"] = sg.KV8(x["cacheK"], x["cacheV"], x["scaleK"], x["scaleV"])
    return state


# ------------------------------------------------------------------ a pass


def run(state):
    case, x = state["case"], state["x"]
    op = case["op"]
    if not own:
        return {"w4": _plain_w4, "w4pack": _plain_pack, "kv8": _plain_kv8, "attend": _plain_attend}[op](state, case, x)
    sg = state["sg"]
    if op == "w4":
        return sg.gemm_w4(x["A"], state["W"])
    if op == "w4pack":
        W = sg.quantize_w4(x["W"], group=case["group"], zeros=case["zeros"], scale_dtype=TYPES[case["stype"]])
        return [sg.dequantize_w4(W, TYPES[case["out"]]), W.scales] + ([W.zeros] if case["zeros"] else [])
    if op == "kv8":
        cache = state["cache"]
        sg.kv8_write(cache, x["newK"], x["newV"], x["table"], x["lens"], x["starts"], max_new=case["new"])
        K, V = sg.kv8_read(cache, x["table"], x["lens"], state["back"], rows=state["back_rows"],
                           dtype=TYPES[case["out"]], max_new=case["back"])
        return [K, V, cache.Ks, cache.Vs]
    return sg.kv8_attend(x["Q"], state["cache"], x["table"], x["lens"], x["starts"], scale=case["dim"] ** -0.5,
                         causal=case["causal"], window=case["window"], max_new=case["new"])


def _unpacked(codes, K):
    """The 4-bit codes of each row, the lower half of a byte first."""
    return torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)[:, :K]


def _plain_w4(state, case, x):
    K, g = case["K"], case["group"]
    q = _unpacked(x["codes"], K).float()
    z = 8.0 if x["zeros"] is None else x["zeros"].float().repeat_interleave(g, dim=1)[:, :K]
    W = (q - z) * x["scales"].float().repeat_interleave(g, dim=1)[:, :K]
    return torch.matmul(x["A"].float(), W.t())


def _plain_pack(state, case, x):
    N, K, g = case["N"], case["K"], case["group"]
    groups, stype = -(-K // g), TYPES[case["stype"]]
    w = torch.zeros(N, groups * g, dtype=torch.float32, device="cuda")
    w[:, :K] = x["W"]
    w = w.view(N, groups, g)
    if case["zeros"]:
        lo, hi = w.amin(dim=2).clamp(max=0), w.amax(dim=2).clamp(min=0)
        s = ((hi - lo).double() / 15).float().to(stype)
        d = s.double()
        z = torch.where(d > 0, (-lo.double() / d).round(), torch.full_like(d, 8)).clamp(0, 15)
    else:
        s = (w.abs().amax(dim=2).double() / 7).float().to(stype)
        d, z = s.double(), torch.full((N, groups), 8.0, dtype=torch.float64, device="cuda")
    # In 64 bits: a quotient next to a half has to fall on its own side.
    r = torch.where(d[:, :, None] > 0, (w.double() / d[:, :, None]).round(), torch.zeros(1, dtype=torch.float64, device="cuda"))
    q = (r + z[:, :, None]).clamp(0, 15)
    back = ((q - z[:, :, None]).float() * s.float()[:, :, None]).view(N, groups * g)[:, :K].to(TYPES[case["out"]])
    return [back, s] + ([z.to(torch.uint8)] if case["zeros"] else [])


def _slots(table, lens, starts, rows, T):
    """Page and place in it of each of the sequences' last rows."""
    i = torch.arange(rows, device="cuda")
    b = torch.searchsorted(starts[1:].long(), i, right=True)
    position = lens[b] - (starts[b + 1] - i)
    return table[b, position // T].long(), position % T


def _plain_kv8(state, case, x):
    T = case["block"]
    page, place = _slots(x["table"], x["lens"], x["starts"], x["rows"], T)
    touched = x["table"].view(-1)[state["touched"]].long()
    old = torch.arange(T, device="cuda")[None, :] < state["kept"][:, None]  # older tokens of the touched pages
    for name in ("K", "V"):
        new, codes, scales = x["new" + name].float(), x["cache" + name], x["scale" + name]
        amax = torch.zeros_like(scales)
        amax.scatter_reduce_(0, page[:, None].expand(-1, scales.shape[1]), new.abs().amax(dim=2), "amax")
        before = scales[touched] * (state["kept"] > 0)[:, None]
        after = torch.maximum(before, _scale_of(amax[touched]))
        ratio = torch.where(after > 0, before / after, torch.ones_like(after))
        bytes_ = codes.view(torch.uint8)
        was = bytes_[touched]
        moved = (was.view(torch.float8_e4m3fn).float() * ratio[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        bytes_[touched] = torch.where(old[:, None, :, None], moved, was)
        scales[touched] = after
        s = scales[page]
        inverse = torch.where(s > 0, 1 / s, torch.zeros_like(s))
        bytes_[page, :, place] = (new * inverse[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    page, place = _slots(x["table"], x["lens"], state["back"], state["back_rows"], T)
    out = []
    for name in ("K", "V"):
        codes = x["cache" + name].view(torch.uint8)[page, :, place].view(torch.float8_e4m3fn).float()
        out.append((codes * x["scale" + name][page][:, :, None]).to(TYPES[case["out"]]))
    return out + [x["scaleK"], x["scaleV"]]


def _plain_attend(state, case, x):
    """All sequences at once, padded to the longest."""
    B, H, D, T, R = case["seqs"], case["heads"], case["dim"], case["block"], case["ratio"]
    n, rows = max(x["new"]), x["rows"]
    table = x["table"].clamp(min=0).long()
    L = table.shape[1] * T

    def dense(name):
        values = x["cache" + name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        values = values * x["scale" + name][table][:, :, :, None, None]
        return values.permute(0, 2, 1, 3, 4).reshape(B * H, L, D)

    count = x["starts"][1:] - x["starts"][:-1]
    i = torch.arange(n, device="cuda")
    source = (x["starts"][:-1, None] + i[None, :]).clamp(max=rows - 1).long()
    Q = x["Q"][source].float().view(B, n, H, R, D).permute(0, 2, 3, 1, 4).reshape(B * H, R * n, D)
    S = torch.matmul(Q, dense("K").transpose(1, 2)).view(B, H, R, n, L) * D ** -0.5
    j = torch.arange(L, device="cuda")[None, None, :]
    seen = j < x["lens"][:, None, None]
    if case["causal"]:
        position = (x["lens"] - count)[:, None, None] + i[None, :, None]
        seen = seen & (j <= position)
        if case["window"]:
            seen = seen & (j > position - case["window"])
    seen = seen.expand(B, n, L)[:, None, None]
    S = torch.where(seen, S, torch.full_like(S[:1, :1, :1, :1, :1], -math.inf))
    P = torch.exp(S - S.amax(dim=4, keepdim=True).clamp(min=-3e38))
    P = P / P.sum(dim=4, keepdim=True).clamp(min=1e-38)
    O = torch.matmul(P.view(B * H, R * n, L), dense("V")).view(B, H, R, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H * R, D)
    return O[(i[None, :] < count[:, None])].contiguous()


# ---------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    x, op = _inputs(case, seed), case["op"]
    if op == "w4":
        K, N = case["K"], case["N"]
        k = torch.arange(K, device="cuda")
        q = ((x["codes"][:, k // 2].int() >> (4 * (k % 2))[None, :]) & 15).double()
        group = k // case["group"]
        z = 8.0 if x["zeros"] is None else x["zeros"].double()[:, group]
        return x["A"].double() @ ((q - z) * x["scales"].double()[:, group]).T
    if op == "w4pack":
        return _exact_pack(case, x)
    if op == "kv8":
        return _exact_kv8(case, x)
    return _exact_attend(case, x)


def _exact_pack(case, x):
    w, g = x["W"].double(), case["group"]
    back, scales, zeros = torch.empty_like(w), [], []
    for k in range(0, case["K"], g):
        part = w[:, k:k + g]
        if case["zeros"]:
            top, low = torch.relu(part.max(dim=1).values), -torch.relu((-part).max(dim=1).values)
            span = (top - low).float().double() / 15  # the span is a float32 by definition
        else:
            top, low = part.abs().max(dim=1).values, None
            span = top / 7
        s = span.float().to(TYPES[case["stype"]]).double()
        safe = torch.where(s > 0, s, torch.ones_like(s))
        z = torch.full_like(s, 8) if low is None else torch.where(s > 0, torch.round(-low / safe), torch.full_like(s, 8)).clamp(0, 15)
        q = torch.where(s[:, None] > 0, torch.round(part / safe[:, None]), torch.zeros_like(part)) + z[:, None]
        back[:, k:k + g] = (q.clamp(0, 15) - z[:, None]) * s[:, None]
        scales.append(s)
        zeros.append(z.to(torch.uint8))
    return [back, torch.stack(scales, dim=1)] + ([torch.stack(zeros, dim=1)] if case["zeros"] else [])


def _two_to(e):
    """2**e as doubles, exactly, by their bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round8(v):
    """Doubles rounded to e4m3 (bias 7, 3 bits behind the point, no infinities), ties to the even code."""
    step = _two_to(torch.frexp(v.abs())[1].clamp(min=-5) - 4)
    return torch.round(v / step) * step


def _exact_kv8(case, x):
    H, T = case["heads"], case["block"]
    table, out = x["table"].cpu().tolist(), []
    for name in ("K", "V"):
        held = x["cache" + name].double()
        scales = x["scale" + name].double()
        first, rows = 0, []
        for b, (l, n) in enumerate(zip(x["length"], x["new"])):
            new = x["new" + name][first:first + n].double().transpose(0, 1)  # heads, rows, dim
            first += n
            for p in range((l - n) // T, -(-l // T)):
                lo, hi = max(l - n, p * T), min(l, p * T + T)
                part, page, kept = new[:, lo - (l - n):hi - (l - n)], table[b][p], lo - p * T
                top = part.abs().amax(dim=(1, 2))
                need = torch.where(top > 0, _two_to(torch.ceil(torch.log2(top.clamp(min=1e-37) / 448))), torch.zeros_like(top))
                s = need if kept == 0 else torch.maximum(need, scales[page])
                safe = torch.where(s > 0, s, torch.ones_like(s))[:, None, None]
                held[page, :, :kept] = _round8(held[page, :, :kept] * (scales[page][:, None, None] / safe))
                held[page, :, kept:kept + hi - lo] = _round8(part / safe)
                scales[page] = s
            ids = torch.tensor(table[b][:-(-l // T)], device="cuda")
            dense = (held[ids] * scales[ids][:, :, None, None]).transpose(1, 2).reshape(-1, H, case["dim"])
            rows.append(dense[l - min(case["back"], l):l])
        out.append((torch.cat(rows), scales))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_attend(case, x):
    H, D, T, R = case["heads"], case["dim"], case["block"], case["ratio"]
    out, first = [], 0
    for b, (l, n) in enumerate(zip(x["length"], x["new"])):
        ids = x["table"][b, :-(-l // T)].long()
        K, V = ((x["cache" + m].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * x["scale" + m].double()[ids][:, :, None, None])
                .transpose(0, 1).reshape(H, -1, D)[:, :l] for m in ("K", "V"))
        Q = x["Q"][first:first + n].double()
        first += n
        o = torch.empty(n, H * R, D, dtype=torch.float64, device="cuda")
        distance = torch.arange(l - n, l, device="cuda")[:, None] - torch.arange(l, device="cuda")[None, :]
        hidden = torch.zeros_like(distance, dtype=torch.bool)
        if case["causal"]:
            hidden = distance < 0
            if case["window"]:
                hidden = hidden | (distance >= case["window"])
        for h in range(H * R):
            score = (Q[:, h] @ K[h // R].T) / math.sqrt(D)
            o[:, h] = torch.softmax(score.masked_fill(hidden, -math.inf), dim=1) @ V[h // R]
        out.append(o)
    return torch.cat(out)
