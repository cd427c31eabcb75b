"""Operators between the packed projections of a served layer, as measured cases: rotary positions, the quantised cache
of keys and values, and the attention of new tokens over it.

Each case is one pass through one operator: `gptq_rotary` (positions turned into rotations of a token's heads),
`gptq_cache_write` with `gptq_cache_read` (keys and values quantised into pages, and read back) and
`gptq_cache_attention` (one new token of every request over its pages).  With `own` false, `run` computes them from
elementary torch operations in 32 bits (64 for angles and for values on a rounding border); with `own` true it calls
the library.

A page holds `ps` tokens of every head: for each head a block of bytes [keys][values][key scales][value scales], the
scales (fp32, one per token) only for 8 and 4 bits.  `Dp` is the stored head size.  Keys: a row of Dp values per token.
Values: per eight tokens Dp x 8 values, the eight tokens of a dimension side by side; with 4 bits a byte holds
dimensions 2i (low) and 2i + 1 of one token.  Codes are two's complement, value = scale * code.
"""
import hashlib
import math
import random

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"


def listed():
    return [
        # the next token of one request, query and key heads of an 8B-shaped layer: nothing but latency
        dict(name="rotary_one_token", op="rotary", T=1, H=40, D=128, rot=128, interleaved=False, kind="none",
             dtype=BF16, far=131072),
        # a prompt batch whose positions lie far out, frequencies stretched for a long context: memory traffic
        dict(name="rotary_prompt_far", op="rotary", T=8192, H=40, D=128, rot=128, interleaved=False, kind="ramp",
             dtype=BF16, far=1048576),
        # neighbouring pairs, part of an odd-sized head, 32-bit rows
        dict(name="rotary_partial_f32", op="rotary", T=2111, H=11, D=80, rot=32, interleaved=True, kind="linear",
             dtype=F32, far=32768),
        # the new tokens of 64 requests, scattered over their pages: latency
        dict(name="cache_decode_8bit", op="cache", T=64, H=8, D=128, bits=8, ps=16, dtype=BF16, pad=0, runs=64),
        # prompts written in 4 bits: memory traffic, and the arithmetic of exact rounding
        dict(name="cache_prompt_4bit", op="cache", T=16384, H=8, D=128, bits=4, ps=64, dtype=BF16, pad=0, runs=5),
        # a padded batch of ragged prompts with 32-bit rows, odd head counts and pages
        dict(name="cache_odd_f32", op="cache", T=1531, H=5, D=96, bits=8, ps=48, dtype=F32, pad=37, runs=9),
        # prompts of wide heads kept in bf16
        dict(name="cache_prompt_bf16", op="cache", T=4096, H=4, D=256, bits=16, ps=32, dtype=BF16, pad=0, runs=3),
        # one request with a short context: the smallest call, latency
        dict(name="attend_one_short", op="attend", R=1, most=777, spread="even", Hq=32, H=8, D=128, bits=8, ps=16,
             window=0, dtype=BF16),
        # a served batch of ragged contexts, 8 bits
        dict(name="attend_64_ragged_8bit", op="attend", R=64, most=8192, spread="ragged", Hq=32, H=8, D=128, bits=8,
             ps=64, window=0, dtype=BF16),
        # one long context beside short ones, 4 bits, 70B-shaped heads: its length has to be shared out
        dict(name="attend_long_4bit", op="attend", R=5, most=131072, spread="one_long", Hq=64, H=8, D=128, bits=4,
             ps=64, window=0, dtype=BF16),
        # 32-bit rows, as many key heads as query heads, odd head size and pages, a sliding window, an empty request
        dict(name="attend_window_f32", op="attend", R=13, most=3001, spread="ragged", Hq=12, H=12, D=80, bits=16,
             ps=48, window=1000, dtype=F32),
        # many requests of like lengths kept in bf16: memory traffic
        dict(name="attend_256_bf16", op="attend", R=256, most=2048, spread="even", Hq=32, H=4, D=128, bits=16, ps=16,
             window=0, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "attend", "attend"])
    dtype = BF16 if rng.random() < 0.7 else F32
    D = rng.choice([32, 64, 64, 72, 80, 96, 104, 128, 128, 128, 192, 256])
    ps = rng.choice([16, 16, 32, 48, 64, 64, 128, 256])
    bits = rng.choice([4, 8, 8, 16])
    while True:
        if op == "rotary":
            T, H = _log(rng, 1, 16384), _log(rng, 1, 64)
            if T * H * D <= 8192 * 40 * 128:
                return dict(op=op, T=T, H=H, D=D, rot=rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]),
                            interleaved=rng.random() < 0.4, kind=rng.choice(["none", "linear", "base", "ramp", "bands"]),
                            dtype=dtype, far=_log(rng, 1024, 1048576))
        elif op == "cache":
            T, H = _log(rng, 1, 16384), _log(rng, 1, 32)
            if T * H * D <= 16384 * 8 * 128:
                return dict(op=op, T=T, H=H, D=D, bits=bits, ps=ps, dtype=dtype, pad=rng.choice([0, 0, 1, 29]),
                            runs=_log(rng, 1, T))
        else:
            R, most, H = _log(rng, 1, 256), _log(rng, 1, 131072), _log(rng, 1, 16)
            case = dict(op=op, R=R, most=most, spread=rng.choice(["even", "ragged", "ragged", "one_long"]),
                        Hq=H * rng.choice([1, 2, 4, 4, 5, 7, 8, 16, 20]), H=H, D=D, bits=bits, ps=ps,
                        window=rng.choice([0, 0, 0, _log(rng, 1, most)]), dtype=dtype)
            # R * most bounds the plain form, which pads every request to the longest
            if R * most * H * D <= 64 * 8192 * 8 * 128 and case["Hq"] <= 128 and work(case)["bytes"] <= 1.0e9:
                return case


def _fixed(case):
    """Random choices that are part of the case itself (lengths of requests, how a batch splits into runs)."""
    text = ",".join("%s=%s" % kv for kv in sorted(case.items()) if kv[0] != "name")
    return random.Random(int(hashlib.sha256(text.encode()).hexdigest()[:12], 16))


def _lengths(case):
    rng, most, R = _fixed(case), case["most"], case["R"]
    if case["spread"] == "even":
        out = [max(1, int(most * rng.uniform(0.9, 1.0))) for _ in range(R)]
    elif case["spread"] == "ragged":
        out = [int(most * rng.random() ** 2) for _ in range(R)]
    else:
        out = [int(most / 64 * rng.random()) for _ in range(R)]
    out[rng.randrange(R)] = most
    if R > 4 and case["spread"] != "even":
        out[out.index(min(out))] = 0                # a slot of the batch without a request
    return out


def _visible(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lengths(case)]


def _type(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _stored(D):
    return min(n for n in (64, 96, 128, 192, 256) if n >= D)


def _block(case):
    """Bytes of a head's part of a page."""
    ps, bits = case["ps"], case["bits"]
    return 2 * ps * _stored(case["D"]) * bits // 8 + (8 * ps if bits < 16 else 0)


def _frequencies(rot, kind):
    """Radians per position of every pair, and the factor on cos and sin."""
    base, factor, original = 500000.0, 8.0, 8192.0
    if kind == "base":
        base *= factor ** (rot / max(rot - 2, 1))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        f = [v / factor for v in f]
    elif kind == "ramp":                            # pairs that turn often stay, those that hardly turn are stretched
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        keep = [1.0 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [v * k + v / factor * (1 - k) for v, k in zip(f, keep)]
    elif kind == "bands":
        smooth = [min(max((original * v / (2 * math.pi) - 1.0) / 3.0, 0.0), 1.0) for v in f]
        f = [v * (s + (1 - s) / factor) for v, s in zip(f, smooth)]
    return f, (0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def _rows(gen, shape, dtype):
    """Normal rows with a few strong dimensions, as keys have them."""
    c = torch.exp(0.3 * torch.randn(shape[-1], generator=gen, device="cuda"))
    c[torch.randint(0, shape[-1], (2,), generator=gen, device="cuda")] *= 6.0
    return (torch.randn(*shape, generator=gen, device="cuda") * c).to(dtype)


def _codes(x, bits):
    """Scale and codes of rows (last dimension): the symmetric grid over [-absmax, absmax], ties to even."""
    m = x.float().abs().amax(-1)
    s = (m.double() / (2.0 ** (bits - 1) - 0.5)).float().clamp(min=2.0 ** -126)
    fine = torch.isfinite(m)
    c = torch.round(x.double() / s.double().unsqueeze(-1)).clamp(-2.0 ** (bits - 1), 2.0 ** (bits - 1) - 1)
    return torch.where(fine, s, math.nan), torch.where(fine.unsqueeze(-1), c, 0.0).to(torch.int8)


def _parts(pages, case):
    """Views of the pages' bytes: key rows, value octets, key scales, value scales."""
    ps, bits, Dp = case["ps"], case["bits"], _stored(case["D"])
    n = ps * Dp * bits // 8
    keys = pages[..., :n].unflatten(-1, (ps, n // ps))
    unit = 2 if bits == 16 else 1
    values = pages[..., n:2 * n].unflatten(-1, (ps // 8, n // ps // unit, 8, unit))
    if bits == 16:
        return keys, values, None, None
    return (keys, values, pages[..., 2 * n:2 * n + 4 * ps].unflatten(-1, (ps, 4)),
            pages[..., 2 * n + 4 * ps:].unflatten(-1, (ps, 4)))


def _to_bytes(x, bits, Dp):
    """Rows as bytes (bf16, bytes, or two dimensions in a byte), and their scales."""
    if bits == 16:
        scale, c = None, x.to(torch.bfloat16)
    else:
        scale, c = _codes(x, bits)
    c = torch.nn.functional.pad(c, (0, Dp - x.shape[-1]))
    if bits == 4:
        return scale, (c[..., 0::2] & 15 | c[..., 1::2] << 4).view(torch.uint8)
    return scale, c.view(torch.uint8)


def _from_bytes(b, bits):
    if bits == 16:
        return b.view(torch.bfloat16).float()
    c = b.view(torch.int8)
    if bits == 8:
        return c.float()
    return torch.stack([(c << 4) >> 4, c >> 4], -1).flatten(-2).float()


def _put(pages, case, slots, k, v):
    ps, bits, Dp = case["ps"], case["bits"], _stored(case["D"])
    keys, values, ks, vs = _parts(pages, case)
    page, at = slots // ps, slots % ps
    scale, b = _to_bytes(k, bits, Dp)
    keys[page, :, at] = b
    if scale is not None:
        ks[page, :, at] = scale.unsqueeze(-1).view(torch.uint8)
    scale, b = _to_bytes(v, bits, Dp)
    values[page, :, at // 8, :, at % 8] = b.unflatten(-1, (-1, values.shape[-1]))
    if scale is not None:
        vs[page, :, at] = scale.unsqueeze(-1).view(torch.uint8)


def _get(pages, case, slots):
    ps, bits, D = case["ps"], case["bits"], case["D"]
    keys, values, ks, vs = _parts(pages, case)
    page, at = slots // ps, slots % ps
    k = _from_bytes(keys[page, :, at], bits)
    v = _from_bytes(values[page, :, at // 8, :, at % 8].flatten(-2), bits)
    if bits < 16:
        k = k * ks[page, :, at].view(torch.float32)
        v = v * vs[page, :, at].view(torch.float32)
    return k[..., :D], v[..., :D]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    op, s, dtype, D = case["op"], {"case": case}, _type(case), case["D"]
    if op == "rotary":
        T = case["T"]
        s["x"] = _rows(gen, (T, case["H"], D), dtype)
        # requests one after the other, each with its own run of positions
        start = torch.randint(0, max(1, case["far"] - T), (1 + T // 512,), generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        s["positions"] = (start[t // 512] + t % 512).to(torch.int32)
        f, s["factor"] = _frequencies(case["rot"], case["kind"])
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["out"] = torch.empty_like(s["x"])
        return s
    H, ps = case["H"], case["ps"]
    if op == "cache":
        T, rng, n = case["T"], _fixed(case), min(case["runs"], case["T"])
        cuts = [0] + sorted(rng.sample(range(1, T), n - 1)) + [T] if n > 1 else [0, T]
        per = [-(-(cuts[i + 1] - cuts[i]) // ps) + 1 for i in range(n)]
        order = torch.randperm(sum(per), generator=gen, device="cuda")
        slots, used = [], 0
        for i in range(n):                          # a run of tokens continues its request's pages somewhere in the first
            at = rng.randrange(ps) + torch.arange(cuts[i + 1] - cuts[i], device="cuda")
            slots.append(order[used + at // ps] * ps + at % ps)
            used += per[i]
        s["n"] = T
        s["slots"] = torch.cat(slots + [torch.full((case["pad"],), -1, device="cuda")]).to(torch.int32)
        s["k"] = _rows(gen, (T + case["pad"], H, D), dtype)
        s["v"] = _rows(gen, (T + case["pad"], H, D), dtype)
        s["pages"] = torch.zeros(sum(per), H, _block(case), dtype=torch.uint8, device="cuda")
        return s
    R, lengths = case["R"], _lengths(case)
    s["q"] = _rows(gen, (R, case["Hq"], D), dtype)
    s["lengths"] = _ints(lengths)
    per = [-(-n // ps) for n in lengths]
    P = sum(per) + 3                                # pages that nobody uses are part of a pool
    order = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    s["table"] = torch.full((R, max(per) + 1), -1, dtype=torch.int32, device="cuda")
    filled, used = torch.zeros(P, device="cuda", dtype=torch.int32), 0
    for r in range(R):
        s["table"][r, :per[r]] = order[used:used + per[r]]
        if per[r]:
            filled[order[used:used + per[r]].long()] = ps
            filled[order[used + per[r] - 1].long()] = lengths[r] - (per[r] - 1) * ps
        used += per[r]
    s["pages"] = torch.zeros(P, H, _block(case), dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 25) // (ps * H * D))
    for i in range(0, P, some):
        page = torch.arange(i, min(P, i + some), device="cuda")
        slots = (page.unsqueeze(1) * ps + torch.arange(ps, device="cuda")).flatten()
        k, v = (_rows(gen, (slots.numel(), H, D), torch.bfloat16) for _ in range(2))
        stale = slots % ps >= filled[slots // ps]   # slots that no token has reached hold anything
        k[stale] = math.nan
        v[stale] = math.nan
        _put(s["pages"], case, slots, k, v)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


def _run_plain(s):
    case = s["case"]
    op, D = case["op"], case["D"]
    if op == "rotary":
        x, rot = s["x"].float(), case["rot"]
        angle = s["positions"].double().unsqueeze(1) * s["freqs"]
        cos = (torch.cos(angle) * s["factor"]).float().unsqueeze(1)
        sin = (torch.sin(angle) * s["factor"]).float().unsqueeze(1)
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., rot:]], -1).to(_type(case))
    if op == "cache":
        n = s["n"]
        slots = s["slots"][:n].long()
        _put(s["pages"], case, slots, s["k"][:n], s["v"][:n])
        k, v = _get(s["pages"], case, slots)
        return {n_: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, case["pad"])).to(_type(case)) for n_, x in (("k", k), ("v", v))}
    R, H, ps, bits = case["R"], case["H"], case["ps"], case["bits"]
    g = case["Hq"] // H
    blocks = s["pages"][s["table"][:, :-1].clamp(min=0).long()]             # R x pages x H x bytes
    keys, values, ks, vs = _parts(blocks, case)
    L = blocks.shape[1] * ps
    k = _from_bytes(keys, bits)                                              # R x pages x H x ps x Dp
    v = _from_bytes(values.permute(0, 1, 2, 3, 5, 4, 6).flatten(-2).contiguous(), bits).flatten(3, 4)
    if bits < 16:
        k = k * ks.contiguous().view(torch.float32)
        v = v * vs.contiguous().view(torch.float32)
    k = k[..., :D].transpose(1, 2).reshape(R, H, L, D)
    v = v[..., :D].transpose(1, 2).reshape(R, H, L, D)
    at = torch.arange(L, device=k.device)
    n = s["lengths"].unsqueeze(1)
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    v = torch.where(seen[:, None, :, None], v, 0.0)
    score = (s["q"].float().view(R, H, g, D) @ k.transpose(2, 3)) * s["scale"]
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    whole = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(whole == 0, 1.0, whole)
    lse = torch.where(whole == 0, -math.inf, top + torch.log(whole))
    return {"out": out.view(R, H * g, D).to(_type(case)), "lse": lse.view(R, H * g)}


def _run_own(s):
    import post_weight_quantization_09_amd as G
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        return G.gptq_rotary(s["x"], s["positions"], s["freqs"], interleaved=case["interleaved"], factor=s["factor"],
                             out=s["out"])
    if op == "cache":
        G.gptq_cache_write(s["k"], s["v"], s["pages"], s["slots"], case["bits"])
        k, v = G.gptq_cache_read(s["pages"], s["slots"], case["D"], case["bits"], _type(case))
        return {"k": k, "v": v}
    ws = s.get("workspace")
    if ws is None:                                  # kept by the program beside its other buffers
        need = G.gptq_attention_workspace_bytes(case["R"], case["Hq"], case["H"], case["D"])
        ws = s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        s["lse"] = torch.empty(case["R"], case["Hq"], device="cuda")
    out = G.gptq_cache_attention(s["q"], s["pages"], s["table"], s["lengths"], case["bits"], scale=s["scale"],
                                 window=case["window"], lse=s["lse"], workspace=ws)
    return {"out": out, "lse": s["lse"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, D, size = case["op"], case["D"], 2 if case["dtype"] == BF16 else 4
    if op == "rotary":
        T, H, rot = case["T"], case["H"], case["rot"]
        return {"bytes": 2 * T * H * D * size + 4 * T + 4 * rot, "flops": 3.0 * T * H * rot}
    kept = D * case["bits"] // 8 + (4 if case["bits"] < 16 else 0)
    if op == "cache":
        T, H = case["T"], case["H"]
        return {"bytes": 4 * T * H * (D * size + kept) + 2 * case["pad"] * H * D * size + 8 * (T + case["pad"]),
                "flops": 6.0 * T * H * D}
    seen = sum(_visible(case))
    return {"bytes": 2 * seen * case["H"] * kept + case["R"] * case["Hq"] * (2 * D * size + 4)
            + 4 * sum(-(-n // case["ps"]) for n in _visible(case)) + 4 * case["R"], "flops": 4.0 * seen * case["Hq"] * D}


def _rounded64(x, bits):
    """A row kept in `bits` bits, as the values it stands for: x is an array of float64."""
    if bits == 16:
        return torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    half = 2.0 ** (bits - 1)
    scale = np.maximum((np.abs(x).max(-1, keepdims=True) / (half - 0.5)).astype(np.float32), np.float32(2.0 ** -126))
    scale = scale.astype(np.float64)
    return np.minimum(np.rint(x / scale), half - 1) * scale


def _tokens64(s, r, first, last):
    """Keys and values of tokens [first, last) of request r from the pages' bytes, H x tokens x D in 64 bits."""
    case = s["case"]
    ps, bits, D, Dp = case["ps"], case["bits"], case["D"], _stored(case["D"])
    t, (P, H, size), flat = torch.arange(first, last, device="cuda"), s["pages"].shape, s["pages"].view(-1)
    begin = (s["table"][r][t // ps].long().view(-1, 1) * H + torch.arange(H, device="cuda")).unsqueeze(2) * size
    row, n = Dp * bits // 8, ps * Dp * bits // 8
    at, d = (t % ps).view(-1, 1, 1), torch.arange(D, device="cuda").view(1, 1, -1)

    def take(where, count):
        """Little-endian whole numbers of `count` bytes at `where` in the blocks of every token's page."""
        out = 0
        for i in range(count):
            out = out | flat[begin + where + i].long() << 8 * i
        return out

    def real(bits32):
        return torch.where(bits32 >= 1 << 31, bits32 - (1 << 32), bits32).to(torch.int32).view(torch.float32).double()

    def signed(c, b):
        return torch.where(c >= 1 << (b - 1), c - (1 << b), c).double()

    if bits == 16:
        k, v = real(take(at * row + 2 * d, 2) << 16), real(take(n + ((at // 8 * Dp + d) * 8 + at % 8) * 2, 2) << 16)
    else:
        if bits == 8:
            k, v = signed(take(at * row + d, 1), 8), signed(take(n + (at // 8 * Dp + d) * 8 + at % 8, 1), 8)
        else:
            k = signed(take(at * row + d // 2, 1) >> 4 * (d % 2) & 15, 4)
            v = signed(take(n + (at // 8 * (Dp // 2) + d // 2) * 8 + at % 8, 1) >> 4 * (d % 2) & 15, 4)
        k, v = k * real(take(2 * n + 4 * at, 4)), v * real(take(2 * n + 4 * ps + 4 * at, 4))
    return k.transpose(0, 1), v.transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "rotary":
        x, rot = s["x"].double().cpu().numpy(), case["rot"]
        z = np.exp(1j * s["positions"].cpu().numpy().astype(np.float64)[:, None, None] * s["freqs"].cpu().numpy())
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        turned = (x[..., first] + 1j * x[..., second]) * z * s["factor"]
        out = x.copy()
        out[..., first], out[..., second] = turned.real, turned.imag
        return out
    if op == "cache":
        n, out = s["n"], {}
        for name in ("k", "v"):
            x = s[name].double().cpu().numpy()
            out[name] = np.zeros_like(x)
            out[name][:n] = _rounded64(x[:n], case["bits"])
        return out
    R, H, Hq = case["R"], case["H"], case["Hq"]
    out = torch.zeros(R, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, (n, seen) in enumerate(zip(_lengths(case), _visible(case))):
        q = s["q"][r].double().view(H, Hq // H, D)
        parts = []
        for t in range(n - seen, n, 8192):          # tokens in pieces, joined by their log sums
            k, v = _tokens64(s, r, t, min(n, t + 8192))
            x = (q.unsqueeze(2) * k.unsqueeze(1)).sum(-1) if k.shape[1] < 64 else q @ k.transpose(1, 2).contiguous()
            x = x * s["scale"]
            parts.append((torch.logsumexp(x, -1), torch.softmax(x, -1) @ v))
        if parts:
            logs = torch.stack([p[0] for p in parts])
            share = torch.softmax(logs, 0)
            out[r] = sum(w.unsqueeze(-1) * p[1] for w, p in zip(share, parts)).view(Hq, D)
            lse[r] = torch.logsumexp(logs, 0).view(Hq)
    return {"out": out, "lse": lse}
