"""Edges of rotary positions, the cache and the attention over it: the largest and smallest queries, infinities, far angles,
the join's forms, packed projections around them.

Bounds are those of test_context.py unless a test says otherwise.
"""
import math
from fractions import Fraction

import pytest
import torch

import post_weight_quantization_09_amd as g
from test_context import BF16, DEV, F32, U, attend64, check_attention, filled, gen_rows, ints, values64

gpu = pytest.mark.gpu


def written(k, v, bits, ps=16):
    """Pages in order of the tokens, and their table."""
    P = -(-k.shape[0] // ps)
    pages = torch.zeros(P, k.shape[1], g.gptq_cache_block_bytes(ps, k.shape[2], bits), dtype=torch.uint8, device=DEV)
    g.gptq_cache_write(k.to(DEV), v.to(DEV), pages, torch.arange(k.shape[0], dtype=torch.int32, device=DEV), bits)
    return pages, torch.arange(P, dtype=torch.int32, device=DEV)[None]


def held(x, bits, ps=16):
    """What those pages hold, in 64 bits."""
    x = torch.nn.functional.pad(values64(x, bits), (0, 0, 0, 0, 0, -x.shape[0] % ps))
    return x.view(-1, ps, *x.shape[1:])


def assert_near(out, ref, bound, dtype):
    unit = 2.0 ** -8 if dtype == BF16 else U
    off = (out.cpu().double() - ref).abs()
    assert (off <= unit * ref.abs() + (1 + unit) * bound + 1e-30).all(), off.max()


# ------------------------------------------------------------------------------------------------ the size of queries

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("scale", [2.0 ** -126, -2.0 ** -130])
def test_attention_of_queries_up_to_the_largest_number(scale, bits, dtype):
    """Every row's largest element is the type's largest number; the scale, also one below the smallest normal number, brings the
    scores back to tens."""
    q = gen_rows((4, 4, 64), F32, 1)
    q = (q / q.abs().amax(-1, keepdim=True) * 2.0 ** 100).double() * (torch.finfo(dtype).max * 2.0 ** -100)
    q = q.to(dtype)
    assert q.isfinite().all() and (q.abs().amax(-1) >= torch.finfo(dtype).max * (1 - 2.0 ** -20)).all()
    check_attention([33, 100, 1, 64], 4, 2, 64, 16, bits, dtype, scale=scale, q=q)


@gpu
@pytest.mark.parametrize("bits,dtype", [(16, BF16), (16, F32), (8, BF16), (8, F32), (4, F32)])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 127, -3.3e38])
def test_attention_of_zero_keys_under_large_queries_and_scales(scale, bits, dtype):
    """Scores are zero although scale times the largest query passes the largest number: an even mean of the values.  (4 bits
    under bf16 rows are left out: their scores are within 20 u 31 steps of sum |q|, a step of zeros is 2^-126, and 2^247 times
    that is no zero.)"""
    k, v = torch.zeros(70, 2, 64, dtype=BF16), gen_rows((70, 2, 64), BF16, 2)
    pages, table = written(k, v, bits)
    for size in (1.0, 2.0 ** 120):
        q = (gen_rows((1, 4, 64), F32, 3) * size).to(dtype)
        lse = torch.empty(1, 4, device=DEV)
        out = g.gptq_cache_attention(q.to(DEV), pages, table, ints([70]), bits, scale, lse=lse)
        ref, _, bound, _ = attend64(torch.zeros_like(q), held(k, bits), held(v, bits), table.cpu(), [70], 16, 1.0, 0, dtype, bits)
        assert_near(out, ref, bound, dtype)
        assert (lse.cpu().double() - math.log(70)).abs().max() <= 80 * U


# ------------------------------------------------------------------------------------------- probabilities in all bits

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_attention_to_one_token_gives_its_value(bits, dtype):
    """The probability is 1: the output is the value s c rounded once, whatever the scale's bits.  Its sum is at most three products
    of eight-bit parts, each addition off by at most 2 u of what it holds: s c, or with 4 bits under bf16 rows s (c + 24), at most
    31 s, and the excess 24 s, taken off at the end: 3 * 2 u (31 + 24) s + u 8 s < 344 u s."""
    n, H, D = 64, 4, 128
    k, v = gen_rows((n, H, D), BF16, 1), gen_rows((n, H, D), F32, 2)
    pages, _ = written(k.to(F32), v, bits)
    # a request for every token: its page, as many tokens as reach it, a window of one
    at = torch.arange(n, dtype=torch.int32, device=DEV)
    table, lengths = (at // 16)[:, None].contiguous(), at % 16 + 1
    out = g.gptq_cache_attention(gen_rows((n, H, D), dtype, 3).to(DEV), pages, table, lengths, bits, window=1).cpu()
    ref = values64(v, bits)
    off = 8 * U * ref.abs()
    if bits == 4 and dtype == BF16:
        off = 344 * U * ref.abs().amax(-1, keepdim=True) / 7             # a row's largest code is 7, or -8 (then s is less)
    low, high = (ref - off).float().to(dtype), (ref + off).float().to(dtype)
    if dtype == F32:
        low, high = ref - off, ref + off
    assert ((out >= low) & (out <= high)).all(), int(((out < low) | (out > high)).sum())


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_of_a_dimension_of_zeros_is_zero(dtype):
    """4 bits under bf16 rows: what the codes are raised by is taken off again by the same sums, whatever the probabilities."""
    lengths, H, D = [1, 40, 3000, 700], 2, 128
    k, v = gen_rows((3776, H, D), BF16, 1), gen_rows((3776, H, D), BF16, 2)
    v[..., [0, 5, 62, 127]] = 0.0
    pages, table = written(k, v, 4)
    tables = torch.zeros(4, 188, dtype=torch.int32, device=DEV)
    first = 0
    for r, n in enumerate(lengths):
        tables[r, :-(-n // 16)] = table[0, first:first + -(-n // 16)]
        first += -(-n // 16)
    out = g.gptq_cache_attention(gen_rows((4, 8, D), dtype, 3).to(DEV), pages, tables, ints(lengths), 4)
    assert not out[..., [0, 5, 62, 127]].any() and out.any(-1).all()


# ------------------------------------------------------------------------------------------------- what is not finite

@gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_attention_of_a_query_that_is_not_finite(bits, dtype, value):
    """NaN in its own row, also where every key meets the infinity with the sign that makes all scores -infinity; zeros where there
    is nothing to attend to."""
    lengths, H, D = [70, 0, 1, 3000], 2, 64
    k, v = gen_rows((3168, H, D), BF16, 1), gen_rows((3168, H, D), BF16, 2)
    k[..., 5] = -k[..., 5].abs() - 1.0                                # never a code of zero
    k[..., 6] = k[..., 5].abs()
    pages, table = written(k, v, bits)
    tables = torch.stack([table[0, :188], table[0, :188], table[0, 2:190], table[0, 5:193]])
    q = gen_rows((4, 4, D), dtype, 3)
    call = lambda x, lse: g.gptq_cache_attention(x.to(DEV), pages, tables, ints(lengths), bits, lse=lse).cpu()  # noqa: E731
    logs, clean_logs = torch.empty(4, 4, device=DEV), torch.empty(4, 4, device=DEV)
    clean = call(q, clean_logs)
    for d in (5, 6):
        bad = q.clone()
        bad[:, 1, d] = value
        out = call(bad, logs)
        assert out[[0, 2, 3], 1].isnan().all() and logs[[0, 2, 3], 1].isnan().all()
        assert not out[1].any() and (logs[1] == -math.inf).all()
        assert torch.equal(out[:, [0, 2, 3]], clean[:, [0, 2, 3]]) and torch.equal(logs[:, [0, 2, 3]], clean_logs[:, [0, 2, 3]])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 33, 70, 3000])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_attention_of_an_infinite_key(n, dtype, value):
    """16 bits, the last token's key: a score of -infinity leaves its token out, as if the length were one less, and one of
    +infinity makes the row NaN; also where q holds a number of few bits there (whose lower parts are zeros), or a zero."""
    H, D, d = 1, 64, 9
    k, v = gen_rows((n, H, D), BF16, 1), gen_rows((n, H, D), BF16, 2)
    k[-1, 0, d] = value
    pages, table = written(k, v, 16)
    q = gen_rows((1, 9, D), dtype, 3)
    sign = 1.0 if value > 0 else -1.0
    q[0, :9, d] = torch.tensor([-1.0, -0.3333333, -1.0 - 2.0 ** -9, -2.0 ** -30, 1.0, 0.3333333, 1.0 + 2.0 ** -9, 2.0 ** 30, 0.0]).to(dtype) * sign
    lse = torch.empty(1, 9, device=DEV)
    out = g.gptq_cache_attention(q.to(DEV), pages, table, ints([n]), 16, lse=lse).cpu()
    assert out[0, 4:].isnan().all() and lse[0, 4:].isnan().all()
    fine = torch.nan_to_num(held(k, 16), nan=0.0, posinf=0.0, neginf=0.0)
    ref, ref_lse, bound, lse_bound = attend64(q[:, :4], fine, held(v, 16), table.cpu(), [n - 1], 16, D ** -0.5, 0, dtype, 16)
    assert_near(out[:, :4], ref, bound, dtype)
    if n == 1:
        assert (lse[0, :4] == -math.inf).all() and not out[:, :4].any()
    else:
        assert ((lse.cpu()[:, :4].double() - ref_lse).abs() <= lse_bound + U).all()


# ---------------------------------------------------------------------------------------------------------- far angles

def pi_times(scale):
    """pi * scale as a whole number, off by a few units: 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        total, power, i = 0, scale // n, 1
        while power:
            total += power // i if i % 4 == 1 else -(power // i)
            power //= n * n
            i += 2
        return total
    return 16 * atan(5) - 4 * atan(239)


TURN = Fraction(2 * pi_times(10 ** 60), 10 ** 60)       # of a double's product with a position, up to 2^51: wrong by 2^-140 of a turn


def rotary_exactly(x, positions, freqs, factor):
    """Halves turned by angles reduced in rationals, and the bound without any term of the angle's size."""
    half = len(freqs)
    angle = torch.tensor([[2 * math.pi * float(Fraction(p) * Fraction(f) / TURN % 1) for f in freqs.tolist()] for p in positions.tolist()],
                         dtype=torch.float64)[:, None]
    a, b = x.double()[..., :half], x.double()[..., half:]
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    size = (11 * U * factor * (a.abs() + b.abs())).repeat(1, 1, 2)
    return torch.cat([a * c - b * s, b * c + a * s], -1), size


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotary_angles_are_exact_at_any_position(dtype):
    """Every 32-bit position and frequencies up to 2^20: the fraction of a turn has fp32's last places."""
    positions = torch.tensor([0, 1, -1, 2 ** 17 + 3, 2 ** 24 + 1, 2 ** 30 - 5, 2 ** 31 - 1, -(2 ** 31), -(2 ** 31) + 12345, 1999999973], dtype=torch.int32)
    for freqs, factor in ((g.gptq_rotary_frequencies(64)[0], 1.0), (torch.tensor([2.0 ** 20, -(2.0 ** 20) / 3, 1.0, 0.7, 12345.678, 2.0 * math.pi, 0.0, -1e-9], dtype=torch.float64), 1.25)):
        x = gen_rows((10, 3, 2 * len(freqs)), dtype, 1)
        y = g.gptq_rotary(x.to(DEV), positions.to(DEV), freqs.to(DEV), factor=factor)
        ref, bound = rotary_exactly(x, positions, freqs, factor)
        assert_near(y, ref, bound, dtype)


# -------------------------------------------------------------------------------------------------------- frequencies

def test_frequencies_of_a_ramp_between_its_ends():
    """Pair by pair: as they are up to the last of at least `high` turns, stretched from the first of at most `low` on, and between
    them in even steps from one to the other."""
    for rot, base, factor, original, low, high in ((128, 500000.0, 8.0, 8192.0, 1.0, 32.0), (64, 10000.0, 40.0, 4096.0, 1.0, 32.0),
                                                   (96, 10000.0, 2.5, 1000.0, 2.0, 3.0), (18, 1e6, 4.0, 32768.0, 0.5, 100.0)):
        plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
        turns = [original * f / (2 * math.pi) for f in plain]
        first = max([i for i in range(rot // 2) if turns[i] >= high], default=0)
        last = min([i for i in range(rot // 2) if turns[i] <= low], default=None)
        assert last is not None
        ramp, m = g.gptq_rotary_frequencies(rot, base, "ramp", factor, original, low, high)
        for i, f in enumerate(plain):
            share = min(max((i - first) / (last - first), 0.0), 1.0)
            want = f * (1 - share) + f / factor * share
            assert abs(ramp[i].item() / want - 1) < 1e-13, (rot, i)
        assert abs(m - (0.1 * math.log(factor) + 1.0)) < 1e-7


def test_frequencies_of_a_ramp_that_every_pair_is_behind():
    """Even the fastest pair makes at most `low` turns: all of them are stretched."""
    for original in (1.0, 4.0, 2 * math.pi * 0.999):
        plain, ramp = g.gptq_rotary_frequencies(64)[0], g.gptq_rotary_frequencies(64, 10000.0, "ramp", 4.0, original)[0]
        assert torch.allclose(ramp, plain / 4, rtol=1e-14, atol=0)


def test_frequencies_of_a_base_that_is_none_are_refused():
    for rot, base, factor in ((2, 1e200, 1e60), (64, 1e300, 1e10), (4, 10.0, 1e155)):
        with pytest.raises(g.GptqError):
            g.gptq_rotary_frequencies(rot, base, "base", factor)


# ------------------------------------------------------------------------------------------------------------ the join

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,Hq,H", [(64, 3, 1), (80, 4, 2), (128, 17, 1), (160, 2, 1), (256, 5, 1)])
def test_attention_join_of_few_rows_over_a_long_context(D, Hq, H, dtype):
    """A row's parts joined by several workgroups, each a slice of the stored dimensions (which need not divide a workgroup)."""
    check_attention([20000, 0, 33, 1500], Hq, H, D, 32, 8, dtype, seed=D)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 96, 256])
def test_attention_of_short_requests_under_a_wide_table(D, dtype):
    """Columns for 20000 tokens and lengths of a few: few parts, or none, where many were possible."""
    check_attention([1, 100, 0, 700, 33], 4, 2, D, 16, 8, dtype, seed=D, extra=1250)
    check_attention([300], 4, 1, D, 16, 16, dtype, window=40, seed=D, extra=1250)


# ------------------------------------------------------------------------------------------------- the size of values

@gpu
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** -100])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_attention_of_the_largest_and_smallest_keys_and_values(bits, dtype, size):
    k, v = ((gen_rows((75, 2, 64), F32, i) * size).to(BF16) for i in (1, 2))
    pages, table = written(k, v, bits)
    q = gen_rows((1, 4, 64), dtype, 3)
    out = g.gptq_cache_attention(q.to(DEV), pages, table, ints([75]), bits, 0.125 / size)
    ref, _, bound, _ = attend64(q, held(k, bits), held(v, bits), table.cpu(), [75], 16, 0.125 / size, 0, dtype, bits)
    unit = 2.0 ** -8 if dtype == BF16 else U
    assert ((out.cpu().double() - ref).abs() <= unit * ref.abs() + (1 + unit) * bound).all()


# ------------------------------------------------------------------------------------------------------------ together

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_a_prompt_as_requests_of_one_table_row(bits, dtype):
    """Every token of a prompt attends to what is before it: as a request of its own, all with the same row of the table."""
    n, D = 75, 64
    pages, k, v, table = filled([n], 2, D, 16, bits, 1)
    q, lengths = gen_rows((n, 4, D), dtype, 2), list(range(1, n + 1))
    out = g.gptq_cache_attention(q.to(DEV), pages, table.to(DEV).expand(n, -1), ints(lengths), bits)
    ref, _, bound, _ = attend64(q, k, v, table.expand(n, -1), lengths, 16, D ** -0.5, 0, dtype, bits)
    assert_near(out, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_between_packed_projections(bits, dtype):
    """A layer's step from its input to the output of its last projection; every call against 64 bits of what it was given."""
    from test_serve import close, layer, packed_on, rows_of, slack
    R, K, Hq, H, D, ps = 9, 192, 6, 2, 64, 16
    before = [33, 0, 5, 100, 16, 15, 31, 64, 1]
    codes, scales, W, s = layer(K, (Hq + 2 * H) * D, 4, 64, 1)
    codes_o, scales_o, W_o, s_o = layer(Hq * D, K, 4, 64, 2)
    pages, keys, values, table = filled(before, H, D, ps, bits, 3, stale=0.0, spare=R)
    free = [p for p in range(pages.shape[0]) if not (table == p).any()]
    for r, n in enumerate(before):
        if n % ps == 0:
            table[r, n // ps] = free.pop()
    slots = [int(table[r, n // ps]) * ps + n % ps for r, n in enumerate(before)]
    lengths = [n + 1 for n in before]
    freqs, factor = g.gptq_rotary_frequencies(D, 500000.0, "bands", 8.0)
    x = rows_of(R, K, dtype, 4)

    qkv = g.gptq_adapter_matmul(x.to(DEV), packed_on(codes, 4, DEV)[0], scales[0].to(DEV), 4, groupsize=64)
    close(qkv, x.double() @ W[0], slack(x, s[0], 4, dtype, K), dtype)
    heads = qkv.view(R, Hq + 2 * H, D)
    given = heads.cpu()
    turned = heads[:, :Hq + H]
    g.gptq_rotary(turned, ints(before), freqs.to(DEV), factor=factor, out=turned)
    assert_near(turned, *rotary_exactly(given[:, :Hq + H], torch.tensor(before), freqs, factor), dtype)
    assert torch.equal(heads[:, Hq + H:].cpu(), given[:, Hq + H:])
    g.gptq_cache_write(heads[:, Hq:Hq + H], heads[:, Hq + H:], pages, ints(slots), bits)
    out = g.gptq_cache_attention(heads[:, :Hq], pages, table.to(DEV), ints(lengths), bits)
    for where, rows in ((keys, heads[:, Hq:Hq + H]), (values, heads[:, Hq + H:])):
        where.view(-1, H, D)[slots] = values64(rows.cpu(), bits)
    ref, _, bound, _ = attend64(heads[:, :Hq].cpu(), keys, values, table, lengths, ps, D ** -0.5, 0, dtype, bits)
    assert_near(out, ref, bound, dtype)
    y = g.gptq_adapter_matmul(out.view(R, Hq * D), packed_on(codes_o, 4, DEV)[0], scales_o[0].to(DEV), 4, groupsize=64)
    rows = out.view(R, Hq * D).cpu()
    close(y, rows.double() @ W_o[0], slack(rows, s_o[0], 4, dtype, Hq * D), dtype)
