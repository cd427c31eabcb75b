"""Edges of the serving calls: buffers on other streams, views, steering lists out of order, skewed loads, extreme values.

Bounds are those of test_serve.py unless a test says otherwise.
"""
import math

import numpy as np
import pytest
import torch

import post_weight_quantization_09_amd as g
from test_serve import BF16, DEV, F32, close, layer, packed_on, rows_of, slack

gpu = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------------------------------------- streams

def behind_a_busy_stream(call, at_most):
    """`call(stream)` on a stream that is still busy, then blocks of every size up to `at_most` bytes taken from the current
    stream's memory and filled with ones: none of them may be the call's."""
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    out = call(st)
    held = []
    size = 512
    while size <= at_most:
        held += [torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]
        size *= 2
    st.synchronize()
    torch.cuda.synchronize()
    return out


@gpu
@pytest.mark.parametrize("M", [3, 70, 1500])
def test_products_on_another_stream_with_their_own_buffers(M):
    K, N = 256, 4096 if M > 1000 else 64
    codes, scales, W, s = layer(K, N, 4, 0, 1)
    p, sc, X = packed_on(codes, 4, DEV), scales.to(DEV), rows_of(M, K, BF16, 1)
    A = torch.ones(1, 8, K, dtype=BF16, device=DEV)
    B = torch.zeros(1, N, 8, dtype=BF16, device=DEV)
    Xd, off, al, ad = X.to(DEV), ints([0, M]), torch.ones(1, device=DEV), ints([0])
    for call in (lambda st: g.gptq_expert_matmul(Xd, p, sc, off, 4, stream=st),
                 lambda st: g.gptq_adapter_matmul(Xd, p[0], sc[0], 4, A=A, B=B, alpha=al, requests=off, adapter=ad, stream=st)):
        y = behind_a_busy_stream(call, 64 << 20)
        close(y, X.double() @ W[0], slack(X, s[0], 4, BF16, K), BF16)


@gpu
def test_routing_and_joining_on_another_stream_with_their_own_buffers():
    T, E, topk = 700, 16, 2
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    want = g.gptq_route(x, topk)
    got = behind_a_busy_stream(lambda st: g.gptq_route(x, topk, stream=st), 1 << 20)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    Y = rows_of(T * topk, 64, BF16, 2).to(DEV)
    want = g.gptq_combine(Y, got["positions"], got["weights"])
    assert torch.equal(want, behind_a_busy_stream(lambda st: g.gptq_combine(Y, got["positions"], got["weights"], stream=st), 1 << 20))


@gpu
def test_buffers_of_a_call_belong_to_its_stream():
    """What a call allocates comes from its stream's memory: once released it goes to no other stream."""
    x, st = torch.randn(300, 8, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    out = g.gptq_route(x, 2, stream=st)["weights"]
    st.synchronize()
    at, like = out.data_ptr(), out.shape
    del out
    mine = [torch.empty(like, device=DEV) for _ in range(8)]
    assert all(t.data_ptr() != at for t in mine)
    with torch.cuda.stream(st):
        theirs = [torch.empty(like, device=DEV) for _ in range(8)]
    assert any(t.data_ptr() == at for t in theirs)


@gpu
def test_quantising_on_another_stream_with_its_own_buffers():
    K, N = 256, 96
    gen = torch.Generator().manual_seed(4)
    W, X = torch.randn(K, N, generator=gen).to(DEV), torch.randn(2048, K, generator=gen).to(BF16).to(DEV)

    def run(st):
        H = torch.zeros(K, K, device=DEV)
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        g.gptq_accumulate_hessian(H, X, stream=st)
        perm = g.gptq_act_order(H, stream=st)
        dead, _, _ = g.gptq_prepare(H, 0.01, stream=st, sync=False)
        q = g.gptq_quantize_layer(W, H, 4, dead=dead, perm=perm, stream=st, check=False)
        return H, q["codes"], q["scales"], g.gptq_pack_codes(q["codes"], 4, stream=st)

    want = run(None)
    torch.cuda.synchronize()
    for a, b in zip(want, behind_a_busy_stream(run, 64 << 20)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------------------------- views

@gpu
@pytest.mark.parametrize("M", [2, 20])
def test_expanded_adapters_are_refused(M):
    """A view that repeats rows has no leading dimension: read as dense it would run out of its memory."""
    K, N, r = 64, 32, 8
    X, p, s = rows_of(M, K, BF16, 1).to(DEV), torch.zeros(8, N, dtype=torch.int32, device=DEV), torch.ones(N, device=DEV)
    full = dict(A=torch.zeros(1, r, K, dtype=BF16, device=DEV), B=torch.zeros(1, N, r, dtype=BF16, device=DEV),
                alpha=torch.ones(1, device=DEV), requests=ints([0, M]), adapter=ints([0]))
    assert bool((g.gptq_adapter_matmul(X, p, s, 4, **full) == g.gptq_adapter_matmul(X, p, s, 4)).all())
    two = dict(full, alpha=torch.ones(2, device=DEV), A=full["A"].repeat(2, 1, 1), B=full["B"].repeat(2, 1, 1))
    z = lambda *shape: torch.zeros(*shape, dtype=BF16, device=DEV)
    for args in (dict(full, A=z(1, 1, K).expand(1, r, K)), dict(full, B=z(1, 1, r).expand(1, N, r)),
                 dict(full, B=z(1, N, 1).expand(1, N, r)), dict(full, A=z(1, r, 1).expand(1, r, K)),
                 dict(full, A=z(r * K).as_strided((1, r, K), (r * K, K - 1, 1))),
                 dict(two, A=z(1, r, K).expand(2, r, K)), dict(two, B=z(1, N, r).expand(2, N, r)),
                 dict(full, A=z(r, K)), dict(full, A=z(K)), dict(full, A=z(1, K, r).transpose(1, 2))):
        with pytest.raises(ValueError):
            g.gptq_adapter_matmul(X, p, s, 4, **args)


@gpu
@pytest.mark.parametrize("M", [2, 20])
def test_adapters_with_dimensions_of_size_one(M):
    """Any stride is right along a dimension of size one (rank 1, one adapter)."""
    K, N = 72, 32
    codes, scales, W, s = layer(K, N, 4, 0, 2)
    X, gen = rows_of(M, K, BF16, 1), torch.Generator().manual_seed(1)
    a, b = torch.randn(K, generator=gen).to(BF16), torch.randn(N, generator=gen).to(BF16)
    A = torch.empty(5, K, dtype=BF16, device=DEV)[2].copy_(a).as_strided((1, 1, K), (1, 3, 1))
    wide = torch.zeros(N, 7, dtype=BF16, device=DEV)
    wide[:, 3] = b.to(DEV)
    B = wide[:, 3:4].as_strided((1, N, 1), (2, 7, 5), 3)
    y = g.gptq_adapter_matmul(X.to(DEV), packed_on(codes, 4, DEV)[0], scales[0].to(DEV), 4, A=A, B=B,
                              alpha=torch.ones(1, device=DEV), requests=ints([0, M]), adapter=ints([0]))
    inner = X.double() @ a.double()[:, None]
    term = (X.double().abs() @ a.double().abs()[:, None]) * b.double().abs()
    # A x: at most 64 roundings of 2^-24 on a term's way; 2^-16 covers them many times over
    close(y, X.double() @ W[0] + inner * b.double(), slack(X, s[0], 4, BF16, K) + 2.0 ** -16 * term, BF16)


# ---------------------------------------------------------------------------------------------------- steering lists

@gpu
def test_offsets_out_of_order_over_many_experts_keep_to_the_tile_list():
    """8192 of 16384 experts claim all of 2^25 rows: 2^31 row tiles and more, of which the list holds its share."""
    M, K, N, E = 1 << 25, 8, 4, 1 << 14
    X = torch.zeros(M, K, dtype=BF16, device=DEV)
    p, s = torch.zeros(E, 1, N, dtype=torch.int32, device=DEV), torch.ones(E, N, device=DEV)
    off = ints([0]).repeat(E + 1)
    off[1::2] = M
    out = torch.full((M + 2, N), 5.0, dtype=BF16, device=DEV)
    need = g.gptq_matmul_workspace_bytes(BF16, M, K, N, experts=E)
    ws = torch.empty(need + 4096, dtype=torch.uint8, device=DEV)
    ws[need:] = 0xA5
    g.gptq_expert_matmul(X, p, s, off, 4, out=out[1:M + 1], workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((out[0] == 5).all()) and bool((out[M + 1] == 5).all()) and bool((ws[need:] == 0xA5).all())
    assert bool((out[1:M + 1] == 0).all())           # expert 0 owns every row, and its rows of X are zero


# ---------------------------------------------------------------------------------------------------------- numerics

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,N", [([1, 2], 70), ([5, 3], 70), ([30, 40], 70), ([900, 600], 4102), ([1] * 1000 + [2] * 200, 4102)])
def test_inner_products_of_adapters_keep_all_their_bits(lengths, N, dtype):
    """A x = (1 + 2^-9 + 2^-20, 1 + 2^-9) with B = (1, -1): 2^-20, exactly, which 16 bits of A x would lose."""
    K, M = 40, sum(lengths)
    codes = torch.full((K, N), 8, dtype=torch.uint8, device=DEV)     # a layer of zeros
    x = torch.zeros(M, K, device=DEV)
    x[:, 0], x[:, 17], x[:, 39] = 1, 2.0 ** -9, 2.0 ** -20
    A = torch.zeros(1, 2, K, device=DEV)
    A[0, 0], A[0, 1, :20] = 1, 1
    B = torch.tensor([1.0, -1.0], device=DEV).expand(1, N, 2).to(BF16).contiguous()
    y = g.gptq_adapter_matmul(x.to(dtype), g.gptq_pack_codes(codes, 4), torch.ones(N, device=DEV), 4, A=A.to(BF16), B=B,
                              alpha=torch.ones(1, device=DEV), requests=ints(np.concatenate([[0], np.cumsum(lengths)]).tolist()),
                              adapter=ints([0] * len(lengths)))
    assert bool((y == 2.0 ** -20).all()), (y.min().item(), y.max().item())


# The largest values: what the products hold on the way must not overflow where the result does not.
@gpu
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_fp32_rows_with_one_value_up_to_the_largest(M):
    """x = +-max and a little below in one place: a bf16 part rounded from it would be infinite."""
    K, N = 8, 4100 if M > 1000 else 70
    gen = torch.Generator().manual_seed(M)
    codes = torch.randint(7, 10, (K, N), generator=gen).to(torch.uint8)
    X = torch.randn(M, K, generator=gen)
    r = torch.arange(M)
    X[r, r % K] = torch.finfo(F32).max * (1 - (r % 5) * 2.0 ** -10) * ((r % 2) * 2.0 - 1)
    s = torch.full((K, N), 2.0 ** -20, dtype=torch.float64)
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes[None], 4, DEV), torch.full((1, N), 2.0 ** -20, device=DEV), ints([0, M]), 4)
    close(y, X.double() @ (s * (codes.double() - 8)), slack(X, s, 4, F32, K), F32)


@gpu
@pytest.mark.parametrize("lengths", [[1], [30], [900, 700]])
def test_inner_products_of_adapters_up_to_the_largest_value(lengths):
    """A x = max in fp32, where bf16 would round to infinity; B = 2^-20."""
    K, N, M = 8, 4100 if len(lengths) > 1 else 70, sum(lengths)
    x = torch.zeros(M, K, device=DEV)
    x[:, 0] = torch.finfo(F32).max
    A, B = torch.zeros(1, 1, K, dtype=BF16, device=DEV), torch.full((1, N, 1), 2.0 ** -20, dtype=BF16, device=DEV)
    A[0, 0, 0] = 1
    y = g.gptq_adapter_matmul(x, g.gptq_pack_codes(torch.full((K, N), 8, dtype=torch.uint8, device=DEV), 4),
                              torch.ones(N, device=DEV), 4, A=A, B=B, alpha=torch.ones(1, device=DEV),
                              requests=ints([0] + np.cumsum(lengths).tolist()), adapter=ints([0] * len(lengths)))
    want = torch.finfo(F32).max * 2.0 ** -20
    # three products of parts, added up in fp32
    assert bool(((y.double() - want).abs() <= 3 * 2.0 ** -24 * want).all())


@gpu
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_fp32_rows_up_to_the_largest_value(M):
    """x = +-max: a bf16 part rounded from it would be infinite.  Weights 2^-20 (c - 8) with c - 8 in {-1, 0, 1}."""
    K, N = 8, 4100 if M > 1000 else 70
    gen = torch.Generator().manual_seed(M)
    codes = torch.randint(7, 10, (K, N), generator=gen).to(torch.uint8)
    sign = torch.randint(0, 2, (M, K), generator=gen) * 2.0 - 1
    X = sign * torch.finfo(F32).max
    X[:, 1:4] *= 0.999                               # on both sides of the last value that bf16 rounds down
    X[:, 4:] *= 2.0 ** -30
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes[None], 4, DEV), torch.full((1, N), 2.0 ** -20, device=DEV), ints([0, M]), 4)
    W = 2.0 ** -20 * (codes.double() - 8)
    close(y, X.double() @ W, slack(X, torch.full((K, N), 2.0 ** -20, dtype=torch.float64), 4, F32, K), F32)


@gpu
@pytest.mark.parametrize("bits,groupsize", [(2, 0), (3, 32), (4, 128), (5, 64), (6, 0)])
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_bf16_rows_up_to_the_largest_value(M, bits, groupsize):
    """Every x is +-max, and a third of the rows have one sign alone: 128 codes at the top of the grid, unscaled, pass it."""
    K, N = 300, 4100 if M > 1000 else 70
    codes, scales, W, s = layer(K, N, bits, groupsize, M)
    X = torch.randint(0, 2, (M, K), generator=torch.Generator().manual_seed(M)) * 2.0 - 1
    X[::3] = 1
    X = (X * torch.finfo(BF16).max).to(BF16)
    W, s, scales = W * 2.0 ** -12, s * 2.0 ** -12, scales * 2.0 ** -12
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes, bits, DEV), scales.to(DEV), ints([0, M]), bits, groupsize=groupsize)
    close(y, X.double() @ W[0], slack(X, s[0], bits, BF16, K), BF16)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_small_values(M, dtype):
    """Rows of about 2^-80 and a scale of 2^-6: no product falls below the normal numbers."""
    K, N = 300, 4100 if M > 1000 else 70
    codes, scales, W, s = layer(K, N, 4, 64, M)
    X = (rows_of(M, K, F32, 1) * 2.0 ** -80).to(dtype)
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes, 4, DEV), scales.to(DEV), ints([0, M]), 4, groupsize=64)
    y, ref = y.double().cpu() * 2.0 ** 80, X.double() @ W[0] * 2.0 ** 80
    close(y, ref, slack(X, s[0], 4, dtype, K) * 2.0 ** 80, dtype)


# -------------------------------------------------------------------------------------------------- many tokens routed

def route_on_device(x, topk):
    """The definition by sorts on the GPU: experts, offsets, rows, positions."""
    T, E = x.shape
    v, ex = torch.sort(x, dim=1, descending=True, stable=True)
    v, ex = v[:, :topk], ex[:, :topk]
    ex = torch.where(v > -math.inf, ex, torch.full_like(ex, E))
    flat = ex.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)
    n = int(counts[:E].sum())
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=x.device)
    rows = torch.where(torch.arange(order.numel(), device=x.device) < n, order // topk, -1)
    return (torch.where(ex < E, ex, -1), torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)]), rows,
            torch.where(flat < E, pos, -1).view(T, topk))


# Around 1024 blocks of 64 tokens (or blocks^2 experts = 2^27) and groups of 64 blocks, where the placing of the rows changes.
@gpu
@pytest.mark.parametrize("T,E,topk", [(65536, 128, 2), (65536, 129, 2), (65537, 5, 2), (69632, 64, 3), (69633, 64, 3),
                                      (32768, 9, 2), (32769, 9, 2), (36864, 130, 1), (36865, 64, 8), (262144 + 63, 33, 3),
                                      (300001, 1, 1), (40000, 1023, 4), (1 << 20, 8, 2)])
def test_route_of_many_tokens(T, E, topk):
    x = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(T))
    x[T // 3:T // 2, :E // 2 + 1] = -math.inf        # a stretch of tokens with few experts, or none
    need = g.gptq_workspace_bytes(g.GPTQ_CALL_ROUTE, E, 0, T)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    out = g.gptq_route(x, topk, workspace=ws[:need])
    ex, off, rows, pos = route_on_device(x, min(topk, E))
    assert torch.equal(out["experts"].long(), ex) and torch.equal(out["offsets"].long(), off)
    assert torch.equal(out["rows"].long(), rows) and torch.equal(out["positions"].long(), pos)
    assert bool((ws[need:] == 0xA5).all())


@gpu
def test_route_takes_time_in_proportion_to_its_tokens():
    """Four times the tokens: four times the time, not sixteen."""
    def us(T):
        x = torch.randn(T, 64, device=DEV)
        ws = torch.empty(g.gptq_workspace_bytes(g.GPTQ_CALL_ROUTE, 64, 0, T), dtype=torch.uint8, device=DEV)
        best = math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.gptq_route(x, 2, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert us(1 << 21) < 8 * us(1 << 19)


# ---------------------------------------------------------------------------------- long requests beside single tokens

def mixed(lengths, ids, K, N, rank, dtype, seed=0):
    """A call's tensors, and its result and bound in 64 bits, for adapters that repeat among many requests."""
    M, n = sum(lengths), 5
    codes, scales, W, s = layer(K, N, 4, 128, seed)
    X, gen = rows_of(M, K, dtype, seed + 1), torch.Generator().manual_seed(seed + 2)
    A = (torch.randn(n, rank, K, generator=gen) / math.sqrt(K)).to(BF16)
    B = (torch.randn(n, N, rank, generator=gen) * 0.3).to(BF16)
    alpha = torch.rand(n, generator=gen) + 0.5
    owner = torch.tensor(np.repeat(ids, lengths))
    ref, bound = X.double() @ W[0], slack(X, s[0], 4, dtype, K)
    for a in range(n):
        r = owner == a
        x, al = X[r].double(), alpha[a].double()
        inner = x.abs() @ A[a].double().abs().t()
        # A x: an fp32 sum of at most (16 + K / 256 + 16) roundings on a term's way; times alpha, times B: 8 more
        ref[r] += al * (x @ A[a].double().t()) @ B[a].double().t()
        bound[r] += (16 + -(-K // 256) + 16 + 8) * 2.0 ** -24 * al * inner @ B[a].double().abs().t()
    call = dict(X=X.to(DEV), packed=packed_on(codes, 4, DEV)[0], scales=scales[0].to(DEV), bits=4, groupsize=128, A=A.to(DEV),
                B=B.to(DEV), alpha=alpha.to(DEV), requests=ints([0] + np.cumsum(lengths).tolist()), adapter=ints(ids))
    return call, ref, bound


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,N", [([1] * 40 + [700] + [1] * 60, 70), ([700] + [1] * 200, 70), ([1] * 200 + [65, 300], 70),
                                       ([1] * 600 + [1500] + [0] * 700 + [1] * 30, 70), ([5] * 300, 70),
                                       ([1] * 255 + [3841], 4100), ([2500] + [1] * 30 + [0] * 5, 4100),
                                       ([1] * 1100 + [2000, 33, 1000] + [2] * 5, 4100)])
def test_adapter_matmul_long_requests_beside_single_tokens(lengths, N, dtype):
    ids = [(3 * i) % 6 - 1 for i in range(len(lengths))]
    ids[int(np.argmax(lengths))] = 2
    call, ref, bound = mixed(lengths, ids, 333, N, 20, dtype)
    close(g.gptq_adapter_matmul(**call), ref, bound, dtype)


@gpu
def test_a_long_request_beside_single_tokens_is_shared_out():
    """The same rows with one adapter, as 256 requests of 16 and as one of 3841 beside 255 of one: alike in time."""
    K, M, n = 4096, 4096, 256
    X, p = torch.randn(M, K, device=DEV).to(BF16), torch.zeros(K // 8, 64, dtype=torch.int32, device=DEV)
    A, B = torch.zeros(1, 16, K, dtype=BF16, device=DEV), torch.zeros(1, 64, 16, dtype=BF16, device=DEV)
    s, al, ad = torch.ones(64, device=DEV), torch.ones(1, device=DEV), ints([0] * n)
    ws = torch.empty(g.gptq_matmul_workspace_bytes(BF16, M, K, 64, rank=16), dtype=torch.uint8, device=DEV)

    def us(lengths):
        req = ints([0] + np.cumsum(lengths).tolist())
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                g.gptq_adapter_matmul(X, p, s, 4, A=A, B=B, alpha=al, requests=req, adapter=ad, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert us([1] * 255 + [3841]) < 3 * us([16] * 256)


# ------------------------------------------------------------------------------------------------------------- limits

@gpu
def test_more_requests_than_one_launch_has_threads_for():
    """2^23 requests and more, nearly all of them empty."""
    K, N, n = 64, 32, (1 << 23) + 70
    codes, scales, W, s = layer(K, N, 4, 0, 2)
    X = rows_of(40, K, BF16, 1)
    A = torch.ones(2, 3, K, dtype=BF16, device=DEV)
    B = torch.ones(2, N, 3, dtype=BF16, device=DEV)
    req = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    req[1 << 22:] = 5
    req[n - 3:] = 39
    ad = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    ad[(1 << 22) - 1], ad[n - 4] = 0, 1              # rows 0 .. 4 and 5 .. 38
    y = g.gptq_adapter_matmul(X.to(DEV), packed_on(codes, 4, DEV)[0], scales[0].to(DEV), 4, A=A, B=B,
                              alpha=torch.tensor([1.0, -2.0], device=DEV), requests=req, adapter=ad)
    ref, x = X.double() @ W[0], X.double()
    ref[:5] += 3 * x[:5].sum(1, keepdim=True)
    ref[5:39] -= 6 * x[5:39].sum(1, keepdim=True)
    close(y, ref, slack(X, s[0], 4, BF16, K) + 40 * 2.0 ** -24 * 6 * x.abs().sum(1, keepdim=True), BF16)


def test_sizes_past_a_launch_are_refused():
    """The tile launch's threads: an argument error, not one of the launch."""
    from test_serve import expert_args
    assert expert_args(M=1 << 30, xr=8, rows=0x100000, K=64, N=32) == g.GPTQ_ERR_ARG
    assert g.gptq_matmul_workspace_bytes(BF16, 1 << 30, 64, 32, experts=2) == 0
    assert expert_args(M=(1 << 30) - 64 * 5, xr=8, rows=0x100000, wsb=0) == g.GPTQ_ERR_ARG
    assert expert_args(M=(1 << 30) - 64 * 6, xr=8, rows=0x100000, wsb=0) == g.GPTQ_ERR_WORKSPACE
    assert expert_args(M=128, xr=128, E=1 << 14, N=1 << 22, ldp=1 << 22, ps=1 << 25, ss=1 << 22, ldy=1 << 22, wsb=0) != g.GPTQ_ERR_ARG


@gpu
def test_gradients_are_refused():
    X = torch.zeros(4, 64, dtype=BF16, device=DEV)
    p, s, off = torch.zeros(8, 32, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV), ints([0, 4])
    A, B = torch.zeros(1, 8, 64, dtype=BF16, device=DEV), torch.zeros(1, 32, 8, dtype=BF16, device=DEV)
    x, w, pos = torch.randn(4, 8, device=DEV), torch.ones(4, 1, device=DEV), ints([[0], [1], [2], [3]])
    al, ad = torch.ones(1, device=DEV), ints([0])
    for t, call in ((X, lambda t: g.gptq_adapter_matmul(t, p, s, 4)), (s, lambda t: g.gptq_adapter_matmul(X, p, t, 4)),
                    (A, lambda t: g.gptq_adapter_matmul(X, p, s, 4, A=t, B=B, alpha=al, requests=off, adapter=ad)),
                    (B, lambda t: g.gptq_adapter_matmul(X, p, s, 4, A=A, B=t, alpha=al, requests=off, adapter=ad)),
                    (al, lambda t: g.gptq_adapter_matmul(X, p, s, 4, A=A, B=B, alpha=t, requests=off, adapter=ad)),
                    (X, lambda t: g.gptq_expert_matmul(t, p[None], s[None], off, 4)), (x, lambda t: g.gptq_route(t, 1)),
                    (X, lambda t: g.gptq_combine(t, pos, w)), (w, lambda t: g.gptq_combine(X, pos, t))):
        call(t)
        leaf = t.clone().requires_grad_()
        with pytest.raises(ValueError):
            call(leaf)
        with pytest.raises(ValueError):
            call(leaf * 1)
        call(leaf.detach())
        with torch.no_grad():
            call(leaf)


# ------------------------------------------------------------------------- adapters: buffers, repeats, graphs, bad lists

# few rows; tens of rows; prompts (one product per run of rows); short requests (by distinct adapter, through Z)
PATHS = [([1, 2, 0, 3], 70), ([20, 0, 9, 13], 70), ([900, 5, 600], 4100), ([1] * 700 + [2] * 200, 4100)]


def ids_of(lengths):
    return [(3 * i + 1) % 6 - 1 for i in range(len(lengths))]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,N", PATHS)
@pytest.mark.parametrize("rank", [3, 70])
def test_adapter_matmul_on_a_workspace_of_the_stated_size(lengths, N, rank, dtype):
    """Filled with NaN, nothing past its end is touched, and two calls give the same bits."""
    call, ref, bound = mixed(lengths, ids_of(lengths), 333, N, rank, dtype)
    need = g.gptq_matmul_workspace_bytes(dtype, sum(lengths), 333, N, rank=rank)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    y = g.gptq_adapter_matmul(**call, workspace=ws[:need])
    close(y, ref, bound, dtype)
    assert bool((ws[need:] == 0xFF).all())
    ws[:need] = 0x7F
    assert torch.equal(y, g.gptq_adapter_matmul(**call, workspace=ws[:need]))
    assert torch.equal(y, g.gptq_adapter_matmul(**call))


@gpu
@pytest.mark.parametrize("lengths,N", PATHS)
def test_adapter_matmul_in_a_graph(lengths, N):
    call, ref, bound = mixed(lengths, ids_of(lengths), 333, N, 20, BF16)
    ws = torch.empty(g.gptq_matmul_workspace_bytes(BF16, sum(lengths), 333, N, rank=20), dtype=torch.uint8, device=DEV)
    want = g.gptq_adapter_matmul(**call)
    close(want, ref, bound, BF16)
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gptq_adapter_matmul(**call, out=out, workspace=ws)
    first = call["X"].clone()
    for i in range(3):
        call["X"].copy_(first if i == 1 else first * (i + 2))
        call["adapter"].copy_(call["adapter"].flip(0))           # other adapters, other lengths, the same graph
        call["requests"].copy_(call["requests"][-1] - call["requests"].flip(0))
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g.gptq_adapter_matmul(**call))


@gpu
@pytest.mark.parametrize("lengths,N", PATHS)
@pytest.mark.parametrize("how", ["outside", "swapped", "wild"])
def test_adapter_matmul_keeps_to_its_rows(lengths, N, how):
    """Requests outside [0, M] or out of order, adapters that do not exist: nothing outside the buffers, lists in order right."""
    n, M = len(lengths), sum(lengths)
    call, ref, bound = mixed(lengths, ids_of(lengths), 96, N, 20, BF16)
    plain = g.gptq_adapter_matmul(**{k: call[k] for k in ("X", "packed", "scales", "bits", "groupsize")})
    full = g.gptq_adapter_matmul(**call)
    req = call["requests"].clone()
    gen = torch.Generator().manual_seed(n)
    if how == "outside":
        req[0], req[n] = -7, M + 1000
    elif how == "swapped":
        req = req.flip(0)
    else:
        req = torch.randint(-2 ** 31, 2 ** 31 - 1, (n + 1,), generator=gen).to(torch.int32).to(DEV)
        call["adapter"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), generator=gen).to(torch.int32).to(DEV)
    call["requests"] = req.contiguous()
    need = g.gptq_matmul_workspace_bytes(BF16, M, 96, N, rank=20)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    guard = torch.full((M + 2, N), 5.0, dtype=BF16, device=DEV)
    g.gptq_adapter_matmul(**call, out=guard[1:M + 1], workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((guard[0] == 5).all()) and bool((guard[M + 1] == 5).all()) and bool((ws[need:] == 0xFF).all())
    if how == "outside":
        assert torch.equal(guard[1:M + 1], full)
    if how == "wild":                                # no adapter exists: the plain product
        assert torch.equal(guard[1:M + 1], plain)


# ---------------------------------------------------------------------------------- skewed experts, far-away addresses

# By the average these are few rows (16), tens of rows (64) and many; one expert has nearly all of them.
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,M,N", [(128, 2048, 70), (128, 2049, 70), (64, 4096, 130), (8, 1200, 4100)])
def test_expert_matmul_skewed(E, M, N, dtype):
    K, bits = 96, 4
    counts = [0] * E
    counts[E // 3], counts[E // 2], counts[E - 1] = M - M // 8 - 3, M // 8, 3
    codes, scales, W, s = layer(K, N, bits, 32, 5, E=E)
    X, off = rows_of(M, K, dtype, 1), np.concatenate([[0], np.cumsum(counts)])
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes, bits, DEV), scales.to(DEV), ints(off.tolist()), bits, groupsize=32)
    ref, bound = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for e in np.nonzero(counts)[0]:
        r = slice(off[e], off[e + 1])
        ref[r], bound[r] = X[r].double() @ W[e], slack(X[r], s[e], bits, dtype, K)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("bits,K,groupsize", [(4, 256, 64), (6, 32, 0), (3, 70, 32), (5, 160, 128)])
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_words_at_the_end_of_the_largest_layer(M, bits, K, groupsize):
    """2^30 words of one layer, 4 GiB: the channels are a view whose rows are as far apart as that allows."""
    N = 4100 if M > 1000 else 70
    nw = (K * bits + 31) // 32
    ldp = (1 << 30) // nw
    whole = torch.empty(nw * ldp, dtype=torch.int32, device=DEV)
    packed = whole.view(nw, ldp)[:, ldp - N:]
    codes, scales, W, s = layer(K, N, bits, groupsize, M)
    packed.copy_(packed_on(codes, bits, DEV)[0])
    X = rows_of(M, K, BF16, 1)
    y = g.gptq_adapter_matmul(X.to(DEV), packed, scales[0].to(DEV), bits, groupsize=groupsize)
    close(y, X.double() @ W[0], slack(X, s[0], bits, BF16, K), BF16)


@gpu
@pytest.mark.parametrize("M", [3, 40, 1500])
def test_experts_past_four_gigabytes(M):
    """The words, rows and results of the last experts lie beyond 32-bit offsets."""
    E, K, N = 9, 64, 4100 if M > 1000 else 70
    codes, scales, W, s = layer(K, N, 4, 0, M, E=E)
    stride = 1 << 28                                 # words: 1 GiB an expert
    packed = torch.empty((E - 1) * stride + 8 * N, dtype=torch.int32, device=DEV).as_strided((E, 8, N), (stride, N, 1))
    packed.copy_(packed_on(codes, 4, DEV))
    ld = -(-(1 << 32) // M) + 64
    X, wide = rows_of(M, K, BF16, 1), torch.empty(M * ld, dtype=BF16, device=DEV).view(M, ld)
    wide[:, 7:7 + K] = X.to(DEV)
    out = torch.empty(M * ld, dtype=BF16, device=DEV).view(M, ld)[:, 1:1 + N] if ld > N else None
    off = [0] * 7 + [M // 3, M // 2, M]              # experts 6, 7 and 8
    y = g.gptq_expert_matmul(wide[:, 7:7 + K], packed, scales.to(DEV), ints(off), 4, out=out)
    ref = torch.cat([X[off[e]:off[e + 1]].double() @ W[e] for e in (6, 7, 8)])
    bound = torch.cat([slack(X[off[e]:off[e + 1]], s[e], 4, BF16, K) for e in (6, 7, 8)])
    close(y, ref, bound, BF16)


@gpu
def test_workspaces_that_are_no_memory_of_their_own_are_refused():
    """A view that repeats one byte, or skips some, has fewer bytes than its elements say."""
    K = 128
    X, p, s = torch.zeros(70, K, dtype=BF16, device=DEV), torch.zeros(K // 8, 32, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV)
    H, off = torch.eye(K, device=DEV), ints([0, 70])
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(1 << 24), torch.empty(1 << 25, dtype=torch.uint8, device=DEV)[::2],
               torch.empty(1 << 24, dtype=torch.uint8)):
        for call in (lambda: g.gptq_adapter_matmul(X, p, s, 4, workspace=ws), lambda: g.gptq_route(X, 2, workspace=ws),
                     lambda: g.gptq_expert_matmul(X, p[None], s[None], off, 4, workspace=ws),
                     lambda: g.gptq_prepare(H, 0.01, workspace=ws), lambda: g.gptq_accumulate_hessian(H, X, workspace=ws)):
            with pytest.raises(ValueError):
                call()
    assert torch.equal(H, torch.eye(K, device=DEV))


@gpu
def test_calls_on_tensors_of_a_gpu_that_is_not_the_current_one(monkeypatch):
    """Every call makes its tensors' GPU the current one first; another current GPU is only made believe here."""
    from post_weight_quantization_09_amd import _binding
    now, entered = [7], []

    class Stream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)
            now.append(self.stream.device.index)

        def __exit__(self, *a):
            now.pop()

    K = 128
    X, x = torch.randn(70, K, device=DEV).to(BF16), torch.randn(70, 8, device=DEV)
    p, s, off = torch.zeros(K // 8, 32, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV), ints([0, 70])
    pos, w = ints([[i] for i in range(70)]), torch.ones(70, 1, device=DEV)
    W, codes = torch.randn(K, 32, device=DEV), torch.zeros(K, 32, dtype=torch.uint8, device=DEV)
    H = torch.zeros(K, K, device=DEV)
    g.gptq_accumulate_hessian(H, X)
    U = H.clone()
    dead, _, _ = g.gptq_prepare(U, 0.01)
    ws = torch.zeros(g.gptq_workspace_bytes(g.GPTQ_CALL_ROUTE, 8, 0, 70), dtype=torch.uint8, device=DEV)
    calls = [lambda: g.gptq_route(x, 2, workspace=ws)["rows"], lambda: g.gptq_device_status(ws), lambda: g.gptq_combine(X, pos, w),
             lambda: g.gptq_adapter_matmul(X, p, s, 4), lambda: g.gptq_expert_matmul(X, p[None], s[None], off, 4),
             lambda: g.gptq_quantize_layer(W, U, 4, dead=dead)["codes"], lambda: g.gptq_pack_codes(codes, 4),
             lambda: g.gptq_unpack_codes(p, K, 4)["codes"], lambda: g.gptq_hadamard_rotate(X),
             lambda: g.gptq_act_order(H.clone()), lambda: g.gptq_prepare(H.clone(), 0.01)[0],
             lambda: g.gptq_accumulate_hessian(H=H.clone(), X=X)]
    want = [c() for c in calls]
    monkeypatch.setattr(_binding, "_device_now", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    for call, before in zip(calls, want):
        entered.clear()
        after = call()
        assert [st.device for st in entered] == [torch.device(DEV)] and now == [7]
        assert torch.equal(before, after) if torch.is_tensor(before) else before == after
