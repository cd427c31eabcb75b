"""Serving the packed layers: routing, experts' products, the join, adapters.

The products are compared with the definition in 64 bits.  Bounds, elementwise, from the kernels' arithmetic:
  * the output's one rounding: 2^-8 |y| for bf16 (8 significant bits, to nearest), 2^-24 |y| for fp32;
  * fp32 sums: every term of a row's sum meets at most n roundings of 2^-24 on its way: those of its 128-k chunk (at most
    16: four steps of a matrix product that adds 32 terms pairwise in up to four levels), one per chunk and one per wave.
    The terms are x s (c - z), for bf16 rows with the excess of the codes: x s (2^b + c) and x s 1.5 2^b, at most
    3.5 2^b s |x| together;
  * the adapters' inner sums are fp32 too; for bf16 rows they enter the second product with 16 bits (two bf16 parts,
    2^-17 of the term).
The 2-norm of the error is held to 2^-8 (bf16: no element is rounded by more) and, for fp32, to 1e-6: n roundings of
random sign on partial sums no larger than a few times the result.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_09_amd as g

gpu = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def layer(K, N, bits, groupsize, seed, dev="cpu", E=1):
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 1 << bits, (E, K, N), generator=gen, dtype=torch.int64).to(torch.uint8)
    codes[:, :, 0] = 0                                   # a channel at each end of the grid
    codes[:, :, -1] = (1 << bits) - 1
    groups = -(-K // groupsize) if groupsize else 1
    scales = (0.01 + 0.02 * torch.rand(E, groups, N, generator=gen))
    s = scales.double().repeat_interleave(groupsize, 1)[:, :K] if groupsize else scales.double()
    return codes, scales if groupsize else scales[:, 0], s * (codes.double() - 2.0 ** (bits - 1)), s.expand(E, K, N)


def packed_on(codes, bits, dev):
    return torch.stack([g.gptq_pack_codes(c.to(dev), bits) for c in codes])


def rows_of(M, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K, generator=gen) * torch.exp(0.5 * torch.randn(K, generator=gen))).to(dtype)


def slack(x, s, bits, dtype, K):
    """Elementwise bound of the product's error before the output's rounding."""
    n = 16 + -(-K // 128) + 16
    if dtype == F32:
        return n * 2.0 ** -24 * (x.double().abs() @ (s * 2.0 ** (bits - 1)))
    return n * 2.0 ** -24 * (x.double().abs() @ (s * 3.5 * 2.0 ** bits))


def close(y, ref, bound, dtype):
    y = y.double().cpu()
    unit = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    assert y.shape == ref.shape
    bad = (y - ref).abs() > unit * ref.abs() + (1 + unit) * bound + 1e-30
    assert not bad.any(), (int(bad.sum()), (y - ref)[bad][:4], ref[bad][:4])
    if ref.norm() > 0:
        rel = ((y - ref).norm() / ref.norm()).item()
        assert rel <= (2.0 ** -8 if dtype == BF16 else 1e-6), rel


def silu(v):
    return v / (1.0 + torch.exp(-v))


# ---------------------------------------------------------------------------------------------------------- experts

def expert_case(counts, K, N, bits, groupsize, dtype, swiglu=False, gather=False, lead=0, trail=0, seed=0, out=None,
                pad=0):
    E = len(counts)
    codes, scales, W, s = layer(K, N, bits, groupsize, seed, E=E)
    offsets = [lead]
    for c in counts:
        offsets.append(offsets[-1] + c)
    M = offsets[-1] + trail
    gen = torch.Generator().manual_seed(seed + 1)
    T = max(1, M // 2) if gather else M
    X = rows_of(T, K + pad, dtype, seed + 2)[:, :K]
    rows = torch.randint(0, T, (M,), generator=gen, dtype=torch.int32) if gather else None
    src = X[rows.long()] if gather else X
    width = N // 2 if swiglu else N
    ref, bound = torch.zeros(M, width, dtype=torch.float64), torch.zeros(M, width, dtype=torch.float64)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        y, b = src[r].double() @ W[e], slack(src[r], s[e], bits, dtype, K)
        if swiglu:
            gt, up = y[:, :width], y[:, width:]
            # |silu'| <= 1.1; the exponential and the quotient add a few roundings of the value itself
            b = 1.1 * b[:, :width] * up.abs() + silu(gt).abs() * b[:, width:] + 1.1 * b[:, :width] * b[:, width:] \
                + 2.0 ** -20 * (silu(gt) * up).abs()
            y = silu(gt) * up
        ref[r], bound[r] = y, b
    Xd = X.to(DEV) if pad == 0 else rows_of(T, K + pad, dtype, seed + 2).to(DEV)[:, :K]
    y = g.gptq_expert_matmul(Xd, packed_on(codes, bits, DEV), scales.to(DEV),
                             torch.tensor(offsets, dtype=torch.int32, device=DEV), bits,
                             rows=None if rows is None else rows.to(DEV), groupsize=groupsize, swiglu=swiglu, out=out)
    return y, ref, bound


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("groupsize", [0, 32, 64, 128])
def test_expert_matmul_few_rows(bits, groupsize, dtype):
    y, ref, bound = expert_case([1, 0, 17, 5], 32 * bits + 67, 70, bits, groupsize, dtype, seed=bits)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("groupsize", [0, 32, 64, 128])
def test_expert_matmul_many_rows(bits, groupsize, dtype):
    y, ref, bound = expert_case([130, 0, 1, 200], 32 * bits + 67, 301, bits, groupsize, dtype, seed=bits)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", [[3, 1], [40, 60], [150, 140]])
@pytest.mark.parametrize("N", [4, 6, 62, 130, 516])
def test_expert_matmul_gated(N, counts, dtype):
    y, ref, bound = expert_case(counts, 192, N, 4, 64, dtype, swiglu=True, gather=True, seed=N)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("K", [1, 2, 7, 31, 32, 33, 127, 128, 129, 1000])
@pytest.mark.parametrize("counts", [[1], [70]])
@pytest.mark.parametrize("bits", [3, 4])
def test_expert_matmul_lengths(K, counts, bits):
    y, ref, bound = expert_case(counts, K, 9, bits, 32, BF16, seed=K)
    close(y, ref, bound, BF16)


@gpu
@pytest.mark.parametrize("counts,lead,trail", [([0, 0, 0], 2, 3), ([0, 0, 0], 0, 0), ([5, 4, 0], 3, 9),
                                               ([90, 0, 120], 70, 65), ([300], 0, 1)])
def test_expert_matmul_rows_of_no_expert_are_zero(counts, lead, trail):
    M = lead + sum(counts) + trail
    out = torch.full((M, 40), float("nan"), dtype=BF16, device=DEV)
    y, ref, bound = expert_case(counts, 96, 40, 4, 0, BF16, lead=lead, trail=trail, out=out)
    close(y, ref, bound, BF16)
    assert y.data_ptr() == out.data_ptr()
    for z in (y[:lead], y[M - trail:]):
        assert bool((z == 0).all())


@gpu
@pytest.mark.parametrize("counts", [[12, 7], [150, 100]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_expert_matmul_strided_rows_and_output(counts, dtype):
    M = sum(counts)
    wide = torch.full((M, 77), 9.0, dtype=dtype, device=DEV)
    y, ref, bound = expert_case(counts, 200, 50, 4, 64, dtype, pad=3, out=wide[:, 5:55])
    close(y, ref, bound, dtype)
    assert bool((wide[:, :5] == 9).all()) and bool((wide[:, 55:] == 9).all())


@gpu
@pytest.mark.parametrize("M", [6, 200])
def test_expert_matmul_rows_out_of_range_give_zeros(M):
    codes, scales, W, s = layer(64, 32, 4, 0, 3)
    X = rows_of(5, 64, BF16, 1)
    rows = torch.arange(M, dtype=torch.int32) % 5
    rows[1], rows[3], rows[M - 1] = -1, 5, 2 ** 31 - 1
    y = g.gptq_expert_matmul(X.to(DEV), packed_on(codes, 4, DEV), scales.to(DEV),
                             torch.tensor([0, M], dtype=torch.int32, device=DEV), 4, rows=rows.to(DEV))
    ok = (rows >= 0) & (rows < 5)
    src = X[rows.clamp(0, 4).long()].double() * ok[:, None]
    close(y, src @ W[0], slack(src, s[0], 4, BF16, 64), BF16)
    assert bool((y[~ok.to(DEV)] == 0).all())


@gpu
@pytest.mark.parametrize("M", [20, 200])
@pytest.mark.parametrize("offsets", [[-5, 3, 10, 400], [7, 3, 9, 2], [0, 2 ** 31 - 1, -9, 4]])
def test_expert_matmul_keeps_to_its_rows(M, offsets):
    """Offsets outside [0, M] or out of order never reach outside the buffers; rows that are in order are right."""
    codes, scales, W, s = layer(64, 32, 4, 0, 3, E=3)
    X = rows_of(M, 64, BF16, 1)
    guard = torch.full((M + 2, 32), 5.0, dtype=BF16, device=DEV)
    g.gptq_expert_matmul(X.to(DEV), packed_on(codes, 4, DEV), scales.to(DEV),
                         torch.tensor(offsets, dtype=torch.int32, device=DEV), 4, out=guard[1:M + 1])
    torch.cuda.synchronize()
    assert bool((guard[0] == 5).all()) and bool((guard[M + 1] == 5).all())
    if offsets[0] == -5:
        ref = torch.cat([X[:3].double() @ W[0], X[3:10].double() @ W[1], X[10:].double() @ W[2]])
        bound = torch.cat([slack(X[:3], s[0], 4, BF16, 64), slack(X[3:10], s[1], 4, BF16, 64), slack(X[10:], s[2], 4, BF16, 64)])
        close(guard[1:M + 1], ref, bound, BF16)


# More workgroups than CUs: four waves share K.
@gpu
@pytest.mark.parametrize("dtype,bits,groupsize,swiglu", [(BF16, 4, 128, False), (BF16, 3, 64, False), (BF16, 5, 32, True),
                                                         (BF16, 2, 0, True), (F32, 4, 0, False), (F32, 6, 64, True)])
def test_expert_matmul_tens_of_rows_wide(dtype, bits, groupsize, swiglu):
    y, ref, bound = expert_case([40, 65, 0, 33, 1], 709, 5450, bits, groupsize, dtype, swiglu=swiglu, gather=True, seed=9)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("M", [9, 150])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_expert_matmul_non_finite_rows_stay_alone(M, dtype):
    codes, scales, W, s = layer(160, 48, 4, 0, 5)
    X = rows_of(M, 160, dtype, 1)
    Xb = X.clone()
    Xb[2, 7], Xb[5, 100] = float("nan"), float("inf")
    p, sc, off = packed_on(codes, 4, DEV), scales.to(DEV), torch.tensor([0, M], dtype=torch.int32, device=DEV)
    a = g.gptq_expert_matmul(X.to(DEV), p, sc, off, 4)
    b = g.gptq_expert_matmul(Xb.to(DEV), p, sc, off, 4)
    others = [r for r in range(M) if r not in (2, 5)]
    assert torch.equal(a[others], b[others])
    assert bool(torch.isnan(b[2]).all()) and not bool(torch.isfinite(b[5]).any())


@gpu
@pytest.mark.parametrize("counts", [[8, 8], [100, 90]])
def test_expert_matmul_repeats_bit_for_bit_and_in_a_graph(counts):
    codes, scales, W, s = layer(512, 256, 4, 128, 7, E=2)
    M = sum(counts)
    X, p, sc = rows_of(M, 512, BF16, 1).to(DEV), packed_on(codes, 4, DEV), scales.to(DEV)
    off = torch.tensor([0, counts[0], M], dtype=torch.int32, device=DEV)
    ws = torch.empty(g.gptq_matmul_workspace_bytes(BF16, M, 512, 256, experts=2) + 256, dtype=torch.uint8, device=DEV)
    ref = g.gptq_expert_matmul(X, p, sc, off, 4, groupsize=128)
    ws.fill_(0xFF)
    out = torch.empty_like(ref)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        g.gptq_expert_matmul(X, p, sc, off, 4, groupsize=128, out=out, workspace=ws)
    for i in range(3):
        out.fill_(float("nan"))
        X2 = rows_of(M, 512, BF16, 50 + i).to(DEV)
        keep = X.clone()
        X.copy_(X2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g.gptq_expert_matmul(X2, p, sc, off, 4,
                                                     groupsize=128))
        X.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# Enough tiles for the kernel of many rows: 64-row tiles, and 112-row tiles where an expert has several of them.
TILE_CASES = [[300, 0, 500, 1, 250], [600, 1300]]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", TILE_CASES)
@pytest.mark.parametrize("bits,groupsize", [(2, 0), (2, 32), (3, 64), (3, 128), (4, 0), (4, 32), (4, 64), (4, 128), (5, 0),
                                            (5, 32), (6, 64), (6, 128)])
def test_expert_matmul_tiles(bits, groupsize, counts, dtype):
    y, ref, bound = expert_case(counts, 135, 4201, bits, groupsize, dtype, gather=True, lead=3, trail=70, seed=bits)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", TILE_CASES)
@pytest.mark.parametrize("K", [1, 128, 260])
def test_expert_matmul_tiles_gated(K, counts, dtype):
    y, ref, bound = expert_case(counts, K, 4202, 4, 64, dtype, swiglu=True, seed=K)
    close(y, ref, bound, dtype)


@gpu
def test_expert_matmul_tiles_repeat_and_graph():
    codes, scales, W, s = layer(256, 4096, 4, 128, 7, E=2)
    X, p, sc = rows_of(1900, 256, BF16, 1).to(DEV), packed_on(codes, 4, DEV), scales.to(DEV)
    off = torch.tensor([0, 900, 1900], dtype=torch.int32, device=DEV)
    ref = g.gptq_expert_matmul(X, p, sc, off, 4, groupsize=128)
    out, ws = torch.empty_like(ref), torch.empty(g.gptq_matmul_workspace_bytes(BF16, 1900, 256, 4096, experts=2),
                                                 dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gptq_expert_matmul(X, p, sc, off, 4, groupsize=128, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(0x7F)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(ref, g.gptq_expert_matmul(X, p, sc, off, 4, groupsize=128))


# ---------------------------------------------------------------------------------------------------------- adapters

def adapter_case(lengths, ids, K, N, bits, groupsize, rank, dtype, n_adapters=3, lead=0, trail=0, seed=0, slices=False):
    codes, scales, W, s = layer(K, N, bits, groupsize, seed)
    offsets = [lead]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    M = offsets[-1] + trail
    X = rows_of(M, K, dtype, seed + 2)
    gen = torch.Generator().manual_seed(seed + 3)
    A = (torch.randn(n_adapters, rank, K, generator=gen) / math.sqrt(K)).to(BF16)
    B = (torch.randn(n_adapters, N, rank, generator=gen) * 0.3).to(BF16)
    alpha = torch.rand(n_adapters, generator=gen) + 0.5
    ref, bound = X.double() @ W[0], slack(X, s[0], bits, dtype, K)
    n = 16 + -(-K // 256) + 16
    for i, a in enumerate(ids):
        if 0 <= a < n_adapters:
            r = slice(offsets[i], offsets[i + 1])
            x, al = X[r].double(), alpha[a].double()
            ref[r] += al * (x @ A[a].double().t()) @ B[a].double().t()
            inner = x.abs() @ A[a].double().abs().t()
            err = n * 2.0 ** -24 * inner + (2.0 ** -16 if dtype == BF16 else 2.0 ** -23) * (x @ A[a].double().t()).abs()
            bound[r] += al * (err + 2.0 ** -18 * inner * (dtype == BF16)) @ B[a].double().abs().t() \
                + 8 * 2.0 ** -24 * al * inner @ B[a].double().abs().t()
    Ad, Bd = A.to(DEV), B.to(DEV)
    if slices:                                      # adapters inside larger tensors, at odd strides
        big = torch.zeros(n_adapters, rank + 1, K + 3, dtype=BF16, device=DEV)
        big[:, :rank, :K] = Ad
        Ad = big[:, :rank, :K]
        big = torch.zeros(n_adapters, N, rank + 5, dtype=BF16, device=DEV)
        big[:, :, 1:rank + 1] = Bd
        Bd = big[:, :, 1:rank + 1]
    y = g.gptq_adapter_matmul(X.to(DEV), packed_on(codes, bits, DEV)[0], scales[0].to(DEV), bits, groupsize=groupsize,
                              A=Ad, B=Bd, alpha=alpha.to(DEV),
                              requests=torch.tensor(offsets, dtype=torch.int32, device=DEV),
                              adapter=torch.tensor(ids, dtype=torch.int32, device=DEV))
    return y, ref, bound


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rank", [1, 3, 8, 16, 17, 40, 64, 128])
@pytest.mark.parametrize("lengths", [[1], [1, 1, 1, 1, 1], [20, 0, 9, 3], [130, 7, 40, 31]])
def test_adapter_matmul_ranks(lengths, rank, dtype):
    ids = [(2 * i + 1) % 3 if i != 2 else -1 for i in range(len(lengths))]
    y, ref, bound = adapter_case(lengths, ids, 200, 70, 4, 0, rank, dtype, seed=rank)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("bits,groupsize", [(2, 32), (3, 0), (5, 64), (6, 128)])
@pytest.mark.parametrize("lengths", [[2, 3], [100, 90]])
def test_adapter_matmul_widths(lengths, bits, groupsize):
    y, ref, bound = adapter_case(lengths, [0, 1], 300, 131, bits, groupsize, 16, BF16, seed=bits)
    close(y, ref, bound, BF16)


@gpu
@pytest.mark.parametrize("n", [33, 64, 200])
def test_adapter_matmul_many_requests_of_one_token(n):
    ids = [(7 * i) % 11 - 1 for i in range(n)]      # 9 is past the last adapter
    y, ref, bound = adapter_case([1] * n, ids, 256, 96, 4, 128, 16, BF16, n_adapters=9)
    close(y, ref, bound, BF16)


# Prompts (A x in parts of K, one product per run of rows) and single tokens (by distinct adapter) in the many-rows kernel.
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,K,rank", [([900, 0, 130, 500], 2100, 24), ([700, 30, 800], 4099, 70),
                                            ([1] * 400 + [3] * 300, 200, 9), ([40] * 35, 333, 128), ([1300], 1, 3)])
def test_adapter_matmul_tiles(lengths, K, rank, dtype):
    ids = [(5 * i + 1) % 8 - 1 for i in range(len(lengths))]
    y, ref, bound = adapter_case(lengths, ids, K, 4102, 4, 128, rank, dtype, n_adapters=6, lead=2, trail=5, seed=rank)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("K", [1, 5, 7, 8, 9, 31, 33, 511, 513, 4103])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", [[1, 2, 4], [5, 17]])
def test_adapter_matmul_lengths(K, lengths, dtype):
    y, ref, bound = adapter_case(lengths, [0, 2, 1][:len(lengths)], K, 37, 4, 0, 12, dtype, seed=K)
    close(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("lead,trail,lengths", [(3, 4, [2, 5]), (0, 0, [0, 0, 0]), (70, 80, [100, 0, 30])])
def test_adapter_matmul_rows_of_no_request(lead, trail, lengths):
    if lead + trail + sum(lengths) == 0:
        lead = 5
    y, ref, bound = adapter_case(lengths, [1, 0, 2][:len(lengths)], 96, 40, 4, 0, 8, BF16, lead=lead, trail=trail)
    close(y, ref, bound, BF16)


@gpu
@pytest.mark.parametrize("lengths", [[3, 4], [120, 50]])
def test_adapter_matmul_strided_adapters(lengths):
    y, ref, bound = adapter_case(lengths, [2, 0], 100, 60, 4, 0, 13, BF16, slices=True)
    close(y, ref, bound, BF16)


# Infinities and NaN in one request's adapter or rows reach no row of another request, whatever kernel takes them.
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,N", [([1] * 6, 70), ([20, 9, 3, 12], 70), ([500, 3, 90, 700], 3900), ([1] * 700 + [2] * 200, 3900)])
def test_adapter_matmul_non_finite_requests_stay_alone(lengths, N, dtype):
    K, rank, n = 168, 20, 3
    codes, scales, W, s = layer(K, N, 4, 0, 3)
    ids = [i % n for i in range(len(lengths))]
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    M = int(offsets[-1])
    owner = torch.tensor(np.repeat(ids, lengths))
    X, A, B = rows_of(M, K, dtype, 1), rows_of(n * rank, K, BF16, 2).view(n, rank, K), rows_of(n * N, rank, BF16, 3).view(n, N, rank)
    args = (packed_on(codes, 4, DEV)[0], scales[0].to(DEV), 4)

    def run(X, A, B):
        return g.gptq_adapter_matmul(X.to(DEV), *args, A=A.to(DEV), B=B.to(DEV), alpha=torch.ones(n, device=DEV),
                                     requests=torch.tensor(offsets, dtype=torch.int32, device=DEV),
                                     adapter=torch.tensor(ids, dtype=torch.int32, device=DEV)).cpu()

    fine = run(X, A, B)
    bad = B.clone()
    bad[1, ::7, 3], bad[1, 1::7, 19] = math.inf, math.nan
    y = run(X, A, bad)
    assert torch.equal(y[owner != 1], fine[owner != 1])
    mine = y[owner == 1]
    assert not mine[:, ::7].isfinite().any() and mine[:, 1::7].isnan().all() and mine[:, 2::7].isfinite().all()
    bad = A.clone()
    bad[1, 5, 100] = math.nan
    y = run(X, bad, B)
    assert torch.equal(y[owner != 1], fine[owner != 1]) and y[owner == 1].isnan().all()
    bad = X.clone()
    bad[M - 1, 7] = math.nan
    y = run(bad, A, B)
    assert torch.equal(y[:-1], fine[:-1]) and y[-1].isnan().all()


@gpu
@pytest.mark.parametrize("M", [1, 3, 70])
def test_adapter_matmul_without_adapters_is_the_dequantised_product(M):
    K, N = 320, 128
    codes, scales, W, s = layer(K, N, 4, 0, 11)
    p, X = packed_on(codes, 4, DEV)[0], rows_of(M, K, BF16, 2)
    y = g.gptq_adapter_matmul(X.to(DEV), p, scales[0].to(DEV), 4)
    close(y, X.double() @ W[0], slack(X, s[0], 4, BF16, K), BF16)
    back = g.gptq_unpack_codes(p, K, 4, scales=scales[0].to(DEV))["W_hat"].double().cpu()
    assert (back - W[0]).abs().max() <= 2.0 ** -24 * W[0].abs().max()


# ---------------------------------------------------------------------------------------------------- route, combine

def route_reference(x, topk, renorm):
    T, E = x.shape
    w, ex = np.zeros((T, topk)), np.full((T, topk), -1, np.int64)
    for t in range(T):
        if not (x[t] < np.inf).all():
            continue
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:topk]
        if order:
            p = np.exp(x[t] - x[t].max())
            ex[t, :len(order)] = order
            w[t, :len(order)] = p[order] / (p[order].sum() if renorm else p.sum())
    rows, pos, off = np.full(T * topk, -1, np.int64), np.full((T, topk), -1, np.int64), [0]
    for e in range(E):
        t, j = np.nonzero(ex == e)
        pos[t, j] = off[-1] + np.arange(len(t))
        rows[off[-1]:off[-1] + len(t)] = t
        off.append(off[-1] + len(t))
    return w, ex, np.array(off), rows, pos


def check_route(out, x, topk, renorm):
    w, ex, off, rows, pos = route_reference(x, topk, renorm)
    for k, v in (("experts", ex), ("offsets", off), ("rows", rows), ("positions", pos)):
        assert np.array_equal(out[k].cpu().numpy(), v), k
    # exp of an fp32 difference (2 ulp), a sum of at most 1024 positive terms in a tree of ten levels, a quotient
    assert np.abs(out["weights"].cpu().numpy() - w).max() <= 2.0 ** -19


@gpu
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 8, 2), (5, 3, 5), (64, 64, 8), (65, 65, 3), (130, 256, 32),
                                      (1000, 1024, 4), (4097, 128, 8)])
def test_route(T, E, topk, dtype, renorm):
    x = (torch.randn(T, E, generator=torch.Generator().manual_seed(T + E)) * 2).to(dtype)
    x[:, 0] = x[:, E // 2]                           # ties; bf16 has many more
    out = g.gptq_route(x.to(DEV), topk, renorm=renorm)
    check_route(out, x.double().numpy(), topk, renorm)


# Experts around the lanes' shares, choices around the 16 that 16 lanes keep.
@gpu
@pytest.mark.parametrize("T,E,topk", [(63, 16, 16), (70, 17, 2), (200, 33, 16), (200, 33, 17), (130, 100, 1), (129, 127, 5),
                                      (67, 129, 7), (66, 200, 20)])
def test_route_lanes(T, E, topk):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T + E)).mul(4).round().div(4)     # ties
    check_route(g.gptq_route(x.to(DEV), topk), x.double().numpy(), topk, False)


@gpu
def test_route_of_many_blocks_of_tokens():
    T, E = 131200, 1024
    x = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x[:, 512:] -= 1                                  # experts of unlike shares
    out = g.gptq_route(x, 1)
    top = x.max(1, keepdim=True).values
    ex = (x == top).int().argmax(1)                  # the first of equal ones
    order = ex.sort(stable=True).indices
    assert torch.equal(out["experts"][:, 0].long(), ex)
    assert torch.equal(out["rows"].long(), order)
    assert torch.equal(out["offsets"].long()[1:], torch.bincount(ex, minlength=E).cumsum(0))
    assert torch.equal(out["rows"][out["positions"][:, 0].long()].long(), torch.arange(T, device=DEV))


@gpu
@pytest.mark.parametrize("T", [3, 200])
def test_route_masks(T):
    x = torch.randn(T, 40, generator=torch.Generator().manual_seed(1))
    x[:, 3:30] = -math.inf
    x[1] = -math.inf                                 # nothing left
    x[2, :39] = -math.inf                            # one left
    x[0] = torch.finfo(torch.float32).min            # the type's lowest value is a value
    x[0, 5] = -0.0
    x[0, 7] = 0.0                                    # equal to -0.0: the lower index first
    out = g.gptq_route(x.to(DEV), 4, renorm=True)
    check_route(out, x.double().numpy(), 4, True)
    assert out["experts"][0, :2].tolist() == [5, 7]


@gpu
@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_route_reports_non_finite_logits(T, value):
    x = torch.randn(T, 16, generator=torch.Generator().manual_seed(1))
    x[T - 1, 4] = value
    ws = torch.empty(g.gptq_workspace_bytes(g.GPTQ_CALL_ROUTE, 16, 0, T), dtype=torch.uint8, device=DEV)
    out = g.gptq_route(x.to(DEV), 3, workspace=ws)
    assert g.gptq_device_status(ws) == g.GPTQ_ERR_NONFINITE
    check_route(out, x.double().numpy(), 3, False)
    out = g.gptq_route(torch.nan_to_num(x, 0.0, 0.0).to(DEV), 3, workspace=ws)
    assert g.gptq_device_status(ws) == g.GPTQ_OK


@gpu
def test_route_of_no_tokens():
    out = g.gptq_route(torch.empty(0, 8, device=DEV), 2)
    assert out["offsets"].tolist() == [0] * 9 and out["rows"].numel() == 0


@gpu
def test_route_strided_logits():
    x = torch.randn(70, 50, generator=torch.Generator().manual_seed(1))
    out = g.gptq_route(x.to(DEV)[:, 7:40], 3)
    check_route(out, x[:, 7:40].double().numpy(), 3, False)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,topk,N", [(1, 1, 1), (3, 2, 64), (50, 8, 4096), (7, 3, 1001), (2, 32, 2056)])
def test_combine(T, topk, N, dtype):
    gen = torch.Generator().manual_seed(N)
    M = T * topk
    Y = torch.randn(M, N, generator=gen).to(dtype)
    pos = torch.randperm(M, generator=gen).to(torch.int32).view(T, topk)
    w = torch.rand(T, topk, generator=gen)
    gone = torch.rand(T, topk, generator=gen) < 0.3
    Y[pos[gone].long()] = float("nan")               # what is left out is not read
    pos[gone] = torch.where(torch.rand(int(gone.sum()), generator=gen) < 0.5, -1, M).to(torch.int32)
    w[gone] = float("nan")
    out = g.gptq_combine(Y.to(DEV), pos.to(DEV), w.to(DEV)).double().cpu()
    terms = torch.where(gone, 0.0, w).double()[:, :, None] * torch.nan_to_num(Y[pos.clamp(0, M - 1).long()].double())
    terms[gone] = 0.0
    unit = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    ref = terms.sum(1)
    assert ((out - ref).abs() <= unit * ref.abs() + (topk + 1) * 2.0 ** -24 * (1 + unit) * terms.abs().sum(1)).all()


# ------------------------------------------------------------------------------------------------------------ wholes

@gpu
@pytest.mark.parametrize("T", [3, 150])
def test_a_routed_layer_of_quantised_experts(T):
    """quantise -> pack -> route -> experts (gated) -> experts -> combine, against the same codes in 64 bits."""
    E, K, I, topk = 4, 128, 96, 2
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=gen).to(BF16)
    layers = {}
    for name, k, n in (("up", K, 2 * I), ("down", I, K)):
        p, s, ref = [], [], []
        for e in range(E):
            W = torch.randn(k, n, generator=gen) * 0.1
            cal = torch.randn(512, k, generator=gen).to(BF16).to(DEV)
            H = torch.zeros(k, k, device=DEV)
            g.gptq_accumulate_hessian(H, cal)
            dead, _, _ = g.gptq_prepare(H, 0.01)
            q = g.gptq_quantize_layer(W.to(DEV), H, 4, dead=dead)
            p.append(g.gptq_pack_codes(q["codes"], 4))
            s.append(q["scales"])
            ref.append(q["scales"].double().cpu() * (q["codes"].double().cpu() - 8))
        layers[name] = (torch.stack(p), torch.stack(s), ref)
    logits = torch.randn(T, E, generator=gen)
    r = g.gptq_route(logits.to(DEV), topk, renorm=True)
    h = g.gptq_expert_matmul(x.to(DEV), layers["up"][0], layers["up"][1], r["offsets"], 4, rows=r["rows"], swiglu=True)
    y = g.gptq_expert_matmul(h, layers["down"][0], layers["down"][1], r["offsets"], 4)
    out = g.gptq_combine(y, r["positions"], r["weights"]).double().cpu()
    w, ex, _, _, _ = route_reference(logits.double().numpy(), topk, True)
    want = torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for j in range(topk):
            u = x[t].double() @ layers["up"][2][ex[t, j]]
            want[t] += w[t, j] * ((silu(u[:I]) * u[I:]) @ layers["down"][2][ex[t, j]])
    # three bf16 roundings in a row, each at most 2^-8 of a value
    assert ((out - want).norm() / want.norm()).item() <= 3 * 2.0 ** -8


@gpu
@pytest.mark.parametrize("T", [4, 100])
def test_act_order_groups_in_processing_order(T):
    """A layer in act-order with scales re-estimated in the loop: codes[perm] with X[:, perm]."""
    K, N, gs = 256, 64, 64
    gen = torch.Generator().manual_seed(9)
    W, cal = torch.randn(K, N, generator=gen) * 0.1, torch.randn(1024, K, generator=gen).to(BF16).to(DEV)
    H = torch.zeros(K, K, device=DEV)
    g.gptq_accumulate_hessian(H, cal)
    perm = g.gptq_act_order(H)
    dead, _, _ = g.gptq_prepare(H, 0.01)
    gi = torch.empty(K, dtype=torch.int32, device=DEV)
    what = torch.empty(K, N, device=DEV)
    q = g.gptq_quantize_layer(W.to(DEV), H, 4, dead=dead, perm=perm, groupsize=gs, g_idx=gi, W_hat=what)
    X = rows_of(T, K, BF16, 1)
    p = g.gptq_pack_codes(q["codes"][perm.long()].contiguous(), 4)
    y = g.gptq_adapter_matmul(X.to(DEV)[:, perm.long()].contiguous(), p, q["scales"], 4, groupsize=gs)
    s = q["scales"].double().cpu()[gi.cpu().long()]
    ref = X.double() @ (s * (q["codes"].double().cpu() - 8))
    close(y, ref, slack(X, s, 4, BF16, K), BF16)


@gpu
def test_serving_on_another_stream():
    codes, scales, W, s = layer(256, 64, 4, 0, 1)
    p, sc = packed_on(codes, 4, DEV)[0], scales[0].to(DEV)
    X = rows_of(20, 256, BF16, 1)
    st = torch.cuda.Stream()
    Xd = X.to(DEV)
    torch.cuda.synchronize()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = torch.empty(20, 64, dtype=BF16, device=DEV)
    g.gptq_adapter_matmul(Xd, p, sc, 4, out=out, workspace=ws, stream=st)
    st.synchronize()
    close(out, X.double() @ W[0], slack(X, s[0], 4, BF16, 256), BF16)


# ---------------------------------------------------------------------------------------------------------- refusals

FAKE = 0x100000                                      # never dereferenced: the arguments are refused first


def expert_args(**kw):
    a = dict(X=FAKE, dt=1, xr=8, ldx=64, rows=None, M=8, off=FAKE, E=2, packed=FAKE, ldp=32, ps=8 * 32, K=64, N=32,
             bits=4, sc=FAKE, ss=32, gs=0, flags=0, Y=2 * FAKE, ldy=32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return g.load().gptq_expert_matmul(*a.values(), None)


@pytest.mark.parametrize("wrong", [dict(X=None), dict(dt=2), dict(xr=7), dict(ldx=63), dict(M=-1), dict(off=None),
                                   dict(E=0), dict(E=1 << 15), dict(packed=None), dict(ldp=31), dict(ps=255), dict(K=0),
                                   dict(N=3), dict(bits=1), dict(bits=7), dict(sc=None), dict(ss=31), dict(gs=16),
                                   dict(gs=32, ss=63), dict(flags=2), dict(Y=None), dict(Y=FAKE), dict(ldy=31),
                                   dict(flags=1, N=31)])
def test_expert_matmul_refuses(wrong):
    assert expert_args(**wrong) == g.GPTQ_ERR_ARG


def test_expert_matmul_workspace():
    assert expert_args(M=2000, xr=2000, ws=None) == g.GPTQ_ERR_WORKSPACE
    assert expert_args(M=2000, xr=2000, ws=FAKE + 16) == g.GPTQ_ERR_WORKSPACE
    need = g.gptq_matmul_workspace_bytes(BF16, 2000, 64, 32, experts=2)
    assert need > 0 and expert_args(M=2000, xr=2000, wsb=need - 1) == g.GPTQ_ERR_WORKSPACE
    assert expert_args(M=0, ws=None, X=None, Y=None) == g.GPTQ_OK
    assert g.gptq_matmul_workspace_bytes(BF16, 0, 64, 32) == 0
    assert g.gptq_matmul_workspace_bytes(BF16, 8, 64, 32, rank=129) == 0
    assert g.gptq_matmul_workspace_bytes(F32, 4000, 64, 32) > g.gptq_matmul_workspace_bytes(BF16, 4000, 64, 32)


def adapter_args(**kw):
    a = dict(X=FAKE, dt=1, M=8, ldx=64, packed=FAKE, ldp=32, K=64, N=32, bits=4, sc=FAKE, gs=0, A=FAKE, lda=64,
             sa=16 * 64, B=FAKE, ldb=16, sb=32 * 16, alpha=FAKE, n=2, rank=16, req=FAKE, ad=FAKE, nr=2, Y=2 * FAKE,
             ldy=32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return g.load().gptq_adapter_matmul(*a.values(), None)


@pytest.mark.parametrize("wrong", [dict(X=None), dict(dt=7), dict(ldx=63), dict(bits=8), dict(gs=100), dict(N=2),
                                   dict(A=None), dict(B=None), dict(alpha=None), dict(req=None), dict(ad=None),
                                   dict(rank=0), dict(rank=129), dict(lda=63), dict(ldb=15), dict(sa=1000),
                                   dict(sb=511), dict(n=-1), dict(nr=-1), dict(ldy=31), dict(Y=FAKE)])
def test_adapter_matmul_refuses(wrong):
    assert adapter_args(**wrong) == g.GPTQ_ERR_ARG


def test_adapter_matmul_workspace():
    assert adapter_args(ws=None) == g.GPTQ_ERR_WORKSPACE
    need = g.gptq_matmul_workspace_bytes(BF16, 8, 64, 32, rank=16)
    assert adapter_args(wsb=need - 1) == g.GPTQ_ERR_WORKSPACE
    assert adapter_args(M=0, ws=None) == g.GPTQ_OK


@gpu
def test_combine_more_tokens_than_one_launch_takes():
    T, N = (1 << 23) + 5, 4
    Y = torch.arange(16, dtype=F32, device=DEV).view(4, N)
    pos = (torch.arange(T, dtype=torch.int32, device=DEV) % 5 - 1).view(T, 1)
    w = torch.arange(T, dtype=F32, device=DEV).view(T, 1) % 64
    out = g.gptq_combine(Y, pos, w)
    ref = torch.where(pos < 0, torch.zeros((), device=DEV), w * Y[pos.clamp(min=0).long().view(-1)])
    assert torch.equal(out, ref)                     # products of small integers: exact


def test_route_refuses():
    lib = g.load()

    def call(**kw):
        a = dict(x=FAKE, dt=0, T=4, E=8, ld=8, topk=2, flags=0, w=FAKE, e=FAKE, o=FAKE, r=FAKE, p=FAKE, ws=FAKE,
                 wsb=1 << 20)
        a.update(kw)
        return lib.gptq_route(*a.values(), None)

    for wrong in (dict(x=None), dict(dt=3), dict(T=-1), dict(E=0), dict(E=1025), dict(ld=7), dict(topk=0),
                  dict(topk=33), dict(flags=2), dict(w=None), dict(e=None), dict(o=None), dict(r=None), dict(p=None)):
        assert call(**wrong) == g.GPTQ_ERR_ARG, wrong
    assert call(ws=None) == g.GPTQ_ERR_WORKSPACE
    assert call(T=1000, wsb=256) == g.GPTQ_ERR_WORKSPACE


def test_combine_refuses():
    lib = g.load()

    def call(**kw):
        a = dict(Y=FAKE, dt=1, M=8, ldy=32, p=FAKE, w=FAKE, T=4, topk=2, N=32, out=2 * FAKE, ldo=32)
        a.update(kw)
        return lib.gptq_combine(*a.values(), None)

    for wrong in (dict(Y=None), dict(dt=9), dict(M=-1), dict(ldy=31), dict(p=None), dict(w=None), dict(T=-1),
                  dict(topk=0), dict(topk=33), dict(N=0), dict(out=None), dict(out=FAKE), dict(ldo=31)):
        assert call(**wrong) == g.GPTQ_ERR_ARG, wrong
    assert call(T=0) == g.GPTQ_OK


@gpu
def test_binding_refuses():
    X = torch.zeros(4, 64, dtype=BF16, device=DEV)
    p, s = torch.zeros(8, 32, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    ok = g.gptq_adapter_matmul(X, p, s, 4)
    assert ok.shape == (4, 32)
    for bad in (lambda: g.gptq_adapter_matmul(X.half(), p, s, 4), lambda: g.gptq_adapter_matmul(X, p, s, 3),
                lambda: g.gptq_adapter_matmul(X, p.t(), s, 4), lambda: g.gptq_adapter_matmul(X, p, s.double(), 4),
                lambda: g.gptq_adapter_matmul(X, p, s[:31], 4), lambda: g.gptq_adapter_matmul(X.cpu(), p, s, 4),
                lambda: g.gptq_adapter_matmul(X, p, s, 4, groupsize=32),
                lambda: g.gptq_adapter_matmul(X, p, s, 4, A=torch.zeros(1, 8, 64, dtype=BF16, device=DEV)),
                lambda: g.gptq_expert_matmul(X, p, s, off, 4),
                lambda: g.gptq_expert_matmul(X, p[None], s[None], off.long(), 4),
                lambda: g.gptq_expert_matmul(X, p[None], s[None], off[:1], 4),
                lambda: g.gptq_expert_matmul(X, p[None], s[None], off, 4, out=torch.empty(4, 31, dtype=BF16, device=DEV)),
                lambda: g.gptq_route(X[0], 2), lambda: g.gptq_route(X, 0),
                lambda: g.gptq_combine(X, off[None], s[None])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g.GptqError):
        g.gptq_adapter_matmul(X, p, s, 4, out=X[:, :32])
