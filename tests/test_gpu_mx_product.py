"""The product of MX operands kernel by kernel: shapes that the dispatch sends to each of them, with a reduction of
whole stages and not, ragged M and N, against the float64 oracle. u = 2^-24 is half a step of fp32."""
import numpy as np
import pytest
import torch

import bit_routed_expert_amd as moe
from oracle import mx

from gpu_helpers import dev

pytestmark = pytest.mark.gpu

# (M, N, K) by kernel: rows, 16 and 32 and 64 to a workgroup; the reduction split among the waves, 32 x 32 and
# 32 x 64; tiles of 32 x 32, 64 x 64, 64 x 128, 128 x 128 and 256 x 256
SHAPES = [(5, 130, 544), (3, 70, 1024), (20, 530, 160), (100, 77, 224), (20, 70, 512),
          (90, 1990, 1056), (64, 1000, 768), (129, 2000, 1024), (64, 5000, 288),
          (250, 2050, 1056), (250, 2050, 1024), (333, 2050, 2080), (520, 1800, 1024),
          (1500, 1700, 416), (1500, 1700, 512), (2050, 2047, 416), (2050, 2047, 512), (2050, 2047, 1056),
          (4100, 3301, 288), (4097, 3330, 512)]


U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_e4m3_sums_keep_small_terms_beside_large_ones(gpu, M, N, K):
    """Each 8 neighbours of a row of A hold 448 and -448, which the weights (equal for both) cancel, and one element
    of a row is j * 2^-9, j = 1 .. 7: what is left is j * 2^-9 w, of 5 bits, so both types hold it. Partial sums are
    at most 3 * 448 * 6 = 2^13 (at most a pair's halves and their sum at a time), multiples of 2^-10: 23 bits."""
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    ac = np.zeros((M, K), np.uint8)
    swap = rng.integers(0, 2, (M, K // 8), dtype=np.uint8) << 7
    ac[:, 0::8] = 0x7E | swap
    ac[:, 1::8] = 0x7E | (swap ^ 0x80)
    at = rng.integers(0, K // 8, M) * 8 + rng.integers(2, 8, M)
    ac[np.arange(M), at] = rng.integers(1, 8, M) | (rng.integers(0, 2, M) << 7)
    asc = np.full((M, K // 32), 127, np.uint8)
    wc = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    wc[:, 0::4] = (wc[:, 0::4] & 15) * 17                      # the weights of both large elements
    wsc = np.full((N, K // 32), 127, np.uint8)
    want = mx.value(ac, asc, mx.E4M3)[np.arange(M), at][:, None] * mx.value(wc, wsc, mx.E2M1)[:, at].T
    a = [dev(v) for v in (ac, asc, wc, wsc)]
    for out in (moe.OUT_F32, moe.OUT_BF16):
        assert np.array_equal(f64(moe.mx_matmul(*a, a_format=moe.MX_E4M3, out_dtype=out)), want), out


@pytest.mark.parametrize("fmt", [moe.MX_E2M1, moe.MX_E4M3])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bf16_is_the_fp32_result_rounded_once(gpu, M, N, K, fmt):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a = moe.mx_quantize(torch.randn((M, K), generator=g, device="cuda"), fmt)
    w = moe.mx_quantize(torch.randn((N, K), generator=g, device="cuda"), moe.MX_E2M1)
    y = moe.mx_matmul(*a, *w, a_format=fmt, out_dtype=moe.OUT_F32)
    assert torch.equal(moe.mx_matmul(*a, *w, a_format=fmt, out_dtype=moe.OUT_BF16), y.bfloat16())


def operand(rng, R, K, fmt, lo, hi, fields=None):
    """Codes (finite; of e4m3 those of the exponent fields `fields` only) and scale bytes in lo .. hi."""
    if fmt == moe.MX_E2M1:
        codes = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    elif fields is None:
        codes = rng.integers(0, 127, (R, K), dtype=np.uint8) | (rng.integers(0, 2, (R, K), dtype=np.uint8) << 7)
    else:
        codes = ((rng.integers(fields[0], fields[1] + 1, (R, K)) << 3) | rng.integers(0, 8, (R, K)) |
                 (rng.integers(0, 2, (R, K)) << 7)).astype(np.uint8)
    return codes, rng.integers(lo, hi + 1, (R, K // 32), dtype=np.uint8)


@pytest.mark.parametrize("fmt", [moe.MX_E2M1, moe.MX_E4M3])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_values_are_exact_where_fp32_is(gpu, M, N, K, fmt):
    """Scales 1 and 2, e4m3 elements of 1/2 to less than 4: products are multiples of 1/32 of at most 8 * 12 (of 1/4 of
    at most 144 between e2m1), so sums of up to 2080 stay below 2^19 and fp32 holds every partial sum: the exact
    result in any order, and its rounding."""
    rng = np.random.default_rng([M, N, K, fmt])
    ac, asc = operand(rng, M, K, fmt, 127, 128, (6, 8))
    wc, wsc = operand(rng, N, K, moe.MX_E2M1, 127, 128)
    want = mx.value(ac, asc, fmt) @ mx.value(wc, wsc, mx.E2M1).T
    a = [dev(v) for v in (ac, asc, wc, wsc)]
    assert np.array_equal(f64(moe.mx_matmul(*a, a_format=fmt, out_dtype=moe.OUT_F32)), want)
    y16 = moe.mx_matmul(*a, a_format=fmt, out_dtype=moe.OUT_BF16)
    assert torch.equal(y16.cpu(), torch.from_numpy(want).float().bfloat16())


@pytest.mark.parametrize("fmt", [moe.MX_E2M1, moe.MX_E4M3])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_values_under_any_scales(gpu, M, N, K, fmt):
    """Any finite codes, scales over 2^-20 .. 2^20. fp32: the exact terms (two of each element of e4m3) are added with
    at most 2 K roundings, each half a step of a partial sum that is at most the sum of the terms' magnitudes (those
    of both halves of an element too). bf16: that and one rounding."""
    rng = np.random.default_rng([M, N, K, fmt, 1])
    ac, asc = operand(rng, M, K, fmt, 107, 147)
    wc, wsc = operand(rng, N, K, moe.MX_E2M1, 107, 147)
    a, w = mx.value(ac, asc, fmt), mx.value(wc, wsc, mx.E2M1)
    want, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    d = [dev(v) for v in (ac, asc, wc, wsc)]
    err = 2 * K * U * mag
    y = f64(moe.mx_matmul(*d, a_format=fmt, out_dtype=moe.OUT_F32))
    assert np.all(np.abs(y - want) <= err)
    y = f64(moe.mx_matmul(*d, a_format=fmt, out_dtype=moe.OUT_BF16))
    assert np.all(np.abs(y - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


def test_every_kernel_in_two_captured_graphs(gpu):
    """All of the shapes, both formats, in two graphs on their own operands, replayed in turn with eager calls
    between: every replay gives the eager results."""
    g = torch.Generator(device="cuda").manual_seed(11)
    sets = []
    for _ in range(2):
        calls = []
        for M, N, K in SHAPES:
            w = moe.mx_quantize(torch.randn((N, K), generator=g, device="cuda"), moe.MX_E2M1)
            for fmt in (moe.MX_E2M1, moe.MX_E4M3):
                calls.append((*moe.mx_quantize(torch.randn((M, K), generator=g, device="cuda"), fmt), *w, fmt))
        sets.append(calls)

    def run(calls):
        return [moe.mx_matmul(*c[:4], a_format=c[4], out_dtype=moe.OUT_F32 if i % 3 else moe.OUT_BF16) for i, c in enumerate(calls)]

    eager = [run(c) for c in sets]
    graphs, outs = [], []
    for c in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(c))
        graphs.append(graph)
    for rep in range(3):
        for i in (0, 1):
            for o in outs[i]:
                o.zero_()
            graphs[i].replay()
            run(sets[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], eager[i])), (rep, i)
