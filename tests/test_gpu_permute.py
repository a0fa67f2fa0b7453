"""Rows in expert order and back, and the gradients, against the float64 oracle (oracle/mx.py)."""
import numpy as np
import pytest
import torch

import bit_routed_expert_amd as moe
from oracle import mx

from gpu_helpers import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.double().cpu().numpy()


def draw_ids(rng, T, top_k, E, invalid=0.1):
    ids = rng.integers(0, E, (T, top_k))
    if E > 2:
        ids = np.where(rng.random((T, top_k)) < 0.3, E // 2, ids)          # a popular expert, twice in a token too
    bad = rng.random((T, top_k)) < invalid
    return np.where(bad, rng.choice([-1, E, 2**31 - 1, -2**31], (T, top_k)), ids).astype(np.int32)


def check_order(ids, E, offsets, perm, pos):
    wo, wp, wpos = mx.order(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), wo)
    assert np.array_equal(perm.cpu().numpy(), wp)
    assert np.array_equal(pos.cpu().numpy(), wpos)


CASES = [(1, 1, 1), (1, 8, 256), (3, 2, 1), (5, 8, 256), (64, 8, 256), (100, 8, 300), (128, 8, 1024), (129, 8, 64), (33, 32, 7),
         (400, 4, 256), (513, 8, 16), (2000, 8, 256), (3001, 6, 1000), (9000, 2, 2), (300, 32, 50),
         (1001, 16, 30), (6001, 1, 1024)]


@pytest.mark.parametrize("T,top_k,E", CASES)
def test_permute(gpu, T, top_k, E):
    rng = np.random.default_rng(T + top_k + E)
    ids = draw_ids(rng, T, top_k, E)
    x = torch.from_numpy(rng.standard_normal((T, 72))).bfloat16().cuda()
    rows, offsets, perm, pos = moe.moe_w2_permute(x, dev(ids), E)
    check_order(ids, E, offsets, perm, pos)
    o2, p2 = moe.moe_w2_route(dev(ids), E)
    assert torch.equal(o2, offsets) and torch.equal(p2, perm)
    want = x[perm.long() // top_k]
    want[int(offsets[-1]):] = 0
    assert torch.equal(rows, want)


@pytest.mark.parametrize("shape,dtype", [((1,), torch.uint8), ((7,), torch.uint8), ((33,), torch.bfloat16), ((5,), torch.float32),
                                         ((4096,), torch.bfloat16), ((6144,), torch.float32), ((2, 24), torch.float16),
                                         ((4104,), torch.float16), ((96,), torch.float8_e4m3fn), ((1, 3), torch.int64),
                                         ((50001,), torch.uint8)])
@pytest.mark.parametrize("T", [3, 300, 701])
def test_permute_rows_of_any_type(gpu, T, shape, dtype):
    rng = np.random.default_rng(T)
    ids = draw_ids(rng, T, 6, 20)
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    x = torch.from_numpy(rng.integers(0, 256, (T, n), dtype=np.uint8)).view(dtype).reshape(T, *shape).cuda()
    rows, offsets, perm, pos = moe.moe_w2_permute(x, dev(ids), 20)
    check_order(ids, 20, offsets, perm, pos)
    raw = x.view(torch.uint8).reshape(T, n)
    want = raw[perm.long() // 6]
    want[int(offsets[-1]):] = 0
    assert rows.shape == (6 * T, *shape) and torch.equal(rows.view(torch.uint8).reshape(6 * T, n), want)


def test_permute_no_tokens_and_no_valid_ids(gpu):
    x = torch.ones((0, 64), device="cuda")
    rows, offsets, perm, pos = moe.moe_w2_permute(x, torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert rows.shape == (0, 64) and offsets.tolist() == [0] * 10 and pos.shape == (0, 4)
    for T in (2, 700):
        x = torch.ones((T, 64), device="cuda")
        ids = torch.full((T, 4), -5, dtype=torch.int32, device="cuda")
        rows, offsets, perm, pos = moe.moe_w2_permute(x, ids, 9)
        assert not rows.any() and offsets.tolist() == [0] * 10
        assert torch.equal(pos.flatten(), -1 - torch.arange(4 * T, dtype=torch.int32, device="cuda"))
        assert not moe.moe_w2_unpermute(rows + float("nan"), pos, None).any()
        d_rows, d_w = moe.moe_w2_unpermute_backward(x * float("nan"), rows, pos, None)
        assert not d_rows.any() and not d_w.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 8, 33, 264, 2048, 4100, 6144])
@pytest.mark.parametrize("T,top_k", [(1, 1), (1, 8), (2, 32), (37, 6), (300, 8)])
def test_back_and_gradients(gpu, T, top_k, K, dtype):
    check_back_and_gradients(T, top_k, K, dtype)


@pytest.mark.parametrize("K", [5, 264, 2056])
@pytest.mark.parametrize("T,top_k", [(513, 1), (600, 2), (520, 7), (700, 32)])
def test_gradients_of_a_token_together(gpu, T, top_k, K):
    """Batches whose pairs no longer have a workgroup each."""
    check_back_and_gradients(T, top_k, K, torch.bfloat16)


def check_back_and_gradients(T, top_k, K, dtype):
    """y: top_k products and sums (2 top_k roundings of partial sums at most the sum of magnitudes), one to
    the type. d_rows: a product in fp32, one rounding to the type. d_w: K products and sums."""
    rng = np.random.default_rng(T + K)
    ids = draw_ids(rng, T, top_k, 16)
    _, _, pos = mx.order(ids, 16)
    w = rng.standard_normal((T, top_k)).astype(np.float32)
    w[pos < 0] = np.nan                                              # weights of no expert: never used
    rows = torch.from_numpy(rng.standard_normal((T * top_k, K))).to(dtype)
    rows[torch.from_numpy(-1 - pos[pos < 0]).long()] = float("nan")  # nor their rows
    g_rows, g_pos, g_w = rows.cuda(), dev(pos), dev(w)
    for weights, gw in ((w, g_w), (None, None)):
        want, mag = mx.unpermute(f64(rows), pos, weights)
        y = f64(moe.moe_w2_unpermute(g_rows, g_pos, gw))
        assert np.all(np.abs(y - want) <= 2 * top_k * U * mag + HALF[dtype] * (np.abs(want) + 2 * top_k * U * mag) + TINY[dtype])
        if weights is None:
            assert np.array_equal(y, f64(moe.moe_w2_permute_backward(g_rows, g_pos)))
        dy = torch.from_numpy(rng.standard_normal((T, K))).to(dtype)
        d_rows, d_w = moe.moe_w2_unpermute_backward(dy.cuda(), g_rows, g_pos, gw)
        here = pos >= 0
        wt = np.where(here, 1.0 if weights is None else np.where(here, w, 0), 0.0)
        row = np.where(here, pos, -1 - pos)
        want_rows = np.zeros((T * top_k, K))
        want_rows[row.reshape(-1)] = (wt[..., None] * f64(dy)[:, None]).reshape(-1, K)
        assert np.all(np.abs(f64(d_rows) - want_rows) <= (HALF[dtype] + 2 * U) * np.abs(want_rows) + TINY[dtype])
        v = np.where(here[..., None], f64(rows)[row], 0.0) * f64(dy)[:, None]
        assert np.all(np.abs(f64(d_w) - v.sum(-1)) <= K * U * np.abs(v).sum(-1))
        assert not d_w.cpu().numpy()[~here].any()


def test_gradients_against_differences(gpu):
    """<dy, y(rows + e, w) - y> = <d_rows, e> and <dy, y(rows, w + e) - y> = <d_w, e> (y is linear in each), and
    <d_sorted, permute(x + e) - permute(x)> = <permute_backward(d_sorted), e>, on fp32 rows. Values are
    multiples of 1/8 (1/4 for e) of at most 4: every sum of products is exact in fp32, and so are both sides."""
    rng = np.random.default_rng(6)
    T, top_k, K, E = 50, 4, 24, 8
    grid = lambda *s: dev((rng.integers(-32, 33, s) / 8).astype(np.float32))
    ids = dev(draw_ids(rng, T, top_k, E))
    x, w, dy = grid(T, K), grid(T, top_k), grid(T, K)
    rows, _, _, pos = moe.moe_w2_permute(x, ids, E)
    d_rows, d_w = moe.moe_w2_unpermute_backward(dy, rows, pos, w)
    y = moe.moe_w2_unpermute(rows, pos, w)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    e = grid(T * top_k, K)
    assert dot(dy, moe.moe_w2_unpermute(rows + e, pos, w) - y) == dot(d_rows, e)
    e = grid(T, top_k)
    assert dot(dy, moe.moe_w2_unpermute(rows, pos, w + e) - y) == dot(d_w, e)
    e, d_sorted = grid(T, K), grid(T * top_k, K)
    assert dot(d_sorted, moe.moe_w2_permute(x + e, ids, E)[0] - rows) == dot(moe.moe_w2_permute_backward(d_sorted, pos), e)


def test_positions_outside_the_rows_are_ignored(gpu):
    """pos is device data: entries outside the rows contribute nothing and write nothing."""
    T, top_k, K = 4, 2, 40
    rows = torch.ones((8, K), device="cuda")
    pos = torch.tensor([[0, 8], [2**31 - 1, 3], [-9, -2**31], [6, 7]], dtype=torch.int32, device="cuda")
    y = moe.moe_w2_unpermute(rows, pos, None)
    assert y[:, 0].tolist() == [1, 1, 0, 2]
    d_rows = torch.full((8, K), 5.0, device="cuda")
    _, d_w = moe.moe_w2_unpermute_backward(torch.ones((T, K), device="cuda"), rows, pos, None, d_rows=d_rows)
    assert d_rows[:, 0].tolist() == [1, 5, 5, 1, 5, 5, 1, 1]
    assert d_w.tolist() == [[K, 0], [0, K], [0, 0], [K, K]]


def test_unaligned_views(gpu):
    """Row buffers that start off 16 bytes (rows of an odd size cut from a larger tensor)."""
    rng = np.random.default_rng(3)
    T, top_k, K = 60, 2, 64
    ids = dev(draw_ids(rng, T, top_k, 8))
    big = torch.randn(T * K + 1, device="cuda").bfloat16()
    x = big[1:].view(T, K)
    out = torch.empty(T * top_k * K + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T * top_k, K)
    rows, _, _, pos = moe.moe_w2_permute(x, ids, 8, rows=out)
    want, _, _, _ = moe.moe_w2_permute(x.clone(), ids, 8)
    assert torch.equal(rows, want)
    w = torch.rand((T, top_k), device="cuda")
    assert torch.equal(moe.moe_w2_unpermute(rows, pos, w), moe.moe_w2_unpermute(want, pos, w))
    got, want = moe.moe_w2_unpermute_backward(x, rows, pos, w), moe.moe_w2_unpermute_backward(x.clone(), want, pos, w)
    assert torch.equal(got[0], want[0])
    mag = float(x.double().square().sum(1).max())             # rows are copies of dy: each side is within K U mag
    torch.testing.assert_close(got[1], want[1], rtol=0, atol=2 * K * U * mag)


def test_large_rows_equal_those_of_smaller_calls(gpu):
    """Row buffers larger than the last cache go past it; copies, sums and gradients of each token are those of a
    call with the token alone (rows of 8 bits, so that sums are exact in any order)."""
    T, top_k, K, E = 2400, 8, 8200, 16
    x = torch.randint(-8, 9, (T, K), device="cuda").bfloat16()
    ids = torch.randint(-1, E, (T, top_k), device="cuda", dtype=torch.int32)
    w = torch.randint(1, 5, (T, top_k), device="cuda").float()
    rows, offsets, perm, pos = moe.moe_w2_permute(x, ids, E)
    d_rows, d_w = moe.moe_w2_unpermute_backward(x, rows, pos, w)
    y = moe.moe_w2_unpermute(rows, pos, w)
    for t in (0, 1, 1234, T - 1):
        one, _, _, at = moe.moe_w2_permute(x[t:t + 1], ids[t:t + 1], E)
        row = torch.where(pos[t] >= 0, pos[t], -1 - pos[t]).long()
        row1 = torch.where(at[0] >= 0, at[0], -1 - at[0]).long()
        assert torch.equal(rows[row], one[row1])
        assert torch.equal(y[t:t + 1], moe.moe_w2_unpermute(one, at, w[t:t + 1]))
        got, got_w = moe.moe_w2_unpermute_backward(x[t:t + 1], one, at, w[t:t + 1])
        assert torch.equal(d_rows[row], got[row1]) and torch.equal(d_w[t:t + 1], got_w)


@pytest.mark.parametrize("K", [1, 9, 33, 64, 2049, 4100])
@pytest.mark.parametrize("T,top_k", [(40, 3), (600, 5)])
def test_gradient_over_its_rows(gpu, T, top_k, K):
    """d_rows in the memory of rows: the same bits as elsewhere."""
    rng = np.random.default_rng(K)
    ids = dev(draw_ids(rng, T, top_k, 8))
    x, dy = [torch.from_numpy(rng.standard_normal((T, K))).bfloat16().cuda() for _ in range(2)]
    rows, _, _, pos = moe.moe_w2_permute(x, ids, 8)
    w = torch.from_numpy(rng.random((T, top_k))).float().cuda()
    want, want_w = moe.moe_w2_unpermute_backward(dy, rows, pos, w)
    got, got_w = moe.moe_w2_unpermute_backward(dy, rows, pos, w, d_rows=rows)
    assert got.data_ptr() == rows.data_ptr() and torch.equal(got, want) and torch.equal(got_w, want_w)


def test_beyond_32_bit_offsets(gpu):
    """2.3e9 values in the rows: copies, sums and gradients at both ends and between."""
    T, top_k, K, E = 65536, 8, 4352, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, K), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(-1, E, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
    rows, offsets, perm, pos = moe.moe_w2_permute(x, ids, E)
    n = int(offsets[-1])
    for at in (0, n // 2, n - 1000, n):
        got = rows[at:at + 1000]
        want = x[perm[at:at + 1000].long() // top_k]
        assert torch.equal(got, want if at < n else torch.zeros_like(want))
    y = moe.moe_w2_unpermute(rows, pos, None)
    count = (pos >= 0).sum(1, keepdim=True)
    for at in (0, T - 1000):
        want = (x[at:at + 1000].float() * count[at:at + 1000]).bfloat16()
        assert torch.equal(y[at:at + 1000], want)         # k copies of 8 bits: exact in fp32, rounded once
    d_rows, d_w = moe.moe_w2_unpermute_backward(x, rows, pos, None)
    for at in (0, n - 1000, n):
        assert torch.equal(d_rows[at:at + 1000], rows[at:at + 1000])
    sq = x[-100:].double().square().sum(1, keepdim=True) * (pos[-100:] >= 0)
    assert bool(((d_w[-100:].double() - sq).abs() <= K * U * sq).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [513, 517, 519, 1025, 1031, 2050, 4097, 4103])
@pytest.mark.parametrize("T,top_k", [(61, 3), (520, 5)])
def test_gradient_over_its_rows_whose_last_chunk_is_another_waves(gpu, T, top_k, K, dtype):
    """Rows whose last 8 values begin in the last lane of one wave and end in the first of the next, in the same step
    of both or in neighbouring ones: over rows or not, d_w is the product with rows as they were (multiples of 1/8 of
    at most 1, so that sums of K products are exact in any order) and d_rows w dy."""
    rng = np.random.default_rng(K + T)
    ids = dev(draw_ids(rng, T, top_k, 8))
    x, dy = [torch.from_numpy(rng.integers(-8, 9, (T, K)) / 8).to(dtype).cuda() for _ in range(2)]
    rows, _, _, pos = moe.moe_w2_permute(x, ids, 8)
    w = torch.from_numpy(rng.integers(1, 4, (T, top_k)) * 64.0).float().cuda()      # far from what rows hold
    here = pos >= 0
    row = torch.where(here, pos, -1 - pos).long()
    want_w = torch.where(here, (x.double() * dy.double()).sum(1)[:, None], 0.0).float()
    want = torch.zeros_like(rows)
    want[row.flatten()] = (torch.where(here, w, 0.0)[..., None] * dy.float()[:, None]).to(dtype).flatten(0, 1)
    for d_rows in (None, rows):                                                      # rows last: they are lost
        got, got_w = moe.moe_w2_unpermute_backward(dy, rows, pos, w, d_rows=d_rows)
        assert torch.equal(got_w, want_w) and torch.equal(got, want)
