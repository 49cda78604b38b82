"""GPU parity of the four-bit token operators (HIP through the C ABI) against
the float64 oracle on the same inputs, at the sizes, strides, places and pages
where they can go wrong, and a run of them together.

Tolerances, from the arithmetic (a rounding is off by at most half a step:
2^-8 relative in bfloat16, 2^-24 in float32; a float32 sum is counted at a whole
step, 2^-23, an addition, as the matrix pipes' order and rounding inside one
instruction are their own):
 quantise, append, read   none: codes, scales and their values are equal.
 linear     weights are exact in bfloat16. A sum of K products goes through K/32
            instructions, at most 32 additions inside one and at most 16 joins:
            (K/32 + 48) 2^-23 sum |x w|; the activations have slopes up to 1.13
            and are evaluated to 2^-20 |z|; residual and output round once each.
 attention  probabilities round to bfloat16, p_i (1 + e_i) with |e_i| <= 2^-8, in
            the product and in the sum: out is off by sum_i p_i e_i (v_i - out),
            at most 2^-8 (weighted mean of |v| + |out|); scores (D <= 128: 4
            instructions, 32 additions, two roundings of the scaled score) to
            38 2^-23 sum |q k|, which exp passes on as a relative error, twice
            (sum and product); 1e-5 for the float32 sums over the keys and the
            joins. Probabilities below 2^-126 of the largest are 0 in float32:
            less than 2^17 keys times 2^8 times that, 2^-101.
Outputs round to their type at the end.
"""
import numpy as np
import pytest
import torch

from oracle import fp4 as of, tokens as ot

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def gkd():
    import prompt_conditioned_keypoint_amd as m
    m.load()
    assert torch.cuda.is_available()
    return m


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(gen, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def arr(t):
    return None if t is None else t.cpu().numpy()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rounded(y, tol, dtype):
    return tol + STEP[dtype] * (np.abs(y) + tol)


def same(a, b):
    """Equal values, NaN with NaN."""
    return torch.equal(torch.nan_to_num(a.float(), nan=12345.0), torch.nan_to_num(b.float(), nan=12345.0))


# ---------------------------------------------------------------- quantise
def hard_values(dtype):
    """Ties, border values, far exponents, zeros and values that are not finite."""
    r = np.random.default_rng(1)
    rows = []
    for e in (-140, -126, -125, -124, -60, -2, 0, 1, 30, 122, 124):
        mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        near = np.concatenate([mids, mids * (1 + 2.0 ** -7), mids * (1 - 2.0 ** -8), [6.0, 6.9, 0.0, -0.0]])
        near = np.concatenate([near, -near])[:31]
        for top in (4.0, 6.0, 6.96875, 7.0, 3.5):
            rows.append(np.concatenate([near, [top]]) * 2.0 ** e)
        rows.append(r.standard_normal(32) * 2.0 ** e)
    rows.append(np.zeros(32))
    for bad in (np.inf, -np.inf, np.nan):
        rows.append(np.where(np.arange(32) == 17, bad, 1.0))
    rows.append(np.where(np.arange(32) == 3, 3.0e38, 1e30))
    x = torch.from_numpy(np.array(rows)).to(torch.float32).cuda()
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise_hard_values(gkd, dtype):
    x = hard_values(dtype)
    codes, scales = gkd.quantize_fp4(x)
    wc, ws = of.quantise(np64(x))
    assert np.array_equal(arr(scales), ws)
    assert np.array_equal(arr(codes), wc)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (7, 5, 64), (33, 4096), (1000, 1056), (0, 64)])
def test_quantise_shapes(gkd, dtype, shape):
    x = randn(rng(3), *shape, dtype=dtype)
    codes, scales = gkd.quantize_fp4(x)
    assert codes.shape == shape[:-1] + (shape[-1] // 2,) and scales.shape == shape[:-1] + (shape[-1] // 32,)
    sub = (slice(None, 40),) + (slice(None),) * (len(shape) - 1)
    wc, ws = of.quantise(np64(x)[sub])
    assert np.array_equal(arr(codes)[sub], wc) and np.array_equal(arr(scales)[sub], ws)


def test_quantise_strided_rows_and_given_outputs(gkd):
    x = randn(rng(4), 6, 9, 128)[:, :, 32:96]
    codes, scales = torch.full((6, 9, 32), 7, dtype=U8, device="cuda"), torch.empty(6, 9, 2, dtype=U8, device="cuda")
    got = gkd.quantize_fp4(x, codes, scales)
    assert got[0] is codes and got[1] is scales
    want = gkd.quantize_fp4(x.contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    for bad in (lambda: gkd.quantize_fp4(x[..., :40]), lambda: gkd.quantize_fp4(x, codes[:5]),
                lambda: gkd.quantize_fp4(x.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gkd.quantize_fp4(x.half())


def test_read_gives_every_code_of_every_scale(gkd):
    """All 256 scale bytes with all 16 codes, exactly (rounded and past its range as
    bfloat16 has it)."""
    codes = torch.zeros(16, 2, 1, 32, 32, dtype=U8, device="cuda")
    codes[:, :, :, :, :8] = torch.arange(8, device="cuda", dtype=U8) * 2 * 17 + 16
    codes[:, :, :, :, 16:24] = torch.arange(8, device="cuda", dtype=U8) * 2 * 17 + 16
    scales = torch.arange(256, device="cuda", dtype=torch.int32).reshape(8, 1, 1, 32, 1).repeat(2, 2, 1, 1, 2).to(U8)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    k, v = gkd.cache_read(codes, scales, table, 256)
    want, _ = of.read(arr(codes), arr(scales), arr(table), 256)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want.astype(np.float32)).to(BF)
    assert same(k.cpu(), want) and same(v.cpu(), want)


# ------------------------------------------------------------------ append
def new_cache(pages, Hk, page, D, fill=None, seed=0):
    if fill is None:
        g = rng(seed + 100)
        return (torch.randint(0, 256, (pages, 2, Hk, page, D // 2), generator=g, device="cuda").to(U8),
                torch.randint(120, 129, (pages, 2, Hk, page, D // 32), generator=g, device="cuda").to(U8))
    return (torch.full((pages, 2, Hk, page, D // 2), fill, dtype=U8, device="cuda"),
            torch.full((pages, 2, Hk, page, D // 32), fill, dtype=U8, device="cuda"))


def check_append(gkd, B, T, Hk, D, page, L, table=None, start=None, count=None, dtype=BF, seed=0, split=False):
    print(f"[append] B={B} T={T} Hk={Hk} D={D} page={page} L={L} {start} {count} {dtype}", flush=True)
    g = rng(seed)
    pages = B * L + 2
    codes, scales = new_cache(pages, Hk, page, D, seed=seed)
    if table is None:
        table = torch.randperm(pages, generator=g, device="cuda")[:B * L].reshape(B, L).to(torch.int32)
    if split:  # one projection's rows: keys, then values, with something beside them
        rows = randn(g, B, T, 2 * Hk * D + 32, dtype=dtype)
        k, v = rows[..., :Hk * D].unflatten(2, (Hk, D)), rows[..., Hk * D:2 * Hk * D].unflatten(2, (Hk, D))
    else:
        k, v = randn(g, B, T, Hk, D, dtype=dtype), randn(g, B, T, Hk, D, dtype=dtype)
    wc, ws = of.append(np64(k), np64(v), arr(codes), arr(scales), arr(table), arr(start), arr(count))
    gkd.cache_append(k, v, codes, scales, table, start=start, count=count)
    assert np.array_equal(arr(codes), wc) and np.array_equal(arr(scales), ws)
    # and back, into places with something in them
    ko, vo = torch.full((2, B, T, Hk, D), 7.0, dtype=BF, device="cuda")
    gkd.cache_read(codes, scales, table, T, start=start, count=count, k_out=ko, v_out=vo)
    kw, vw = of.read(wc, ws, arr(table), T, arr(start), arr(count))
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        assert np.array_equal(np64(ko)[b, :n], kw[b, :n]) and np.array_equal(np64(vo)[b, :n], vw[b, :n])
        assert bool((ko[b, n:] == 7).all()) and bool((vo[b, n:] == 7).all())
    kn, vn = gkd.cache_read(codes, scales, table, T, start=start, count=count)
    assert np.array_equal(np64(kn), kw) and np.array_equal(np64(vn), vw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hk,page,L", [(1, 1, 1, 32, 1), (3, 1, 5, 64, 2), (2, 45, 3, 32, 2), (5, 7, 2, 96, 1),
                                           (1, 130, 8, 256, 1)])
def test_append_and_read(gkd, B, T, Hk, D, page, L, dtype):
    check_append(gkd, B, T, Hk, D, page, L, dtype=dtype, seed=T)


@pytest.mark.parametrize("D", [64, 128])
def test_append_ragged_places(gkd, D):
    check_append(gkd, 4, 20, 2, D, 32, 3, start=ints(0, 25, 70, 31), count=ints(20, 1, 0, 13), split=True)
    # places before the first and behind the last; counts past T and below 0
    check_append(gkd, 4, 20, 2, D, 32, 3, start=ints(-7, 90, 96, 2**31 - 5), count=ints(20, 20, 20, 50), dtype=F32)
    check_append(gkd, 2, 20, 3, D, 64, 1, start=ints(-2**31, 50), count=ints(-1, 99), split=True)
    # columns without a page, or with one that the cache does not have
    check_append(gkd, 2, 90, 2, D, 32, 3, table=torch.tensor([[1, -1, 6], [8, 2, 2**31 - 1]], dtype=torch.int32,
                                                              device="cuda"), start=ints(3, 0))


def test_append_takes_hard_values(gkd):
    x = hard_values(F32)
    n = len(x) // 2 * 2
    k = x[:n].reshape(1, n // 2, 1, 64)
    codes, scales = new_cache(4, 1, 32, 64, 0)
    table = ints(2, 0, 3)[None]
    gkd.cache_append(k, -k, codes, scales, table)
    wc, ws = of.append(np64(k), -np64(k), np.zeros_like(arr(codes)), np.zeros_like(arr(scales)), arr(table))
    assert np.array_equal(arr(codes), wc) and np.array_equal(arr(scales), ws)


def test_append_and_read_without_room(gkd):
    k = randn(rng(0), 2, 3, 2, 64)
    codes, scales = new_cache(0, 2, 32, 64, 0)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    gkd.cache_append(k, k, codes, scales, table)               # no pages: dropped
    a, b = gkd.cache_read(codes, scales, table, 3)
    assert a.shape == (2, 3, 2, 64) and not a.any() and not b.any()
    codes, scales = new_cache(2, 2, 32, 64, 5)
    gkd.cache_append(k, k, codes, scales, table[:, :0])        # no columns: dropped
    assert bool((codes == 5).all()) and not gkd.cache_read(codes, scales, table[:, :0], 3)[0].any()
    gkd.cache_append(k[:, :0], k[:, :0], codes, scales, table)
    assert bool((codes == 5).all())
    assert gkd.cache_read(codes, scales, table[:0], 3)[0].shape == (0, 3, 2, 64)


# ------------------------------------------------------------------ linear
def linear_tol(y, size, K, dtype, residual):
    tol = 1.13 * (K / 32 + 48) * 2.0 ** -23 * size + 2.0 ** -20 * size
    if residual is not None:
        tol = tol + 2.0 ** -23 * (np.abs(y) + np.abs(residual))
    return rounded(y, tol, dtype)


def check_linear(gkd, M, K, N, act="none", bias=True, residual=True, out=BF, seed=0):
    print(f"[linear_fp4] M={M} K={K} N={N} {act} bias={bias} residual={residual} {out}", flush=True)
    g = rng(seed)
    x = randn(g, M, K)
    codes, scales = gkd.quantize_fp4(randn(g, N, K, scale=K ** -0.5, dtype=F32))
    b = randn(g, N) if bias else None
    r = randn(g, M, N, dtype=out) if residual else None
    y = gkd.linear_fp4(x, codes, scales, bias=b, residual=r, act=act, out_dtype=out)
    assert y.dtype == out and y.shape == (M, N)
    want, size = ot.linear(np64(x), of.values(arr(codes), arr(scales)), np64(b), np64(r), act)
    err = np.abs(np64(y) - want)
    assert np.all(err <= linear_tol(want, size, K, out, np64(r))), err.max()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "quick_gelu", "silu"])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear_activations(gkd, act, out):
    check_linear(gkd, 70, 192, 136, act, out=out)
    check_linear(gkd, 3, 192, 136, act, out=out, residual=False)


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 31, 33, 48, 64, 65, 96, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("K,N", [(32, 16), (288, 257), (1024, 130), (96, 1), (2080, 300)])
def test_linear_ragged_sizes(gkd, M, K, N):
    check_linear(gkd, M, K, N, seed=M)
    check_linear(gkd, M, K, N, "silu", bias=False, residual=False, out=F32, seed=M)


@pytest.mark.parametrize("M,K,N", [(1, 16384, 64), (13, 16384, 4095), (37, 1024, 4096), (128, 8192, 1030),
                                   (1, 1024, 16385), (80, 4096, 1024), (1100, 512, 1000), (3000, 96, 70), (9, 65536, 33)])
def test_linear_large(gkd, M, K, N):
    check_linear(gkd, M, K, N, "gelu", seed=N)


# rows and weights for which work goes by tiles of 32, 64 and 128 rows, with K split and
# not, with rows of scales that are whole words and not
TILES = [(20, 2048, 9000), (31, 4128, 9001), (17, 8224, 4100), (63, 544, 16390), (50, 4096, 4100), (50, 4128, 8200),
         (128, 8192, 1030), (130, 8224, 2050), (1500, 544, 2050), (2000, 1024, 1030)]


@pytest.mark.parametrize("M,K,N", TILES)
def test_linear_tiles(gkd, M, K, N):
    check_linear(gkd, M, K, N, "silu", seed=N)
    check_linear(gkd, M, K, N, bias=False, residual=False, out=F32, seed=M)


# and a K of one step of the tiles
@pytest.mark.parametrize("M,K,N", [(20, 256, 16390), (32, 96, 16385), (64, 160, 8190), (50, 256, 16385), (1024, 32, 1025),
                                   (400, 96, 2050), (257, 256, 4099), (1100, 224, 1030)])
def test_linear_tiles_of_one_step(gkd, M, K, N):
    check_linear(gkd, M, K, N, "silu", seed=N)
    check_linear(gkd, M, K, N, bias=False, residual=False, out=F32, seed=M)


@pytest.mark.parametrize("M,K,N", [(31, 4128, 9001), (50, 4128, 8200), (130, 8224, 2050), (63, 544, 16390)])
def test_linear_tiles_stay_within_their_arrays(gkd, M, K, N):
    g = rng(11)
    x = randn(g, M, K)
    codes, scales = gkd.quantize_fp4(randn(g, N, K, scale=1 / 32, dtype=F32))
    want = gkd.linear_fp4(x, codes, scales)
    buf = torch.full((M + 2, K + 24), float("nan"), dtype=BF, device="cuda")
    buf[1:-1, 8:8 + K] = x
    cb = torch.full((N + 2, K // 2), 0x77, dtype=U8, device="cuda")
    sb = torch.full((N + 32, K // 32), 255, dtype=U8, device="cuda")
    cb[1:-1], sb[16:-16] = codes, scales
    for out in (BF, F32):
        y = torch.full((M + 2, N + 3), 7.0, dtype=out, device="cuda")
        got = gkd.linear_fp4(buf[1:-1, 8:8 + K], cb[1:-1], sb[16:-16], out=y[1:-1, 1:-2])
        assert torch.equal(got.to(BF), want)
        y[1:-1, 1:-2] = 7
        assert bool((y == 7).all())
    # a group of NaN reaches its column alone, a NaN in a row its row
    sb[16 + 7, K // 32 - 1] = 255
    x[2, K - 1] = float("nan")
    nan = torch.isnan(gkd.linear_fp4(x, cb[1:-1], sb[16:-16]))
    assert bool(nan[:, 7].all()) and bool(nan[2].all()) and int(nan.sum()) == M + N - 1


def test_linear_reads_nothing_beside_its_rows(gkd):
    g = rng(5)
    for M in (3, 40, 130):
        K, N = 160, 70
        x = randn(g, M, K)
        codes, scales = gkd.quantize_fp4(randn(g, N, K))
        want = gkd.linear_fp4(x, codes, scales)
        buf = torch.full((M + 2, K + 24), float("nan"), dtype=BF, device="cuda")
        buf[1:-1, 8:8 + K] = x
        # the weights lie in a larger array whose other groups are NaN
        cb = torch.full((N + 2, K // 2), 0x77, dtype=U8, device="cuda")
        sb = torch.full((N + 32, K // 32), 255, dtype=U8, device="cuda")
        cb[1:-1], sb[16:-16] = codes, scales
        out = torch.full((M + 2, N + 3), 7.0, dtype=BF, device="cuda")
        got = gkd.linear_fp4(buf[1:-1, 8:8 + K], cb[1:-1], sb[16:-16], out=out[1:-1, 1:-2])
        assert torch.equal(got, want)
        out[1:-1, 1:-2] = 7
        assert bool((out == 7).all())


def test_linear_groups_of_nan_and_rows_of_nan_stay_where_they_are(gkd):
    g = rng(6)
    for M in (5, 60, 150):
        x = randn(g, M, 256)
        codes, scales = gkd.quantize_fp4(randn(g, 50, 256))
        want = gkd.linear_fp4(x, codes, scales)
        scales[7, 3] = 255
        x[2, 9] = float("nan")
        y = gkd.linear_fp4(x, codes, scales)
        nan = torch.isnan(y)
        assert bool(nan[:, 7].all()) and bool(nan[2].all())
        rest = torch.ones(M, 50, dtype=torch.bool, device="cuda")
        rest[2], rest[:, 7] = False, False
        assert not nan[rest].any() and torch.equal(y[rest], want[rest])


def test_linear_strided_rows_and_in_place_residual(gkd):
    g = rng(7)
    M, K, N = 45, 64, 36
    xs = randn(g, 3, 15, 2 * K)
    x = xs[:, :, K:]
    codes, scales = gkd.quantize_fp4(randn(g, N, K))
    for out in (BF, F32):
        buf = torch.full((3, 15, N + 5), 7.0, dtype=out, device="cuda")
        y = buf[:, :, :N]
        y.copy_(randn(g, 3, 15, N))
        r = np64(y).reshape(M, N)
        got = gkd.linear_fp4(x, codes, scales, residual=y, out=y)
        assert got.data_ptr() == buf.data_ptr()
        want, size = ot.linear(np64(x).reshape(M, K), of.values(arr(codes), arr(scales)), None, r)
        assert np.all(np.abs(np64(y).reshape(M, N) - want) <= linear_tol(want, size, K, out, r))
        assert bool((buf[:, :, N:] == 7).all())


def test_linear_equals_that_of_bf16_weights(gkd):
    """The weights are exact in bfloat16: gkd_linear of their values differs by the
    order of its sums alone."""
    g = rng(8)
    x = randn(g, 37, 1024)
    codes, scales = gkd.quantize_fp4(randn(g, 512, 1024, scale=1 / 32))
    w = torch.from_numpy(of.values(arr(codes), arr(scales))).to(BF).cuda()
    a, b = gkd.linear_fp4(x, codes, scales, out_dtype=F32), gkd.linear(x, w, out_dtype=F32)
    size = np.abs(np64(x)) @ np.abs(np64(w)).T
    assert np.all(np.abs(np64(a) - np64(b)) <= 2 * (1024 / 32 + 48) * 2.0 ** -23 * size)


def test_linear_weights_past_32_bit_offsets(gkd):
    """600 rows of 2^22 - 32 values: codes past 2^30 bytes, values past 2^31."""
    K, N = (1 << 22) - 32, 1100
    codes = torch.zeros(N, K // 2, dtype=U8, device="cuda")
    scales = torch.full((N, K // 32), 127, dtype=U8, device="cuda")
    codes[:, 0], codes[:, -1] = 0x2, (torch.arange(N, device="cuda") % 7).to(U8) * 16
    x = torch.zeros(2, K, dtype=BF, device="cuda")
    x[0, 0], x[1, -1] = 3, 1
    y = gkd.linear_fp4(x, codes, scales, out_dtype=F32)
    sizes = torch.tensor(of.SIZES[:7], dtype=F32, device="cuda")
    assert bool((y[0] == 3).all()) and torch.equal(y[1], sizes[torch.arange(N, device="cuda") % 7])


@pytest.mark.parametrize("M", [2, 20])
def test_linear_codes_past_32_bits(gkd, M):
    """2100 rows of 2^22 - 32 weights: codes past 2^32 bytes, for the few rows' kernel and for
    tiles with K split."""
    K, N = (1 << 22) - 32, 2100
    assert N * (K // 2) > 1 << 32 and (gkd.linear_fp4_workspace_size(M, N, K) > 0) == (M > 16)
    codes = torch.zeros(N, K // 2, dtype=U8, device="cuda")
    scales = torch.full((N, K // 32), 127, dtype=U8, device="cuda")
    n, m = torch.arange(N, device="cuda"), torch.arange(M, device="cuda")
    codes[:, 0], codes[:, -1] = (n % 5).to(U8), (n % 7).to(U8) * 16
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[:, 0], x[:, -1] = m % 4, 1 + m % 3
    y = gkd.linear_fp4(x, codes, scales, out_dtype=F32)
    sizes = torch.tensor(of.SIZES, dtype=F32, device="cuda")
    assert torch.equal(y, (m % 4)[:, None] * sizes[n % 5] + (1 + m % 3)[:, None] * sizes[n % 7])


@pytest.mark.parametrize("K,N,split", [(1024, 130, False), (8192, 1030, True), (544, 16390, False)])
def test_linear_rows_past_32_bits(gkd, K, N, split):
    """Rows of x and of the output that lie 2^22 - 8 and 2^22 elements apart: the last ones past
    2^31 elements; the few rows' kernel, tiles with K split and without."""
    M, g = 600, rng(N)
    assert (gkd.linear_fp4_workspace_size(M, N, K) > 0) == split
    x = randn(g, M, K)
    codes, scales = gkd.quantize_fp4(randn(g, N, K, scale=K ** -0.5, dtype=F32))
    wide = torch.empty(M * (1 << 22), dtype=BF, device="cuda").as_strided((M, K), ((1 << 22) - 8, 1))
    wide.copy_(x)
    far = torch.empty(M * (1 << 22), dtype=F32, device="cuda").as_strided((M, N + 1), (1 << 22, 1))
    far.fill_(7)
    got = gkd.linear_fp4(wide, codes, scales, act="silu", out=far[:, :N])
    assert torch.equal(got, gkd.linear_fp4(x, codes, scales, act="silu", out_dtype=F32))
    assert bool((far[:, N] == 7).all())


def test_linear_empty_and_refusals(gkd):
    codes, scales = gkd.quantize_fp4(torch.zeros(8, 64, dtype=BF, device="cuda"))
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    assert gkd.linear_fp4(x[:0], codes, scales).shape == (0, 8)
    assert gkd.linear_fp4(x, codes[:0], scales[:0]).shape == (4, 0)
    for bad in (lambda: gkd.linear_fp4(x[:, :32], codes, scales), lambda: gkd.linear_fp4(x, codes, scales[:4]),
                lambda: gkd.linear_fp4(x, codes, scales[:, :1]), lambda: gkd.linear_fp4(x, codes[:, ::2], scales),
                lambda: gkd.linear_fp4(x, codes, scales, act="tanh"),
                lambda: gkd.linear_fp4(x, codes, scales, out=torch.empty(4, 9, dtype=BF, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        gkd.linear_fp4(x.float(), codes, scales)
    with pytest.raises(gkd.GkdError) as e:
        gkd.linear_fp4(x[:1].expand(4, 64), codes, scales)
    assert e.value.status == 2
    with pytest.raises(gkd.GkdError) as e:  # rows that start off 16-byte places
        gkd.linear_fp4(torch.zeros(4, 68, dtype=BF, device="cuda")[:, :64], codes, scales)
    assert e.value.status == 7


# --------------------------------------------------------------- attention
def attention_tol(out, mean_abs, worst):
    rel = 2 * 38 * 2.0 ** -23 * worst + 1e-5
    return rounded(out, 2.0 ** -8 * (mean_abs + np.abs(out)) + rel * mean_abs + 2.0 ** -101, BF)


def attn_inputs(B, Tq, Hq, Hk, D, page, L, seed=0, pages=None, spread=1.0):
    g = rng(seed)
    pages = B * L + 3 if pages is None else pages
    codes, scales = gkd_quantised(g, pages, Hk, page, D, spread)
    table = torch.randperm(pages, generator=g, device="cuda")[:B * L].reshape(B, L).to(torch.int32)
    return randn(g, B, Tq, Hq, D), codes, scales, table


def gkd_quantised(g, pages, Hk, page, D, spread=1.0):
    import prompt_conditioned_keypoint_amd as gkd
    v = torch.randn(pages, 2, Hk, page, D, generator=g, device="cuda")
    v = v * torch.exp2(torch.randint(-2, 3, (pages, 2, Hk, page, D // 32, 1), generator=g, device="cuda") *
                       spread).expand(-1, -1, -1, -1, -1, 32).flatten(-2)
    return gkd.quantize_fp4(v)


def check_attention(gkd, q, codes, scales, table, length=None, q_len=None, causal=False, **kw):
    B, Tq, Hq, D = q.shape
    print(f"[cache_attention] q={tuple(q.shape)} cache={tuple(codes.shape)} table={tuple(table.shape)} "
          f"length={None if length is None else length.tolist()} q_len={None if q_len is None else q_len.tolist()} "
          f"causal={causal}", flush=True)
    got = gkd.cache_attention(q, codes, scales, table, length=length, q_len=q_len, causal=causal, **kw)
    want, mean_abs, worst = of.attention(np64(q), arr(codes), arr(scales), arr(table), arr(length), arr(q_len), causal,
                                         kw.get("scale"))
    err = np.abs(np64(got) - want)
    assert np.all(err <= attention_tol(want, mean_abs, worst)), (err.max(), np.unravel_index(err.argmax(), err.shape))
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Tq,Hq,Hk,page,L", [
    (1, 1, 1, 1, 32, 1), (3, 1, 8, 2, 64, 3), (2, 1, 16, 16, 32, 5), (2, 5, 4, 4, 64, 2), (1, 17, 3, 3, 96, 2),
    (2, 3, 14, 2, 32, 4), (1, 40, 2, 1, 64, 3), (1, 33, 8, 1, 128, 2), (1, 1, 20, 1, 256, 2), (2, 65, 1, 1, 32, 3)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_shapes(gkd, B, Tq, Hq, Hk, D, page, L, causal):
    q, codes, scales, table = attn_inputs(B, Tq, Hq, Hk, D, page, L, seed=Tq)
    check_attention(gkd, q, codes, scales, table, causal=causal)
    length = torch.randint(0, L * page + 1, (B,), generator=rng(Tq + 1), device="cuda").to(torch.int32)
    q_len = torch.randint(0, Tq + 1, (B,), generator=rng(Tq + 2), device="cuda").to(torch.int32)
    check_attention(gkd, q, codes, scales, table, length, q_len, causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160])
def test_attention_lengths(gkd, D, n):
    q, codes, scales, table = attn_inputs(2, 3, 4, 2, D, 32, 5, seed=n)
    # what lies behind the last token is not a number
    for b in range(2):
        for i in range(n, 160):
            scales[int(table[b, i // 32]), :, :, i % 32] = 255
    for causal in (False, True):
        got = check_attention(gkd, q, codes, scales, table, ints(n, n), causal=causal)
        if n == 0:
            assert not got.any()
    # more queries than tokens: the first ones see none
    if n in (1, 2):
        got = gkd.cache_attention(q, codes, scales, table, length=ints(n, n), causal=True)
        assert not got[:, :3 - n].any() and bool(got[:, 3 - n:].any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_long(gkd, D, causal):
    q, codes, scales, table = attn_inputs(3, 1, 8, 2, D, 64, 70, seed=1, spread=0.5)
    check_attention(gkd, q, codes, scales, table, ints(4480, 4001, 70), causal=causal)
    q, codes, scales, table = attn_inputs(1, 20, 8, 4, D, 128, 60, seed=2, spread=0.5)
    check_attention(gkd, q, codes, scales, table, ints(7333), causal=causal)
    q, codes, scales, table = attn_inputs(1, 2, 3, 1, D, 32, 1100, seed=3, spread=0.5)
    check_attention(gkd, q, codes, scales, table, ints(35001), causal=causal)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_rows(gkd, D):
    q, codes, scales, table = attn_inputs(2, 80, 4, 4, D, 64, 10, seed=4)
    check_attention(gkd, q, codes, scales, table, ints(576, 640), ints(80, 11))
    q, codes, scales, table = attn_inputs(1, 150, 6, 2, D, 64, 5, seed=5)
    check_attention(gkd, q, codes, scales, table, ints(300), causal=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Tq,Hq,Hk", [(90, 1, 6, 3), (45, 10, 9, 3), (30, 20, 6, 3), (20, 36, 6, 3), (70, 65, 4, 1)])
def test_attention_more_tiles_than_compute_units(gkd, B, Tq, Hq, Hk, D, causal):
    """One, two, three and more tiles of 16 rows of a key head, all of them or as many as a
    sequence has."""
    q, codes, scales, table = many_pages(B, Tq, Hq, Hk, D, 5, seed=Tq)
    length = torch.randint(0, 161, (B,), generator=rng(B), device="cuda").to(torch.int32)
    q_len = torch.randint(0, Tq + 1, (B,), generator=rng(B + 1), device="cuda").to(torch.int32)
    length[0], q_len[0], length[1], q_len[2] = 160, Tq, 0, 0
    table[3:9, 1] = -1
    check_attention(gkd, q, codes, scales, table, length, q_len, causal)


def many_pages(B, Tq, Hq, Hk, D, L, seed):
    """Room for 32 L tokens a sequence on a few pages, so that columns share them: keys are
    few to look at, and how the work is cut goes by the room."""
    g = rng(seed)
    codes, scales = gkd_quantised(g, 50, Hk, 32, D, 0.5)
    return randn(g, B, Tq, Hq, D), codes, scales, torch.randint(0, 50, (B, L), generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Tq,Hq,Hk", [(1, 1, 8, 1), (6, 1, 4, 2), (3, 9, 6, 3), (5, 40, 2, 2), (2, 70, 2, 1)])
def test_attention_room_for_many_tokens(gkd, B, Tq, Hq, Hk, D, causal):
    q, codes, scales, table = many_pages(B, Tq, Hq, Hk, D, 170, seed=Tq)
    length = torch.randint(0, 700, (B,), generator=rng(B), device="cuda").to(torch.int32)
    q_len = torch.randint(0, Tq + 1, (B,), generator=rng(B + 1), device="cuda").to(torch.int32)
    length[-1], q_len[-1] = 5440, Tq
    check_attention(gkd, q, codes, scales, table, length, q_len, causal)
    # columns without a page, whole steps of them
    table[:, 1:4], table[-1, 60:160], table[-1, 8] = -1, 50, 2**31 - 1
    check_attention(gkd, q, codes, scales, table, length, None, causal)
    # idle sequences around one, and none at all
    length[:-1] = 0
    check_attention(gkd, q, codes, scales, table, length, None, causal)
    length[-1] = 0
    assert not check_attention(gkd, q, codes, scales, table, length, None, causal).any()


def test_attention_many_sequences_with_room(gkd):
    for B in (1024, 1025):
        q, codes, scales, table = many_pages(B, 1, 2, 1, 64, 270, seed=B)
        length = torch.randint(0, 40, (B,), generator=rng(B), device="cuda").to(torch.int32)
        length[3], length[-1], length[700:720] = 2000, 8640, 0
        check_attention(gkd, q, codes, scales, table, length)


def test_attention_short_tiles_beside_a_long_one(gkd):
    """One sequence of 960 rows and 120000 tokens, and 23 of one to three tokens: more tiles
    than one share lists at a time."""
    B, Tq, H, D = 24, 960, 4, 128
    q, codes, scales, table = many_pages(B, Tq, H, H, D, 3750, seed=31)
    length = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    length[::3], length[12] = 1, 120000
    length[1::3] = 3
    out = gkd.cache_attention(q, codes, scales, table, length=length)
    rows = [0, 47, 48, 500, 959]
    for b in (0, 1, 11, 12, 13, 23):
        want, mean_abs, worst = of.attention(np64(q[b:b + 1, rows]), arr(codes), arr(scales), arr(table[b:b + 1]),
                                             arr(length[b:b + 1]))
        assert np.all(np.abs(np64(out[b:b + 1, rows]) - want) <= attention_tol(want, mean_abs, worst)), b
    # a row's result is that of its sequence by itself, up to how its keys are cut: the short
    # ones are one step, which is never cut
    for b in (0, 1, 11, 13, 23):
        alone = gkd.cache_attention(q[b:b + 1], codes, scales, table[b:b + 1, :1], length=length[b:b + 1])
        assert torch.equal(out[b:b + 1], alone), b


def test_attention_a_long_sequence_among_many_tiles(gkd):
    """More than four times as many tiles as stay resident, and room for one sequence to
    outlast them: its keys are shared, the short ones are as they are by themselves."""
    B, H, D, L = 600, 8, 128, 1100
    assert gkd.cache_attention_workspace_size(B, 1, H, H, D, 32, L) > 0
    q, codes, scales, table = many_pages(B, 1, H, H, D, L, seed=51)
    length = torch.randint(0, 33, (B,), generator=rng(52), device="cuda").to(torch.int32)
    length[0], length[200], length[201], length[599] = 4000, 35011, 0, 700
    out = gkd.cache_attention(q, codes, scales, table, length=length)
    for b in (0, 200, 599):
        want, mean_abs, worst = of.attention(np64(q[b:b + 1]), arr(codes), arr(scales), arr(table[b:b + 1]),
                                             arr(length[b:b + 1]))
        assert np.all(np.abs(np64(out[b:b + 1]) - want) <= attention_tol(want, mean_abs, worst)), b
    alone = gkd.cache_attention(q, codes, scales, table[:, :1].contiguous(), length=length.clamp_max(32))
    one_step = length <= 32
    assert torch.equal(out[one_step], alone[one_step])


@pytest.mark.parametrize("causal", [False, True])
def test_attention_many_rows_of_one_key_head(gkd, causal):
    """As many tiles, all of one key head: they are spread over the whole GPU."""
    Tq, Hq, D, L = 9300, 16, 64, 260
    assert gkd.cache_attention_workspace_size(1, Tq, Hq, 1, D, 32, L) > 0
    q, codes, scales, table = many_pages(1, Tq, Hq, 1, D, L, seed=53)
    q_len, length = 9290, 8300
    out = torch.full_like(q, 7)
    gkd.cache_attention(q, codes, scales, table, length=ints(length), q_len=ints(q_len), causal=causal, out=out)
    assert bool((out[:, q_len:] == 7).all())
    for t in (0, 1, 900, 989, 990, 991, 992, 1021, 5000, 9288, 9289):
        sees = length - q_len + t + 1 if causal else length
        if sees <= 0:
            assert not out[:, t].any(), t
            continue
        want, mean_abs, worst = of.attention(np64(q[:, t:t + 1]), arr(codes), arr(scales), arr(table), np.array([sees]))
        assert np.all(np.abs(np64(out[:, t:t + 1]) - want) <= attention_tol(want, mean_abs, worst)), t


@pytest.mark.parametrize("B,Hk,L,long", [(2500, 1, 520, {0: 700, 3: 16600, 1026: 5000, 2499: 90}),
                                         (10500, 4, 4300, {7: 1000, 5003: 17000, 10498: 5000})])
def test_attention_shares_many_sequences(gkd, B, Hk, L, long):
    """Several sequences an entry of the running sum, more than one listing's pieces a share."""
    assert gkd.cache_attention_workspace_size(B, 1, Hk, Hk, 64, 32, L) > 0
    q, codes, scales, table = many_pages(B, 1, Hk, Hk, 64, L, seed=B)
    length = torch.randint(0, 33, (B,), generator=rng(B), device="cuda").to(torch.int32)
    length[100:108], length[1030:1033] = 0, 0
    for b, n in long.items():
        length[b] = n
    out = gkd.cache_attention(q, codes, scales, table, length=length)
    for b in long:
        want, mean_abs, worst = of.attention(np64(q[b:b + 1]), arr(codes), arr(scales), arr(table[b:b + 1]),
                                             arr(length[b:b + 1]))
        assert np.all(np.abs(np64(out[b:b + 1]) - want) <= attention_tol(want, mean_abs, worst)), b
    alone = gkd.cache_attention(q, codes, scales, table[:, :1].contiguous(), length=length.clamp_max(32))
    one_step = length <= 32
    assert torch.equal(out[one_step], alone[one_step])


def test_attention_lengths_are_clamped(gkd):
    q, codes, scales, table = attn_inputs(3, 2, 2, 1, 64, 32, 2, seed=6)
    check_attention(gkd, q, codes, scales, table, ints(1000, -5, 2**31 - 1), ints(-3, 9, 1))
    check_attention(gkd, q, codes, scales, table, ints(1000, -5, 64), ints(2, 9, -2**31), causal=True)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_pages_that_are_not_there(gkd, D):
    q, codes, scales, table = attn_inputs(3, 2, 4, 2, D, 32, 6, seed=7)
    table[0, 1], table[1, 0], table[1, 5] = -1, codes.shape[0], 2**31 - 1
    table[2] = -7
    for causal in (False, True):
        got = check_attention(gkd, q, codes, scales, table, ints(150, 192, 190), causal=causal)
        assert not got[2].any()
    empty = gkd.cache_attention(q, codes[:0], scales[:0], table)
    assert not empty.any()
    assert not gkd.cache_attention(q, codes, scales, table[:, :0]).any()


def test_attention_sequences_share_pages(gkd):
    q, codes, scales, table = attn_inputs(4, 1, 4, 2, 128, 64, 6, seed=8)
    table[1:, :4] = table[0, :4]
    check_attention(gkd, q, codes, scales, table, ints(384, 300, 256, 257))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_rows_that_are_not_in_use(gkd, D):
    q, codes, scales, table = attn_inputs(3, 9, 4, 2, D, 32, 40, seed=9)
    q_len, length = ints(9, 0, 4), ints(1280, 700, 5)
    want = check_attention(gkd, q, codes, scales, table, length, q_len)
    q[1], q[2, 4:] = float("nan"), float("nan")
    out = torch.full((3, 9, 4, D + 8), 7.0, dtype=BF, device="cuda")
    got = gkd.cache_attention(q, codes, scales, table, length=length, q_len=q_len, out=out[..., :D])
    assert bool((out[1] == 7).all()) and bool((out[2, 4:] == 7).all()) and bool((out[..., D:] == 7).all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[2, :4], want[2, :4])


def test_attention_strided_queries(gkd):
    g = rng(10)
    _, codes, scales, table = attn_inputs(2, 1, 6, 2, 64, 64, 3, seed=10)
    q = randn(g, 2, 5, 6 * 64 + 64)[..., 32:32 + 6 * 64].unflatten(2, (6, 64))
    a = check_attention(gkd, q, codes, scales, table, ints(190, 77))
    b = gkd.cache_attention(q.contiguous(), codes, scales, table, length=ints(190, 77))
    assert torch.equal(a, b)
    t = randn(g, 6, 2, 5, 64).permute(1, 2, 0, 3)  # heads outermost
    check_attention(gkd, t, codes, scales, table, ints(190, 77), causal=True)
    e = randn(g, 1, 1, 1, 64).expand(2, 5, 6, 64)  # one query for all
    check_attention(gkd, e, codes, scales, table, ints(190, 77))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_large_scores_keep_their_largest(gkd, D):
    """Scores far out: the row is the value of the one key that leads."""
    q, codes, scales, table = attn_inputs(1, 2, 4, 2, D, 32, 4, seed=11)
    for scale in (1e6, 1e20, 1e30):
        got = gkd.cache_attention(q, codes, scales, table, scale=scale)
        assert bool(torch.isfinite(got).all())
        k, v = (np64(t)[0] for t in gkd.cache_read(codes, scales, table, 128))
        for t in range(2):
            for h in range(4):
                s = k[:, h // 2] @ np64(q)[0, t, h]
                first, second = np.argsort(-s)[:2]
                if s[first] - s[second] > 1e-3 * abs(s[first]):  # far past float32's rounding of the score
                    assert np.array_equal(np64(got)[0, t, h], v[first, h // 2])


@pytest.mark.parametrize("D", [64, 128])
def test_attention_large_scores_in_parts(gkd, D):
    """As above, the keys in parts that are joined, with what lies behind them not a number."""
    q, codes, scales, table = attn_inputs(2, 2, 4, 2, D, 32, 140, seed=21)
    assert gkd.cache_attention_workspace_size(2, 2, 4, 2, D, 32, 140) > 0
    n = 4433
    flat = table.long().flatten(1)
    for b in range(2):
        scales[flat[b, n // 32], :, :, n % 32:] = 255
        scales[flat[b, n // 32 + 1:]] = 255
    length = ints(n, n)
    check_attention(gkd, q, codes, scales, table, length)
    for scale in (1e6, 1e20, 1e30):
        got = gkd.cache_attention(q, codes, scales, table, length=length, scale=scale)
        assert bool(torch.isfinite(got).all())
        k, v = (np64(t) for t in gkd.cache_read(codes, scales, table, n))
        for b in range(2):
            for t in range(2):
                for h in range(4):
                    s = k[b, :, h // 2] @ np64(q)[b, t, h]
                    first, second = np.argsort(-s)[:2]
                    if s[first] - s[second] > 1e-3 * abs(s[first]):
                        assert np.array_equal(np64(got)[b, t, h], v[b, first, h // 2])
    q2 = q * 30
    q2[1, 1, 2] = q[1, 1, 2]
    a, b = (gkd.cache_attention(x, codes, scales, table, length=length) for x in (q, q2))
    assert torch.equal(a[1, 1, 2], b[1, 1, 2])


def test_attention_small_scale_is_the_mean(gkd):
    q, codes, scales, table = attn_inputs(1, 1, 2, 1, 64, 32, 3, seed=12)
    check_attention(gkd, q, codes, scales, table, ints(90), scale=1e-30)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_rising_scores_move_the_reference_point(gkd, D):
    """Keys that grow from step to step: every step passes the reference point."""
    q, codes, scales, table = attn_inputs(2, 3, 4, 2, D, 32, 40, seed=13)
    rows = torch.arange(1280, device="cuda") // 40  # 32 steps of the scale
    unit = (100 + rows).clamp_max(130).to(U8)
    for b in range(2):
        for c in range(40):
            scales[table[b, c].long(), 0] = unit[32 * c:32 * c + 32, None]
    check_attention(gkd, q, codes, scales, table, ints(1280, 1111), scale=1.0)
    check_attention(gkd, q, codes, scales, table, ints(1280, 1111), causal=True, scale=1.0)
    for b in range(2):
        for c in range(40):
            scales[table[b, c].long(), 0] = unit.flip(0)[32 * c:32 * c + 32, None]
    check_attention(gkd, q, codes, scales, table, ints(1280, 1111), scale=1.0)


def test_attention_a_row_does_not_depend_on_the_rows_beside_it(gkd):
    q, codes, scales, table = attn_inputs(3, 4, 8, 2, 128, 64, 6, seed=14)
    length = ints(300, 384, 100)
    a = gkd.cache_attention(q, codes, scales, table, length=length)
    q2 = q * 30
    q2[1, 2] = q[1, 2]
    b = gkd.cache_attention(q2, codes, scales, table, length=length)
    assert torch.equal(a[1, 2], b[1, 2])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [30, 400])
def test_attention_a_row_does_not_depend_on_far_rows_beside_it(gkd, D, L):
    """Every other row's scores pass 2^24 in magnitude, of either sign: the rows between them
    keep every bit of their results, though their own scores are far enough out (element 0
    adds 2^20 or so to each) for a rounded product to show."""
    g = rng(L)
    kv = torch.randn(6 * L, 2, 2, 32, D, generator=g, device="cuda")
    kv[:, 0, :, :, :32] = 0
    kv[:, 0, :, :, 0] = 1
    codes, scales = gkd.quantize_fp4(kv)
    table = torch.randperm(6 * L, generator=g, device="cuda").reshape(6, L).to(torch.int32)
    q = randn(g, 6, 6, 8, D)
    q[..., 0] = 2.0 ** 22
    length = torch.tensor([32 * L, 32 * L - 40, 17 * L, 500, 31 * L, 900], dtype=torch.int32, device="cuda")
    a = gkd.cache_attention(q, codes, scales, table, length=length)
    for factor in (2.0 ** 10, -2.0 ** 10):
        q2 = q.clone()
        q2[:, 1::2, ::3] *= factor
        q2[:, 0::2, 1::3] *= factor
        b = gkd.cache_attention(q2, codes, scales, table, length=length)
        kept = (q2 == q).all(-1)
        assert torch.equal(a[kept], b[kept])
        assert bool(torch.isfinite(b).all())


def test_attention_pages_past_32_bit_offsets(gkd):
    """A pool of more than 2^32 bytes of codes: the last page lies past them."""
    page, Hk, D = 1024, 16, 128
    per = 2 * Hk * page * D // 2
    pages = (1 << 32) // per + 40
    codes = torch.empty(pages, 2, Hk, page, D // 2, dtype=U8, device="cuda")
    scales = torch.empty(pages, 2, Hk, page, D // 32, dtype=U8, device="cuda")
    q, c, s, _ = attn_inputs(1, 1, Hk, Hk, D, page, 2, seed=15, pages=2)
    codes[-2:], scales[-2:] = c, s
    near = gkd.cache_attention(q, c, s, ints(0, 1)[None], length=ints(1500))
    far = gkd.cache_attention(q, codes, scales, ints(pages - 2, pages - 1)[None], length=ints(1500))
    assert torch.equal(near, far)
    k, v = randn(rng(1), 1, 3, Hk, D), randn(rng(2), 1, 3, Hk, D)
    gkd.cache_append(k, v, c, s, ints(0, 1)[None], start=ints(1022))
    gkd.cache_append(k, v, codes, scales, ints(pages - 2, pages - 1)[None], start=ints(1022))
    assert torch.equal(codes[-2:], c) and torch.equal(scales[-2:], s)
    a = gkd.cache_read(c, s, ints(0, 1)[None], 5, start=ints(1021))
    b = gkd.cache_read(codes, scales, ints(pages - 2, pages - 1)[None], 5, start=ints(1021))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def named_values(gkd, B, Hk, D, page, L, name):
    """A cache whose keys are zeros and whose value at token j has a 1 at element name(j), with
    a table in no order."""
    table = torch.randperm(B * L, generator=rng(L), device="cuda").reshape(B, L).to(torch.int32)
    j = torch.arange(L * page, device="cuda")
    v = (name(j)[:, None] == torch.arange(D, device="cuda")).to(BF)
    c, s = gkd.quantize_fp4(v)
    codes = torch.zeros(B * L, 2, Hk, page, D // 2, dtype=U8, device="cuda")
    scales = torch.full((B * L, 2, Hk, page, D // 32), 127, dtype=U8, device="cuda")
    for b in range(B):
        codes[table[b].long(), 1] = c.view(L, 1, page, -1)
        scales[table[b].long(), 1] = s.view(L, 1, page, -1)
    return codes, scales, table


NAMED = [  # B, Tq, Hq, Hk, page, L, lengths, q_len: one row, several tiles, one to three of 16 rows together
    (3, 1, 8, 2, 64, 70, (4480, 4001, 70), None), (1, 20, 8, 4, 128, 60, (7333,), None),
    (1, 2, 3, 1, 32, 1100, (35001,), None), (6, 1, 16, 16, 64, 36, (2304, 1, 0, 33, 2000, 640), None),
    (3, 40, 8, 8, 64, 200, (12800, 6401, 31), (40, 17, 9)), (2, 30, 16, 4, 64, 150, (9600, 9543), (30, 29)),
    (5, 80, 16, 16, 64, 36, (2304, 77, 2303, 1000, 5), (80, 3, 65, 80, 16)), (1, 300, 8, 2, 128, 100, (12790,), None),
    (1, 1, 8, 2, 128, 1500, (191999,), None)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("by_step", [True, False])
@pytest.mark.parametrize("B,Tq,Hq,Hk,page,L,lengths,q_len", NAMED)
def test_attention_counts_every_key_once(gkd, B, Tq, Hq, Hk, page, L, lengths, q_len, by_step, D):
    """Queries of zeros see all keys alike, and an output element is the share of the keys that
    name it, by their step of 32 or by their place in every step. Sums are whole numbers in
    float32, and their quotient is rounded three times. Up to 94 steps name an element: one
    that is left out, or taken twice, changes it by more than two roundings."""
    unit = 32 if by_step else 1
    codes, scales, table = named_values(gkd, B, Hk, D, page, L, lambda j: j // unit % D)
    q = torch.zeros(B, Tq, Hq, D, dtype=BF, device="cuda")
    length = ints(*lengths)
    rows = torch.full((B,), Tq, device="cuda") if q_len is None else ints(*q_len)
    t, d = torch.arange(Tq, device="cuda"), torch.arange(D, device="cuda")
    for causal in (False, True):
        out = gkd.cache_attention(q, codes, scales, table, length=length, q_len=None if q_len is None else ints(*q_len),
                                  causal=causal)
        n = (length[:, None] - rows[:, None] + t + 1).clamp_min(0) if causal else length[:, None].expand(B, Tq)
        n = torch.where(t < rows[:, None], n, 0).double()[..., None]               # keys that a row sees
        per = unit * D
        count = (n / per).floor() * unit + (n % per - unit * d).clamp(0, unit)     # those that name each element
        want = (count / n.clamp_min(1))[:, :, None]
        err = (out.double() - want).abs()
        assert bool((err <= want * (2.0 ** -8 + 2.0 ** -22)).all()), err.max()


@pytest.mark.parametrize("D", [64, 128])
def test_attention_largest_values(gkd, D):
    """Values of up to 1e24, one step after another passing the reference point's slack."""
    q, codes, scales, table = attn_inputs(2, 3, 4, 2, D, 32, 140, seed=25)
    scales[:, 1] = 127 + 77
    scales[:, 0] = scales[:, 0] // 8 * 8
    assert 6 * 2.0 ** 77 < 1e24
    check_attention(gkd, q, codes, scales, table, ints(4470, 33), causal=True)


def test_attention_refusals(gkd):
    q, codes, scales, table = attn_inputs(2, 1, 4, 2, 64, 32, 2, seed=16)
    assert gkd.cache_attention(q[:0], codes, scales, table[:0]).shape == (0, 1, 4, 64)
    assert gkd.cache_attention(q[:, :0], codes, scales, table).shape == (2, 0, 4, 64)
    for bad in (lambda: gkd.cache_attention(q, codes, scales, table[:1]),
                lambda: gkd.cache_attention(q, codes, scales[:, :1], table),
                lambda: gkd.cache_attention(q, codes, scales, table.long()),
                lambda: gkd.cache_attention(q, codes, scales, table, length=ints(1)),
                lambda: gkd.cache_attention(q[..., :32], codes, scales, table),
                lambda: gkd.cache_attention(q.float(), codes, scales, table),
                lambda: gkd.cache_attention(q, codes[..., ::2], scales, table),
                lambda: gkd.cache_attention(q, codes.cpu(), scales, table)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for status, bad in ((5, lambda: gkd.cache_attention(q[:, :, :3], codes, scales, table)),
                        (4, lambda: gkd.cache_attention(q, codes, scales, table, scale=0.0)),
                        (4, lambda: gkd.cache_attention(q, codes, scales, table, scale=float("nan"))),
                        (2, lambda: gkd.cache_attention(q, codes, scales, table,
                                                        out=q[:1].clone().expand(2, 1, 4, 64)))):
        with pytest.raises(gkd.GkdError) as e:
            bad()
        assert e.value.status == status


# ------------------------------------------------- streams, graphs, together
def test_calls_run_on_the_current_stream(gkd):
    q, codes, scales, table = attn_inputs(2, 1, 8, 2, 128, 64, 20, seed=17)
    k = randn(rng(3), 2, 1, 2, 128)
    start, length = ints(700, 900), ints(701, 901)
    c2, s2 = codes.clone(), scales.clone()
    gkd.cache_append(k, k, c2, s2, table, start=start)
    want = gkd.cache_attention(q, c2, s2, table, length=length)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        gkd.cache_append(k, k, codes, scales, table, start=start)
        got = gkd.cache_attention(q, codes, scales, table, length=length)
    st.synchronize()
    assert torch.equal(got, want)


def test_calls_take_their_place_on_a_busy_stream(gkd):
    """Long work on a stream that writes the inputs last: a call that ran on any other stream
    would take the old ones."""
    B, H, D, page, L = 2, 2, 128, 64, 130
    q, codes, scales, table = attn_inputs(B, 1, 8, H, D, page, L, seed=61)
    assert gkd.cache_attention_workspace_size(B, 1, 8, H, D, page, L) > 0
    g = rng(62)
    new = dict(q=randn(g, B, 1, 8, D), k=randn(g, B, 3, H, D), x=randn(g, 128, 8192), w=randn(g, 1030, 8192, scale=1 / 64),
               start=ints(5000, 900), length=ints(5003, 903))
    assert gkd.linear_fp4_workspace_size(128, 1030, 8192) > 0

    def calls(s, c, sc):
        wc, ws = gkd.quantize_fp4(s["w"])
        gkd.cache_append(s["k"], s["k"], c, sc, table, start=s["start"])
        return (gkd.cache_attention(s["q"], c, sc, table, length=s["length"]), gkd.linear_fp4(s["x"], wc, ws),
                gkd.cache_attention(s["q"], c, sc, table[:, :4].contiguous()), wc, ws,
                *gkd.cache_read(c, sc, table, 3, start=s["start"]))

    c2, s2 = codes.clone(), scales.clone()
    want = calls(new, c2, s2)
    old = {n: torch.zeros_like(t) for n, t in new.items()}
    a = torch.randn(4096, 4096, device="cuda").to(BF)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        calls(old, codes.clone(), scales.clone())  # (the stream's memory is there from here on)
        a @ a / 64
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        busy = a
        for _ in range(60):
            busy = busy @ a / 64
        for n in old:
            old[n].copy_(new[n])
        got = calls(old, codes, scales)
        ended = st.query()
    st.synchronize()
    assert not ended  # the calls were made while the work was under way
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


def test_captured_step_follows_its_inputs(gkd):
    """A decoding step captured once and replayed while its inputs change in place,
    with other work between the replays: every replay equals the eager step."""
    B, Hq, Hk, D, page, L, K = 3, 8, 2, 128, 64, 12, 1024
    g = rng(18)
    q, codes, scales, table = attn_inputs(B, 1, Hq, Hk, D, page, L, seed=18)
    wc, ws = gkd.quantize_fp4(randn(g, 512, Hq * D, scale=1 / 32))
    k, v = randn(g, B, 1, Hk, D), randn(g, B, 1, Hk, D)
    start = ints(100, 300, 511)
    work = torch.empty(max(1, gkd.cache_attention_workspace_size(B, 1, Hq, Hk, D, page, L)), dtype=U8, device="cuda")
    lwork = torch.empty(max(1, gkd.linear_fp4_workspace_size(B, 512, Hq * D)), dtype=U8, device="cuda")
    out, y = torch.empty_like(q), torch.empty(B, 512, dtype=BF, device="cuda")
    length = start + 1

    def step(c, s, o, z):
        gkd.cache_append(k, v, c, s, table, start=start)
        gkd.cache_attention(q, c, s, table, length=length, out=o, workspace=work)
        gkd.linear_fp4(o.view(B, -1), wc, ws, act="silu", out=z, workspace=lwork)

    step(codes, scales, out, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(codes, scales, out, y)
    for i in range(4):
        start.add_(1)
        length.add_(1)
        q.copy_(randn(g, *q.shape))
        k.copy_(randn(g, *k.shape))
        v.copy_(randn(g, *v.shape))
        c2, s2, o2, y2 = codes.clone(), scales.clone(), torch.empty_like(out), torch.empty_like(y)
        step(c2, s2, o2, y2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(codes, c2) and torch.equal(scales, s2), i
        assert torch.equal(out, o2) and torch.equal(y, y2), i


def test_captured_steps_of_long_caches_and_two_streams(gkd):
    """Two captured steps with workspaces of their own, replayed side by side on two streams
    while their inputs change between the replays."""
    B, Hq, Hk, D, L = 3, 8, 2, 64, 200
    need = gkd.cache_attention_workspace_size(B, 2, Hq, Hk, D, 32, L), gkd.linear_fp4_workspace_size(128, 1030, 8192)
    assert min(need) > 0
    g = rng(40)
    wc, ws = gkd.quantize_fp4(randn(g, 1030, 8192, scale=1 / 64))
    sets = []
    for i in range(2):
        q, codes, scales, table = many_pages(B, 2, Hq, Hk, D, L, seed=41 + i)
        length, x = ints(6400, 1000 * i + 17, 90), randn(g, 128, 8192)
        work = [torch.empty(n, dtype=U8, device="cuda") for n in need]
        out, y = torch.empty_like(q), torch.empty(128, 1030, dtype=BF, device="cuda")

        def step(q=q, codes=codes, scales=scales, table=table, length=length, x=x, work=work, out=out, y=y):
            gkd.cache_attention(q, codes, scales, table, length=length, causal=True, out=out, workspace=work[0])
            gkd.linear_fp4(x, wc, ws, out=y, workspace=work[1])

        step()
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=st):
            step()
        sets.append((q, codes, scales, table, length, x, out, y, st, graph))
    for n in range(3):
        for q, _, _, _, length, x, out, y, _, _ in sets:
            length.sub_(5)
            q.copy_(randn(g, *q.shape))
            x.copy_(randn(g, *x.shape))
            out.fill_(7)
            y.fill_(7)
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s[8]):
                s[9].replay()
        torch.cuda.synchronize()
        for q, codes, scales, table, length, x, out, y, _, _ in sets:
            assert torch.equal(out, gkd.cache_attention(q, codes, scales, table, length=length, causal=True)), n
            assert torch.equal(y, gkd.linear_fp4(x, wc, ws)), n


def test_results_do_not_change_from_call_to_call(gkd):
    q, codes, scales, table = attn_inputs(2, 2, 8, 2, 64, 64, 100, seed=19)
    x = randn(rng(4), 50, 2048)
    wc, ws = gkd.quantize_fp4(randn(rng(5), 1000, 2048))
    a = gkd.cache_attention(q, codes, scales, table), gkd.linear_fp4(x, wc, ws, out_dtype=F32)
    for _ in range(5):
        b = gkd.cache_attention(q, codes, scales, table), gkd.linear_fp4(x, wc, ws, out_dtype=F32)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_block_of_four_bit_operators_together(gkd):
    """Tokens of an image stored, then prompt rows through a block: projections with
    four-bit weights, positions, attention over the stored image, projection and
    residual, two feed-forward layers. Each step against the oracle on its inputs."""
    g = rng(20)
    C, H, D, T, R, page = 256, 4, 64, 149, 11, 32
    L = (T + page - 1) // page
    tokens, prompts = randn(g, 2, T, C), randn(g, 2, R, C)
    weight = {n: gkd.quantize_fp4(randn(g, *s, scale=s[1] ** -0.5, dtype=F32)) for n, s in
              dict(kv=(2 * C, C), q=(C, C), o=(C, C), up=(4 * C, C), down=(C, 4 * C)).items()}
    pos = torch.rand(T, 2, generator=g, device="cuda") * 24
    freqs = torch.stack([torch.linspace(1, 0.1, 32, device="cuda") * m for m in (0, 1)])
    codes, scales = new_cache(2 * L, H, page, D, 255)
    table = torch.randperm(2 * L, generator=g, device="cuda").reshape(2, L).to(torch.int32)

    def linear(x, name, act="none", residual=None, out=BF):
        c, s = weight[name]
        y = gkd.linear_fp4(x, c, s, act=act, residual=residual, out_dtype=out)
        n, k = c.shape[0], 2 * c.shape[1]
        r = None if residual is None else np64(residual).reshape(-1, n)
        want, size = ot.linear(np64(x).reshape(-1, k), of.values(arr(c), arr(s)), None, r, act)
        assert np.all(np.abs(np64(y).reshape(-1, n) - want) <= linear_tol(want, size, k, out, r))
        return y

    kv = linear(tokens, "kv").unflatten(-1, (2, H, D))
    k, _ = gkd.qk_norm_rope(kv[:, :, 0], None, pos, freqs)
    gkd.cache_append(k, kv[:, :, 1], codes, scales, table)
    ko, vo = gkd.cache_read(codes, scales, table, T)
    for x, y in ((k, ko), (kv[:, :, 1], vo)):
        assert np.array_equal(np64(y), of.values(*of.quantise(np64(x))))
    q = linear(prompts, "q").unflatten(-1, (H, D))
    length = ints(T, T)
    a = check_attention(gkd, q, codes, scales, table, length, ints(R, 6))
    h = linear(a.flatten(2), "o", residual=prompts.float(), out=F32)
    u = linear(h.to(BF), "up", "gelu")
    y = linear(u, "down", residual=h, out=F32)
    assert bool(torch.isfinite(y).all())
    # the same keys held in bfloat16 give the same attention, but for its own rounding
    b = gkd.prefix_attention(q, None, None, ko, vo, q_len=ints(R, 6))
    want, mean_abs, worst = of.attention(np64(q), arr(codes), arr(scales), arr(table), arr(length), np.array([R, 6]))
    assert np.all(np.abs(np64(a) - np64(b)) <= 2 * attention_tol(want, mean_abs, worst))
